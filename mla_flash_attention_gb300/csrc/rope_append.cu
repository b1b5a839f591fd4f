// Append new tokens to the paged latent cache with the latent's norm and the rope key's
// rotation on the way (mla_cache_append takes rows that are finished).
//
//   row = [w c / sqrt(mean(c^2) + eps) | R(pos) k_rope],  c the 512 latent columns of the raw row
//   bf16 cache: rounded once to bf16; e4m3 cache: scale = max|row| / 448 (1 if all zero), codes =
//   e4m3(clamp(row / scale, +-448)), from the fp32 row, so a value is rounded once there too.
//
// Bound by memory (1152 bytes in, 1152 or 580 out a row) or, for a decode step's few rows, by the
// chain length -> page-table entry -> store.  Sixteen lanes a row, two rows a warp: lane l holds
// latent columns 8 l + 128 i (16-byte loads, 8- or 16-byte stores) and rope columns 4 l .. 4 l + 3;
// all the row's loads are issued at once (in large batches behind its sequence's count), and the page-table
// entry, which waits for the length, is fetched while the row is computed.  65536 rows into an e4m3 cache: 26.2 us (4.3 TB/s of rows in
// and out; into a bf16 cache 24.0 us, 6.3 TB/s), its instructions and the latency of a row's two reductions and scale in about equal
// parts.  With a whole warp a row, scalar arithmetic, a division for every code and the table entry
// awaited first it was 36 us.  (Blocks of two warps at 64 registers: with four 27.0, at 56
// registers 29.5.)
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "rope.cuh"

namespace mla {
namespace rope_append {

constexpr int kDl = 512, kDc = kDl + rope::kDr, kPage = 64;
constexpr int kWarps = 2;

struct Params {
  const uint16_t* c_new;  // rows of 576, row_stride elements apart
  long long row_stride;
  const uint16_t* w;  // [512] or null
  float eps;
  const int* positions;  // [B, T, axes], or null with one axis: a token's place in its sequence
  const unsigned long long* turns;  // [axes][32]
  int axes;
  void* cache;
  float* kv_scale;
  const int *page_table, *cache_lens, *new_lens;
  int rows, T, max_pages, num_pages;
  unsigned int* err;
};

// e4m3 codes of two values, low byte first; satfinite is the clamp to +-448, a NaN stays one.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t codes;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(codes) : "f"(hi), "f"(lo));
  return codes;
}
__device__ __forceinline__ uint32_t e4m3x2(uint64_t v) { return e4m3x2(ptx::f2_lo(v), ptx::f2_hi(v)); }

__device__ __forceinline__ uint64_t bf16x2_to_f2(uint32_t w) {
  return ptx::f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// sum / maximum over the 16 lanes of a row
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// kDrop: rows of padding are passed over before they are read.
template <bool kFp8, bool kPairs, bool kAxes, bool kDrop>
__global__ void __launch_bounds__(kWarps * 32, 16) rope_append_kernel(const Params p) {
  wait_for_stream();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int id = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * 2 + (lane >> 4);
  // a half-warp without a row to write stays for the other one's shuffles
  const bool in_range = id < p.rows;
  const int b = in_range ? static_cast<unsigned>(id) / static_cast<unsigned>(p.T) : 0, t = id - b * p.T;
  uint4 lat[4] = {};
  uint2 rp = make_uint2(0, 0);
  int L = 0, n = 0, pos = 0;
  if (in_range) {
    L = __ldg(p.cache_lens + b);
    n = p.new_lens ? __ldg(p.new_lens + b) : p.T;
  }
  if constexpr (kDrop) {
    if (!__any_sync(0xffffffffu, t < n)) return;
  }
  if (in_range) {
    if (!kAxes && p.positions) pos = __ldg(p.positions + id);
    const uint16_t* src = p.c_new + (long long)id * p.row_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) lat[i] = __ldg(reinterpret_cast<const uint4*>(src) + l + 16 * i);
    rp = __ldg(reinterpret_cast<const uint2*>(src + kDl) + l);
  }
  // lane l makes cos and sin of frequencies 2l and 2l + 1
  const ulonglong2* turns_l = reinterpret_cast<const ulonglong2*>(p.turns) + l;
  ulonglong2 turns = make_ulonglong2(0, 0);  // several axes: the phases themselves
  if constexpr (kAxes) {
#pragma unroll
    for (int a = 0; a < rope::kMaxAxes; ++a) {
      if (!in_range || a >= p.axes) break;
      const ulonglong2 of = __ldg(turns_l + a * (rope::kFreqs / 2));
      const int at = __ldg(p.positions + (long long)id * p.axes + a);
      turns.x += rope::phase(at, of.x);
      turns.y += rope::phase(at, of.y);
    }
  } else {
    turns = *turns_l;
  }
  const int place = static_cast<int>(max(min((long long)L - n + t, 0x7fffffffLL), -1LL));
  // rows t >= n are padding; of a sequence with fewer cached tokens than new ones the first have
  // no place; more new tokens than rows are refused
  bool write = t < n && (place >= 0 || n > p.T);
  if (!__any_sync(0xffffffffu, write)) return;
  const unsigned pg = static_cast<unsigned>(place) / kPage;
  int page = -1;  // on its way while the row is computed
  if (write && n <= p.T && pg < static_cast<unsigned>(p.max_pages))
    page = __ldg(p.page_table + (long long)b * p.max_pages + pg);

  uint64_t x[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i][0] = bf16x2_to_f2(lat[i].x);
    x[i][1] = bf16x2_to_f2(lat[i].y);
    x[i][2] = bf16x2_to_f2(lat[i].z);
    x[i][3] = bf16x2_to_f2(lat[i].w);
  }
  if (p.w) {
    uint64_t s2[2] = {ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) s2[k & 1] = ptx::fma2(x[i][k], x[i][k], s2[k & 1]);
    s2[0] = ptx::add2(s2[0], s2[1]);
    const float r = rsqrtf(row_sum(ptx::f2_lo(s2[0]) + ptx::f2_hi(s2[0])) * (1.f / kDl) + p.eps);
    const uint64_t r2 = ptx::f2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.w) + l + 16 * i);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] = ptx::mul2(ptx::mul2(x[i][k], r2), bf16x2_to_f2(ww[k]));
    }
  }
  // Rope columns 4l .. 4l + 3: two pairs, or the same half of four pairs (lanes 0..7 the first, lanes
  // 8..15 the second).
  if (!kAxes && !p.positions) pos = place;
  float c[2], s[2];
  rope::cos_sin(kAxes ? turns.x : rope::phase(pos, turns.x), c[0], s[0]);
  rope::cos_sin(kAxes ? turns.y : rope::phase(pos, turns.y), c[1], s[1]);
  const float a[4] = {__uint_as_float(rp.x << 16), __uint_as_float(rp.x & 0xffff0000u), __uint_as_float(rp.y << 16),
                      __uint_as_float(rp.y & 0xffff0000u)};
  float y[4];
  if constexpr (kPairs) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      y[2 * i] = a[2 * i] * c[i] - a[2 * i + 1] * s[i];
      y[2 * i + 1] = a[2 * i + 1] * c[i] + a[2 * i] * s[i];
    }
  } else {
    const float sign = l < 8 ? -1.f : 1.f;
    const int from = (lane & 16) + 2 * (l & 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float ci = __shfl_sync(0xffffffffu, c[i & 1], from + (i >> 1));
      const float si = __shfl_sync(0xffffffffu, s[i & 1], from + (i >> 1));
      const float other = __shfl_xor_sync(0xffffffffu, a[i], 8);
      y[i] = a[i] * ci + sign * (other * si);
    }
  }
  if (write && (page < 0 || page >= p.num_pages)) {
    if (l == 0) latch_error(p.err, kErrBadPage);
    write = false;
  }
  const long long dst = (long long)page * kPage + static_cast<unsigned>(place) % kPage;
  if constexpr (!kFp8) {
    if (!write) return;
    uint16_t* row = static_cast<uint16_t*>(p.cache) + dst * kDc;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(row)[l + 16 * i] =
          make_uint4(ptx::pack_bf16x2(ptx::f2_lo(x[i][0]), ptx::f2_hi(x[i][0])),
                     ptx::pack_bf16x2(ptx::f2_lo(x[i][1]), ptx::f2_hi(x[i][1])),
                     ptx::pack_bf16x2(ptx::f2_lo(x[i][2]), ptx::f2_hi(x[i][2])),
                     ptx::pack_bf16x2(ptx::f2_lo(x[i][3]), ptx::f2_hi(x[i][3])));
    reinterpret_cast<uint2*>(row + kDl)[l] = make_uint2(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]));
  } else {
    float amax = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = ptx::fmax3(amax, fabsf(ptx::f2_lo(x[i][k])), fabsf(ptx::f2_hi(x[i][k])));
    amax = row_max(amax);
    if (!write) return;  // the last shuffle is behind
    const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    // Codes of x / scale.  The quotient itself is not needed, only which code is nearest: it lies
    // between x in_lo and x in_hi, where in_lo and in_hi bracket 1 / scale by 2^-21 on either side
    // (four roundings of 2^-24 lie between), so if both round to the same code, that is the
    // quotient's.  Otherwise (a quotient that close to the middle of two codes: about one row in a
    // hundred), or with a scale too near 0 or infinity, the divisions are made.
    const float inv = __fdiv_rn(1.f, scale);
    const float in_lo = inv * (1.f - 0x1p-21f), in_hi = inv * (1.f + 0x1p-21f);
    const uint64_t lo2 = ptx::f2(in_lo, in_lo), hi2 = ptx::f2(in_hi, in_hi);
    const uint64_t y2[2] = {ptx::f2(y[0], y[1]), ptx::f2(y[2], y[3])};
    auto value = [&](int k) { return k < 16 ? x[k >> 2][k & 3] : y2[k - 16]; };
    uint32_t codes[9], off = !(scale > 1e-30f && scale < 1e30f);  // four codes a word
#pragma unroll
    for (int k = 0; k < 9; ++k) {
      codes[k] = e4m3x2(ptx::mul2(value(2 * k), lo2)) | e4m3x2(ptx::mul2(value(2 * k + 1), lo2)) << 16;
      off |= codes[k] ^ (e4m3x2(ptx::mul2(value(2 * k), hi2)) | e4m3x2(ptx::mul2(value(2 * k + 1), hi2)) << 16);
    }
    if (off != 0) {
#pragma unroll
      for (int k = 0; k < 9; ++k) {
        const uint64_t u = value(2 * k), v = value(2 * k + 1);
        codes[k] = e4m3x2(__fdiv_rn(ptx::f2_lo(u), scale), __fdiv_rn(ptx::f2_hi(u), scale)) |
                   e4m3x2(__fdiv_rn(ptx::f2_lo(v), scale), __fdiv_rn(ptx::f2_hi(v), scale)) << 16;
      }
    }
    uint8_t* row = static_cast<uint8_t*>(p.cache) + dst * kDc;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint2*>(row)[l + 16 * i] = make_uint2(codes[2 * i], codes[2 * i + 1]);
    reinterpret_cast<uint32_t*>(row + kDl)[l] = codes[8];
    if (l == 0) p.kv_scale[dst] = scale;
  }
}

}  // namespace rope_append

cudaError_t launch_rope_append(const void* c_new, long long row_stride, const void* w, float eps,
                               const int* positions, const void* turns, int axes, bool pairs, void* cache, float* kv_scale,
                               const int* page_table, const int* cache_lens, const int* new_lens, int B, int T,
                               int max_pages, int num_pages, bool fp8, unsigned int* err, cudaStream_t stream) {
  using namespace rope_append;
  Params p;
  p.c_new = static_cast<const uint16_t*>(c_new);
  p.row_stride = row_stride;
  p.w = static_cast<const uint16_t*>(w);
  p.eps = eps;
  p.positions = positions;
  p.axes = axes;
  p.turns = static_cast<const unsigned long long*>(turns);
  p.cache = cache;
  p.kv_scale = kv_scale;
  p.page_table = page_table;
  p.cache_lens = cache_lens;
  p.new_lens = new_lens;
  p.rows = B * T;
  p.T = T;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.err = err;
  const int grid = (p.rows + 2 * kWarps - 1) / (2 * kWarps);
  // Rows of padding are passed over where the rows are three times what stands on a GPU of 152 SMs at once, which hides the
  // length that this waits for (8 sequences of up to 8191 new rows, 44 % of the rows padding, 3 axes, from DRAM: bf16 21.5, so
  // 17.6 us; e4m3 23.5, so 21.7; with the rows in L2 20.4, so 14.4, and 21.0, so 18.5; 16384 rows the same either way; 64 to
  // 4096 rows 0.3 us more)
  const bool drop = new_lens && p.rows >= 32768;
  auto pick = [&](auto fp8_, auto pairs_) {
    constexpr bool f = decltype(fp8_)::value, r = decltype(pairs_)::value;
    return drop ? (axes > 1 ? rope_append_kernel<f, r, true, true> : rope_append_kernel<f, r, false, true>)
                : (axes > 1 ? rope_append_kernel<f, r, true, false> : rope_append_kernel<f, r, false, false>);
  };
  const std::true_type yes;
  const std::false_type no;
  auto kernel = fp8 ? (pairs ? pick(yes, yes) : pick(yes, no)) : (pairs ? pick(no, yes) : pick(no, no));
  // (a programmatic dependent: calls of 128 x 7 rows in a row take 3.3 instead of 6.2 us, of 65536 rows
  // 26.2 instead of 28.7)
  return launch_dependent(kernel, grid, kWarps * 32, stream, p);
}

}  // namespace mla
