// Append new tokens to the paged latent cache with the latent's norm and the rope key's
// rotation on the way (mla_cache_append takes rows that are finished).
//
//   row = [w c / sqrt(mean(c^2) + eps) | R(pos) k_rope],  c the 512 latent columns of the raw row
//   bf16 cache: rounded once to bf16; e4m3 cache: scale = max|row| / 448 (1 if all zero), codes =
//   e4m3(clamp(row / scale, +-448)), from the fp32 row, so a value is rounded once there too.
//
// Bound by memory (1152 bytes in, 1152 or 580 out a row) or, for a decode step's few rows, by the
// chain length -> page-table entry -> store.  One warp a row: lane l holds latent columns 8l and
// 256 + 8l on (16-byte loads, 8- or 16-byte stores) and rope columns 2l, 2l + 1; the row's loads
// are issued before the length, and the page-table entry is fetched while they are in flight.
#include <algorithm>

#include "common.cuh"
#include "rope.cuh"

namespace mla {
namespace rope_append {

constexpr int kDl = 512, kDc = kDl + rope::kDr, kPage = 64;
constexpr int kWarps = 4;

struct Params {
  const uint16_t* c_new;  // rows of 576, row_stride elements apart
  long long row_stride;
  const uint16_t* w;  // [512] or null
  float eps;
  const int* positions;  // [B, T] or null: a token's place in its sequence
  const unsigned long long* turns;
  void* cache;
  float* kv_scale;
  const int *page_table, *cache_lens, *new_lens;
  int rows, T, max_pages, num_pages;
  unsigned int* err;
};

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi, float scale) {
  // satfinite is the clamp to +-448; a NaN stays one
  uint16_t codes;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(codes) : "f"(__fdiv_rn(hi, scale)), "f"(__fdiv_rn(lo, scale)));
  return codes;
}

template <bool kFp8, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32) rope_append_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const int id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= p.rows) return;
  const int b = id / p.T, t = id - b * p.T;
  const uint16_t* src = p.c_new + (long long)id * p.row_stride;
  const uint4 lat[2] = {__ldg(reinterpret_cast<const uint4*>(src) + lane),
                        __ldg(reinterpret_cast<const uint4*>(src) + 32 + lane)};
  const uint32_t rp = __ldg(reinterpret_cast<const uint32_t*>(src + kDl) + lane);
  const long long L = __ldg(p.cache_lens + b);
  const int n = p.new_lens ? __ldg(p.new_lens + b) : p.T;
  if (t >= n) return;  // padding behind the sequence's last new token
  const long long place = L - n + t;
  if (place < 0 && n <= p.T) return;  // fewer cached tokens than new ones: nothing to write for this one
  const long long pg = place / kPage;
  const int page = n <= p.T && pg < p.max_pages ? __ldg(p.page_table + (long long)b * p.max_pages + pg) : -1;
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) latch_error(p.err, kErrBadPage);
    return;
  }
  const long long dst = (long long)page * kPage + place % kPage;

  float x[2][8];
  rope::unpack8(lat[0], x[0]);
  rope::unpack8(lat[1], x[1]);
  if (p.w) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(x[i][k], x[i][k], ss);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(ss * (1.f / kDl) + p.eps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[8];
      rope::unpack8(__ldg(reinterpret_cast<const uint4*>(p.w) + 32 * i + lane), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i][k] = x[i][k] * r * w[k];
    }
  }
  // rope columns 2l, 2l + 1: one pair, or the same half of the pairs of two frequencies
  float c, s;
  const int pos = p.positions ? __ldg(p.positions + id) : static_cast<int>(place);
  rope::cos_sin(pos, __ldg(p.turns + lane), c, s);
  const float a0 = __uint_as_float(rp << 16), a1 = __uint_as_float(rp & 0xffff0000u);
  float y0, y1;
  if constexpr (kPairs) {
    y0 = a0 * c - a1 * s;
    y1 = a1 * c + a0 * s;
  } else {
    const int f = (2 * lane) & 31;
    const float c0 = __shfl_sync(0xffffffffu, c, f), s0 = __shfl_sync(0xffffffffu, s, f);
    const float c1 = __shfl_sync(0xffffffffu, c, f + 1), s1 = __shfl_sync(0xffffffffu, s, f + 1);
    const float o0 = __shfl_xor_sync(0xffffffffu, a0, 16), o1 = __shfl_xor_sync(0xffffffffu, a1, 16);
    const float sign = lane < 16 ? -1.f : 1.f;
    y0 = a0 * c0 + sign * (o0 * s0);
    y1 = a1 * c1 + sign * (o1 * s1);
  }
  if constexpr (!kFp8) {
    uint16_t* row = static_cast<uint16_t*>(p.cache) + dst * kDc;
    reinterpret_cast<uint4*>(row)[lane] = rope::pack8(x[0]);
    reinterpret_cast<uint4*>(row)[32 + lane] = rope::pack8(x[1]);
    reinterpret_cast<uint32_t*>(row + kDl)[lane] = ptx::pack_bf16x2(y0, y1);
  } else {
    float amax = fmaxf(fabsf(y0), fabsf(y1));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[i][k]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    uint8_t* row = static_cast<uint8_t*>(p.cache) + dst * kDc;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w[k] = e4m3x2(x[i][4 * k], x[i][4 * k + 1], scale) |
               static_cast<uint32_t>(e4m3x2(x[i][4 * k + 2], x[i][4 * k + 3], scale)) << 16;
      reinterpret_cast<uint2*>(row)[32 * i + lane] = make_uint2(w[0], w[1]);
    }
    reinterpret_cast<uint16_t*>(row + kDl)[lane] = e4m3x2(y0, y1, scale);
    if (lane == 0) p.kv_scale[dst] = scale;
  }
}

}  // namespace rope_append

cudaError_t launch_rope_append(const void* c_new, long long row_stride, const void* w, float eps,
                               const int* positions, const void* turns, bool pairs, void* cache, float* kv_scale,
                               const int* page_table, const int* cache_lens, const int* new_lens, int B, int T,
                               int max_pages, int num_pages, bool fp8, unsigned int* err, cudaStream_t stream) {
  using namespace rope_append;
  Params p;
  p.c_new = static_cast<const uint16_t*>(c_new);
  p.row_stride = row_stride;
  p.w = static_cast<const uint16_t*>(w);
  p.eps = eps;
  p.positions = positions;
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
  const int grid = (p.rows + kWarps - 1) / kWarps;
  if (fp8 && pairs)
    rope_append_kernel<true, true><<<grid, kWarps * 32, 0, stream>>>(p);
  else if (fp8)
    rope_append_kernel<true, false><<<grid, kWarps * 32, 0, stream>>>(p);
  else if (pairs)
    rope_append_kernel<false, true><<<grid, kWarps * 32, 0, stream>>>(p);
  else
    rope_append_kernel<false, false><<<grid, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
