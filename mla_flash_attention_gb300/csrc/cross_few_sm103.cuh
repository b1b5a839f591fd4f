// Cross attention of at most eight queries a sequence (a decode step's token, a few drafted ones or beams), and of more in
// small calls, part of cross_sm103.cu: loads straight into registers instead of tiles.
//
// Such a call does 2 to 16 operations a byte of K and V, so their bytes bound it, and a tile of 128 rows would be
// padding but for these rows: nothing is staged.  A CTA has one (batch, head) and a run of `chunk` keys, of which each
// of its eight warps takes 16 at a time with all their loads on their way, keeps its own maxima, sums and O, and
// these are joined at the end.  Two CTAs an SM have 160 KB of loads in flight.  Loads of keys that do not exist are left
// out, so ragged lengths cost nothing beyond them.
//   one query: fp32 products, eight lanes a key (16 columns of nope and 8 of rope each, three shuffles a score),
//     weights in fp32.  64 sequences x 32 heads, up to 1500 keys: 128 us (155 as tiles; the keys' bytes take 120); 64
//     x 128 x 1000 keys 624 us (7.0 TB/s; 679 as tiles); 1 x 8 x 77 3.1 us (6.2).
//   two to eight (a CTA each eight of more): 16 keys x 8 rows mma.sync, whose rate does here (28 of them for 16 keys):
//     scores as K Q', so that the rows fill the narrow side, and O' += V' P', P' being the scores' own registers
//     transposed.  As Q K' with the rows on the wide side, half of it empty and twice the products, they took 158 instead of
//     133 us.  64 x 32 x up to 1500 keys, 8 rows: 137 us (159 as tiles); 8 x 32 x 300 8.7 us.
// Eight heads a CTA, a warp each, with shorter runs, took 134-140 us for the first.
#pragma once

namespace mla {
namespace sm103_cross {

constexpr int kFewRows = 8;  // queries of a block
constexpr int kFewWarps = 8, kFewStep = 16 * kFewWarps;  // keys of a step

__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// the k-th pair of eight bf16 values
__device__ __forceinline__ uint64_t pair_of(const uint4& v, int k) {
  const uint32_t w = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
  return ptx::f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Row r of the result, four columns a lane: the output, or this share's part of it.
__device__ __forceinline__ void finish_row(const Params& p, int b, int h, int bh, int share, int r, int lane, const float4& a,
                                           float lse2) {
  if (p.n_split > 1) {
    const size_t slot = (static_cast<size_t>(bh) * p.n_split + share) * p.Sq + r;
    float4* dst = reinterpret_cast<float4*>(p.part_o + slot * 128) + lane;
    if (MLA_STORE_OK(dst, p.part_o, p.part_o_bytes, p.err)) *dst = a;
    if (lane == 0 && MLA_STORE_OK(p.part_lse + slot, p.part_lse, p.part_lse_bytes, p.err)) p.part_lse[slot] = lse2;
  } else {
    uint2* dst = reinterpret_cast<uint2*>(p.out + ((static_cast<size_t>(b) * p.Sq + r) * p.H + h) * 128) + lane;
    if (MLA_STORE_OK(dst, p.out, p.out_bytes, p.err)) *dst = make_uint2(ptx::pack_bf16x2(a.x, a.y), ptx::pack_bf16x2(a.z, a.w));
    float* lse_at = p.lse + static_cast<size_t>(bh) * p.Sq + r;
    if (lane == 0 && MLA_STORE_OK(lse_at, p.lse, p.lse_bytes, p.err)) *lse_at = lse2 * kLn2;
  }
}

__global__ void __launch_bounds__(kFewWarps * 32, 2)
    one_row_kernel(const uint16_t* __restrict__ q_nope, const uint16_t* __restrict__ q_rope,
                   const uint16_t* __restrict__ k_nope, const uint16_t* __restrict__ k_rope,
                   const uint16_t* __restrict__ v, const Params p) {
  __shared__ float joined[kFewWarps][DV + 4];  // each warp's O, maximum, sum
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 7, group = lane >> 3;
  const int heads = p.B * p.H, share = blockIdx.x / static_cast<unsigned>(heads), bh = blockIdx.x - share * heads;
  const int b = bh / p.H, h = bh - b * p.H;
  const unsigned len = key_len(p, b), first = static_cast<unsigned>(share) * p.chunk, end = min(first + p.chunk, len);
  if (p.n_split > 1 && first >= len) return;  // (the join passes over it)

  uint64_t q[12], o[8];  // columns 8 c.., 64 + 8 c.. of nope, 8 c.. of rope; 8 c.., 64 + 8 c.. of O, of this group's keys
  {
    const uint4 x[3] = {load_once(q_nope + static_cast<size_t>(bh) * 128 + 8 * c),
                        load_once(q_nope + static_cast<size_t>(bh) * 128 + 64 + 8 * c),
                        load_once(q_rope + static_cast<size_t>(bh) * 64 + 8 * c)};
#pragma unroll
    for (int k = 0; k < 12; ++k) q[k] = pair_of(x[k >> 2], k & 3);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = ptx::f2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (unsigned key0 = first + warp * 16; key0 < end; key0 += kFewStep) {
    uint4 kk[4][3], vv[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const unsigned key = key0 + 4 * u + group;
      const bool live = key < end;
      const size_t bk = static_cast<size_t>(b) * p.Sk + key, row = (bk * p.H + h) * 128 + 8 * c;
      kk[u][0] = live ? load_once(k_nope + row) : zero;
      kk[u][1] = live ? load_once(k_nope + row + 64) : zero;
      kk[u][2] = live ? __ldg(reinterpret_cast<const uint4*>(k_rope + bk * 64 + 8 * c)) : zero;
      vv[u][0] = live ? load_once(v + row) : zero;
      vv[u][1] = live ? load_once(v + row + 64) : zero;
    }
    float s[4], top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint64_t sum[2] = {ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f)};
#pragma unroll
      for (int k = 0; k < 12; ++k) sum[k & 1] = ptx::fma2(q[k], pair_of(kk[u][k >> 2], k & 3), sum[k & 1]);
      sum[0] = ptx::add2(sum[0], sum[1]);
      s[u] = ptx::f2_lo(sum[0]) + ptx::f2_hi(sum[0]);
    }
#pragma unroll
    for (int off = 1; off < 8; off *= 2)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], off);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (key0 + 4 * u + group >= end) s[u] = -INFINITY;
      top = fmaxf(top, s[u]);
    }
    top *= p.scale_log2;
    if (__any_sync(0xffffffffu, top > m)) {
      const float to = fmaxf(m, top), keep = ptx::ex2(m - (to == -INFINITY ? 0.f : to));
      m = to;
      l *= keep;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = ptx::mul2(o[k], ptx::f2(keep, keep));
    }
    const float neg_m = m == -INFINITY ? 0.f : -m;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      s[u] = ptx::ex2(fmaf(s[u], p.scale_log2, neg_m));
      l += s[u];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = ptx::fma2(ptx::f2(s[u], s[u]), pair_of(vv[u][k >> 2], k & 3), o[k]);
  }
  // the four groups
#pragma unroll
  for (int off = 8; off < 32; off *= 2) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, off), to = fmaxf(m, m2), ref = to == -INFINITY ? 0.f : to;
    const float keep = ptx::ex2(m - ref), other = ptx::ex2(m2 - ref);
    m = to;
    l = l * keep + __shfl_xor_sync(0xffffffffu, l, off) * other;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint64_t o2 = __shfl_xor_sync(0xffffffffu, o[k], off);
      o[k] = ptx::fma2(o[k], ptx::f2(keep, keep), ptx::mul2(o2, ptx::f2(other, other)));
    }
  }
  if (group == 0) {
    float* to = joined[warp];
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      *reinterpret_cast<float4*>(to + (k >> 2) * 64 + 8 * c + 2 * (k & 3)) =
          make_float4(ptx::f2_lo(o[k]), ptx::f2_hi(o[k]), ptx::f2_lo(o[k + 1]), ptx::f2_hi(o[k + 1]));
    if (c == 0) {
      to[DV] = m;
      to[DV + 1] = l;
    }
  }
  __syncthreads();
  // the eight warps' results, in their order: four columns a lane
  if (warp > 0) return;
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, joined[w][DV]);
  const float ref = top == -INFINITY ? 0.f : top;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    const float e = ptx::ex2(joined[w][DV] - ref);
    const float4 x = reinterpret_cast<const float4*>(joined[w])[lane];
    sum += joined[w][DV + 1] * e;
    a = make_float4(a.x + x.x * e, a.y + x.y * e, a.z + x.z * e, a.w + x.w * e);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum, lse2 = sum == 0.f ? -INFINITY : top + __log2f(sum);
  finish_row(p, b, h, bh, share, 0, lane, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv), lse2);
}

// an 8 x 8 matrix of 16-bit values, two of a row a lane, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

constexpr int kPadQ = 28;  // 16-byte pieces of a query row in shared memory: rows of a quarter-warp's loads on other banks

__global__ void __launch_bounds__(kFewWarps * 32, 2)
    eight_rows_kernel(const uint16_t* __restrict__ q_nope, const uint16_t* __restrict__ q_rope,
                      const uint16_t* __restrict__ k_nope, const uint16_t* __restrict__ k_rope,
                      const uint16_t* __restrict__ v, const Params p) {
  __shared__ uint4 qs[8 * kPadQ];
  __shared__ float joined[kFewWarps][8][DV + 4];  // each warp's O, maximum, sum
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const unsigned item = blockIdx.x / p.row_blocks, heads = p.B * p.H;
  const int row0 = (blockIdx.x - item * p.row_blocks) * kFewRows, share = item / heads, bh = item - share * heads;
  const int b = bh / p.H, h = bh - b * p.H;
  const unsigned len = key_len(p, b), first = static_cast<unsigned>(share) * p.chunk, end = min(first + p.chunk, len);
  if (p.n_split > 1 && first >= len) return;  // (the join passes over it)
  if (threadIdx.x < 8 * 24) {
    const int r = threadIdx.x / 24, x = threadIdx.x - 24 * r;
    uint4 val = make_uint4(0, 0, 0, 0);
    if (row0 + r < p.Sq) {
      const size_t row = (static_cast<size_t>(b) * p.Sq + row0 + r) * p.H + h;
      val = x < 16 ? load_once(q_nope + row * 128 + 8 * x) : load_once(q_rope + row * 64 + 8 * (x - 16));
    }
    qs[r * kPadQ + x] = val;
  }
  __syncthreads();
  float o[8][4] = {};  // O': columns 8 g + i and 64 + 8 g + i, rows 2 t and 2 t + 1 each
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {};  // of rows 2 t, 2 t + 1; the sums of this lane's keys
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (unsigned key0 = first + warp * 16; key0 < end; key0 += kFewStep) {
    uint4 kk[2][6], vv[4][2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const unsigned key = key0 + 8 * n + g;
      const bool live = key < end;
      const size_t bk = static_cast<size_t>(b) * p.Sk + key, row = (bk * p.H + h) * 128 + 8 * t;
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[n][j] = live ? load_once(k_nope + row + 32 * j) : zero;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        kk[n][4 + j] = live ? __ldg(reinterpret_cast<const uint4*>(k_rope + bk * 64 + 8 * t + 32 * j)) : zero;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const unsigned key = key0 + 2 * t + (n & 1) + 8 * (n >> 1);
      const bool live = key < end;
      const size_t row = ((static_cast<size_t>(b) * p.Sk + key) * p.H + h) * 128 + 8 * g;
      vv[n][0] = live ? load_once(v + row) : zero;
      vv[n][1] = live ? load_once(v + row + 64) : zero;
    }
    // S' (16 keys x 8 rows): the 16 bytes of a lane serve two steps of the contraction, whose order is Q's as well
    float s[4] = {}, s1[4] = {};
#pragma unroll
    for (int j = 0; j < 6; ++j) {
      const uint4 q = qs[g * kPadQ + 4 * j + t];
      ptx::mma_16x8(s, kk[0][j].x, kk[1][j].x, kk[0][j].y, kk[1][j].y, q.x, q.y);
      ptx::mma_16x8(s1, kk[0][j].z, kk[1][j].z, kk[0][j].w, kk[1][j].w, q.z, q.w);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[x] += s1[x];
      if (key0 + 8 * (x >> 1) + g >= end) s[x] = -INFINITY;
    }
    float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
    for (int off = 4; off < 32; off *= 2)
#pragma unroll
      for (int r = 0; r < 2; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], off));
    top[0] *= p.scale_log2;
    top[1] *= p.scale_log2;
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float to = fmaxf(m[r], top[r]), keep = ptx::ex2(m[r] - (to == -INFINITY ? 0.f : to));
        m[r] = to;
        l[r] *= keep;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i][r] *= keep;
          o[i][2 + r] *= keep;
        }
      }
    }
    // A weight enters the products as two bf16 terms, its upper half and the rest rounded, which gives it to 2^-15 and not 2^-8
    // (with one term O was off by 0.0023 of itself, RMS, where its own rounding is 0.0017) and takes no time here: 64 x 32 x
    // up to 1500 keys, 2 rows 134.4, so 135.0 us, 8 rows 137.2 either way.  The rest is taken 2^-20 of the weight too large,
    // so that neither term is 0: times an infinite value both are that.
    uint32_t w[2], rest[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float x = ptx::ex2(fmaf(s[2 * n], p.scale_log2, m[0] == -INFINITY ? 0.f : -m[0]));
      const float y = ptx::ex2(fmaf(s[2 * n + 1], p.scale_log2, m[1] == -INFINITY ? 0.f : -m[1]));
      w[n] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
      rest[n] = ptx::pack_bf16x2(fmaf(x, 0x1p-20f, x - __uint_as_float(__float_as_uint(x) & 0xffff0000u)),
                                 fmaf(y, 0x1p-20f, y - __uint_as_float(__float_as_uint(y) & 0xffff0000u)));
      l[0] += x;
      l[1] += y;
      w[n] = transposed(w[n]);  // keys 2 t, 2 t + 1 of row g
      rest[n] = transposed(rest[n]);
    }
    // O' += V' P': column i of a lane's 16 bytes in both halves of the row
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      auto word = [&](const uint4& x) { return (i & 6) == 0 ? x.x : (i & 6) == 2 ? x.y : (i & 6) == 4 ? x.z : x.w; };
      const uint32_t pick = i & 1 ? 0x7632 : 0x5410;
      const uint32_t a[4] = {__byte_perm(word(vv[0][0]), word(vv[1][0]), pick), __byte_perm(word(vv[0][1]), word(vv[1][1]), pick),
                             __byte_perm(word(vv[2][0]), word(vv[3][0]), pick), __byte_perm(word(vv[2][1]), word(vv[3][1]), pick)};
      ptx::mma_16x8(o[i], a[0], a[1], a[2], a[3], w[0], w[1]);
      ptx::mma_16x8(o[i], a[0], a[1], a[2], a[3], rest[0], rest[1]);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int off = 4; off < 32; off *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
    float* to = joined[warp][2 * t + r];
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4*>(to + 64 * half + 8 * g + i) = make_float4(
            o[i][2 * half + r], o[i + 1][2 * half + r], o[i + 2][2 * half + r], o[i + 3][2 * half + r]);
    if (g == 0) {
      to[DV] = m[r];
      to[DV + 1] = l[r];
    }
  }
  __syncthreads();
  // the eight warps' results, in their order: a warp a row, four columns a lane
  if (row0 + warp >= p.Sq) return;
  float ref = -INFINITY, sum = 0.f;
  for (int k = 0; k < kFewWarps; ++k) ref = fmaxf(ref, joined[k][warp][DV]);
  const float top = ref;
  if (ref == -INFINITY) ref = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kFewWarps; ++k) {
    const float* from = joined[k][warp];
    const float e = ptx::ex2(from[DV] - ref);
    const float4 x = reinterpret_cast<const float4*>(from)[lane];
    sum += from[DV + 1] * e;
    a = make_float4(a.x + x.x * e, a.y + x.y * e, a.z + x.z * e, a.w + x.w * e);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum, lse2 = sum == 0.f ? -INFINITY : top + __log2f(sum);
  finish_row(p, b, h, bh, share, row0 + warp, lane, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv), lse2);
}

}  // namespace sm103_cross
}  // namespace mla
