// Cross attention of at most four queries a sequence (a decode step's token, a few drafted ones), part of
// cross_sm103.cu: plain loads and fp32 products instead of tiles.
//
// Such a call does 2 to 8 operations a byte of K and V, so it is bound by their bytes, and a tile of 128 rows would be
// padding but for these: no tensor cores, no staging.  Eight lanes take a key (16 columns of nope and 8 of rope each; a
// score is their sum by three shuffles), the four groups of a warp neighbouring keys, kKeys of them at a time with
// all their loads on their way; each group keeps its own maximum, sum and 16 columns of O a lane, joined at the end.
// A warp has one (batch, head) and a run of `chunk` keys; eight warps of a CTA have eight heads (whose keys lie side by
// side, 2 KB a token), or in calls too small for that each an eighth of one head's run.  Weights stay in fp32.
#pragma once

namespace mla {
namespace sm103_cross {

constexpr int kFewRows = 4;    // most queries a sequence of this form
constexpr int kFewWarps = 8;

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

template <int kRows, int kKeys>
__global__ void __launch_bounds__(kFewWarps * 32, kRows == 1 ? 2 : 1)
    few_rows_kernel(const uint16_t* __restrict__ q_nope, const uint16_t* __restrict__ q_rope,
                    const uint16_t* __restrict__ k_nope, const uint16_t* __restrict__ k_rope,
                    const uint16_t* __restrict__ v, const Params p) {
  __shared__ float joined[kFewWarps][kRows][DV + 2];  // each warp's O, maximum, sum
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 7, group = lane >> 3;
  const int heads = p.B * p.H, share = blockIdx.x / static_cast<unsigned>(heads), bh = blockIdx.x - share * heads;
  const int b = bh / p.H, h = bh - b * p.H;
  const unsigned len = key_len(p, b), first = static_cast<unsigned>(share) * p.chunk, end = min(first + p.chunk, len);
  if (p.n_split > 1 && first >= len) return;  // (the join passes over it)

  uint64_t q[kRows][12], o[kRows][8];  // columns 8c.., 64 + 8c.. of nope, 8c.. of rope; 8c.., 64 + 8c.. of O
  float m[kRows], l[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const size_t row = (static_cast<size_t>(b) * p.Sq + min(r, p.Sq - 1)) * p.H + h;
    const uint4 x[3] = {load_once(q_nope + row * 128 + 8 * c), load_once(q_nope + row * 128 + 64 + 8 * c),
                        load_once(q_rope + row * 64 + 8 * c)};
#pragma unroll
    for (int k = 0; k < 12; ++k) q[r][k] = pair_of(x[k >> 2], k & 3);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[r][k] = ptx::f2(0.f, 0.f);
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  constexpr int kStep = 4 * kKeys * kFewWarps;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (unsigned key0 = first + warp * 4 * kKeys; key0 < end; key0 += kStep) {
    uint4 kk[kKeys][3], vv[kKeys][2];
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const unsigned key = key0 + 4 * u + group;
      const bool live = key < end;
      const size_t bk = static_cast<size_t>(b) * p.Sk + key, row = (bk * p.H + h) * 128 + 8 * c;
      kk[u][0] = live ? load_once(k_nope + row) : zero;
      kk[u][1] = live ? load_once(k_nope + row + 64) : zero;
      kk[u][2] = live ? __ldg(reinterpret_cast<const uint4*>(k_rope + bk * 64 + 8 * c)) : zero;
      vv[u][0] = live ? load_once(v + row) : zero;
      vv[u][1] = live ? load_once(v + row + 64) : zero;
    }
    float s[kRows][kKeys];
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      uint64_t sum[kRows][2];
#pragma unroll
      for (int r = 0; r < kRows; ++r) sum[r][0] = sum[r][1] = ptx::f2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 12; ++k) {
        const uint64_t x = pair_of(kk[u][k >> 2], k & 3);
#pragma unroll
        for (int r = 0; r < kRows; ++r) sum[r][k & 1] = ptx::fma2(q[r][k], x, sum[r][k & 1]);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint64_t both = ptx::add2(sum[r][0], sum[r][1]);
        s[r][u] = ptx::f2_lo(both) + ptx::f2_hi(both);
      }
    }
#pragma unroll
    for (int off = 1; off < 8; off *= 2)
#pragma unroll
      for (int u = 0; u < kKeys; ++u)
#pragma unroll
        for (int r = 0; r < kRows; ++r) s[r][u] += __shfl_xor_sync(0xffffffffu, s[r][u], off);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        if (key0 + 4 * u + group >= end) s[r][u] = -INFINITY;
        top = fmaxf(top, s[r][u]);
      }
      top *= p.scale_log2;
      if (__any_sync(0xffffffffu, top > m[r])) {
        const float to = fmaxf(m[r], top), keep = ptx::ex2(m[r] - (to == -INFINITY ? 0.f : to));
        const uint64_t keep2 = ptx::f2(keep, keep);
        m[r] = to;
        l[r] *= keep;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[r][k] = ptx::mul2(o[r][k], keep2);
      }
      const float neg_m = m[r] == -INFINITY ? 0.f : -m[r];
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        s[r][u] = ptx::ex2(fmaf(s[r][u], p.scale_log2, neg_m));
        l[r] += s[r][u];
      }
    }
#pragma unroll
    for (int u = 0; u < kKeys; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t x = pair_of(vv[u][k >> 2], k & 3);
#pragma unroll
        for (int r = 0; r < kRows; ++r) o[r][k] = ptx::fma2(ptx::f2(s[r][u], s[r][u]), x, o[r][k]);
      }
  }
  // the four groups
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int off = 8; off < 32; off *= 2) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[r], off), to = fmaxf(m[r], m2), ref = to == -INFINITY ? 0.f : to;
      const float keep = ptx::ex2(m[r] - ref), other = ptx::ex2(m2 - ref);
      const uint64_t keep2 = ptx::f2(keep, keep), other2 = ptx::f2(other, other);
      m[r] = to;
      l[r] = l[r] * keep + __shfl_xor_sync(0xffffffffu, l[r], off) * other;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t o2 = __shfl_xor_sync(0xffffffffu, o[r][k], off);
        o[r][k] = ptx::fma2(o[r][k], keep2, ptx::mul2(o2, other2));
      }
    }
  // the eight warps' results, in their order: a warp a row, four columns a lane
  if (group == 0) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float* to = joined[warp][r];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<float2*>(to + (k >> 2) * 64 + 8 * c + 2 * (k & 3)) = make_float2(ptx::f2_lo(o[r][k]), ptx::f2_hi(o[r][k]));
      if (c == 0) {
        to[DV] = m[r];
        to[DV + 1] = l[r];
      }
    }
  }
  __syncthreads();
  if (warp >= p.Sq || warp >= kRows) return;
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, joined[w][warp][DV]);
  const float ref = top == -INFINITY ? 0.f : top;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    const float* from = joined[w][warp];
    const float e = ptx::ex2(from[DV] - ref);
    const float2 x = reinterpret_cast<const float2*>(from)[2 * lane], y = reinterpret_cast<const float2*>(from)[2 * lane + 1];
    sum += from[DV + 1] * e;
    a = make_float4(a.x + x.x * e, a.y + x.y * e, a.z + y.x * e, a.w + y.y * e);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum, lse2 = sum == 0.f ? -INFINITY : top + __log2f(sum);
  a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  if (p.n_split > 1) {
    const size_t slot = (static_cast<size_t>(bh) * p.n_split + share) * p.Sq + warp;
    float4* dst = reinterpret_cast<float4*>(p.part_o + slot * 128) + lane;
    if (MLA_STORE_OK(dst, p.part_o, p.part_o_bytes, p.err)) *dst = a;
    if (lane == 0 && MLA_STORE_OK(p.part_lse + slot, p.part_lse, p.part_lse_bytes, p.err)) p.part_lse[slot] = lse2;
  } else {
    uint2* dst = reinterpret_cast<uint2*>(p.out + ((static_cast<size_t>(b) * p.Sq + warp) * p.H + h) * 128) + lane;
    if (MLA_STORE_OK(dst, p.out, p.out_bytes, p.err)) *dst = make_uint2(ptx::pack_bf16x2(a.x, a.y), ptx::pack_bf16x2(a.z, a.w));
    float* lse_at = p.lse + static_cast<size_t>(bh) * p.Sq + warp;
    if (lane == 0 && MLA_STORE_OK(lse_at, p.lse, p.lse_bytes, p.err)) *lse_at = lse2 * kLn2;
  }
}

}  // namespace sm103_cross
}  // namespace mla
