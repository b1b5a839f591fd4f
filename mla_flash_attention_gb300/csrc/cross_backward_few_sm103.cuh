// Gradient of cross attention for few queries and keys (at most 64 queries a sequence), part of cross_backward_sm103.cu: 128-row
// tiles would be padding but for these, and a unit of tiles takes 6 us however little there is in it (53 x 56 heads, 29
// queries, up to 9 keys 242 us, so 79; 26 x 15 heads, 3 queries, up to 112 keys 45, so 21; 11 x 48, 18 queries, 165 keys 98, so
// 79).  Bound by latency: a step is a load, three barriers and chains of 20 products, 7 us of two CTAs an SM, so that long
// keys stay with the tiles.
//
// A CTA has one (batch, head) and a run of keys, 64 at a time; Q and dO stay in shared memory.  For each 64 keys
//   S' = K Q', dP' = V dO' in pieces of 16 keys x 16 queries, P' = exp2(.. - LSE) and dS' = P' * (dP' - D) to shared memory
//   as bf16 (as the form by tiles has them: a row has one precision in both); dV = P' dO and dK = dS' Q in pieces of 16 keys
//   x 64 columns, written at once; dQ += dS K in pieces of 16 x 64 that stay in registers of a warp each,
// all by mma.sync on ldmatrix fragments (rows of an odd number of 16 bytes: no bank conflicts), scores formed once.  D
// is made by the CTA itself.  The rope key's gradient and, where a (batch, head) has several CTAs, dQ go to
// the sum kernel in fp32.
#pragma once

namespace mla {
namespace sm103_cross_bwd {

constexpr int kFewRows = 64;  // most queries of this form
constexpr int kFewKeys = 64;  // keys of a step

template <int kRows>
struct FewSmem {
  static constexpr int kStride3 = 400, kStride2 = 272, kStrideP = (kRows + 8) * 2;  // bytes of a row of Q | K, of dO | V, of P'
  static constexpr int kQ = 0, kDo = kQ + kRows * kStride3, kK = kDo + kRows * kStride2, kV = kK + kFewKeys * kStride3,
                       kP = kV + kFewKeys * kStride2, kDs = kP + kFewKeys * kStrideP, kVec = kDs + kFewKeys * kStrideP,
                       kBytes = kVec + 2 * kRows * 4;
};

struct FewInputs {
  const uint16_t *qn, *qr, *kn, *kr, *v, *out, *dout;
  const float* lse;
};

// A lane's part of a row of 64 columns (2 t, 2 t + 1 of each eight) times mul as bf16: neighbouring lanes exchange every
// other eight, so that a store of the warp covers whole sectors.
__device__ __forceinline__ void store_piece(uint16_t* row, const float (&acc)[8][4], int half, float mul, int t, bool live,
                                            const uint16_t* to, size_t bytes, unsigned int* err) {
#pragma unroll
  for (int n = 0; n < 8; n += 2) {
    const uint32_t x = ptx::pack_bf16x2(acc[n][2 * half] * mul, acc[n][2 * half + 1] * mul);
    const uint32_t y = ptx::pack_bf16x2(acc[n + 1][2 * half] * mul, acc[n + 1][2 * half + 1] * mul);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, t & 1 ? x : y, 1);
    uint2* dst = reinterpret_cast<uint2*>(row + 8 * (n + (t & 1)) + 4 * (t >> 1));
    if (live && MLA_STORE_OK(dst, to, bytes, err)) *dst = t & 1 ? make_uint2(other, y) : make_uint2(x, other);
  }
}

template <int kRows>
__global__ void __launch_bounds__(256, 2) few_rows_kernel(const FewInputs in, const Params p) {
  using L = FewSmem<kRows>;
  extern __shared__ __align__(16) unsigned char few_smem[];
  unsigned char* sm = few_smem;
  const uint32_t base = ptx::smem_u32(sm);
  wait_for_stream();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const unsigned bh = blockIdx.x / p.n_ks;
  const int share = blockIdx.x - bh * p.n_ks, b = bh / p.H, h = bh - b * p.H;
  const long long first = (long long)share * p.few_chunk;
  const int len = key_len(p, b), end = static_cast<int>(min(first + p.few_chunk, (long long)len));
  // zeros for the keys of this run behind the last
  for (long long key = max(first, (long long)len) + warp; key < min(first + p.few_chunk, (long long)p.Sk); key += 8) {
    const size_t row = ((size_t)b * p.Sk + key) * p.H + h;
    uint4* to = reinterpret_cast<uint4*>((lane < 16 ? p.dv : p.dk_nope) + row * 128) + (lane & 15);
    if (MLA_STORE_OK(to, lane < 16 ? p.dv : p.dk_nope, p.k_bytes, p.err)) *to = make_uint4(0, 0, 0, 0);
  }
  if (first >= len && p.n_ks > 1) return;

  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto get = [](const uint16_t* x) { return __ldg(reinterpret_cast<const uint4*>(x)); };
  for (int i = tid; i < kRows * 24; i += 256) {
    const int r = i / 24, x = i - 24 * r;
    const size_t row = ((size_t)b * p.Sq + r) * p.H + h;
    *reinterpret_cast<uint4*>(sm + L::kQ + r * L::kStride3 + 16 * x) =
        r >= p.Sq ? zero : x < 16 ? get(in.qn + row * 128 + 8 * x) : get(in.qr + row * 64 + 8 * (x - 16));
  }
  // dO, and D = rowsum(dO * O): 16 lanes a row
  float* nl = reinterpret_cast<float*>(sm + L::kVec);
  float* dd = nl + kRows;
  for (int r = tid >> 4; r < kRows; r += 16) {
    const int x = lane & 15;
    const size_t row = ((size_t)b * p.Sq + r) * p.H + h;
    const uint4 a = r < p.Sq ? get(in.dout + row * 128 + 8 * x) : zero, o = r < p.Sq ? get(in.out + row * 128 + 8 * x) : zero;
    *reinterpret_cast<uint4*>(sm + L::kDo + r * L::kStride2 + 16 * x) = a;
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, ow[4] = {o.x, o.y, o.z, o.w};
    float d = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      d = fmaf(__uint_as_float(aw[j] & 0xffff0000u), __uint_as_float(ow[j] & 0xffff0000u),
               fmaf(__uint_as_float(aw[j] << 16), __uint_as_float(ow[j] << 16), d));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (x == 0) {
      const float of = r < p.Sq ? __ldg(in.lse + (size_t)bh * p.Sq + r) : -INFINITY;
      nl[r] = of == -INFINITY ? -INFINITY : -of * 1.4426950408889634f;
      dd[r] = d;
    }
  }

  // rows of the fragments: of A (16 x 16 at row, column) and of B from rows [n][k]; both from rows [k][m or n] by transposing
  const int ar = lane & 15, ac = (lane >> 4) * 16, br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 16;
  constexpr int kQueryStrips = kRows / 16;
  constexpr bool kSteps = kRows <= 32;  // more rows: no more keys than a step's, dQ a product like the others
  const bool has_dq = kSteps && warp < 3 * kQueryStrips;
  const int dq_strip = warp / 3, dq_block = warp - 3 * dq_strip;
  float dq[8][4] = {};
  auto add_dq = [&](float (&acc)[8][4], int strip, int block, int strips) {  // dS K of one step
    for (int k = 0; k < strips; ++k) {
      uint32_t a[4];
      ptx::ldmatrix_x4<true>(a, base + L::kDs + (16 * k + br) * L::kStrideP + 32 * strip + bc);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t kb[4];
        ptx::ldmatrix_x4<true>(kb, base + L::kK + (16 * k + ar) * L::kStride3 + 128 * block + 32 * n + ac);
        ptx::mma_16x8(acc[2 * n], a[0], a[1], a[2], a[3], kb[0], kb[1]);
        ptx::mma_16x8(acc[2 * n + 1], a[0], a[1], a[2], a[3], kb[2], kb[3]);
      }
    }
  };
  auto store_dq = [&](const float (&acc)[8][4], int strip, int block) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int q = 16 * strip + g + 8 * half;
      if (p.n_ks > 1) {
        if (q >= p.Sq) continue;
        float* row = p.part_q + (((size_t)bh * p.n_ks + share) * p.Sq + q) * 192 + 64 * block + 2 * t;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          float2* dst = reinterpret_cast<float2*>(row + 8 * n);
          if (MLA_STORE_OK(dst, p.part_q, p.part_q_bytes, p.err))
            *dst = make_float2(acc[n][2 * half] * p.scale, acc[n][2 * half + 1] * p.scale);
        }
      } else {
        const size_t at = ((size_t)b * p.Sq + q) * p.H + h;
        uint16_t* to = block < 2 ? p.dq_nope : p.dq_rope;
        store_piece(block < 2 ? to + at * 128 + 64 * block : to + at * 64, acc, half, p.scale, t, q < p.Sq, to,
                    block < 2 ? p.q_bytes : p.q_bytes / 2, p.err);
      }
    }
  };
  for (long long k0l = first; k0l < end; k0l += kFewKeys) {
    const int k0 = static_cast<int>(k0l), strips = (min(kFewKeys, end - k0) + 15) / 16;
    __syncthreads();  // (the keys before are done with)
    const size_t row0 = ((size_t)b * p.Sk + k0) * p.H + h;
#pragma unroll
    for (int i = 0; i < kFewKeys * 40 / 256; ++i) {
      const int at = i * 256 + tid, key = at / 40, x = at - 40 * key;
      if (key >= 16 * strips) break;
      uint4 val = zero;
      if (k0 + key < end) {
        const size_t row = row0 + (size_t)key * p.H;
        val = x < 16 ? get(in.kn + row * 128 + 8 * x)
                     : x < 24 ? get(in.kr + ((size_t)b * p.Sk + k0 + key) * 64 + 8 * (x - 16)) : get(in.v + row * 128 + 8 * (x - 24));
      }
      *reinterpret_cast<uint4*>(sm + (x < 24 ? L::kK + key * L::kStride3 + 16 * x : L::kV + key * L::kStride2 + 16 * (x - 24))) = val;
    }
    __syncthreads();
    for (int task = warp; task < strips * kQueryStrips; task += 8) {
      const int strip = task / kQueryStrips, qs = task - strip * kQueryStrips;
      float s[2][4] = {}, dp[2][4] = {}, s1[2][4] = {}, dp1[2][4] = {};  // (two chains each)
      uint32_t a[4], bq[4];
#pragma unroll
      for (int k = 0; k < 12; ++k) {
        ptx::ldmatrix_x4<false>(a, base + L::kK + (16 * strip + ar) * L::kStride3 + 32 * k + ac);
        ptx::ldmatrix_x4<false>(bq, base + L::kQ + (16 * qs + br) * L::kStride3 + 32 * k + bc);
        ptx::mma_16x8(k & 1 ? s1[0] : s[0], a[0], a[1], a[2], a[3], bq[0], bq[1]);
        ptx::mma_16x8(k & 1 ? s1[1] : s[1], a[0], a[1], a[2], a[3], bq[2], bq[3]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ptx::ldmatrix_x4<false>(a, base + L::kV + (16 * strip + ar) * L::kStride2 + 32 * k + ac);
        ptx::ldmatrix_x4<false>(bq, base + L::kDo + (16 * qs + br) * L::kStride2 + 32 * k + bc);
        ptx::mma_16x8(k & 1 ? dp1[0] : dp[0], a[0], a[1], a[2], a[3], bq[0], bq[1]);
        ptx::mma_16x8(k & 1 ? dp1[1] : dp[1], a[0], a[1], a[2], a[3], bq[2], bq[3]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[j][x] += s1[j][x];
          dp[j][x] += dp1[j][x];
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = 16 * qs + 8 * j + 2 * t;
        const float2 n2 = *reinterpret_cast<const float2*>(nl + q), d2 = *reinterpret_cast<const float2*>(dd + q);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int key = 16 * strip + g + 8 * half;
          const bool live = k0 + key < end;
          const float x = live && q < p.Sq ? ptx::ex2(fmaf(s[j][2 * half], p.scale_log2, n2.x)) : 0.f;
          const float y = live && q + 1 < p.Sq ? ptx::ex2(fmaf(s[j][2 * half + 1], p.scale_log2, n2.y)) : 0.f;
          const float dx = live && q < p.Sq ? x * (dp[j][2 * half] - d2.x) : 0.f;
          const float dy = live && q + 1 < p.Sq ? y * (dp[j][2 * half + 1] - d2.y) : 0.f;
          *reinterpret_cast<uint32_t*>(sm + L::kP + key * L::kStrideP + 2 * q) = ptx::pack_bf16x2(x, y);
          *reinterpret_cast<uint32_t*>(sm + L::kDs + key * L::kStrideP + 2 * q) = ptx::pack_bf16x2(dx, dy);
        }
      }
    }
    __syncthreads();
    if (has_dq) add_dq(dq, dq_strip, dq_block, strips);
    // pieces 0, 1 of a strip: dV; 2, 3: dK nope; 4: dK rope
    for (int task = 7 - warp; task < 5 * strips + (kSteps ? 0 : 3 * kQueryStrips); task += 8) {
      __syncwarp();  // (lanes of no key or query stored nothing of the task before)
      if (!kSteps && task >= 5 * strips) {
        float acc[8][4] = {};
        const int piece = task - 5 * strips;
        add_dq(acc, piece / 3, piece % 3, strips);
        store_dq(acc, piece / 3, piece % 3);
        continue;
      }
      const int strip = task / 5, piece = task - 5 * strip;
      const uint32_t from = base + (piece < 2 ? L::kP : L::kDs);
      const uint32_t with = base + (piece < 2 ? L::kDo + 128 * piece : L::kQ + 128 * (piece - 2));
      const int stride = piece < 2 ? L::kStride2 : L::kStride3;
      float acc[8][4] = {};
#pragma unroll
      for (int k = 0; k < kQueryStrips; ++k) {
        uint32_t a[4];
        ptx::ldmatrix_x4<false>(a, from + (16 * strip + ar) * L::kStrideP + 32 * k + ac);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          uint32_t w[4];
          ptx::ldmatrix_x4<true>(w, with + (16 * k + ar) * stride + 32 * n + ac);
          ptx::mma_16x8(acc[2 * n], a[0], a[1], a[2], a[3], w[0], w[1]);
          ptx::mma_16x8(acc[2 * n + 1], a[0], a[1], a[2], a[3], w[2], w[3]);
        }
      }
      const float mul = piece < 2 ? 1.f : p.scale;
      uint16_t* to = piece < 2 ? p.dv : p.dk_nope;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int key = k0 + 16 * strip + g + 8 * half;
        if (piece == 4) {
          if (key >= end) continue;
          float* row = p.part_rope + ((size_t)bh * p.Sk + key) * 64 + 2 * t;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            float2* dst = reinterpret_cast<float2*>(row + 8 * n);
            if (MLA_STORE_OK(dst, p.part_rope, p.part_rope_bytes, p.err))
              *dst = make_float2(acc[n][2 * half] * mul, acc[n][2 * half + 1] * mul);
          }
        } else {
          store_piece(to + (((size_t)b * p.Sk + key) * p.H + h) * 128 + 64 * (piece & 1), acc, half, mul, t, key < end, to,
                      p.k_bytes, p.err);
        }
      }
    }
  }
  if (has_dq) store_dq(dq, dq_strip, dq_block);
  if (!kSteps && len == 0)  // zeros
    for (int piece = warp; piece < 3 * kQueryStrips; piece += 8) store_dq(dq, piece / 3, piece % 3);
}

}  // namespace sm103_cross_bwd
}  // namespace mla
