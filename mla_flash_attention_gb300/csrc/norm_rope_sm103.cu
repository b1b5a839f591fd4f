// Norms of queries and keys for each head with the position rotation in the same pass, the
// step between the projections and mla_prefill / mla_absorb, and its gradient.
//
//   n(x) = w x / sqrt(mean(x^2) + eps) over the 128 nope (64 rope) columns of one head, x where
//   w is absent; y_nope = n(x_nope), y_rope = R(pos) n(x_rope).
//   Gradient: g = dy (nope), R(pos)' dy (rope); with r = 1 / sqrt(mean(x^2) + eps)
//     dx = r (w g - x r^2 mean(x w g)),   dw = sum over rows and heads of g x r
//   (dx = g where w is absent).
//
// One pass over memory bounds it: 2 bytes in and out an element (forward), 6 (gradient), about
// ten operations each.  A warp takes four heads of one row at a time, every load 16 bytes a
// lane: two loads of 128-wide parts (16 lanes a head) for q and two for k_nope, one of the four
// rope parts (8 lanes a head), all issued before the first is used; the sums are shuffles inside
// the 16 or 8 lanes.  Each lane makes the cos and sin of one of the 32 frequencies and the
// others fetch it by shuffle.  Everything between load and store is fp32, rounded once.
// The gradient's weight sums stay in registers over a warp's whole share of the rows, are joined
// per block in shared memory and written as one partial row of 384 a block; a second kernel adds
// the partial rows in a fixed order, so the result does not depend on the run.
#include <algorithm>

#include "common.cuh"
#include "rope.cuh"

namespace mla {
namespace norm_rope {

constexpr int kDn = 128, kDr = rope::kDr, kDq = kDn + kDr;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kHeads = 4;                       // heads of a row a warp takes at a time
constexpr int kDw = 2 * (kDn + kDr);            // weight gradients: q nope, q rope, k nope, k rope
constexpr int kOffQr = kDn, kOffKn = kDq, kOffKr = kDq + kDn;

struct Params {
  // inputs (any of the three may be absent) and their strides in elements
  const uint16_t *q, *kn, *kr;
  long long q_row, q_head, kn_row, kn_head, kr_row;
  const uint16_t *w_qn, *w_qr, *w_kn, *w_kr;  // null: the part is not normalised
  const int* pos;
  const unsigned long long* turns;
  float eps;
  int H;
  int groups;  // ceil(H / 4)
  int tasks;   // R * groups
  // forward: contiguous outputs; gradient: dx with the operands' strides
  uint16_t *qn_out, *qr_out, *kn_out, *kr_out;
  // gradient: contiguous upstream gradients
  const uint16_t *dqn, *dqr, *dkn;
  const float* dkr;
  float* partial;  // [blocks][384]
  unsigned int* err;
  size_t qn_bytes, qr_bytes, kn_bytes, kr_bytes, partial_bytes;  // for the store checks
};

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}

// sum over the kLanes lanes (8 or 16, aligned) that share a head
template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ uint4 weights8(const uint16_t* w, int chunk) {
  return w ? *reinterpret_cast<const uint4*>(w + 8 * chunk) : make_uint4(0, 0, 0, 0);
}

// x <- n(x) for a part of kLanes * 8 columns
template <int kLanes>
__device__ __forceinline__ void norm8(float (&x)[8], const uint4& wp, bool has_w, float eps) {
  if (!has_w) return;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = group_sum<kLanes>(ss);
  const float r = rsqrtf(ss * (1.f / (8 * kLanes)) + eps);
  float w[8];
  rope::unpack8(wp, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
}

// g <- dx for the upstream gradient g of n(x); dw += g x r where `live`
template <int kLanes>
__device__ __forceinline__ void norm8_grad(float (&g)[8], const float (&x)[8], const uint4& wp, bool has_w,
                                           float eps, bool live, float (&dw)[8]) {
  if (!has_w) return;
  float w[8];
  rope::unpack8(wp, w);
  float ss = 0.f, dot = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ss = fmaf(x[i], x[i], ss);
    dot = fmaf(x[i] * w[i], g[i], dot);
  }
  ss = group_sum<kLanes>(ss);
  dot = group_sum<kLanes>(dot);
  const float r = rsqrtf(ss * (1.f / (8 * kLanes)) + eps);
  const float t = dot * (1.f / (8 * kLanes)) * r * r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (live) dw[i] = fmaf(g[i], x[i] * r, dw[i]);
    g[i] = r * fmaf(-x[i], t, w[i] * g[i]);
  }
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const int c16 = lane & 15, c8 = lane & 7;
  const uint4 w_qn = weights8(p.w_qn, c16), w_qr = weights8(p.w_qr, c8);
  const uint4 w_kn = weights8(p.w_kn, c16), w_kr = weights8(p.w_kr, c8);
  const unsigned long long turns = __ldg(p.turns + lane);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (long long task = blockIdx.x * kWarps + (threadIdx.x >> 5); task < p.tasks; task += gridDim.x * kWarps) {
    const unsigned row32 = static_cast<unsigned>(task) / static_cast<unsigned>(p.groups);
    const int g = static_cast<int>(static_cast<unsigned>(task) - row32 * p.groups), h0 = g * kHeads;
    const long long row = row32;
    const int hn[2] = {h0 + (lane >> 4), h0 + 2 + (lane >> 4)};  // heads of the two nope loads
    const int hr = h0 + (lane >> 3);                             // head of the rope load
    const bool rope_key = p.kr && g == 0;
    uint4 qn[2], kn[2], qr = zero, kr = zero;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      qn[i] = p.q && hn[i] < p.H ? load16(p.q + row * p.q_row + hn[i] * p.q_head + 8 * c16) : zero;
      kn[i] = p.kn && hn[i] < p.H ? load16(p.kn + row * p.kn_row + hn[i] * p.kn_head + 8 * c16) : zero;
    }
    if (p.q && hr < p.H) qr = load16(p.q + row * p.q_row + hr * p.q_head + kDn + 8 * c8);
    if (rope_key && lane < 8) kr = load16(p.kr + row * p.kr_row + 8 * c8);
    float c, s;
    rope::cos_sin(__ldg(p.pos + row), turns, c, s);
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (p.q) {
        rope::unpack8(qn[i], x);
        norm8<16>(x, w_qn, p.w_qn, p.eps);
        uint4* dst = reinterpret_cast<uint4*>(p.qn_out + (row * p.H + hn[i]) * kDn + 8 * c16);
        if (hn[i] < p.H && MLA_STORE_OK(dst, p.qn_out, p.qn_bytes, p.err)) *dst = rope::pack8(x);
      }
      if (p.kn) {
        rope::unpack8(kn[i], x);
        norm8<16>(x, w_kn, p.w_kn, p.eps);
        uint4* dst = reinterpret_cast<uint4*>(p.kn_out + (row * p.H + hn[i]) * kDn + 8 * c16);
        if (hn[i] < p.H && MLA_STORE_OK(dst, p.kn_out, p.kn_bytes, p.err)) *dst = rope::pack8(x);
      }
    }
    if (p.q) {
      rope::unpack8(qr, x);
      norm8<8>(x, w_qr, p.w_qr, p.eps);
      rope::rotate8<kPairs, false>(x, c, s, lane);
      uint4* dst = reinterpret_cast<uint4*>(p.qr_out + (row * p.H + hr) * kDr + 8 * c8);
      if (hr < p.H && MLA_STORE_OK(dst, p.qr_out, p.qr_bytes, p.err)) *dst = rope::pack8(x);
    }
    if (rope_key) {
      rope::unpack8(kr, x);
      norm8<8>(x, w_kr, p.w_kr, p.eps);
      rope::rotate8<kPairs, false>(x, c, s, lane);
      uint4* dst = reinterpret_cast<uint4*>(p.kr_out + row * kDr + 8 * c8);
      if (lane < 8 && MLA_STORE_OK(dst, p.kr_out, p.kr_bytes, p.err)) *dst = rope::pack8(x);
    }
  }
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads) norm_rope_grad_kernel(const Params p) {
  __shared__ float joined[kWarps][kDw];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c16 = lane & 15, c8 = lane & 7;
  const uint4 w_qn = weights8(p.w_qn, c16), w_qr = weights8(p.w_qr, c8);
  const uint4 w_kn = weights8(p.w_kn, c16), w_kr = weights8(p.w_kr, c8);
  const unsigned long long turns = __ldg(p.turns + lane);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float dw_qn[8] = {}, dw_qr[8] = {}, dw_kn[8] = {}, dw_kr[8] = {};
  for (long long task = blockIdx.x * kWarps + warp; task < p.tasks; task += gridDim.x * kWarps) {
    const unsigned row32 = static_cast<unsigned>(task) / static_cast<unsigned>(p.groups);
    const int g = static_cast<int>(static_cast<unsigned>(task) - row32 * p.groups), h0 = g * kHeads;
    const long long row = row32;
    const int hn[2] = {h0 + (lane >> 4), h0 + 2 + (lane >> 4)};
    const int hr = h0 + (lane >> 3);
    const bool rope_key = p.kr && g == 0;
    uint4 qn[2], kn[2], dqn[2], dkn[2], qr = zero, dqr = zero;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool q_in = p.q && hn[i] < p.H, k_in = p.kn && hn[i] < p.H;
      qn[i] = q_in ? load16(p.q + row * p.q_row + hn[i] * p.q_head + 8 * c16) : zero;
      dqn[i] = q_in ? load16(p.dqn + (row * p.H + hn[i]) * kDn + 8 * c16) : zero;
      kn[i] = k_in ? load16(p.kn + row * p.kn_row + hn[i] * p.kn_head + 8 * c16) : zero;
      dkn[i] = k_in ? load16(p.dkn + (row * p.H + hn[i]) * kDn + 8 * c16) : zero;
    }
    if (p.q && hr < p.H) {
      qr = load16(p.q + row * p.q_row + hr * p.q_head + kDn + 8 * c8);
      dqr = load16(p.dqr + (row * p.H + hr) * kDr + 8 * c8);
    }
    float c, s;
    rope::cos_sin(__ldg(p.pos + row), turns, c, s);
    float x[8], d[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool live = hn[i] < p.H;
      if (p.q) {
        rope::unpack8(qn[i], x);
        rope::unpack8(dqn[i], d);
        norm8_grad<16>(d, x, w_qn, p.w_qn, p.eps, live, dw_qn);
        uint4* dst = reinterpret_cast<uint4*>(p.qn_out + row * p.q_row + hn[i] * p.q_head + 8 * c16);
        if (live && MLA_STORE_OK(dst, p.qn_out, p.qn_bytes, p.err)) *dst = rope::pack8(d);
      }
      if (p.kn) {
        rope::unpack8(kn[i], x);
        rope::unpack8(dkn[i], d);
        norm8_grad<16>(d, x, w_kn, p.w_kn, p.eps, live, dw_kn);
        uint4* dst = reinterpret_cast<uint4*>(p.kn_out + row * p.kn_row + hn[i] * p.kn_head + 8 * c16);
        if (live && MLA_STORE_OK(dst, p.kn_out, p.kn_bytes, p.err)) *dst = rope::pack8(d);
      }
    }
    if (p.q) {
      rope::unpack8(qr, x);
      rope::unpack8(dqr, d);
      rope::rotate8<kPairs, true>(d, c, s, lane);
      norm8_grad<8>(d, x, w_qr, p.w_qr, p.eps, hr < p.H, dw_qr);
      uint4* dst = reinterpret_cast<uint4*>(p.qn_out + row * p.q_row + hr * p.q_head + kDn + 8 * c8);
      if (hr < p.H && MLA_STORE_OK(dst, p.qn_out, p.qn_bytes, p.err)) *dst = rope::pack8(d);
    }
    if (rope_key) {
      uint4 kr = zero;
      float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
      if (lane < 8) {
        kr = load16(p.kr + row * p.kr_row + 8 * c8);
        const float4* src = reinterpret_cast<const float4*>(p.dkr + row * kDr + 8 * c8);
        lo = __ldg(src);
        hi = __ldg(src + 1);
      }
      rope::unpack8(kr, x);
      d[0] = lo.x; d[1] = lo.y; d[2] = lo.z; d[3] = lo.w;
      d[4] = hi.x; d[5] = hi.y; d[6] = hi.z; d[7] = hi.w;
      rope::rotate8<kPairs, true>(d, c, s, lane);
      norm8_grad<8>(d, x, w_kr, p.w_kr, p.eps, lane < 8, dw_kr);
      uint4* dst = reinterpret_cast<uint4*>(p.kr_out + row * p.kr_row + 8 * c8);
      if (lane < 8 && MLA_STORE_OK(dst, p.kr_out, p.kr_bytes, p.err)) *dst = rope::pack8(d);
    }
  }
  if (!p.partial) return;
  // the lanes of a warp that hold the same columns, then the block's warps in order
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    dw_qn[i] += __shfl_xor_sync(0xffffffffu, dw_qn[i], 16);
    dw_kn[i] += __shfl_xor_sync(0xffffffffu, dw_kn[i], 16);
    dw_qr[i] += __shfl_xor_sync(0xffffffffu, dw_qr[i], 16);
    dw_qr[i] += __shfl_xor_sync(0xffffffffu, dw_qr[i], 8);
  }
  float* mine = joined[warp];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (lane < 16) {
      mine[8 * lane + i] = dw_qn[i];
      mine[kOffKn + 8 * lane + i] = dw_kn[i];
    }
    if (lane < 8) {
      mine[kOffQr + 8 * lane + i] = dw_qr[i];
      mine[kOffKr + 8 * lane + i] = dw_kr[i];
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < kDw; col += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += joined[w][col];
    float* dst = p.partial + (size_t)blockIdx.x * kDw + col;
    if (MLA_STORE_OK(dst, p.partial, p.partial_bytes, p.err)) *dst = v;
  }
}

// dw[col] = sum of the blocks' partial rows.  A block takes 32 columns, its 32 warps every 32nd
// row each, joined in warp order.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* __restrict__ partial, int rows,
                                                           float* dw_qn, float* dw_qr, float* dw_kn, float* dw_kr) {
  __shared__ float joined[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 4
  for (int r = warp; r < rows; r += 32) v += __ldg(partial + (size_t)r * kDw + col);
  joined[warp][lane] = v;
  __syncthreads();
  if (warp > 0) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) v += joined[w][lane];
  if (col < kOffQr) {
    if (dw_qn) dw_qn[col] = v;
  } else if (col < kOffKn) {
    if (dw_qr) dw_qr[col - kOffQr] = v;
  } else if (col < kOffKr) {
    if (dw_kn) dw_kn[col - kOffKn] = v;
  } else if (dw_kr) {
    dw_kr[col - kOffKr] = v;
  }
}

// Blocks of a persistent launch: at most four (forward) or three (gradient) a SM, what their
// registers leave room for.
constexpr int kForwardBlocks = 4, kGradBlocks = 3;

inline int blocks_for(long long tasks, int per_sm, int sms) {
  return static_cast<int>(std::min<long long>((tasks + kWarps - 1) / kWarps, (long long)per_sm * sms));
}

}  // namespace norm_rope

size_t norm_rope_grad_workspace_bytes(long long rows, int H, int sms) {
  using namespace norm_rope;
  return (size_t)blocks_for(rows * ((H + kHeads - 1) / kHeads), kGradBlocks, sms) * kDw * sizeof(float);
}

namespace {

norm_rope::Params shared_params(const void* q, long long q_row, long long q_head, const void* kn,
                                long long kn_row, long long kn_head, const void* kr, long long kr_row,
                                const void* w_qn, const void* w_qr, const void* w_kn, const void* w_kr,
                                const int* pos, const void* turns, float eps, long long rows, int H,
                                unsigned int* err) {
  norm_rope::Params p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.kn = static_cast<const uint16_t*>(kn);
  p.kr = static_cast<const uint16_t*>(kr);
  p.q_row = q_row;
  p.q_head = q_head;
  p.kn_row = kn_row;
  p.kn_head = kn_head;
  p.kr_row = kr_row;
  p.w_qn = static_cast<const uint16_t*>(w_qn);
  p.w_qr = static_cast<const uint16_t*>(w_qr);
  p.w_kn = static_cast<const uint16_t*>(w_kn);
  p.w_kr = static_cast<const uint16_t*>(w_kr);
  p.pos = pos;
  p.turns = static_cast<const unsigned long long*>(turns);
  p.eps = eps;
  p.H = H;
  p.groups = (H + norm_rope::kHeads - 1) / norm_rope::kHeads;
  p.tasks = static_cast<int>(rows * p.groups);  // the caller keeps rows * groups below 2^31
  p.err = err;
  return p;
}

}  // namespace

cudaError_t launch_norm_rope_sm103(const void* q, long long q_row, long long q_head, const void* kn,
                                   long long kn_row, long long kn_head, const void* kr, long long kr_row,
                                   const void* w_qn, const void* w_qr, const void* w_kn, const void* w_kr,
                                   const int* pos, const void* turns, float eps, bool pairs, long long rows,
                                   int H, void* qn_out, void* qr_out, void* kn_out, void* kr_out, int sms,
                                   unsigned int* err, cudaStream_t stream) {
  using namespace norm_rope;
  Params p = shared_params(q, q_row, q_head, kn, kn_row, kn_head, kr, kr_row, w_qn, w_qr, w_kn, w_kr, pos, turns,
                           eps, rows, H, err);
  p.qn_out = static_cast<uint16_t*>(qn_out);
  p.qr_out = static_cast<uint16_t*>(qr_out);
  p.kn_out = static_cast<uint16_t*>(kn_out);
  p.kr_out = static_cast<uint16_t*>(kr_out);
  p.qn_bytes = (size_t)rows * H * kDn * 2;
  p.qn_bytes -= std::min(p.qn_bytes, testing_out_shrink());
  p.qr_bytes = (size_t)rows * H * kDr * 2;
  p.kn_bytes = (size_t)rows * H * kDn * 2;
  p.kr_bytes = (size_t)rows * kDr * 2;
  const int grid = blocks_for(p.tasks, kForwardBlocks, sms);
  if (pairs)
    norm_rope_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else
    norm_rope_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_grad_sm103(const void* dqn, const void* dqr, const void* dkn, const float* dkr,
                                        const void* q, long long q_row, long long q_head, const void* kn,
                                        long long kn_row, long long kn_head, const void* kr, long long kr_row,
                                        const void* w_qn, const void* w_qr, const void* w_kn, const void* w_kr,
                                        const int* pos, const void* turns, float eps, bool pairs, long long rows,
                                        int H, void* dq, void* dk_nope, void* dk_rope, float* dw_qn, float* dw_qr,
                                        float* dw_kn, float* dw_kr, float* workspace, int sms, unsigned int* err,
                                        cudaStream_t stream) {
  using namespace norm_rope;
  Params p = shared_params(q, q_row, q_head, kn, kn_row, kn_head, kr, kr_row, w_qn, w_qr, w_kn, w_kr, pos, turns,
                           eps, rows, H, err);
  p.dqn = static_cast<const uint16_t*>(dqn);
  p.dqr = static_cast<const uint16_t*>(dqr);
  p.dkn = static_cast<const uint16_t*>(dkn);
  p.dkr = dkr;
  p.qn_out = static_cast<uint16_t*>(dq);
  p.kn_out = static_cast<uint16_t*>(dk_nope);
  p.kr_out = static_cast<uint16_t*>(dk_rope);
  p.qn_bytes = ((rows - 1) * q_row + (H - 1) * q_head + kDq) * 2;
  p.qn_bytes -= std::min(p.qn_bytes, testing_out_shrink());
  p.kn_bytes = ((rows - 1) * kn_row + (H - 1) * kn_head + kDn) * 2;
  p.kr_bytes = ((rows - 1) * kr_row + kDr) * 2;
  const int grid = blocks_for(p.tasks, kGradBlocks, sms);
  const bool weights = dw_qn || dw_qr || dw_kn || dw_kr;
  p.partial = weights ? workspace : nullptr;
  p.partial_bytes = (size_t)grid * kDw * sizeof(float);
  if (pairs)
    norm_rope_grad_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else
    norm_rope_grad_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !weights) return e;
  weight_grad_kernel<<<kDw / 32, 1024, 0, stream>>>(workspace, grid, dw_qn, dw_qr, dw_kn, dw_kr);
  return cudaGetLastError();
}

}  // namespace mla
