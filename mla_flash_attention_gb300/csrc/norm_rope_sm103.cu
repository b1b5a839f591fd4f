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
// ten operations each.  The work is a list of warp tasks of four kinds, walked in a grid stride:
// four (row, head) pairs of q's nope part, the same of k_nope (16 lanes a pair, 16 bytes a lane),
// the rope parts of eight of q's heads in one row (8 lanes a head), one row's rope key.  One kind
// at a time keeps few values live, so that the SM holds enough warps to cover memory's latency:
// 16384 tokens of 128 heads, q and keys, 424 us (6.3 TB/s, 93 % of the measured copy rate); the
// gradient of 4096 tokens of 64 heads 90 us (5.6 TB/s, 82 %).  With q and k_nope of four heads in
// one task the registers (104 and 152 a thread) left too few warps: 520 and 175 us.  A task's
// loads issued while the one before is worked on cost more in registers than they gave (429 and
// 91 us at 64 and 80 registers).
// A rope task has places for eight heads and the rope key's uses 8 of its 32 lanes, so few heads leave
// lanes idle: 131072 tokens of 1 head 69 us against 30 of bytes, 32768 of 4 heads 36 against 26, 16384 of 8
// heads 32 against 25.
// The sums are shuffles inside the 16 or 8 lanes; each lane makes the cos and sin of one of the 32
// frequencies and the others fetch it by shuffle.  Everything between load and store is fp32,
// rounded once.
// The gradient's weight sums stay in registers while a warp's tasks are of one kind, then go to
// the warp's own row in shared memory; a block writes its warps' sum as one partial row of 384, and
// a second kernel adds the partial rows in a fixed order, so the result does not depend on the run.
#include <algorithm>

#include "common.cuh"
#include "rope.cuh"

namespace mla {
namespace norm_rope {

constexpr int kDn = 128, kDr = rope::kDr, kDq = kDn + kDr;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kPairs4 = 4;                      // (row, head) pairs of a nope task
constexpr int kRopeHeads = 8;                   // heads of a rope task
constexpr int kDw = 2 * (kDn + kDr);            // weight gradients: q nope, q rope, k nope, k rope
constexpr int kOffQr = kDn, kOffKn = kDq, kOffKr = kDq + kDn;

// Blocks a SM holds (their registers' share); the grid is at most that many a SM.
constexpr int kForwardBlocks = 5, kGradBlocks = 4;

struct Params {
  // inputs (any of the three may be absent) and their strides in elements
  const uint16_t *q, *kn, *kr;
  long long q_row, q_head, kn_row, kn_head, kr_row;
  const uint16_t *w_qn, *w_qr, *w_kn, *w_kr;  // null: the part is not normalised
  const int* pos;
  const unsigned long long* turns;
  float eps;
  int H;
  unsigned pairs;        // rows * H
  unsigned n_qn, n_kn;   // nope tasks of q and of k_nope
  unsigned n_qr, n_kr;   // rope tasks: rope_groups a row for q, one for the rope key
  unsigned rope_groups;  // ceil(H / 8)
  int q_linear, kn_linear;  // row stride == H * head stride: pair i is i head strides in
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

// Element offset of pair i (row * H + head) in an operand with these strides.
__device__ __forceinline__ long long pair_offset(unsigned i, int H, long long row_stride, long long head_stride,
                                                 int linear) {
  if (linear) return i * head_stride;
  const unsigned row = i / H;
  return row * row_stride + (i - row * H) * head_stride;
}

// The nope tasks u, u + step, ... < n of one operand; returns the first u past them.
template <bool kGrad>
__device__ __forceinline__ unsigned nope_tasks(const Params& p, unsigned u, unsigned n, unsigned step,
                                               const uint16_t* x, long long row_stride, long long head_stride,
                                               int linear, const uint16_t* w, const uint16_t* dy, uint16_t* out,
                                               size_t out_bytes, float* dw_row) {
  if (u >= n) return u;
  const int lane = threadIdx.x & 31, c16 = lane & 15;
  const uint4 w16 = weights8(w, c16), zero = make_uint4(0, 0, 0, 0);
  float dw[8] = {};
  for (; u < n; u += step) {
    unsigned pair[2];
    long long off[2];
    uint4 in[2], up[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      pair[i] = u * kPairs4 + 2 * i + (lane >> 4);
      off[i] = pair_offset(pair[i], p.H, row_stride, head_stride, linear) + 8 * c16;
      in[i] = pair[i] < p.pairs ? load16(x + off[i]) : zero;
      if (kGrad) up[i] = pair[i] < p.pairs ? load16(dy + (size_t)pair[i] * kDn + 8 * c16) : zero;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v[8], g[8];
      rope::unpack8(in[i], v);
      uint4* dst;
      if constexpr (kGrad) {
        rope::unpack8(up[i], g);
        norm8_grad<16>(g, v, w16, w, p.eps, pair[i] < p.pairs, dw);
        dst = reinterpret_cast<uint4*>(out + off[i]);
      } else {
        norm8<16>(v, w16, w, p.eps);
        dst = reinterpret_cast<uint4*>(out + (size_t)pair[i] * kDn + 8 * c16);
      }
      if (pair[i] < p.pairs && MLA_STORE_OK(dst, out, out_bytes, p.err)) *dst = rope::pack8(kGrad ? g : v);
    }
  }
  if (kGrad && dw_row) {  // the two lanes that hold the same columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], 16);
      if (lane < 16) dw_row[8 * lane + i] = dw[i];
    }
  }
  return u;
}

// The rope tasks u, u + step, ... < n: of q (eight heads of a row, groups tasks a row) or of the
// rope key (kKey: one "head" a row, and its upstream gradient in fp32).
template <bool kGrad, bool kPairs, bool kKey>
__device__ __forceinline__ unsigned rope_tasks(const Params& p, unsigned u, unsigned n, unsigned step,
                                               const uint16_t* x, long long row_stride, long long head_stride,
                                               int heads, unsigned groups, const uint16_t* w, const void* dy,
                                               uint16_t* out, size_t out_bytes, float* dw_row) {
  if (u >= n) return u;
  const int lane = threadIdx.x & 31, c8 = lane & 7;
  const uint4 w8 = weights8(w, c8), zero = make_uint4(0, 0, 0, 0);
  const unsigned long long turns = __ldg(p.turns + lane);
  constexpr int kLoads = kKey ? 1 : 2;
  float dw[8] = {};
  for (; u < n; u += step) {
    const unsigned row32 = kKey || groups == 1 ? u : u / groups;
    const int h0 = kKey ? 0 : (u - row32 * groups) * kRopeHeads + (lane >> 3);
    const long long row = row32;
    const bool mine = !kKey || lane < 8;
    uint4 in[kLoads], up[kLoads];
    float4 uk[2] = {};
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int h = h0 + 4 * i;
      const bool live = mine && h < heads;
      in[i] = live ? load16(x + row * row_stride + h * head_stride + 8 * c8) : zero;
      if constexpr (kGrad && kKey) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(dy) + row * kDr + 8 * c8);
        if (live) {
          uk[0] = __ldg(src);
          uk[1] = __ldg(src + 1);
        }
      } else if constexpr (kGrad) {
        up[i] = live ? load16(static_cast<const uint16_t*>(dy) + (row * heads + h) * kDr + 8 * c8) : zero;
      }
    }
    float c, s;
    rope::cos_sin(__ldg(p.pos + row), turns, c, s);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int h = h0 + 4 * i;
      const bool live = mine && h < heads;
      if (!__any_sync(0xffffffffu, live)) break;
      float v[8], d[8];
      rope::unpack8(in[i], v);
      uint4* dst;
      if constexpr (kGrad) {
        if constexpr (kKey) {
          d[0] = uk[0].x; d[1] = uk[0].y; d[2] = uk[0].z; d[3] = uk[0].w;
          d[4] = uk[1].x; d[5] = uk[1].y; d[6] = uk[1].z; d[7] = uk[1].w;
        } else {
          rope::unpack8(up[i], d);
        }
        rope::rotate8<kPairs, true>(d, c, s, lane);
        norm8_grad<8>(d, v, w8, w, p.eps, live, dw);
        dst = reinterpret_cast<uint4*>(out + row * row_stride + h * head_stride + 8 * c8);
      } else {
        norm8<8>(v, w8, w, p.eps);
        rope::rotate8<kPairs, false>(v, c, s, lane);
        dst = reinterpret_cast<uint4*>(out + (row * heads + h) * kDr + 8 * c8);
      }
      if (live && MLA_STORE_OK(dst, out, out_bytes, p.err)) *dst = rope::pack8(kGrad ? d : v);
    }
  }
  if (kGrad && dw_row) {  // the four lanes that hold the same columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], 16);
      dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], 8);
      if (lane < 8) dw_row[8 * lane + i] = dw[i];
    }
  }
  return u;
}

// The four kinds of tasks of warp `u` of `step`.
template <bool kGrad, bool kPairs>
__device__ __forceinline__ void all_tasks(const Params& p, unsigned u, unsigned step, float* dw_row) {
  auto at = [&](int off) { return dw_row ? dw_row + off : nullptr; };
  u = nope_tasks<kGrad>(p, u, p.n_qn, step, p.q, p.q_row, p.q_head, p.q_linear, p.w_qn, p.dqn, p.qn_out, p.qn_bytes,
                        at(0)) - p.n_qn;
  u = nope_tasks<kGrad>(p, u, p.n_kn, step, p.kn, p.kn_row, p.kn_head, p.kn_linear, p.w_kn, p.dkn, p.kn_out,
                        p.kn_bytes, at(kOffKn)) - p.n_kn;
  // (the gradient of q's rope part lies behind its nope part, as in q)
  u = rope_tasks<kGrad, kPairs, false>(p, u, p.n_qr, step, p.q + kDn, p.q_row, p.q_head, p.H, p.rope_groups, p.w_qr,
                                       p.dqr, kGrad ? p.qn_out + kDn : p.qr_out,
                                       kGrad ? p.qn_bytes - 2 * kDn : p.qr_bytes, at(kOffQr)) - p.n_qr;
  rope_tasks<kGrad, kPairs, true>(p, u, p.n_kr, step, p.kr, p.kr_row, 0, 1, 1, p.w_kr, p.dkr, p.kr_out, p.kr_bytes,
                                  at(kOffKr));
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads, kForwardBlocks) norm_rope_kernel(const Params p) {
  const unsigned step = gridDim.x * kWarps;
  wait_for_stream();
  all_tasks<false, kPairs>(p, blockIdx.x * kWarps + (threadIdx.x >> 5), step, nullptr);
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads, kGradBlocks) norm_rope_grad_kernel(const Params p) {
  __shared__ float joined[kWarps][kDw];
  wait_for_stream();
  const int warp = threadIdx.x >> 5;
  const unsigned step = gridDim.x * kWarps;
  float* mine = nullptr;
  if (p.partial) {  // a warp need not meet every kind of task
    mine = joined[warp];
    for (int i = threadIdx.x & 31; i < kDw; i += 32) mine[i] = 0.f;
    __syncwarp();
  }
  all_tasks<true, kPairs>(p, blockIdx.x * kWarps + warp, step, mine);
  if (!p.partial) return;
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
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* partial, int rows,
                                                           float* dw_qn, float* dw_qr, float* dw_kn, float* dw_kr) {
  __shared__ float joined[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  wait_for_stream();  // the partial rows are written
#pragma unroll 4
  for (int r = warp; r < rows; r += 32) v += ptx::ld_l2(partial + (size_t)r * kDw + col);
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

inline unsigned nope_count(long long rows, int H) { return static_cast<unsigned>((rows * H + kPairs4 - 1) / kPairs4); }
inline unsigned rope_count(long long rows, int H) { return static_cast<unsigned>(rows * ((H + kRopeHeads - 1) / kRopeHeads)); }

inline long long task_count(const Params& p) { return (long long)p.n_qn + p.n_kn + p.n_qr + p.n_kr; }

inline int blocks_for(long long tasks, int per_sm, int sms) {
  return static_cast<int>(std::min<long long>((tasks + kWarps - 1) / kWarps, (long long)per_sm * sms));
}

}  // namespace norm_rope

// Partial rows of the largest launch for these sizes (all operands given).
size_t norm_rope_grad_workspace_bytes(long long rows, int H, int sms) {
  using namespace norm_rope;
  const long long tasks = 2LL * nope_count(rows, H) + rope_count(rows, H) + rows;
  return (size_t)blocks_for(tasks, kGradBlocks, sms) * kDw * sizeof(float);
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
  p.pairs = static_cast<unsigned>(rows * H);  // the caller keeps rows * H at most 0x70000000
  p.n_qn = q ? norm_rope::nope_count(rows, H) : 0;
  p.n_kn = kn ? norm_rope::nope_count(rows, H) : 0;
  p.n_qr = q ? norm_rope::rope_count(rows, H) : 0;
  p.n_kr = kr ? static_cast<unsigned>(rows) : 0;
  p.rope_groups = (H + norm_rope::kRopeHeads - 1) / norm_rope::kRopeHeads;
  p.q_linear = q_row == H * q_head;
  p.kn_linear = kn_row == H * kn_head;
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
  const int grid = blocks_for(task_count(p), kForwardBlocks, sms);
  return launch_dependent(pairs ? norm_rope_kernel<true> : norm_rope_kernel<false>, grid, kThreads, stream, p);
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
  const int grid = blocks_for(task_count(p), kGradBlocks, sms);
  const bool weights = dw_qn || dw_qr || dw_kn || dw_kr;
  p.partial = weights ? workspace : nullptr;
  p.partial_bytes = (size_t)grid * kDw * sizeof(float);
  const cudaError_t e = launch_dependent(pairs ? norm_rope_grad_kernel<true> : norm_rope_grad_kernel<false>, grid,
                                         kThreads, stream, p);
  if (e != cudaSuccess || !weights) return e;
  return launch_dependent(weight_grad_kernel, kDw / 32, 1024, stream, static_cast<const float*>(workspace), grid, dw_qn,
                          dw_qr, dw_kn, dw_kr);
}

}  // namespace mla
