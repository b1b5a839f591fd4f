// Cross attention to an encoder's states: queries of one length, keys and values of another, each
// sequence with its own number of keys (tcgen05 + TMEM + TMA, bf16).
//
//   s_ij = scale (qn_i . kn_j + qr_i . kr_j),  lse_i = log sum_{j < n_b} exp(s_ij),
//   o_i = sum_{j < n_b} exp(s_ij - lse_i) v_j
//
// in one pass over the keys with the running maximum and sum, as mla_prefill does; the tile (two
// 128-row score buffers, 128 keys) and the roles of the warps are that kernel's.  What differs:
//   - A CTA is persistent and walks work units of (batch, head, row block, share of the keys): the next
//     unit's keys are on their way, and its first scores are formed, while this one's last rows are
//     stored.  With encoder lengths of ten tiles a CTA a unit spent a fifth of its time on its two ends.
//   - Up to eight rows (decode steps), and small calls, take no tiles: cross_few_sm103.cuh.
//   - Row blocks of up to 128 rows (short prompts) give both score buffers the same rows and every other key
//     tile each (`by_keys`): each softmax warpgroup keeps its own maximum, sum and output accumulator and the
//     two are joined at the end.  Such blocks are bound by the keys' bytes: four ring slots instead of three
//     then take the shared memory that the second query tile would.
//   - Few units (few rows, long keys) are split along the keys; a second kernel joins the shares by their
//     log-sum-exp.
//   - Keys behind a sequence's last are masked, and the value rows there zeroed in shared memory before
//     the product (0 * NaN is NaN): what stands in a padded batch does not matter.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace sm103_cross {

constexpr int BM = 128, BN = 128, DV = 128;
constexpr int kChunk = 128 * 128;   // one 128-row x 128-byte swizzled chunk
constexpr int kQTile = 3 * kChunk;  // nope (2 chunks) + rope (1 chunk)
constexpr int kSlot = 2 * kChunk;   // a K_nope or V tile
constexpr int kThreads = 384;
// registers per thread after the run-time hand-off, as in the prefill: 128 producer/MMA threads drop to
// kRegsLow, 256 softmax threads rise to kRegsHigh; the launch must provide their average
constexpr int kRegsLow = 56, kRegsHigh = 224;
constexpr int kRegsAtLaunch = ((128 * kRegsLow + 256 * kRegsHigh + kThreads - 1) / kThreads + 7) / 8 * 8;
static_assert(kRegsAtLaunch * kThreads <= 65536, "register hand-off exceeds the SM's file");
constexpr float kLn2 = 0.69314718055994531f;

// Shared memory: one query tile and four K/V slots, or two and three; 224 KB either way.
template <bool kOneTile>
struct Smem {
  static constexpr int kQTiles = kOneTile ? 1 : 2, kRing = kOneTile ? 4 : 3, kRope = kOneTile ? 3 : 2;
  static constexpr int kOffRing = kQTiles * kQTile, kOffRope = kOffRing + kRing * kSlot;
  static constexpr int kBytes = kOffRope + kRope * kChunk, kAlloc = kBytes + 1024;
};

struct Params {
  int B, H, Sq, Sk;
  int nrb;        // row blocks of a (batch, head)
  int n_split;    // shares of the keys of a row block
  int units;      // B * H * nrb * n_split
  int chunk, row_blocks;  // few rows: keys of a share; blocks of eight rows
  unsigned shift;  // 1: see Walk
  int slot_rows;  // rows of a partial result
  float scale_log2;
  const int* key_lens;  // or null: Sk everywhere
  uint16_t* out;
  float* lse;
  float *part_o, *part_lse;  // [B * H * nrb * n_split][slot_rows](128): O / l, and log2 of the sum of exponentials
  unsigned int* err;
  size_t out_bytes, lse_bytes, part_o_bytes, part_lse_bytes;  // for the store checks
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t ring_full[4], ring_empty[4], rope_full[3], rope_empty[3];
  uint64_t s_full[2], p_full[2][2], o_done[2];  // p_full[t][h]: keys 64h..64h+63 of P_t
  uint64_t o_free;                              // the unit's accumulators were read
  uint64_t stat_full, drained;
  uint32_t tmem_base;
  int abort_flag;
  float m[BM], l[BM], lr[BM];  // by_keys: the second warpgroup's maximum and sums of each row
};
static_assert(Smem<true>::kAlloc + sizeof(Bars) <= 232448 && Smem<false>::kAlloc + sizeof(Bars) <= 232448,
              "shared memory of a CTA");

__device__ __forceinline__ int key_len(const Params& p, int b) {
  return p.key_lens ? min(max(__ldg(p.key_lens + b), 0), p.Sk) : p.Sk;
}
// first key tile of share s
__device__ __forceinline__ int share_begin(int tiles, int s, int n_split) {
  return static_cast<int>(static_cast<long long>(tiles) * s / n_split);
}

// share s of a sequence of len keys holds none
__device__ __forceinline__ bool share_empty(const Params& p, int len, int s) {
  if (p.chunk > 0) return static_cast<long long>(s) * p.chunk >= len;
  const int tiles = (len + BN - 1) / BN;
  return share_begin(tiles, s, p.n_split) == share_begin(tiles, s + 1, p.n_split);
}

struct Unit {
  int b, h, row0, len, tile0, nt;
  bool by_keys;
  // key tiles that score buffer t works on
  __device__ __forceinline__ int steps(int t) const { return by_keys ? (nt + 1 - t) >> 1 : nt; }
};

template <bool kOneTile>
__device__ __forceinline__ Unit unit_of(const Params& p, unsigned id) {
  Unit u;
  const unsigned item = id / p.n_split;
  const int share = id - item * p.n_split;
  const unsigned bh = item / p.nrb;
  u.row0 = kOneTile ? 0 : (item - bh * p.nrb) * 2 * BM;
  u.b = bh / p.H;
  u.h = bh - u.b * p.H;
  u.len = key_len(p, u.b);
  const int tiles = (u.len + BN - 1) / BN;
  u.tile0 = share_begin(tiles, share, p.n_split);
  u.nt = share_begin(tiles, share + 1, p.n_split) - u.tile0;
  u.by_keys = kOneTile || p.Sq - u.row0 <= BM;
  return u;
}

// The units of a CTA: one of every gridDim.x; where the last row block of a (batch, head) is by_keys and the others are
// not, a place further on each time, so that no CTA has the last ones alone and another none (8 x 152 heads, 300
// queries, 640 keys: 290 us, so 248).
struct Walk {
  unsigned id = blockIdx.x, place = blockIdx.x;
  __device__ __forceinline__ void next(const Params& p) {
    const unsigned to = place + p.shift == gridDim.x ? 0 : place + p.shift;
    id += gridDim.x + to - place;
    place = to;
  }
};

template <bool kOneTile>
__global__ void __launch_bounds__(kThreads, 1)
    cross_kernel(const __grid_constant__ CUtensorMap tm_qn, const __grid_constant__ CUtensorMap tm_qr,
                 const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_kr,
                 const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using L = Smem<kOneTile>;
  constexpr uint32_t kRing = L::kRing, kRope = L::kRope;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ Bars bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tm_qn);
    ptx::prefetch_tensormap(&tm_qr);
    ptx::prefetch_tensormap(&tm_kn);
    ptx::prefetch_tensormap(&tm_kr);
    ptx::prefetch_tensormap(&tm_v);
    bars.abort_flag = 0;
    ptx::mbar_init(&bars.q_full, 1);
    ptx::mbar_init(&bars.q_empty, 1);
    for (uint32_t i = 0; i < kRing; ++i) {
      ptx::mbar_init(&bars.ring_full[i], 1);
      ptx::mbar_init(&bars.ring_empty[i], 1);
    }
    for (uint32_t i = 0; i < kRope; ++i) {
      ptx::mbar_init(&bars.rope_full[i], 1);
      ptx::mbar_init(&bars.rope_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&bars.s_full[t], 1);
      ptx::mbar_init(&bars.p_full[t][0], BM / 32);  // one arrival per softmax warp
      ptx::mbar_init(&bars.p_full[t][1], BM / 32);
      ptx::mbar_init(&bars.o_done[t], 1);
    }
    ptx::mbar_init(&bars.stat_full, BM / 32);
    ptx::mbar_init(&bars.o_free, 8);
    ptx::mbar_init(&bars.drained, 1);
    ptx::fence_barrier_init();
  }
  if (warp == 2) ptx::tmem_alloc(&bars.tmem_base, 512);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort_flag;
  wait_for_stream();

  if (warp < 4) {
    ptx::regs_dec<kRegsLow>();
    if (warp == 0 && ptx::elect_one()) {
      // ------------------------------------------------------------ producer
      // K/V tiles go through one ring in the order in which the MMA warp takes them: the scores run
      // `ahead` tiles (one, or two by_keys) before the products with V
      uint32_t n_ring = 0, n_rope = 0, n_q = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, const Unit& u, int key0) {
        const uint32_t s = n_ring % kRing;
        if (!ptx::mbar_wait(&bars.ring_empty[s], ((n_ring / kRing) & 1) ^ 1, abort_flag, p.err)) return ok = false;
        unsigned char* dst = sm + L::kOffRing + s * kSlot;
        ptx::mbar_arrive_expect_tx(&bars.ring_full[s], kSlot);
        ptx::tma_load_4d(dst, map, &bars.ring_full[s], 0, u.h, key0, u.b);
        ptx::tma_load_4d(dst + kChunk, map, &bars.ring_full[s], 64, u.h, key0, u.b);
        ++n_ring;
        return true;
      };
      auto load_k = [&](const Unit& u, int i) {
        const int key0 = (u.tile0 + i) * BN;
        if (!load(&tm_kn, u, key0)) return false;
        const uint32_t s = n_rope % kRope;
        if (!ptx::mbar_wait(&bars.rope_empty[s], ((n_rope / kRope) & 1) ^ 1, abort_flag, p.err)) return ok = false;
        ptx::mbar_arrive_expect_tx(&bars.rope_full[s], kChunk);
        ptx::tma_load_3d(sm + L::kOffRope + s * kChunk, &tm_kr, &bars.rope_full[s], 0, key0, u.b);
        ++n_rope;
        return true;
      };
      for (Walk w; ok && w.id < static_cast<unsigned>(p.units); w.next(p)) {
        const Unit u = unit_of<kOneTile>(p, w.id);
        if (u.nt == 0) continue;
        const int ahead = u.by_keys ? 2 : 1;
        for (int i = 0; i < min(ahead, u.nt); ++i)
          if (!load_k(u, i)) break;
        // the query tiles are free once the last scores of the unit before are done
        if (!ok || !(ok = ptx::mbar_wait(&bars.q_empty, (n_q & 1) ^ 1, abort_flag, p.err))) break;
        const int q_tiles = u.by_keys ? 1 : 2;
        ptx::mbar_arrive_expect_tx(&bars.q_full, q_tiles * kQTile);
        for (int t = 0; t < q_tiles; ++t) {
          unsigned char* q = sm + t * kQTile;
          const int row = u.row0 + t * BM;
          ptx::tma_load_4d(q, &tm_qn, &bars.q_full, 0, u.h, row, u.b);
          ptx::tma_load_4d(q + kChunk, &tm_qn, &bars.q_full, 64, u.h, row, u.b);
          ptx::tma_load_4d(q + 2 * kChunk, &tm_qr, &bars.q_full, 0, u.h, row, u.b);
        }
        ++n_q;
        for (int n = 0; n < u.nt; ++n) {
          if (!load(&tm_v, u, (u.tile0 + n) * BN)) break;
          if (n + ahead < u.nt && !load_k(u, n + ahead)) break;
          // warm L2 with the tile whose ring slots free only as this one's products end
          if (n + ahead + 1 < u.nt) {
            const int key = (u.tile0 + n + ahead + 1) * BN;
            ptx::tma_prefetch_4d(&tm_kn, 0, u.h, key, u.b);
            ptx::tma_prefetch_4d(&tm_kn, 64, u.h, key, u.b);
            ptx::tma_prefetch_3d(&tm_kr, 0, key, u.b);
            ptx::tma_prefetch_4d(&tm_v, 0, u.h, key, u.b);
            ptx::tma_prefetch_4d(&tm_v, 64, u.h, key, u.b);
          }
        }
      }
      // after an abort: copies that nobody waited for land before the CTA leaves
      for (uint32_t v = n_ring > kRing ? n_ring - kRing : 0; v < n_ring; ++v)
        ptx::mbar_wait_drain(&bars.ring_full[v % kRing], (v / kRing) & 1);
      for (uint32_t v = n_rope > kRope ? n_rope - kRope : 0; v < n_rope; ++v)
        ptx::mbar_wait_drain(&bars.rope_full[v % kRope], (v / kRope) & 1);
      if (n_q > 0) ptx::mbar_wait_drain(&bars.q_full, (n_q - 1) & 1);
    } else if (warp == 1 && ptx::elect_one()) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdS = ptx::make_idesc(1, BM, BN, 0, 0);    // Q K', both K-major
      constexpr uint32_t kIdPV = ptx::make_idesc(1, BM, 128, 0, 1);  // P V, V is N-major
      const uint64_t d_q = ptx::sw128_desc(ptx::smem_u32(sm), 16, 1024);
      const uint64_t d_ring = ptx::sw128_desc(ptx::smem_u32(sm + L::kOffRing), 16, 1024);
      const uint64_t d_rope = ptx::sw128_desc(ptx::smem_u32(sm + L::kOffRope), 16, 1024);
      const uint64_t d_v = ptx::sw128_desc(ptx::smem_u32(sm + L::kOffRing), kChunk, 1024);
      // operand descriptors built once; a tile at a byte offset from its base differs only in the
      // start-address field (an opaque add, so that each is formed where it is used)
      auto at = [](uint64_t d, uint32_t bytes) {
        uint64_t r;
        asm volatile("add.u64 %0, %1, %2;" : "=l"(r) : "l"(d), "l"(static_cast<uint64_t>(bytes >> 4)));
        return r;
      };
      uint32_t n_ring = 0, n_rope = 0, n_q = 0, n_step[2] = {0, 0};
      bool ok = true;
      auto take = [&]() -> bool {  // the next ring tile
        const bool w = ptx::mbar_wait(&bars.ring_full[n_ring % kRing], (n_ring / kRing) & 1, abort_flag, p.err);
        return ok = ok && w;
      };
      auto give = [&]() {
        ptx::mma_commit(&bars.ring_empty[n_ring % kRing]);
        ++n_ring;
      };
      auto take_k = [&]() -> bool {
        return take() &&
               (ok = ptx::mbar_wait(&bars.rope_full[n_rope % kRope], (n_rope / kRope) & 1, abort_flag, p.err));
      };
      auto give_k = [&]() {
        give();
        ptx::mma_commit(&bars.rope_empty[n_rope % kRope]);
        ++n_rope;
      };
      // S_t = Q K' of the taken key tile: 8 k-steps over the nope chunks + 4 over the rope chunk
      auto scores = [&](int t, int q_tile) {
        const uint64_t qa = at(d_q, q_tile * kQTile);
        const uint64_t kb = at(d_ring, (n_ring % kRing) * kSlot);
        const uint64_t rb = at(d_rope, (n_rope % kRope) * kChunk);
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          const int c = k >> 2, kk = k & 3;
          ptx::mma_bf16_ss(tmem + t * BN, at(qa, c * kChunk + kk * 32),
                           c < 2 ? at(kb, c * kChunk + kk * 32) : at(rb, kk * 32), kIdS, k > 0);
        }
        ptx::mma_commit(&bars.s_full[t]);
      };
      // O_t (+)= P_t V of the taken value tile, in two halves of 64 keys, each issued as soon as
      // that half of P_t (bf16, over S_t) is in TMEM
      auto product = [&](int t, bool first) -> bool {
        if (first && !(ok = ptx::mbar_wait(&bars.o_free, (n_q & 1) ^ 1, abort_flag, p.err))) return false;
        const uint64_t vb = at(d_v, (n_ring % kRing) * kSlot);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!(ok = ptx::mbar_wait(&bars.p_full[t][hf], n_step[t] & 1, abort_flag, p.err))) return false;
          ptx::tc_fence_after();
#pragma unroll
          for (int k = 4 * hf; k < 4 * hf + 4; ++k)
            ptx::mma_bf16_ts(tmem + 2 * BN + t * 128, tmem + t * BN + k * 8, at(vb, k * 2048), kIdPV,
                             (!first || k > 0) ? 1u : 0u);
        }
        ptx::mma_commit(&bars.o_done[t]);
        ++n_step[t];
        return true;
      };
      for (Walk w; ok && w.id < static_cast<unsigned>(p.units); w.next(p)) {
        const Unit u = unit_of<kOneTile>(p, w.id);
        if (u.nt == 0) continue;
        if (!take_k() || !(ok = ptx::mbar_wait(&bars.q_full, n_q & 1, abort_flag, p.err))) break;
        scores(0, 0);
        if (u.by_keys) {
          give_k();
          if (u.nt > 1) {
            if (!take_k()) break;
            scores(1, 0);
            give_k();
          }
          if (u.nt <= 2) ptx::mma_commit(&bars.q_empty);
          for (int n = 0; n < u.nt; ++n) {
            const int t = n & 1;
            if (!take() || !product(t, n < 2)) break;
            give();
            if (n + 2 < u.nt) {
              if (!take_k()) break;
              scores(t, 0);
              give_k();
              if (n + 3 == u.nt) ptx::mma_commit(&bars.q_empty);
            }
          }
        } else {
          scores(1, 1);
          give_k();
          if (u.nt == 1) ptx::mma_commit(&bars.q_empty);
          for (int n = 0; n < u.nt; ++n) {
            if (!take() || !product(0, n == 0)) break;
            const bool more = n + 1 < u.nt;
            const uint32_t v_slot = n_ring;
            if (more) {  // the next scores of tile 0 ahead of this product of tile 1
              ++n_ring;
              if (!take_k()) break;
              scores(0, 0);
              n_ring = v_slot;
            }
            if (!product(1, n == 0)) break;
            give();
            if (more) {
              scores(1, 1);
              give_k();
              if (n + 2 == u.nt) ptx::mma_commit(&bars.q_empty);
            }
          }
        }
        ++n_q;
      }
      // every MMA issued completes, and every commit arrives, before the CTA gives its memory back
      ptx::mma_commit(&bars.drained);
      ptx::mbar_wait_drain(&bars.drained, 0);
    }
  } else {
    // -------------------------------------------------------------- softmax warpgroups
    ptx::regs_inc<kRegsHigh>();
    const int t = (warp >> 2) - 1;         // score buffer of this warpgroup
    const int r = (warp & 3) * 32 + lane;  // row within the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + t * BN;
    const uint32_t o_addr = tmem + lane_off + 2 * BN;  // O_0; O_1 128 columns on
    uint32_t n_ring = 0, n_stat = 0, n_step[2] = {0, 0};  // steps of both buffers
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      const bool w = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort_flag, p.err));
      if (w) ptx::tc_fence_after();
      return w;
    };
    for (Walk w; ok && w.id < static_cast<unsigned>(p.units); w.next(p)) {
      const Unit u = unit_of<kOneTile>(p, w.id);
      const int row0 = u.by_keys ? u.row0 : u.row0 + t * BM;
      const int i = row0 + r;                              // query
      const bool row_live = i < p.Sq;
      const bool warp_live = row0 + (warp & 3) * 32 < p.Sq;  // a warp of padding rows leaves its scores alone
      uint16_t* out_row = p.out + ((static_cast<size_t>(u.b) * p.Sq + i) * p.H + u.h) * 128;
      float* lse_at = p.lse + (static_cast<size_t>(u.b) * p.H + u.h) * p.Sq + i;
      if (u.nt == 0) {
        // no key: zeros here, or left to the kernel that joins the shares
        if (p.n_split == 1 && row_live && !(u.by_keys && t == 1)) {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            uint4* dst = reinterpret_cast<uint4*>(out_row) + x;
            if (MLA_STORE_OK(dst, p.out, p.out_bytes, p.err)) *dst = make_uint4(0, 0, 0, 0);
          }
          if (MLA_STORE_OK(lse_at, p.lse, p.lse_bytes, p.err)) *lse_at = -INFINITY;
        }
        continue;
      }
      float m = -INFINITY, l = 0.f, lr = 0.f;  // exact row sum (LSE), bf16-rounded sum (O)
      const int steps = u.steps(t);
      for (int j = 0; j < steps; ++j) {
        const uint32_t step = n_step[t] + j;
        if (!(ok = wait(&bars.s_full[t], step & 1))) break;
        const int tile = u.by_keys ? 2 * j + t : j;
        const int lim = u.len - (u.tile0 + tile) * BN;  // keys of this tile below lim exist
        // the value rows behind them are zeroed before P is announced, by whose product takes the tile first
        // (those past Sk are zeros as loaded)
        const bool clean = lim < BN && u.len < p.Sk && (u.by_keys || t == 0);
        if (warp_live) {
          float s[128];
          uint32_t* su = reinterpret_cast<uint32_t*>(s);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            ptx::tmem_ld32(s_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(su + c * 32));
          ptx::tmem_ld_wait();
          if (lim < BN) {
#pragma unroll
            for (int x = 0; x < 128; ++x)
              if (x >= lim) s[x] = -INFINITY;
          }
          // row max: four independent chains of three-input maxima
          float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int x = 4; x < 128; x += 2) mx4[(x >> 1) & 3] = ptx::fmax3(mx4[(x >> 1) & 3], s[x], s[x + 1]);
          const float m_tile = ptx::fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) * p.scale_log2;
          float m_use = m;
          if (j == 0) {
            m_use = m_tile;
          } else {
            const bool grow = m_tile > m + 8.0f;
            if (__any_sync(0xffffffffu, grow)) {
              // O of the product before must be complete before it is rescaled
              if (!(ok = wait(&bars.o_done[t], (step - 1) & 1))) break;
              const float alpha = grow ? ptx::ex2(m - m_tile) : 1.f;
              if (grow) m_use = m_tile;
              uint32_t v[2][32];
#pragma unroll
              for (int c = 0; c < 4; c += 2) {
                const uint32_t o_t = o_addr + t * 128 + c * 32;
                ptx::tmem_ld32(o_t, v[0]);
                ptx::tmem_ld32(o_t + 32, v[1]);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                  v[0][x] = __float_as_uint(__uint_as_float(v[0][x]) * alpha);
                  v[1][x] = __float_as_uint(__uint_as_float(v[1][x]) * alpha);
                }
                ptx::tmem_st32(o_t, v[0]);
                ptx::tmem_st32(o_t + 32, v[1]);
              }
              l *= alpha;
              lr *= alpha;
            }
          }
          m = m_use;
          const float neg_m = m == -INFINITY ? 0.f : -m;
          // as in the prefill: the weights enter the product with V as one bf16 term (a second one, as the forms without
          // tiles have it, would double that product, 1024 of the 2560 clocks of MMAs that bound a step of long prompts),
          // O is normalised by the sum of the rounded weights that the product uses, the LSE is that of the exact ones
          const uint64_t sc2 = ptx::f2(p.scale_log2, p.scale_log2), nm2 = ptx::f2(neg_m, neg_m);
          uint64_t ps2[2] = {ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f)};
          float pr[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const uint64_t a2 = ptx::fma2(ptx::f2(s[c * 64 + 2 * x], s[c * 64 + 2 * x + 1]), sc2, nm2);
              const float p0 = ptx::ex2(ptx::f2_lo(a2));
              const float p1 = ptx::ex2(ptx::f2_hi(a2));
              const uint32_t w = ptx::pack_bf16x2(p0, p1);
              pk[x] = w;
              ps2[x & 1] = ptx::add2(ps2[x & 1], ptx::f2(p0, p1));
              ptx::add_bf16x2(pr[2 * (x & 1)], pr[2 * (x & 1) + 1], w);
            }
            ptx::tmem_st32(s_addr + c * 32, pk);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (!clean && lane == 0) ptx::mbar_arrive(&bars.p_full[t][c]);
          }
          const uint64_t ps_all = ptx::add2(ps2[0], ps2[1]);
          l += ptx::f2_lo(ps_all) + ptx::f2_hi(ps_all);
          lr += (pr[0] + pr[1]) + (pr[2] + pr[3]);
        }
        if (clean) {
          const uint32_t seq = n_ring + 2 * u.nt - 1;  // the unit's last ring tile is its last value tile
          if (!(ok = wait(&bars.ring_full[seq % kRing], (seq / kRing) & 1))) break;
          if (r >= lim) {
            uint4* row = reinterpret_cast<uint4*>(sm + L::kOffRing + (seq % kRing) * kSlot + r * 128);
#pragma unroll
            for (int x = 0; x < 8; ++x) row[x] = row[x + kChunk / 16] = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async();
        }
        if (clean || !warp_live) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&bars.p_full[t][0]);
            ptx::mbar_arrive(&bars.p_full[t][1]);
          }
        }
      }
      if (!ok) break;
      n_ring += 2 * u.nt;
      n_step[0] += u.steps(0);
      n_step[1] += u.steps(1);
      // ------------------------------------------------------------ the unit's rows
      // w0 O_0 + w1 O_1, or w0 O_t of this warpgroup's own rows
      float w0, w1 = 0.f, row_m = m, row_l = l;
      const bool both = u.by_keys && u.nt > 1;
      if (!(u.by_keys && u.steps(t) == 0) && !(ok = wait(&bars.o_done[t], (n_step[t] - 1) & 1))) break;
      if (both && t == 1) {
        // (its last product waited for o_free, so the first warpgroup has read the rows of the unit before)
        bars.m[r] = m;
        bars.l[r] = l;
        bars.lr[r] = lr;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.stat_full);
      }
      if (both && t == 0) {
        if (!(ok = wait(&bars.o_done[1], (n_step[1] - 1) & 1) && wait(&bars.stat_full, n_stat & 1))) break;
        ++n_stat;
        row_m = fmaxf(m, bars.m[r]);
        const float ref = row_m == -INFINITY ? 0.f : row_m;
        const float e0 = ptx::ex2(m - ref), e1 = ptx::ex2(bars.m[r] - ref);
        row_l = l * e0 + bars.l[r] * e1;
        const float sum = lr * e0 + bars.lr[r] * e1, inv = sum == 0.f ? 0.f : 1.f / sum;
        w0 = e0 * inv;
        w1 = e1 * inv;
      } else {
        w0 = lr == 0.f ? 0.f : 1.f / lr;
      }
      const float lse2 = row_l == 0.f ? -INFINITY : row_m + __log2f(row_l);
      const size_t slot = static_cast<size_t>(w.id) * p.slot_rows + (i - u.row0);  // row of a partial result
      if (warp_live && !(u.by_keys && t == 1)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          ptx::tmem_ld32(o_addr + (u.by_keys ? 0 : t * 128) + c * 32, v);
          if (both) {
            uint32_t v1[32];
            ptx::tmem_ld32(o_addr + 128 + c * 32, v1);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x)
              v[x] = __float_as_uint(__uint_as_float(v[x]) * w0 + __uint_as_float(v1[x]) * w1);
          } else {
            ptx::tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * w0);
          }
          if (row_live) {
            if (p.n_split > 1) {
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + slot * 128 + c * 32);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if (MLA_STORE_OK(dst + x, p.part_o, p.part_o_bytes, p.err))
                  dst[x] = make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(out_row + c * 32);
              const float* f = reinterpret_cast<const float*>(v);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (MLA_STORE_OK(dst + x, p.out, p.out_bytes, p.err))
                  dst[x] = make_uint4(
                      ptx::pack_bf16x2(f[8 * x], f[8 * x + 1]), ptx::pack_bf16x2(f[8 * x + 2], f[8 * x + 3]),
                      ptx::pack_bf16x2(f[8 * x + 4], f[8 * x + 5]), ptx::pack_bf16x2(f[8 * x + 6], f[8 * x + 7]));
            }
          }
          __syncwarp();  // the next columns are loaded by the whole warp, rows of padding included
        }
        if (row_live) {
          if (p.n_split > 1) {
            if (MLA_STORE_OK(p.part_lse + slot, p.part_lse, p.part_lse_bytes, p.err)) p.part_lse[slot] = lse2;
          } else if (MLA_STORE_OK(lse_at, p.lse, p.lse_bytes, p.err)) {
            *lse_at = lse2 * kLn2;
          }
        }
      }
      // eight arrivals a unit, by_keys all from the first warpgroup: the second one may have had no tile of
      // this unit and waited for nothing, and would count itself into the unit before
      ptx::tc_fence_before();
      __syncwarp();
      if (u.by_keys ? t == 0 && lane < 2 : lane == 0) ptx::mbar_arrive(&bars.o_free);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace sm103_cross
}  // namespace mla

#include "cross_few_sm103.cuh"

namespace mla {
namespace sm103_cross {

// Joins the shares of a row: with the largest of their log2 sums as reference, weights 2^(lse_s - max)
// over their sum, in the order of the shares.  kWarps warps a row, every kWarps-th share each.
template <int kWarps>
__global__ void __launch_bounds__(256) join_kernel(const Params p) {
  __shared__ float4 joined[8][32];
  __shared__ float2 sums[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % kWarps;
  const long long rows = static_cast<long long>(p.B) * p.H * p.Sq;
  const long long row = static_cast<long long>(blockIdx.x) * (8 / kWarps) + warp / kWarps;
  wait_for_stream();
  const bool live = row < rows;
  const long long bh = live ? row / p.Sq : 0;
  const int i = live ? static_cast<int>(row - bh * p.Sq) : 0, b = static_cast<int>(bh / p.H);
  const int len = live ? key_len(p, b) : 0;
  const int block = i / p.slot_rows, r = i - block * p.slot_rows;
  const size_t first = (static_cast<size_t>(bh) * p.nrb + block) * p.n_split;
  float m = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = part; s < p.n_split; s += kWarps) {
    if (share_empty(p, len, s)) continue;  // no keys of this sequence
    const size_t at = (first + s) * p.slot_rows + r;
    const float lse = ptx::ld_l2(p.part_lse + at);
    const float4 v = ptx::ld_l2(reinterpret_cast<const float4*>(p.part_o + at * 128) + lane);
    const float to = fmaxf(m, lse), ref = to == -INFINITY ? 0.f : to;
    const float keep = exp2f(m - ref), w = exp2f(lse - ref);
    m = to;
    sum = sum * keep + w;
    o = make_float4(o.x * keep + v.x * w, o.y * keep + v.y * w, o.z * keep + v.z * w, o.w * keep + v.w * w);
  }
  if constexpr (kWarps > 1) {
    joined[warp][lane] = o;
    if (lane == 0) sums[warp] = make_float2(m, sum);
    __syncthreads();
    if (part != 0) return;
    for (int w = 1; w < kWarps; ++w) {
      const float2 of = sums[warp + w];
      const float4 v = joined[warp + w][lane];
      const float to = fmaxf(m, of.x), ref = to == -INFINITY ? 0.f : to;
      const float keep = exp2f(m - ref), other = exp2f(of.x - ref);
      m = to;
      sum = sum * keep + of.y * other;
      o = make_float4(o.x * keep + v.x * other, o.y * keep + v.y * other, o.z * keep + v.z * other,
                      o.w * keep + v.w * other);
    }
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint2* dst = reinterpret_cast<uint2*>(p.out + ((static_cast<size_t>(b) * p.Sq + i) * p.H + bh % p.H) * 128) + lane;
  if (MLA_STORE_OK(dst, p.out, p.out_bytes, p.err))
    *dst = make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0 && MLA_STORE_OK(p.lse + row, p.lse, p.lse_bytes, p.err))
    p.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// How a call is cut: row blocks of up to 256 rows (128 where that is all), and each block's keys in
// n_split shares.  A share costs its key tiles and about kEnds of them more for its two ends, the join
// about kJoin; the CTAs work in rounds of one unit each.  Few rows (the form without tiles): runs of whole steps, two
// CTAs an SM that start as others end; where lengths are given they may be ragged, and half a unit more is charged
// for the longest (16 x 8 heads, one row, up to 6000 keys: 44 us, 52 without).
struct Cut {
  bool one_tile;
  int nrb, n_split, slot_rows, chunk;
  long long units;  // of tiles; a partial result each where split
};
constexpr int kEnds = 2, kJoin = 3, kMaxSlots = 4;  // slots: units of a split call, times the SMs

inline Cut few_cut(int B, int H, int Sq, int Sk, bool ragged, int sms) {
  Cut c = {};
  const int blocks = (Sq + kFewRows - 1) / kFewRows;
  const long long items = (long long)B * H * blocks, slots = 2LL * sms;
  const int steps = (Sk + kFewStep - 1) / kFewStep;
  double best = 1e300;
  for (long long s = 1; s <= steps && (s == 1 || items * s <= 4 * slots); ++s) {
    const double unit = (double)((steps + s - 1) / s) + kEnds, rounds = (double)(items * s) / slots;
    const double cost = (ragged ? std::max(rounds, 1.) + 0.5 : std::ceil(rounds)) * unit + (s > 1 ? 2 + s / 32. : 0);
    if (cost < best) {
      best = cost;
      c.chunk = (int)std::min((steps + s - 1) / s * kFewStep, 0x7fffffffLL);
    }
  }
  c.n_split = (int)(((long long)Sk + c.chunk - 1) / c.chunk);
  c.nrb = 1;
  c.slot_rows = Sq;
  c.units = (long long)B * H * c.n_split;
  return c;
}

inline Cut tile_cut(int B, int H, int Sq, int Sk, int sms) {
  Cut c = {};
  c.one_tile = Sq <= BM;
  c.nrb = c.one_tile ? 1 : (Sq + 2 * BM - 1) / (2 * BM);
  c.slot_rows = std::min(Sq, c.one_tile ? BM : 2 * BM);
  const long long items = (long long)B * H * c.nrb;
  const int tiles = (Sk + BN - 1) / BN;
  c.n_split = 1;
  double best = 1e300;
  for (long long s = 1; s <= tiles && (s == 1 || items * s <= (long long)kMaxSlots * sms); ++s) {
    const double rounds = (double)((items * s + sms - 1) / sms);
    const double cost = rounds * ((double)((tiles + s - 1) / s) + kEnds) + (s > 1 ? kJoin : 0);
    if (cost < best) {
      best = cost;
      c.n_split = (int)s;
    }
  }
  c.units = items * c.n_split;
  return c;
}

// Up to eight rows take the form without tiles, more of them, in blocks of eight that read the keys once each, where that is
// expected to be faster.  Microseconds, fitted to calls of 8 to 100 rows: a CTA of few rows has 2.2 beside its keys, of which
// 128 take 1.1 alone and 2.9 with all SMs full; a unit of tiles 3 beside 1.5 a tile (of a share: rounded down), and 1.7 to
// start with.  Measured as tiles and without: 1 x 8 heads x 77 keys, 64 rows 6.9, so 3.6; 8 x 8 x 300, 16 rows 9.2, so 6.2, 48 rows
// 9.2, not 13.3; 64 x 64 x 50, 16 rows 117, so 101, 32 rows 119, not 190.  Next to the border it errs by up to 4 us for tiles, where
// shares take about 3 more than it expects (1 x 8 x 600, 100 rows 12.3, not 8.7) or lengths are ragged (8 x 32 x up to 300, 16 rows
// 15.4, not 12.3).
inline Cut cut_of(int B, int H, int Sq, int Sk, bool ragged, int sms) {
  const Cut few = few_cut(B, H, Sq, Sk, ragged, sms);
  if (Sq <= kFewRows) return few;
  const Cut tiles = tile_cut(B, H, Sq, Sk, sms);
  const double ctas = (double)few.units * ((Sq + kFewRows - 1) / kFewRows), slots = 2. * sms;
  const double keys = (double)std::min(few.chunk, Sk) / kFewStep, full = std::min(ctas / slots, 1.);
  const double t_few = std::ceil(ctas / slots) * (keys * (1.1 + 1.8 * full) + 2.2) + (few.n_split > 1 ? 2.2 : 0);
  const double t_tiles = 1.7 + std::ceil((double)tiles.units / sms) * ((Sk + BN - 1) / BN / tiles.n_split * 1.5 + 3) +
                         (tiles.n_split > 1 ? 3 : 0);
  return t_few < t_tiles && ctas < 0x40000000 ? few : tiles;
}

}  // namespace sm103_cross

// ---------------------------------------------------------------- host side

cudaError_t encode_tensor_map(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* ptr,
                              const uint64_t* dims, const uint64_t* strides, const uint32_t* box);

namespace {

// [B, S, H, d] tensor of bf16, box = 64 columns x 1 head x 128 tokens
bool cross_map(CUtensorMap* m, const void* p, int B, int S, int H, int d) {
  uint64_t dims[4] = {(uint64_t)d, (uint64_t)H, (uint64_t)S, (uint64_t)B};
  uint64_t strides[3] = {(uint64_t)d * 2, (uint64_t)H * d * 2, (uint64_t)S * H * d * 2};
  uint32_t box[4] = {64, 1, 128, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box) == cudaSuccess;
}

size_t part_o_bytes(const sm103_cross::Cut& c) { return (size_t)c.units * c.slot_rows * 128 * sizeof(float); }
size_t part_lse_bytes(const sm103_cross::Cut& c) { return ((size_t)c.units * c.slot_rows * sizeof(float) + 255) / 256 * 256; }

template <bool kOneTile>
cudaError_t launch_cross(const CUtensorMap& tqn, const CUtensorMap& tqr, const CUtensorMap& tkn, const CUtensorMap& tkr,
                         const CUtensorMap& tv, const sm103_cross::Params& p, int sms, cudaStream_t stream) {
  using namespace sm103_cross;
  auto kernel = cross_kernel<kOneTile>;
  // the raised register counts of the softmax warps are drawn from what the CTA was launched with: with
  // fewer than the average the raise would wait forever, so refuse to launch then
  static int regs_ok = 0;  // 0 unknown, 1 checked
  if (!__atomic_load_n(&regs_ok, __ATOMIC_ACQUIRE)) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kRegsAtLaunch) return cudaErrorInvalidDeviceFunction;
    __atomic_store_n(&regs_ok, 1, __ATOMIC_RELEASE);
  }
  static unsigned long long smem_set = 0;
  const cudaError_t e = smem_attr_once(kernel, Smem<kOneTile>::kAlloc, &smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent_smem(kernel, std::min(p.units, sms), kThreads, Smem<kOneTile>::kAlloc, stream, tqn, tqr, tkn,
                               tkr, tv, p);
}

cudaError_t launch_join(const sm103_cross::Params& p, cudaStream_t stream) {
  using namespace sm103_cross;
  // few shares: a warp a row; many: the warps of a block share one
  const long long rows = (long long)p.B * p.H * p.Sq;
  if (p.n_split <= 4) return launch_dependent(join_kernel<1>, (int)((rows + 7) / 8), 256, stream, p);
  return launch_dependent(join_kernel<8>, (int)rows, 256, stream, p);
}

}  // namespace

// Whether the units of such a call can be numbered.
bool cross_fits(int B, int H, int Sq) {
  return (long long)B * H * ((Sq + 255) / 256) <= 0x40000000LL && (double)B * H * Sq <= 8.0e9;
}

size_t cross_workspace_bytes(int B, int H, int Sq, int Sk, int sms) {
  size_t most = 0;  // with and without key lengths
  for (const bool ragged : {false, true}) {
    const sm103_cross::Cut c = sm103_cross::cut_of(B, H, Sq, Sk, ragged, sms);
    if (c.n_split > 1) most = std::max(most, part_o_bytes(c) + part_lse_bytes(c));
  }
  return most;
}

// Of a call's plan, for tests: 0 without tiles, 1 one query tile, 2 two.
int cross_form(int B, int H, int Sq, int Sk, bool ragged, int sms, int* shares) {
  const sm103_cross::Cut c = sm103_cross::cut_of(B, H, Sq, Sk, ragged, sms);
  *shares = c.n_split;
  return c.chunk > 0 ? 0 : c.one_tile ? 1 : 2;
}

cudaError_t launch_cross_sm103(const void* q_nope, const void* q_rope, const void* k_nope, const void* k_rope,
                               const void* v, const int* key_lens, void* out, float* lse, int B, int H, int Sq, int Sk,
                               float softmax_scale, void* workspace, int sms, unsigned int* err, cudaStream_t stream) {
  using namespace sm103_cross;
  const Cut c = cut_of(B, H, Sq, Sk, key_lens != nullptr, sms);
  Params p = {};
  p.B = B;
  p.H = H;
  p.Sq = Sq;
  p.Sk = Sk;
  p.nrb = c.nrb;
  p.n_split = c.n_split;
  p.units = (int)c.units;
  p.chunk = c.chunk;
  p.row_blocks = (Sq + kFewRows - 1) / kFewRows;
  p.shift = c.nrb > 1 && (Sq - 1) % (2 * BM) < BM;
  p.slot_rows = c.slot_rows;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.key_lens = key_lens;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.err = err;
  p.out_bytes = (size_t)B * Sq * H * 128 * 2;
  p.out_bytes -= std::min(p.out_bytes, testing_out_shrink());
  p.lse_bytes = (size_t)B * H * Sq * sizeof(float);
  if (c.n_split > 1) {
    p.part_o_bytes = part_o_bytes(c);
    p.part_lse_bytes = part_lse_bytes(c);
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_o_bytes);
  }
  cudaError_t e;
  if (c.chunk > 0) {
    auto kernel = Sq == 1 ? one_row_kernel : eight_rows_kernel;
    auto in = [](const void* x) { return static_cast<const uint16_t*>(x); };
    e = launch_dependent(kernel, p.units * p.row_blocks, kFewWarps * 32, stream, in(q_nope), in(q_rope), in(k_nope), in(k_rope),
                         in(v), p);
    if (e != cudaSuccess || c.n_split == 1) return e;
    return launch_join(p, stream);
  }
  CUtensorMap tqn, tqr, tkn, tkr, tv;
  uint64_t kr_dims[3] = {64, (uint64_t)Sk, (uint64_t)B};
  uint64_t kr_strides[2] = {64 * 2, (uint64_t)Sk * 64 * 2};
  uint32_t kr_box[3] = {64, BN, 1};
  if (!cross_map(&tqn, q_nope, B, Sq, H, 128) || !cross_map(&tqr, q_rope, B, Sq, H, 64) ||
      !cross_map(&tkn, k_nope, B, Sk, H, 128) || !cross_map(&tv, v, B, Sk, H, 128) ||
      encode_tensor_map(&tkr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, k_rope, kr_dims, kr_strides, kr_box) != cudaSuccess)
    return cudaErrorInvalidValue;
  e = c.one_tile ? launch_cross<true>(tqn, tqr, tkn, tkr, tv, p, sms, stream)
                 : launch_cross<false>(tqn, tqr, tkn, tkr, tv, p, sms, stream);
  if (e != cudaSuccess || c.n_split == 1) return e;
  return launch_join(p, stream);
}

}  // namespace mla
