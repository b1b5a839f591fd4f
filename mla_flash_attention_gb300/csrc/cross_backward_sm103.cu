// Backward pass of cross attention on tcgen05 / TMEM / TMA, bf16 operands: queries and keys of unlike counts, each
// sequence with its own number of keys.
//
// For one (batch, head), with s = scale [Qn|Qr][Kn|Kr]' and P = exp(s - LSE) (the forward's log-sum-exp, so no
// row statistics are recomputed):
//   dV = P' dO,  dP = dO V',  D_i = sum_d dO_id O_id,  dS = P * (dP - D),
//   dQ = scale dS K,  dK = scale dS' Q   (the rope key is shared by the heads: its gradient is the sum over them)
//
// P and dS are rounded to bf16 where they enter products as operands beside bf16 ones, as in the prefill's: gradients are
// off by 0.0024 of themselves, RMS, where their own rounding is 0.0017; a second term of each would add
// 44 % to the MMAs.  The rope key's gradient, the whole sum in fp32, is rounded once and to bf16 like the other gradients.
//
// Two roles of units with the products, tiles and roles of warps of the prefill's backward:
//   key-tile units (b, h, 128 keys): K and V stay in shared memory; query tiles stream by.
//     TMEM: X [0,128) S' = K Q' (keys on lanes), then dP' = V dO'; dV [128,256);
//           dK [256,448) (nope 128 + rope 64); Y [448,512) P', then dS' (bf16 pairs)
//     MMAs per query tile n: dP'(n), dV += P' dO (TS: A = Y), S'(n+1), dK += dS' Q (TS: A = Y)
//   query-tile units (b, h, 128 queries): Q and dO stay; key tiles stream by.
//     TMEM: X [0,128) S = Q K'; [128,256) dP = dO V'; dQ [256,448); Y [448,512) dS (bf16)
//     MMAs per key tile n: S(n+1), dQ += dS K (TS: A = Y), dP(n+1)
// Shared memory (both roles): fixed 3-chunk tile (K | Q) + fixed 2-chunk tile (V | dO), a 2-stage ring of
// streamed 3-chunk tiles (Q | K), one streamed 2-chunk tile (dO | V), and the streamed query tiles'
// -LSE*log2(e) and D vectors (key role).
// Warps: 0 TMA producer, 1 MMA issuer, 2-9 elementwise (TMEM lane quarter = warp % 4, column half =
// (warp - 2) / 4; each half owns 64 score columns and 32 packed columns of Y).
//
// What differs from the prefill's:
//   - CTAs are persistent: encoder lengths make streams of a few tiles, and a unit's two ends took 11 us beside 2 us
//     a tile.  The next unit's tiles are loaded, and its first scores formed, while this one's accumulators are stored;
//     the barriers' phases go on from unit to unit.
//   - In the key role the keys are TMEM lanes, so what stands behind a sequence's last key stays in lanes that are
//     stored as zeros; in the query role those keys' weights and dP are masked and their K rows zeroed in shared
//     memory (0 * NaN is NaN).
//   - Few queries and keys take no tiles: cross_backward_few_sm103.cuh.
//   - The tiles that a CTA streams are cut in shares where few tiles of the one kind meet many of the other.  Shares,
//     and the rope key's gradient of each head, are fp32 partial results that a third kernel adds in a fixed
//     order: gradients do not depend on the run.
//
// Bound by shared memory: a step of the key role (128 keys x 128 queries) reads 240 KB of operands and writes 80, 2500 clocks
// of its bandwidth beside 2560 of MMA work, and takes 3700; of the query role 2300 and 2050, 2750.  2048 queries x 4096
// keys, 64 heads: 870 us (1030 TFLOP/s of the definition's products, 1430 of those done, scores and dP being
// formed in both roles).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace sm103_cross_bwd {

constexpr int BT = 128;                        // rows of every tile (queries or keys)
constexpr int kChunk = BT * 128;               // 128 rows x 64 bf16, 128B-swizzled (16 KB)
constexpr int kOffFix3 = 0;                    // K (key role) | Q (query role): 3 chunks
constexpr int kOffFix2 = kOffFix3 + 3 * kChunk;  // V | dO: 2 chunks
constexpr int kOffRing = kOffFix2 + 2 * kChunk;  // 2 stages x 3 chunks: Q | K
constexpr int kOffOne = kOffRing + 2 * 3 * kChunk;  // dO | V: 2 chunks
constexpr int kOffVec = kOffOne + 2 * kChunk;    // per ring stage: -LSE*log2e [128], D [128]
constexpr int kSmemBytes = kOffVec + 2 * 2 * BT * 4;  // 210 KB
constexpr int kSmemAlloc = kSmemBytes + 1024;
constexpr int kThreads = 320;
constexpr uint32_t kColX = 0, kColDP = 128, kColDV = 128, kColAcc = 256, kColY = 448;

struct Params {
  const float* nlse2;      // [B*H, q_pad]: -LSE * log2(e); -inf for padding rows and rows that saw no key
  const float* dvec;       // [B*H, q_pad]: D = rowsum(dO * O); padding rows hold 0
  uint16_t* dq_nope;       // [B, Sq, H, 128]
  uint16_t* dq_rope;       // [B, Sq, H, 64]
  uint16_t* dk_nope;       // [B, Sk, H, 128]
  uint16_t* dk_rope;       // [B, Sk, 64]
  uint16_t* dv;            // [B, Sk, H, 128]
  const int* key_lens;     // or null: Sk everywhere
  float* part_rope;        // [B*H][n_qs][Sk][64]: dk_rope of one head and share
  float* part_kv;          // n_qs > 1: [key units][128][dV 128 | dK nope 128]
  float* part_q;           // n_ks > 1: [query units][128][192]
  unsigned int* err;
  int B, H, Sq, Sk, q_pad;
  int nqt, nkt;            // query tiles, key tiles of Sk
  int n_query_units;
  int n_qs, n_ks;          // shares of the query tiles (key role) and of the key tiles (query role)
  int few_chunk;           // few queries: keys of a CTA; else 0
  int by_lens;             // units pass over the key tiles that hold no key
  int wide;                // the bf16 gradients are 32-byte aligned
  float scale, scale_log2;
  size_t q_bytes, k_bytes, rope_bytes;                   // of dq_nope (dq_rope half), dk_nope and dv, dk_rope: for the
  size_t part_rope_bytes, part_kv_bytes, part_q_bytes;   // store checks
};

__device__ __forceinline__ int key_len(const Params& p, int b) {
  return p.key_lens ? min(max(__ldg(p.key_lens + b), 0), p.Sk) : p.Sk;
}
// first tile of share s
__device__ __forceinline__ int share_begin(int tiles, int s, int n) {
  return static_cast<int>(static_cast<long long>(tiles) * s / n);
}

struct Bars {
  // one full barrier per 16 KB chunk of a streamed tile, so the MMAs over its first chunk can
  // start while the later ones are still arriving
  uint64_t fix3_full, fix3_empty, fix2_full, fix2_empty, ring_full[2][3], ring_empty[2], one_full[2], one_empty;
  uint64_t s_full, x_read, dp_full, dp_read, p_ready, dv_done, ds_ready, acc_step, acc_done, acc_free, drained;
  uint32_t tmem_base;
  int abort_flag;
};

// D = rowsum(dO * O) and -LSE * log2(e) into vectors padded to whole query tiles.  A warp takes eight rows of a head, 16
// lanes a row, all its loads under way at once (32 rows a warp were too few warps for small batches: 128 rows of
// 152 heads 21 us, so 5).  A row that saw no key (LSE = -inf) gets -inf like the padding, so its weights are 0.
__global__ void __launch_bounds__(256) prep_kernel(const uint16_t* __restrict__ out,
                                                         const uint16_t* __restrict__ d_out,
                                                         const float* __restrict__ lse, float* __restrict__ nlse2,
                                                         float* __restrict__ dvec, int B, int H, int S, int S_pad) {
  wait_for_stream();
  const long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, groups = S_pad / 8;
  if (task >= (long long)B * H * groups) return;
  const int bh = static_cast<int>(task / groups), i0 = static_cast<int>(task - (long long)bh * groups) * 8;
  const int b = bh / H, h = bh - b * H;
  uint4 a[4], o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = i0 + 2 * k + (lane >> 4);
    const size_t ro = (((size_t)b * S + i) * H + h) * 128 + (lane & 15) * 8;
    a[k] = o[k] = make_uint4(0, 0, 0, 0);
    if (i < S) {
      a[k] = __ldg(reinterpret_cast<const uint4*>(d_out + ro));
      o[k] = __ldg(reinterpret_cast<const uint4*>(out + ro));
    }
  }
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
  float mine = 0.f;  // lane 16 r + 2 k: of row 2 k + r
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, y[4] = {o[k].x, o[k].y, o[k].z, o[k].w};
    float d = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) d = fmaf(hi(x[j]), hi(y[j]), fmaf(lo(x[j]), lo(y[j]), d));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if ((lane & 15) == 2 * k) mine = d;
  }
  if ((lane & 15) >= 8 || (lane & 1)) return;
  const int i = i0 + (lane & 15) + (lane >> 4);
  const size_t vo = (size_t)bh * S_pad + i;
  const float of = i < S ? lse[(size_t)bh * S + i] : -INFINITY;
  dvec[vo] = mine;
  nlse2[vo] = of == -INFINITY ? -INFINITY : -of * 1.4426950408889634f;
}

// 32 fp32 accumulator columns (times `mul`) -> 32 bf16 at dst (64 bytes, 16-byte aligned)
__device__ __forceinline__ void store_bf16x32(uint16_t* dst, const uint32_t (&u)[32], float mul) {
  uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint4 w;
    w.x = ptx::pack_bf16x2(__uint_as_float(u[8 * x + 0]) * mul, __uint_as_float(u[8 * x + 1]) * mul);
    w.y = ptx::pack_bf16x2(__uint_as_float(u[8 * x + 2]) * mul, __uint_as_float(u[8 * x + 3]) * mul);
    w.z = ptx::pack_bf16x2(__uint_as_float(u[8 * x + 4]) * mul, __uint_as_float(u[8 * x + 5]) * mul);
    w.w = ptx::pack_bf16x2(__uint_as_float(u[8 * x + 6]) * mul, __uint_as_float(u[8 * x + 7]) * mul);
    d[x] = w;
  }
}

// What one store_row writes, checked as a whole.
struct alignas(16) Row64 {
  uint4 v[4];
};
struct alignas(16) Row128 {
  uint4 v[8];
};

// store_bf16x32 in two whole sectors where dst is 32-byte aligned: a warp's lanes write rows that lie apart, and
// 16 bytes at a time took a request for every half sector.
__device__ __forceinline__ void store_row(uint16_t* dst, const uint32_t (&u)[32], float mul, bool wide, const void* base,
                                          size_t bytes, unsigned int* err) {
  if (!MLA_STORE_OK(reinterpret_cast<Row64*>(dst), base, bytes, err)) return;
  if (!wide) {
    store_bf16x32(dst, u, mul);
    return;
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t w[8];
#pragma unroll
    for (int y = 0; y < 8; ++y)
      w[y] = ptx::pack_bf16x2(__uint_as_float(u[16 * x + 2 * y]) * mul, __uint_as_float(u[16 * x + 2 * y + 1]) * mul);
    ptx::st_v8(dst + 16 * x, w);
  }
}
// 32 fp32 accumulator columns (times `mul`) -> 32 fp32 at dst (32-byte aligned)
__device__ __forceinline__ void store_row(float* dst, const uint32_t (&u)[32], float mul, const void* base, size_t bytes,
                                          unsigned int* err) {
  if (!MLA_STORE_OK(reinterpret_cast<Row128*>(dst), base, bytes, err)) return;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint32_t w[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) w[y] = __float_as_uint(__uint_as_float(u[8 * x + y]) * mul);
    ptx::st_v8(dst + 8 * x, w);
  }
}

struct Maps {
  const CUtensorMap *qn, *qr, *kn, *kr, *v, *dout;
};

// The units of a CTA: every gridDim.x-th, the key-tile units first; if there are more units than CTAs, only the tiles that
// hold keys (with the empty ones in the order, which a CTA passes in no time, other CTAs had more than their share: 8 x 16
// heads, 448 queries, up to 1500 keys 207 us, so 178; 4 x 32 heads, 1024 queries, up to 1024 keys 251, so 198).  Every
// warp walks them by itself, 32 sequences' lengths at a time; where it stands is kept in shared memory, the products'
// loops having no register for it.
struct Walk {
  unsigned id, base;  // base: key-tile units of the sequences before b
  int b;
};
__device__ __forceinline__ bool next_unit(Walk& walk, const Params& p, bool& key_role, int& bh, int& tile, int& share) {
  const int lane = threadIdx.x & 31;
  const unsigned id = walk.id, each = static_cast<unsigned>(p.H) * p.n_qs;  // units of a sequence's key tile
  unsigned base = p.by_lens ? walk.base : static_cast<unsigned>(p.B) * p.nkt * each, at = id, tiles = p.nkt;
  int b = 0;
  key_role = id < base;
  if (p.by_lens) {
    for (b = walk.b; b < p.B; b += 32) {
      const unsigned mine = b + lane < p.B ? (key_len(p, b + lane) + BT - 1) / BT : 0;
      unsigned upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const unsigned low = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += low;
      }
      const unsigned past = __ballot_sync(0xffffffffu, id - base >= upto * each);
      key_role = past != 0xffffffffu;
      if (key_role) {
        const int first = __ffs(~past) - 1;
        tiles = __shfl_sync(0xffffffffu, mine, first);
        at = id - base - (__shfl_sync(0xffffffffu, upto, first) - tiles) * each;
        __syncwarp();
        if (lane == 0) walk.base = base, walk.b = b;
        b += first;
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31) * each;
    }
    if (!key_role) {
      __syncwarp();
      if (lane == 0) walk.base = base, walk.b = b;
    }
  }
  const unsigned shares = key_role ? p.n_qs : p.n_ks;
  if (!key_role) {
    at = id - base;
    tiles = p.nqt;
    if (at >= static_cast<unsigned>(p.n_query_units)) return false;
  }
  const unsigned unit = at / shares, h = unit / tiles;
  share = at - unit * shares;
  tile = unit - h * tiles;
  bh = (key_role ? b * p.H : 0) + h;
  __syncwarp();
  if (lane == 0) walk.id = id + gridDim.x;
  __syncwarp();
  return true;
}

// Where a thread's role stands in the run of units that its CTA works through: steps and units before this
// one (the phases of the barriers go on from unit to unit), and copies under way.
struct Flow {
  uint32_t g = 0, u = 0;
  uint32_t n_fix3 = 0, n_fix2 = 0, n_ring = 0, n_one = 0;
  bool after_key = false;  // the unit before was of the key role
  bool ok = true;
};

// kKeyRole: this CTA owns key tile `tile` and streams query tiles (dK, dV); otherwise it
// owns query tile `tile` and streams key tiles (dQ); share `share` of them.  `unit` numbers the role's units.
template <bool kKeyRole>
__device__ __forceinline__ void bwd_body(const Maps& m, const Params& p, unsigned char* sm,
                                         Bars& bars, int b, int h, int tile, int share, int unit, Flow& f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = key_len(p, b);
  const int of = kKeyRole ? (tile * BT < len ? p.nqt : 0) : (len + BT - 1) / BT, shares = kKeyRole ? p.n_qs : p.n_ks;
  const int t_begin = share_begin(of, share, shares), t_end = share_begin(of, share + 1, shares);
  const int nsteps = t_end - t_begin;
  const uint32_t g = f.g;  // step n of this unit is step g + n of the CTA
  const int rows = kKeyRole ? p.Sk : p.Sq;  // of the owned operand and its gradients
  const int bh = b * p.H + h;
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort_flag;

  if (nsteps == 0) {  // queries without a key: zeros (shares are joined without them)
    const int r = (warp & 3) * 32 + lane, hf = (warp - 2) >> 2, row_idx = tile * BT + r;
    if (!kKeyRole && warp >= 2 && row_idx < rows && shares == 1) {
      const size_t ro = ((size_t)b * rows + row_idx) * p.H + h;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4* wide = reinterpret_cast<uint4*>(p.dq_nope + ro * 128) + 8 * hf;
      uint4* narrow = reinterpret_cast<uint4*>(p.dq_rope + ro * 64) + 4 * hf;
      for (int x = 0; x < 8; ++x)
        if (MLA_STORE_OK(wide + x, p.dq_nope, p.q_bytes, p.err)) wide[x] = zero;
      for (int x = 0; x < 4; ++x)
        if (MLA_STORE_OK(narrow + x, p.dq_rope, p.q_bytes / 2, p.err)) narrow[x] = zero;
    }
    return;
  }

  if (warp == 0) {
    if (ptx::elect_one()) {
      // ------------------------------------------------------------ TMA producer
      const int row0 = tile * BT;
      // the owned tiles, each as soon as the unit before has formed its last products with it
      auto load_fix3 = [&]() -> bool {
        if (!ptx::mbar_wait(&bars.fix3_empty, (f.u & 1) ^ 1, abort_flag, p.err)) return false;
        unsigned char* f3 = sm + kOffFix3;
        ptx::mbar_arrive_expect_tx(&bars.fix3_full, 3 * kChunk);
        const CUtensorMap* nope = kKeyRole ? m.kn : m.qn;
        ptx::tma_load_4d(f3, nope, &bars.fix3_full, 0, h, row0, b);
        ptx::tma_load_4d(f3 + kChunk, nope, &bars.fix3_full, 64, h, row0, b);
        if (kKeyRole)
          ptx::tma_load_3d(f3 + 2 * kChunk, m.kr, &bars.fix3_full, 0, row0, b);
        else
          ptx::tma_load_4d(f3 + 2 * kChunk, m.qr, &bars.fix3_full, 0, h, row0, b);
        ++f.n_fix3;
        return true;
      };
      auto load_fix2 = [&]() -> bool {
        if (!ptx::mbar_wait(&bars.fix2_empty, (f.u & 1) ^ 1, abort_flag, p.err)) return false;
        unsigned char* f2_ = sm + kOffFix2;
        ptx::mbar_arrive_expect_tx(&bars.fix2_full, 2 * kChunk);
        const CUtensorMap* of = kKeyRole ? m.v : m.dout;
        ptx::tma_load_4d(f2_, of, &bars.fix2_full, 0, h, row0, b);
        ptx::tma_load_4d(f2_ + kChunk, of, &bars.fix2_full, 64, h, row0, b);
        ++f.n_fix2;
        return true;
      };
      constexpr int kAhead = 2;  // tiles warmed in L2 ahead of their load
      auto warm = [&](int n) {
        const int r0 = (t_begin + n) * BT;
        if (kKeyRole) {
          ptx::tma_prefetch_4d(m.qn, 0, h, r0, b);
          ptx::tma_prefetch_4d(m.qn, 64, h, r0, b);
          ptx::tma_prefetch_4d(m.qr, 0, h, r0, b);
          ptx::tma_prefetch_4d(m.dout, 0, h, r0, b);
          ptx::tma_prefetch_4d(m.dout, 64, h, r0, b);
          const size_t vo = (size_t)bh * p.q_pad + r0;
          ptx::bulk_prefetch(p.nlse2 + vo, BT * 4);
          ptx::bulk_prefetch(p.dvec + vo, BT * 4);
        } else {
          ptx::tma_prefetch_4d(m.kn, 0, h, r0, b);
          ptx::tma_prefetch_4d(m.kn, 64, h, r0, b);
          ptx::tma_prefetch_3d(m.kr, 0, r0, b);
          ptx::tma_prefetch_4d(m.v, 0, h, r0, b);
          ptx::tma_prefetch_4d(m.v, 64, h, r0, b);
        }
      };
      f.ok = load_fix3();
      for (int n = 0; f.ok && n < nsteps; ++n) {
        const uint32_t step = g + n;
        const int r0 = (t_begin + n) * BT, s = step & 1;
        if (!(f.ok = ptx::mbar_wait(&bars.ring_empty[s], ((step >> 1) & 1) ^ 1, abort_flag, p.err))) break;
        unsigned char* dst = sm + kOffRing + s * 3 * kChunk;
        if (kKeyRole) {
          ptx::mbar_arrive_expect_tx(&bars.ring_full[s][0], kChunk + 2 * BT * 4);
          ptx::mbar_arrive_expect_tx(&bars.ring_full[s][1], kChunk);
          ptx::mbar_arrive_expect_tx(&bars.ring_full[s][2], kChunk);
          ptx::tma_load_4d(dst, m.qn, &bars.ring_full[s][0], 0, h, r0, b);
          ptx::tma_load_4d(dst + kChunk, m.qn, &bars.ring_full[s][1], 64, h, r0, b);
          ptx::tma_load_4d(dst + 2 * kChunk, m.qr, &bars.ring_full[s][2], 0, h, r0, b);
          const size_t vo = (size_t)bh * p.q_pad + r0;
          unsigned char* vec = sm + kOffVec + s * 2 * BT * 4;
          ptx::bulk_load(vec, p.nlse2 + vo, BT * 4, &bars.ring_full[s][0]);
          ptx::bulk_load(vec + BT * 4, p.dvec + vo, BT * 4, &bars.ring_full[s][0]);
        } else {
          for (int c = 0; c < 3; ++c) ptx::mbar_arrive_expect_tx(&bars.ring_full[s][c], kChunk);
          ptx::tma_load_4d(dst, m.kn, &bars.ring_full[s][0], 0, h, r0, b);
          ptx::tma_load_4d(dst + kChunk, m.kn, &bars.ring_full[s][1], 64, h, r0, b);
          ptx::tma_load_3d(dst + 2 * kChunk, m.kr, &bars.ring_full[s][2], 0, r0, b);
        }
        ++f.n_ring;
        if (n == 0 && !(f.ok = load_fix2())) break;
        if (!(f.ok = ptx::mbar_wait(&bars.one_empty, (step & 1) ^ 1, abort_flag, p.err))) break;
        unsigned char* one = sm + kOffOne;
        const CUtensorMap* tm = kKeyRole ? m.dout : m.v;
        ptx::mbar_arrive_expect_tx(&bars.one_full[0], kChunk);
        ptx::mbar_arrive_expect_tx(&bars.one_full[1], kChunk);
        ptx::tma_load_4d(one, tm, &bars.one_full[0], 0, h, r0, b);
        ptx::tma_load_4d(one + kChunk, tm, &bars.one_full[1], 64, h, r0, b);
        ++f.n_one;
        // (behind this step's own loads, which the unit waits for)
        for (int a = n == 0 ? 1 : kAhead; a <= kAhead; ++a)
          if (n + a < nsteps) warm(n + a);
      }
    }
    f.ok = __all_sync(0xffffffffu, f.ok);
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdS = ptx::make_idesc(1, BT, BT, 0, 0);     // both K-major
      constexpr uint32_t kIdDV = ptx::make_idesc(1, BT, 128, 0, 1);   // B N-major, N = 128
      constexpr uint32_t kIdAcc = ptx::make_idesc(1, BT, 192, 0, 1);  // B N-major, N = 192
      const uint32_t base = ptx::smem_u32(sm);
      const uint32_t one = base + kOffOne;
      auto ring_of = [&](int n) { return base + kOffRing + ((g + n) & 1) * 3 * kChunk; };
      // scores over the 192-deep nope+rope contraction (key role: transposed, keys on lanes)
      auto issue_s = [&](int n) -> bool {
        const uint32_t ring = ring_of(n);
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          if ((k & 3) == 0) {  // each 64-deep chunk as soon as it has landed
            if (!ptx::mbar_wait(&bars.ring_full[(g + n) & 1][k >> 2], ((g + n) >> 1) & 1, abort_flag, p.err)) return false;
            ptx::tc_fence_after();
          }
          const uint32_t off = (k >> 2) * kChunk + (k & 3) * 32;
          ptx::mma_bf16_ss(tmem + kColX, ptx::sw128_desc(base + kOffFix3 + off, 16, 1024),
                           ptx::sw128_desc(ring + off, 16, 1024), kIdS, k > 0);
        }
        ptx::mma_commit(&bars.s_full);
        if (n + 1 == nsteps) ptx::mma_commit(&bars.fix3_empty);
        return true;
      };
      // dP = dO V' over d_v = 128 (key role: dP' = V dO' into X; query role: own columns)
      auto issue_dp = [&](int n) -> bool {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if ((k & 3) == 0) {
            if (!ptx::mbar_wait(&bars.one_full[k >> 2], (g + n) & 1, abort_flag, p.err)) return false;
            if (n == 0 && k == 0 && !ptx::mbar_wait(&bars.fix2_full, f.u & 1, abort_flag, p.err)) return false;
            ptx::tc_fence_after();
          }
          const uint32_t off = (k >> 2) * kChunk + (k & 3) * 32;
          ptx::mma_bf16_ss(tmem + (kKeyRole ? kColX : kColDP),
                           ptx::sw128_desc(base + kOffFix2 + off, 16, 1024),
                           ptx::sw128_desc(one + off, 16, 1024), kIdS, k > 0);
        }
        ptx::mma_commit(&bars.dp_full);
        if (n + 1 == nsteps) ptx::mma_commit(&bars.fix2_empty);
        return true;
      };
      // dK += dS' Q (key role) or dQ += dS K: A = dS (bf16 pairs in Y), B = the streamed
      // 192-wide tile, N-major
      auto issue_acc = [&](int n) {
        const uint32_t ring = ring_of(n);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          ptx::mma_bf16_ts(tmem + kColAcc, tmem + kColY + k * 8,
                           ptx::sw128_desc(ring + k * 2048, kChunk, 1024), kIdAcc,
                           (n > 0 || k > 0) ? 1u : 0u);
        ptx::mma_commit(&bars.ring_empty[(g + n) & 1]);
        ptx::mma_commit(&bars.acc_step);
      };
      auto wait = [&](uint64_t* bar, int n) -> bool {
        if (!ptx::mbar_wait(bar, (g + n) & 1, abort_flag, p.err)) return false;
        ptx::tc_fence_after();
        return true;
      };
      // the accumulators of the unit before were read
      auto acc_free = [&]() -> bool {
        if (!ptx::mbar_wait(&bars.acc_free, (f.u & 1) ^ 1, abort_flag, p.err)) return false;
        ptx::tc_fence_after();
        return true;
      };
      // (the score columns were read: dP' of the unit before lay in them, or its dP was read after them)
      bool ok = ptx::mbar_wait(&bars.fix3_full, f.u & 1, abort_flag, p.err) && (g == 0 || wait(&bars.dp_read, -1)) &&
                issue_s(0);
      if (kKeyRole) {
        // per query tile n: dP'(n) | dV(n) | S'(n+1) | dK(n) -- the next scores run while the
        // elementwise warps turn dP'(n) into dS(n)
        for (int n = 0; ok && n < nsteps; ++n) {
          if (!(ok = wait(&bars.x_read, n) && issue_dp(n))) break;
          if (!(ok = wait(&bars.p_ready, n) && (n > 0 || acc_free()))) break;
#pragma unroll
          for (int k = 0; k < 8; ++k)  // dV += P' dO: A = P' (bf16 pairs in Y), B = dO N-major
            ptx::mma_bf16_ts(tmem + kColDV, tmem + kColY + k * 8,
                             ptx::sw128_desc(one + k * 2048, kChunk, 1024), kIdDV,
                             (n > 0 || k > 0) ? 1u : 0u);
          ptx::mma_commit(&bars.dv_done);
          ptx::mma_commit(&bars.one_empty);
          if (n + 1 < nsteps && !(ok = wait(&bars.dp_read, n) && issue_s(n + 1))) break;
          if (!(ok = wait(&bars.ds_ready, n))) break;
          issue_acc(n);
        }
      } else {
        // per key tile n: S(n+1) | dQ(n) | dP(n+1), with dP(0) issued up front
        // (dP's columns are those of dV in the key role)
        if (ok && f.after_key) ok = acc_free();
        if (ok && (ok = issue_dp(0))) ptx::mma_commit(&bars.one_empty);
        for (int n = 0; ok && n < nsteps; ++n) {
          if (n + 1 < nsteps && !(ok = wait(&bars.x_read, n) && issue_s(n + 1))) break;
          if (!(ok = wait(&bars.ds_ready, n) && (n > 0 || acc_free()))) break;
          issue_acc(n);
          if (n + 1 < nsteps) {
            if (!(ok = wait(&bars.dp_read, n) && issue_dp(n + 1))) break;
            ptx::mma_commit(&bars.one_empty);
          }
        }
      }
      if (ok) ptx::mma_commit(&bars.acc_done);
      f.ok = ok;
    }
    f.ok = __all_sync(0xffffffffu, f.ok);
  } else {
    // -------------------------------------------------------------- elementwise warps
    const int q4 = warp & 3, hf = (warp - 2) >> 2;
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t tX = tmem + lane_off + kColX + hf * 64;
    const uint32_t tDP = tmem + lane_off + (kKeyRole ? kColX : kColDP) + hf * 64;
    const uint32_t tY = tmem + lane_off + kColY + hf * 32;
    const int row_idx = tile * BT + r;  // key (key role) or query
    float nl_row = 0.f, d_row = 0.f;
    if (!kKeyRole) {
      nl_row = p.nlse2[(size_t)bh * p.q_pad + row_idx];
      d_row = p.dvec[(size_t)bh * p.q_pad + row_idx];
    }
    const uint64_t sc2 = ptx::f2(p.scale_log2, p.scale_log2);
    // all lanes wait (bounded); the warp goes on only if every lane saw the phase
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      const bool w = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort_flag, p.err));
      if (w) ptx::tc_fence_after();
      return w;
    };
    // one arrival per warp once its TMEM reads / writes are complete
    auto arrive = [&](uint64_t* bar) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
    bool ok = true;
    for (int n = 0; n < nsteps; ++n) {
      const uint32_t step = g + n;
      const int t = t_begin + n, s = step & 1;
      const float* vec = reinterpret_cast<const float*>(sm + kOffVec + s * 2 * BT * 4);
      ok = wait(&bars.s_full, step & 1);
      // the query vectors of this stage arrived with its TMA transaction: observe it directly
      if (kKeyRole && ok) ok = wait(&bars.ring_full[s][0], (step >> 1) & 1);
      if (!ok) break;
      uint32_t u[64];
      ptx::tmem_ld32(tX, *reinterpret_cast<uint32_t(*)[32]>(u));
      ptx::tmem_ld32(tX + 32, *reinterpret_cast<uint32_t(*)[32]>(u + 32));
      ptx::tmem_ld_wait();
      arrive(&bars.x_read);
      // P = exp2(s * scale * log2(e) - LSE * log2(e)), two columns per packed instruction
      float pr[64];
      if (kKeyRole) {
        const float4* nl = reinterpret_cast<const float4*>(vec) + hf * 16;  // per query
#pragma unroll
        for (int x4 = 0; x4 < 16; ++x4) {
          const float4 l4 = nl[x4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = 2 * x4 + e;
            const uint64_t a2 = ptx::fma2(ptx::f2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])), sc2,
                                          e == 0 ? ptx::f2(l4.x, l4.y) : ptx::f2(l4.z, l4.w));
            pr[2 * x] = ptx::ex2(ptx::f2_lo(a2));
            pr[2 * x + 1] = ptx::ex2(ptx::f2_hi(a2));
          }
        }
      } else {
        const uint64_t nl2 = ptx::f2(nl_row, nl_row);
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const uint64_t a2 = ptx::fma2(ptx::f2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])),
                                        sc2, nl2);
          pr[2 * x] = ptx::ex2(ptx::f2_lo(a2));
          pr[2 * x + 1] = ptx::ex2(ptx::f2_hi(a2));
        }
        if ((t + 1) * BT > len) {  // keys past the sequence end
          const int lim = len - t * BT - hf * 64;
#pragma unroll
          for (int x = 0; x < 64; ++x)
            if (x >= lim) pr[x] = 0.f;
        }
      }
      uint32_t pk[32];
      if (kKeyRole) {
        // P' (bf16) into Y once dK(n-1) has consumed the dS' held there
        if (n > 0 && !(ok = wait(&bars.acc_step, (step - 1) & 1))) break;
#pragma unroll
        for (int x = 0; x < 32; ++x) pk[x] = ptx::pack_bf16x2(pr[2 * x], pr[2 * x + 1]);
        ptx::tmem_st32(tY, pk);
        ptx::tmem_st_wait();
        arrive(&bars.p_ready);
      }
      if (!(ok = wait(&bars.dp_full, step & 1))) break;
      ptx::tmem_ld32(tDP, *reinterpret_cast<uint32_t(*)[32]>(u));
      ptx::tmem_ld32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(u + 32));
      ptx::tmem_ld_wait();
      arrive(&bars.dp_read);
      if constexpr (!kKeyRole) {
        if ((t + 1) * BT > len && len < p.Sk) {
          // what stands behind the last key may be NaN: out of dP, and out of the product with K
          const int lim = len - t * BT;
#pragma unroll
          for (int x = 0; x < 64; ++x)
            if (hf * 64 + x >= lim) u[x] = 0u;
          for (int c = 0; c < 3 && ok; ++c) ok = wait(&bars.ring_full[s][c], (step >> 1) & 1);
          if (!ok) break;
          if (r >= lim) {
            for (int c = hf; c < 3; c += 2) {
              uint4* row = reinterpret_cast<uint4*>(sm + kOffRing + (s * 3 + c) * kChunk + r * 128);
              for (int x = 0; x < 8; ++x) row[x] = make_uint4(0, 0, 0, 0);
            }
          }
          ptx::fence_proxy_async();
          __syncwarp();  // (the store of dS is the whole warp's, and the first step has no wait before it)
        }
      }
      // dS = P * (dP - D) as bf16 pairs
      if (kKeyRole) {
        const float4* dd = reinterpret_cast<const float4*>(vec + BT) + hf * 16;  // per query
#pragma unroll
        for (int x4 = 0; x4 < 16; ++x4) {
          const float4 d4 = dd[x4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = 2 * x4 + e;
            const uint64_t ds = ptx::mul2(ptx::f2(pr[2 * x], pr[2 * x + 1]),
                                          ptx::sub2(ptx::f2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])),
                                                    e == 0 ? ptx::f2(d4.x, d4.y) : ptx::f2(d4.z, d4.w)));
            pk[x] = ptx::pack_bf16x2(ptx::f2_lo(ds), ptx::f2_hi(ds));
          }
        }
      } else {
        const uint64_t d2 = ptx::f2(d_row, d_row);
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const uint64_t g = ptx::mul2(ptx::f2(pr[2 * x], pr[2 * x + 1]),
                                       ptx::sub2(ptx::f2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])), d2));
          pk[x] = ptx::pack_bf16x2(ptx::f2_lo(g), ptx::f2_hi(g));
        }
      }
      // dS into Y once its previous reader is done: dV(n) (key role: P' lives there) or
      // dQ(n-1)
      if (kKeyRole) {
        if (!(ok = wait(&bars.dv_done, step & 1))) break;
      } else if (n > 0 && !(ok = wait(&bars.acc_step, (step - 1) & 1))) {
        break;
      }
      ptx::tmem_st32(tY, pk);
      ptx::tmem_st_wait();
      arrive(&bars.ds_ready);
    }
    // ---------------------------------------------------------------- epilogue
    if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.acc_done, f.u & 1, abort_flag, p.err));
    if (ok) {
      ptx::tc_fence_after();
      const bool store = row_idx < rows;
      const size_t ro = ((size_t)b * rows + row_idx) * p.H + h;  // row of a [B, S, H, d] tensor
      if (kKeyRole) {
        // half 0: dV (4 chunks) and rope columns 0..31 of dK; half 1: dK nope (4 chunks) and
        // rope columns 32..63
#pragma unroll
        for (int c = 0; c < 5; ++c) {
          const uint32_t col = hf == 0 ? (c < 4 ? kColDV + 32 * c : kColAcc + 128)
                                       : (c < 4 ? kColAcc + 32 * c : kColAcc + 160);
          uint32_t w[32];
          ptx::tmem_ld32(tmem + lane_off + col, w);
          ptx::tmem_ld_wait();
          if (row_idx >= len) {  // lanes of no key
#pragma unroll
            for (int x = 0; x < 32; ++x) w[x] = 0u;
          }
          const float mul = c < 4 && hf == 0 ? 1.f : p.scale;
          uint16_t* to = hf == 0 ? p.dv : p.dk_nope;
          if (store) {
            if (c == 4)
              store_row(p.part_rope + (((size_t)bh * p.n_qs + share) * p.Sk + row_idx) * 64 + 32 * hf, w, mul, p.part_rope,
                        p.part_rope_bytes, p.err);
            else if (p.n_qs > 1)
              store_row(p.part_kv + ((size_t)unit * BT + r) * 256 + hf * 128 + 32 * c, w, mul, p.part_kv, p.part_kv_bytes,
                        p.err);
            else
              store_row(to + ro * 128 + 32 * c, w, mul, p.wide, to, p.k_bytes, p.err);
          }
          __syncwarp();
        }
      } else {
        // dQ: half 0 takes columns 0..95, half 1 columns 96..191 (nope 0..127, rope 128..191)
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const int cc = hf * 3 + c;
          uint32_t w[32];
          ptx::tmem_ld32(tmem + lane_off + kColAcc + 32 * cc, w);
          ptx::tmem_ld_wait();
          if (store) {
            if (p.n_ks > 1)
              store_row(p.part_q + ((size_t)unit * BT + r) * 192 + 32 * cc, w, p.scale, p.part_q, p.part_q_bytes, p.err);
            else if (cc < 4)
              store_row(p.dq_nope + ro * 128 + 32 * cc, w, p.scale, p.wide, p.dq_nope, p.q_bytes, p.err);
            else
              store_row(p.dq_rope + ro * 64 + 32 * (cc - 4), w, p.scale, p.wide, p.dq_rope, p.q_bytes / 2, p.err);
          }
          __syncwarp();
        }
      }
      arrive(&bars.acc_free);
    }
    f.ok = ok;
  }
  f.g += nsteps;
  ++f.u;
  f.after_key = kKeyRole;
}

__global__ void __launch_bounds__(kThreads, 1)
    cross_bwd_kernel(const __grid_constant__ CUtensorMap tm_qn,
                       const __grid_constant__ CUtensorMap tm_qr,
                       const __grid_constant__ CUtensorMap tm_kn,
                       const __grid_constant__ CUtensorMap tm_kr,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_do, const Params p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ Bars bars;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tm_qn);
    ptx::prefetch_tensormap(&tm_kn);
    bars.abort_flag = 0;
    ptx::mbar_init(&bars.fix3_full, 1);
    ptx::mbar_init(&bars.fix3_empty, 1);
    ptx::mbar_init(&bars.fix2_full, 1);
    ptx::mbar_init(&bars.fix2_empty, 1);
    for (int s = 0; s < 2; ++s) {
      for (int c = 0; c < 3; ++c) ptx::mbar_init(&bars.ring_full[s][c], 1);
      ptx::mbar_init(&bars.ring_empty[s], 1);
    }
    ptx::mbar_init(&bars.one_full[0], 1);
    ptx::mbar_init(&bars.one_full[1], 1);
    ptx::mbar_init(&bars.one_empty, 1);
    ptx::mbar_init(&bars.s_full, 1);
    ptx::mbar_init(&bars.x_read, 8);    // one arrival per elementwise warp
    ptx::mbar_init(&bars.dp_full, 1);
    ptx::mbar_init(&bars.dp_read, 8);
    ptx::mbar_init(&bars.acc_step, 1);
    ptx::mbar_init(&bars.p_ready, 8);
    ptx::mbar_init(&bars.dv_done, 1);
    ptx::mbar_init(&bars.ds_ready, 8);
    ptx::mbar_init(&bars.acc_done, 1);
    ptx::mbar_init(&bars.acc_free, 8);
    ptx::mbar_init(&bars.drained, 1);
    ptx::fence_barrier_init();
  }
  if (warp == 0) ptx::tmem_alloc(&bars.tmem_base, 512);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  wait_for_stream();
  const Maps m{&tm_qn, &tm_qr, &tm_kn, &tm_kr, &tm_v, &tm_do};
  // Within a role the tiles of one (b, h) are consecutive, so CTAs that run together stream the same (b, h)'s
  // tiles and find them in L2.
  Flow f;
  if (p.key_lens && p.n_qs == 1 && warp >= 2) {  // key tiles that no unit has, while the first tiles are on their way
    const int lane = threadIdx.x & 31, each = p.H * 32;  // 16-byte pieces of a key's dV and dK nope
    for (long long row = blockIdx.x * 8LL + warp - 2; row < (long long)p.B * p.Sk; row += gridDim.x * 8LL) {
      const int b = static_cast<int>(row / p.Sk), key = static_cast<int>(row - (long long)b * p.Sk);
      if (key < (key_len(p, b) + BT - 1) / BT * BT) continue;
      for (int i = lane; i < each; i += 32) {
        uint16_t* to = i < each / 2 ? p.dv : p.dk_nope;
        uint4* dst = reinterpret_cast<uint4*>(to + row * p.H * 128) + (i < each / 2 ? i : i - each / 2);
        if (MLA_STORE_OK(dst, to, p.k_bytes, p.err)) *dst = make_uint4(0, 0, 0, 0);
      }
    }
  }
  __shared__ Walk walks[kThreads / 32];
  Walk& walk = walks[warp];
  if (ptx::elect_one()) walk = {blockIdx.x, 0, 0};
  __syncwarp();
  bool key_role;
  int bh, tile, share;
  while (f.ok && next_unit(walk, p, key_role, bh, tile, share)) {
    const int b = bh / p.H, h = bh - b * p.H;
    if (key_role)
      bwd_body<true>(m, p, sm, bars, b, h, tile, share, (bh * p.nkt + tile) * p.n_qs + share, f);
    else
      bwd_body<false>(m, p, sm, bars, b, h, tile, share, (bh * p.nqt + tile) * p.n_ks + share, f);
  }
  // Nothing asynchronous outlives the CTA: commits arrive in its shared memory, and after an abort copies and
  // products may be under way that nobody waits for.
  if (warp < 2 && ptx::elect_one()) {
    if (warp == 1) {
      ptx::mma_commit(&bars.drained);
      ptx::mbar_wait_drain(&bars.drained, 0);
    } else if (!f.ok) {
      if (f.n_fix3 > 0) ptx::mbar_wait_drain(&bars.fix3_full, (f.n_fix3 - 1) & 1);
      if (f.n_fix2 > 0) ptx::mbar_wait_drain(&bars.fix2_full, (f.n_fix2 - 1) & 1);
      for (uint32_t v = f.n_ring > 2 ? f.n_ring - 2 : 0; v < f.n_ring; ++v)
        for (int c = 0; c < 3; ++c) ptx::mbar_wait_drain(&bars.ring_full[v & 1][c], (v >> 1) & 1);
      for (int c = 0; c < 2 && f.n_one > 0; ++c) ptx::mbar_wait_drain(&bars.one_full[c], (f.n_one - 1) & 1);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(bars.tmem_base, 512);
  }
}

// Adds what the units left in fp32.  The rope key's gradient of a key, a sum over heads and shares: 16 threads' loads cover
// its 64 columns, and kGroups such groups (one for four terms or fewer, up to a block's 16) take every kGroups-th
// term each, joined in group order; a block has 16 / kGroups keys at a time (with one key a block, however few terms, the
// gradient of 6 x 1 heads, 6 queries and up to 29241 keys took 274 us, so 118; one thread for all of 152 terms waited 150 loads
// long).  The shares'
// gradients of K and V, and of Q, where those were cut: a thread for four columns of a row.
template <int kGroups>
__global__ void __launch_bounds__(256) sum_kernel(const Params p) {
  __shared__ float4 sums[16][17];
  wait_for_stream();
  auto add = [](float4& a, const float4& v) { a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w); };
  auto put = [&](uint16_t* base, size_t at, size_t bytes, const float4& a) {
    uint2* dst = reinterpret_cast<uint2*>(base + at);
    if (MLA_STORE_OK(dst, base, bytes, p.err)) *dst = make_uint2(ptx::pack_bf16x2(a.x, a.y), ptx::pack_bf16x2(a.z, a.w));
  };
  const int c4 = threadIdx.x & 15, place = threadIdx.x >> 4, terms = p.H * p.n_qs;
  const int group = place % kGroups;
  constexpr int keys = 16 / kGroups;
  for (long long row0 = (long long)blockIdx.x * keys; row0 < (long long)p.B * p.Sk; row0 += (long long)gridDim.x * keys) {
    const long long row = row0 + place / kGroups;
    const int b = static_cast<int>(row / p.Sk), key = static_cast<int>(row - (long long)b * p.Sk);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (b < p.B && key < key_len(p, b)) {
      const float* src = p.part_rope + ((size_t)b * terms * p.Sk + key) * 64 + 4 * c4;
#pragma unroll 4
      for (int k = group; k < terms; k += kGroups)
        add(a, ptx::ld_l2(reinterpret_cast<const float4*>(src + (size_t)k * p.Sk * 64)));
    }
    if constexpr (kGroups > 1) {
      sums[place][c4] = a;
      __syncthreads();
      if (group == 0)
        for (int k = 1; k < kGroups; ++k) add(a, sums[place + k][c4]);
    }
    if (group == 0 && b < p.B) put(p.dk_rope, row * 64 + 4 * c4, p.rope_bytes, a);
    if constexpr (kGroups > 1) __syncthreads();
  }
  const long long n_kv = p.n_qs > 1 ? (long long)p.B * p.Sk * p.H * 64 : 0;
  const long long n_q = p.n_ks > 1 ? (long long)p.B * p.Sq * p.H * 48 : 0;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n_kv + n_q;
       i += (long long)gridDim.x * blockDim.x) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n_kv) {
      const long long bkh = i >> 6;  // (b, key, h)
      const int c = (i & 63) * 4, h = static_cast<int>(bkh % p.H);
      const long long bk = bkh / p.H;
      const int b = static_cast<int>(bk / p.Sk), key = static_cast<int>(bk - (long long)b * p.Sk);
      if (key < key_len(p, b)) {
        const size_t unit = (((size_t)b * p.H + h) * p.nkt + key / BT) * p.n_qs;
#pragma unroll 4
        for (int s = 0; s < p.n_qs; ++s)
          add(a, ptx::ld_l2(reinterpret_cast<const float4*>(p.part_kv + ((unit + s) * BT + key % BT) * 256 + c)));
      }
      put(c < 128 ? p.dv : p.dk_nope, bkh * 128 + (c & 127), p.k_bytes, a);
    } else {
      const long long at = i - n_kv, bqh = at / 48;  // (b, query, h)
      const int c = static_cast<int>(at - bqh * 48) * 4, h = static_cast<int>(bqh % p.H);
      const long long bq = bqh / p.H;
      const int b = static_cast<int>(bq / p.Sq), q = static_cast<int>(bq - (long long)b * p.Sq);
      const int len = key_len(p, b), tiles = (len + BT - 1) / BT, rows = p.few_chunk ? p.Sq : BT;
      const size_t unit = (((size_t)b * p.H + h) * p.nqt + q / BT) * p.n_ks;
#pragma unroll 4
      for (int s = 0; s < p.n_ks; ++s)
        if (p.few_chunk ? (long long)s * p.few_chunk < len : share_begin(tiles, s, p.n_ks) < share_begin(tiles, s + 1, p.n_ks))
          add(a, ptx::ld_l2(reinterpret_cast<const float4*>(p.part_q + ((unit + s) * rows + q % BT) * 192 + c)));
      if (c < 128)
        put(p.dq_nope, bqh * 128 + c, p.q_bytes, a);
      else
        put(p.dq_rope, bqh * 64 + (c - 128), p.q_bytes / 2, a);
    }
  }
}

}  // namespace sm103_cross_bwd
}  // namespace mla

#include "cross_backward_few_sm103.cuh"

namespace mla {
namespace sm103_cross_bwd {

// How a call is cut: the tiles that one CTA streams go in shares where their
// steps would last longer than half of what an SM has to do in all.
struct Cut {
  int nqt, nkt, n_qs, n_ks, few_chunk;
  long long key_units, query_units;
};
constexpr int kLeastSteps = 4;

inline Cut cut_of(int B, int H, int Sq, int Sk, int sms) {
  Cut c = {};
  c.nqt = (Sq + BT - 1) / BT;
  c.nkt = (Sk + BT - 1) / BT;
  // Few queries and keys without tiles (microseconds as tiles and without, 8 | 32 queries: 53 x 56 heads, up to 9 keys 236 | 246, so
  // 35 | 80; 26 x 15 x up to 112 45 | 45, so 21 | 25; 8 x 16 x 1000 81 | 86, not 93 | 110; 33 | 64: 37 x 49 x 13 121 | 128, so 68 | 89;
  // 64 x 64 x 40 270 | 280, not 244 | 286; 11 x 48 x 128 57 | 59, not 97 | 121).  Towards its ends the rule errs where heads fill two
  // CTAs an SM once and a bit: 11 x 48 x 128, 8 queries 54, so 46, but 32 queries 56, and 63 without; 4 x 99 x up to 512, 8
  // queries 92, and 115 without.
  if ((Sq <= 16 && Sk <= 512) || (Sq <= 32 && Sk <= 256) || (Sq <= kFewRows && Sk <= kFewKeys / 2)) {
    // runs of whole steps, two CTAs an SM; a CTA takes about as long as three steps beside its own, a sum of shares as two
    const long long items = (long long)B * H, slots = 2LL * sms;
    const int steps = (Sk + kFewKeys - 1) / kFewKeys;
    double best = 1e300;
    for (long long s = 1; s <= steps && (s == 1 || items * s <= 4 * slots); ++s) {
      const double cost = (double)((items * s + slots - 1) / slots) * ((double)((steps + s - 1) / s) + 3) + (s > 1 ? 2 + s / 16. : 0);
      if (cost < best) {
        best = cost;
        c.few_chunk = (int)std::min((steps + s - 1) / s * kFewKeys, 0x7fffffc0LL);
      }
    }
    c.n_qs = 1;
    c.n_ks = (int)(((long long)Sk + c.few_chunk - 1) / c.few_chunk);
    c.key_units = 0;
    c.query_units = items * c.n_ks;
    return c;
  }
  const double each = (double)B * H * c.nqt * c.nkt / sms;  // half of both roles' steps, an SM
  const double most = each > kLeastSteps ? each : kLeastSteps;
  c.n_qs = c.nqt > most ? (int)(c.nqt / most + 0.999) : 1;
  c.n_ks = c.nkt > most ? (int)(c.nkt / most + 0.999) : 1;
  c.key_units = (long long)B * H * c.nkt * c.n_qs;
  c.query_units = (long long)B * H * c.nqt * c.n_ks;
  return c;
}

}  // namespace sm103_cross_bwd

// ---------------------------------------------------------------- host side

cudaError_t encode_tensor_map(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* ptr,
                              const uint64_t* dims, const uint64_t* strides, const uint32_t* box);

namespace {
// [B, S, H, d] tensor of bf16, box = 64 columns x 1 head x 128 tokens
bool cross_bwd_map(CUtensorMap* m, const void* p, int B, int S, int H, int d) {
  uint64_t dims[4] = {(uint64_t)d, (uint64_t)H, (uint64_t)S, (uint64_t)B};
  uint64_t strides[3] = {(uint64_t)d * 2, (uint64_t)H * d * 2, (uint64_t)S * H * d * 2};
  uint32_t box[4] = {64, 1, sm103_cross_bwd::BT, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box) == cudaSuccess;
}
}  // namespace

// Whether the units of such a call can be numbered.
bool cross_bwd_fits(int B, int H, int Sq, int Sk) {
  return (long long)B * H * ((Sq + 127) / 128 + (long long)((Sk + 127) / 128)) <= 0x40000000LL;
}

namespace {
struct CrossBwdWorkspace {
  size_t nlse2, dvec, rope, kv, q, bytes;  // offsets, and the whole
  CrossBwdWorkspace(const sm103_cross_bwd::Cut& c, int B, int H, int Sq, int Sk) {
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t here = at;
      at += (n + 255) / 256 * 256;
      return here;
    };
    const size_t vec = c.few_chunk ? 0 : (size_t)B * H * c.nqt * sm103_cross_bwd::BT * sizeof(float);
    nlse2 = take(vec);
    dvec = take(vec);
    rope = take((size_t)B * H * c.n_qs * Sk * 64 * sizeof(float));
    kv = take(c.n_qs > 1 ? (size_t)c.key_units * sm103_cross_bwd::BT * 256 * sizeof(float) : 0);
    q = take(c.n_ks > 1 ? (size_t)c.query_units * (c.few_chunk ? Sq : sm103_cross_bwd::BT) * 192 * sizeof(float) : 0);
    bytes = at + 32;
  }
};
}  // namespace

size_t cross_bwd_workspace_bytes(int B, int H, int Sq, int Sk, int sms) {
  return CrossBwdWorkspace(sm103_cross_bwd::cut_of(B, H, Sq, Sk, sms), B, H, Sq, Sk).bytes;
}

// Of a call's plan, for tests: 0 without tiles, 1 by tiles.
int cross_bwd_form(int B, int H, int Sq, int Sk, int sms, int* query_shares, int* key_shares) {
  const sm103_cross_bwd::Cut c = sm103_cross_bwd::cut_of(B, H, Sq, Sk, sms);
  *query_shares = c.n_qs;
  *key_shares = c.n_ks;
  return c.few_chunk > 0 ? 0 : 1;
}

cudaError_t launch_cross_bwd_sm103(const void* q_nope, const void* q_rope, const void* k_nope, const void* k_rope,
                                   const void* v, const int* key_lens, const void* out, const float* lse,
                                   const void* d_out, void* dq_nope, void* dq_rope, void* dk_nope, void* dk_rope,
                                   void* dv, int B, int H, int Sq, int Sk, float softmax_scale, void* workspace, int sms,
                                   unsigned int* err, cudaStream_t stream) {
  using namespace sm103_cross_bwd;
  const Cut c = cut_of(B, H, Sq, Sk, sms);
  const CrossBwdWorkspace w(c, B, H, Sq, Sk);
  CUtensorMap tqn, tqr, tkn, tkr, tv, tdo;
  uint64_t kr_dims[3] = {64, (uint64_t)Sk, (uint64_t)B};
  uint64_t kr_strides[2] = {64 * 2, (uint64_t)Sk * 64 * 2};
  uint32_t kr_box[3] = {64, BT, 1};
  if (c.few_chunk == 0 &&
      (!cross_bwd_map(&tqn, q_nope, B, Sq, H, 128) || !cross_bwd_map(&tqr, q_rope, B, Sq, H, 64) ||
      !cross_bwd_map(&tkn, k_nope, B, Sk, H, 128) || !cross_bwd_map(&tv, v, B, Sk, H, 128) ||
      !cross_bwd_map(&tdo, d_out, B, Sq, H, 128) ||
      encode_tensor_map(&tkr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, k_rope, kr_dims, kr_strides, kr_box) != cudaSuccess))
    return cudaErrorInvalidValue;
  // (the workspace is 16-byte aligned, its parts 32)
  char* base = static_cast<char*>(workspace) + (reinterpret_cast<uintptr_t>(workspace) & 16);
  auto at = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  Params p = {};
  p.nlse2 = at(w.nlse2);
  p.dvec = at(w.dvec);
  p.dq_nope = static_cast<uint16_t*>(dq_nope);
  p.dq_rope = static_cast<uint16_t*>(dq_rope);
  p.dk_nope = static_cast<uint16_t*>(dk_nope);
  p.dk_rope = static_cast<uint16_t*>(dk_rope);
  p.dv = static_cast<uint16_t*>(dv);
  p.err = err;
  p.B = B;
  p.H = H;
  p.Sq = Sq;
  p.nqt = c.nqt;
  p.q_pad = c.nqt * BT;
  p.Sk = Sk;
  p.nkt = c.nkt;
  p.n_qs = c.n_qs;
  p.n_ks = c.n_ks;
  p.few_chunk = c.few_chunk;
  p.key_lens = key_lens;
  const void* grads[] = {dq_nope, dq_rope, dk_nope, dv};
  p.wide = 1;
  for (const void* g : grads) p.wide &= (reinterpret_cast<uintptr_t>(g) & 31) == 0;
  p.q_bytes = (size_t)B * Sq * H * 128 * 2;
  p.q_bytes -= std::min(p.q_bytes, testing_out_shrink());
  p.k_bytes = (size_t)B * Sk * H * 128 * 2;
  p.rope_bytes = (size_t)B * Sk * 64 * 2;
  p.part_rope_bytes = w.kv - w.rope;
  p.part_kv_bytes = w.q - w.kv;
  p.part_q_bytes = w.bytes - 32 - w.q;
  p.part_rope = at(w.rope);
  p.part_kv = at(w.kv);
  p.part_q = at(w.q);
  p.scale = softmax_scale;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.n_query_units = (int)c.query_units;
  const long long units = c.key_units + c.query_units;
  p.by_lens = key_lens && units > sms;
  if (units > 0x7fff0000LL) return cudaErrorInvalidConfiguration;
  cudaError_t e;
  if (c.few_chunk) {
    auto at16 = [](const void* x) { return static_cast<const uint16_t*>(x); };
    const FewInputs in{at16(q_nope), at16(q_rope), at16(k_nope), at16(k_rope), at16(v), at16(out), at16(d_out), lse};
    static unsigned long long few_set[3] = {0, 0, 0};
    const int rows = Sq <= 16 ? 0 : Sq <= 32 ? 1 : 2;
    auto kernel = rows == 0 ? few_rows_kernel<16> : rows == 1 ? few_rows_kernel<32> : few_rows_kernel<64>;
    const int bytes = rows == 0 ? FewSmem<16>::kBytes : rows == 1 ? FewSmem<32>::kBytes : FewSmem<64>::kBytes;
    e = smem_attr_once(kernel, bytes, &few_set[rows]);
    if (e != cudaSuccess) return e;
    e = launch_dependent_smem(kernel, (int)units, 256, bytes, stream, in, p);
    if (e != cudaSuccess) return e;
  } else {
    const long long tasks = (long long)B * H * (p.q_pad / 8);
    if ((tasks + 7) / 8 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    static unsigned long long smem_set = 0;
    e = smem_attr_once(cross_bwd_kernel, kSmemAlloc, &smem_set);
    if (e != cudaSuccess) return e;
    e = launch_dependent(prep_kernel, (int)((tasks + 7) / 8), 256, stream, static_cast<const uint16_t*>(out),
                         static_cast<const uint16_t*>(d_out), lse, at(w.nlse2), at(w.dvec), B, H, Sq, p.q_pad);
    if (e != cudaSuccess) return e;
    e = launch_dependent_smem(cross_bwd_kernel, (int)(units < sms ? units : sms), kThreads, kSmemAlloc, stream, tqn,
                              tqr, tkn, tkr, tv, tdo, p);
    if (e != cudaSuccess) return e;
  }
  const long long cut = (c.n_qs > 1 ? (long long)B * Sk * H * 64 : 0) + (c.n_ks > 1 ? (long long)B * Sq * H * 48 : 0);
  // four terms a group, fewer while there are blocks for it
  const long long keys = (long long)B * Sk, terms = (long long)H * c.n_qs;
  int groups = 1;
  while (groups < 16 && groups < terms && (groups * 4 < terms || keys * groups < 16 * 4LL * sms)) groups *= 2;
  const long long blocks = std::max((keys * groups + 15) / 16, (cut + 255) / 256);
  auto sum = groups == 1   ? sum_kernel<1>
             : groups == 2 ? sum_kernel<2>
             : groups == 4 ? sum_kernel<4>
             : groups == 8 ? sum_kernel<8>
                           : sum_kernel<16>;
  return launch_dependent(sum, (int)std::min(blocks, 8LL * sms), 256, stream, p);
}

}  // namespace mla
