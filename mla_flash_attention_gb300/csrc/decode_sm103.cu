// Absorbed MLA decode over the paged latent cache on tcgen05 / TMEM: split-KV, with the
// log-sum-exp merge of the splits done by the last split of each sequence to finish.
//
// Each work unit (a contiguous range of pages from the split plan) is served by a pair
// of CTAs that differ only in which half of the 512 latent output columns they own:
// O (128 query rows x 512 fp32) is exactly the 512-column TMEM, so one CTA cannot also
// hold the scores.  Both CTAs of a pair compute the full scores S = Q C' (the redundant
// part) and their own half of O += P C[:, half].  Query rows are the (token, head) pairs
// of one sequence, padded to the MMA's M = 128.
//
// Per CTA (8 warps; 12 with the fp8 cache):
//   warp 0      TMA producer: each sequence's Q latent 0..255 (staged in shared memory),
//               then the cache pages (64 keys x 576 columns) -- bf16: in two parts, the
//               five score-only 64-column chunks and the CTA's four value chunks, 128B-
//               swizzled, ready for the MMA; fp8: the whole raw page into the upper half of
//               a stage -- plus L2 prefetch of pages ahead
//   warp 1      MMA issuer: at a sequence change, copies the staged Q latent 0..255 into
//               TMEM (tcgen05.cp) and loads latent 256..511 + rope into shared memory by TMA;
//               then S(g) = Q C(g)' into one of two S buffers (A operand = Q: latent 0..255
//               from TMEM, the rest from shared memory), and O_half += P(g) C(g)[:, half]
//               with P read from TMEM.  S(g+1) and PV(g) are issued in whichever order their
//               inputs arrive.
//   warps 2-3   stage preparation: zero the rows past the sequence end of a partial page;
//   (+ 8-11)    fp8: widen the page to bf16 in place (three lockstep steps of three
//               64-column chunks, 16-byte granules spread over the preparation threads;
//               warps 8-11 exist in the fp8 kernel only, and softmax warps whose 32 rows
//               are all padding of the M = 128 MMA join them) and stage its scales
//   warps 4-7   softmax, one thread per query row; they also write the split's partial
//               (O_half / l, log-sum-exp), column quads of 32 rows per 512-byte store, and,
//               in the CTA that completes a (sequence, column half), merge its splits into
//               the bf16 output and the LSE
// Two further instances serve a tree of drafted tokens (kTree): which of the n newest keys a row
// sees comes from a bit mask a token instead of the diagonal, and the pages that hold drafted keys
// pass through warps 2 and 3, which take non-finite values out of them (a zero weight times such a
// value would reach rows that do not see the key) and flag their keys, so that the rows that see
// them, and no others, come out as NaN.  They also write the rows of items without keys.
// The tree over an fp8 cache (kF8) widens nothing: the e4m3 page is the MMA's operand as it lies.
// Its other operands are sums of two 8-bit terms: a bf16 query, scaled by a power of two into
// [128, 256) at its row's largest value, is two e4m3 terms exactly (8 significant bits, 4 + 4) down to 2^-10
// of that value (2^-17 of it is lost at most); a weight P'' = p ks is hi (e4m3) + lo (e5m2) to 2^-8 of
// itself, as a bf16 weight is (and see kF8StepsPerMass for small weights).  Twice the k-steps at twice the
// rate: the tensor work is bf16's, pages take half the bytes, and four fit instead of two; each page is its
// own stage, released by its PV product.  Warps 8-11 make the query terms.  64 ragged
// sequences of up to 16384 keys, 1 to 13 tokens of 16 heads: 613 us with the pages widened to bf16, 433
// with e4m3 operands (an item's query terms then took 20 us), 344 with the terms made in place from
// TMA loads and items charged in the split plan, 255 with tiles of padding left out, 250 with the ends of
// items shortened, 255 with the range of the weights above (two e4m3 terms before, which lost small
// weights).  A page takes 1.3 us, 2,500 clocks for 2,240 of MMAs.  (Two softmax warpgroups, a key
// half each, were no faster, nor was splitting into terms with integer instructions.)
// TMEM columns: [0,128) Q latent 0..255 (bf16 pairs), [128,256) two S / P buffers of 64,
// [256,512) O half.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "decode_plan.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace sm103_decode {

using decode_plan::Plan;
using decode_plan::SegmentsOf;
using decode_plan::clamp_len;
using decode_plan::make_plan;
constexpr int kPage = decode_plan::kPage;
constexpr int kDl = 512, kDc = 576, kRows = 128;
constexpr int kPageChunk = kPage * 128;       // 64 rows x 64 bf16 (8 KB), 128B-swizzled
constexpr int kStageBytes = 9 * kPageChunk;   // 72 KB
constexpr int kRawChunk = kPage * 64;         // 64 rows x 64 fp8 bytes (4 KB), unswizzled
constexpr int kRawOffset = 9 * kRawChunk;     // fp8 page lands in the upper 36 KB of a stage
constexpr int kStages = 2;
constexpr int kQChunk = kRows * 128;          // 128 rows x 64 bf16 (16 KB)
constexpr int kOffQhi = 0;                    // latent 256..511 (4 chunks) + rope (1 chunk)
constexpr int kOffStage = 5 * kQChunk;        // 80 KB
constexpr int kSmemBytes = kOffStage + kStages * kStageBytes;  // 224 KB
// bf16 pages arrive in two parts: the score-only chunks (the other column half's four latent
// chunks and the rope chunk, 40 KB) into one slot, free again once the score MMAs that read
// them are done, and this CTA's own four latent chunks (32 KB), which the PV product reads
// too, into a ring of three, so that they land two pages ahead of their use.
constexpr int kSPartBytes = 5 * kPageChunk;
constexpr int kVPartBytes = 4 * kPageChunk;
constexpr int kVSlots = 3;
constexpr int kOffSPart = kOffStage;
constexpr int kOffVPart = kOffStage + kSPartBytes;
static_assert(kOffVPart + kVSlots * kVPartBytes <= kSmemBytes, "bf16 page parts fit the stages");
// position of 64-column chunk c (0..8) within its part, for column half `half`: the value
// chunks 4 half .. 4 half + 3 in order; the score-only ones (half 0: 4..8, half 1: 0..3, 8)
__host__ __device__ constexpr int chunk_idx(int c, int half) {
  return ((c >> 2) == half && c < 8) ? c - 4 * half : (half == 0 ? c - 4 : (c < 4 ? c : 4));
}
constexpr int kSmemAlloc = kSmemBytes + 1024;
// kF8: pages of four 128-column chunks (64 rows x 128 bytes, 128B-swizzled) and the rope columns
// (64 rows x 64 bytes, 64B-swizzled), four of them; Q's smem part: latent 256..383 as a hi and a lo
// chunk, latent 384..511 likewise, then one chunk with the rope's hi and lo terms
constexpr int kF8Page = 4 * kPageChunk + kPage * 64;  // 36 KB
constexpr int kF8Stages = 4;
static_assert(kF8Stages * kF8Page <= kStages * kStageBytes, "fp8 tree pages fit the stages");
// Flat pages the tree's split plan charges for an item's start and end (its queries, the epilogue, and
// for fp8 the query terms), at most: a page of keys takes 1.4 us (bf16) and 1.3 us (fp8).  64 ragged
// sequences of up to 16384 keys, fp8: 256, 257, 254 and 261 us for 10, 12, 13 and 16; 16 of up to 8000
// keys and 8 x 128 rows, bf16: 158, 159, 151 and 150 us for 4, 5, 6 and 8.
constexpr int kF8ItemCost = 13, kTreeItemCost = 8;
// registers a thread: 384 threads launched at kF8RegsLaunch, then traded between the warpgroups
constexpr int kF8RegsLaunch = 168, kF8RegsHigh = 232, kF8RegsLow = 136;
static_assert(128 * kF8RegsHigh + 256 * kF8RegsLow <= 384 * kF8RegsLaunch, "register split");
// bf16: 8 warps; fp8: 12 (four more preparation warps)
template <bool kFp8> constexpr int kThreadsOf = kFp8 ? 384 : 256;
template <bool kFp8> constexpr int kPrepOf = kFp8 ? 192 : 64;
// A tree's item in at most this many splits is merged by the split that finishes last, from its
// accumulator and one bulk copy, if there are more items than half the units.  With fewer (few) the merge
// kernel is done sooner than that split, whose unit has nothing else to do meanwhile: 6 ragged
// sequences of up to 1432 keys, 8 x 16 rows, 31 -> 22 us; 160 items of up to 2000 keys, 84 -> 91 us.
constexpr int kFusedSplits = 2;
constexpr int kPrefetchAhead = 4;             // pages warmed in L2 ahead of their load
// Limit of the waits of a role that has nothing to do between an item's start and its last pages, in SM
// clocks: an item of 2^25 pages takes 50 s.  The others wait for a page at a time, each half a second at
// most, and what makes one of them give up ends these waits too (the abort flag).
constexpr long long kItemWait = 200000000000LL;

struct Params {
  const uint16_t* q_latent;  // [B, T, H, 512]
  const uint16_t* q_rope;    // [B, T, H, 64]
  const float* kv_scale;     // [num_pages, 64] (fp8 path)
  const unsigned char* cache_bytes;  // the cache as bytes: page g at g * 64 * 576 * element size
  const int* page_table;
  const int* cache_lens;
  float* part_o;
  float* part_lse;   // [2][n_slots][TQ]: each column half writes its own copy
  // tree: how many items are left to the merge kernel (.x of the first entry, zeroed per call), then
  // {item, first unit, splits} of each, at most one a unit.  They lie in the last of the n_slots
  // slots of part_o, which no split uses (unit c and item v share slot c + v <= G - 1 + B * NQT - 1).
  int4* deferred;
  // tree: at most half as many items as units.  Every item in several splits is left to the merge
  // kernel, and entry 1 + v is item v's, whatever its splits (0: no keys), so that nothing has to be
  // zeroed before this launch; the split kernel is then itself the one that waits for the work ahead.
  int few;
  int* counters;     // [B * NQT][2]: finished splits per (virtual sequence, half), zeroed per call
  uint16_t* out;     // [B, T, H, 512] bf16
  float* lse;        // [B, H, T]
  unsigned int* err;
  int B, H, T, max_pages, num_pages, causal, G;
  int NQT, TQ;  // query tiles per sequence (T*H rows in tiles of 128) and rows per tile
  int n_slots;  // partial slots: G + B * NQT
  float scale_log2;
  // drafted tree: bit j of row t says whether token t sees drafted key j
  const uint32_t* tree_mask;  // [B or 1][T][mask_words]
  long long mask_stride;      // words from one sequence's mask to the next (0: one for all)
  int mask_words;
  const int* new_lens;        // [B] drafted tokens of each sequence, or null (T each)
  int page_box;  // 1: a page is one box of the 3-D cache map (else nine boxes of the 2-D one)
  int item_cost;  // flat pages the split plan charges per work item (see decode_plan.cuh)
  // buffer sizes for the store checks of the bounds-checked build
  size_t out_bytes, lse_bytes, part_o_bytes, part_lse_bytes, counters_bytes;
};

struct F8Bars {
  uint64_t full[kF8Stages], empty[kF8Stages];
  uint64_t q_lo_raw, q_raw;                 // a segment's raw rows landed in the ring and in the query area
  uint64_t q0_sync;                         // first segment: both warpgroups have read their raw rows
  signed char q_exp[2][kRows];              // the power of two a query row was scaled by, by segment parity
  float ks[kRows / 32][kPage], lk[kRows / 32][kPage];  // a page's key scales and their log2, a copy a softmax warp
};
struct NoBars {};
template <bool kF8> struct F8Part { using type = NoBars; };
template <> struct F8Part<true> { using type = F8Bars; };

template <bool kFp8, bool kTree>
struct Bars {
  // stage_ready[s][k]: bf16 pages are ready at once (k = 0); fp8 pages in three parts, k = 0..2
  // covering 64-column chunks 3k..3k+2, as the in-place widening completes them
  uint64_t stage_full[kStages], stage_ready[kStages][3], stage_empty[kStages];
  // bf16 page parts: the score-only slot and the ring of this half's value chunks; a page
  // that ends a sequence part-way is handed to the preparation warps (zero_go) and back once
  // the rows past the end are zeroed (zeroed), one phase each per such page
  uint64_t spart_full, spart_empty;
  uint64_t vpart_full[kVSlots], vpart_empty[kVSlots];
  uint64_t zero_go, zeroed;
  uint64_t s_full[2], p_full[2], o_done, seg_done, conv_sync;
  uint64_t q_free, q_lo_full, q_cp_done, q_hi_full;  // per-sequence Q staging
  uint64_t q0_copied;  // the first sequence's staged Q is in TMEM (one phase per launch)
  uint64_t part_done, merge_go;  // partial written by the 4 softmax warps / merge decision
  uint64_t dec_go;               // the segment's merge path decided
  uint64_t merge_full;           // the other split's partial copied into shared memory
  int merge_last, merge_fast, merge_bulk;
  uint32_t tmem_base;
  int abort_flag;
  Plan plan;
  float kscale[kFp8 && !kTree ? kStages : 1][kFp8 && !kTree ? kPage : 1];
  unsigned char key_nan[kTree ? 2 : 1][kPage];  // tree: 1 where a drafted key holds a non-finite value
  typename F8Part<kFp8 && kTree>::type f8;
};

// with 224 KB of dynamic shared memory and no slack, what the fp8 tree's block has left
static_assert(kSmemBytes + sizeof(Bars<true, true>) <= 227 * 1024, "static shared memory of the fp8 tree");

// Drafted tokens of virtual sequence v: the newest n keys; rows of tokens n .. T - 1 are padding.
__device__ __forceinline__ int drafted(const Params& p, int vseq) { return decode_plan::drafted_of(p, vseq / p.NQT); }

// Bits j .. j + 63 of a row's tree mask, 0 past its words (j >= 0).
__device__ __forceinline__ unsigned long long mask_bits(const uint32_t* row, int words, int j) {
  const int w = j >> 5, sh = j & 31;
  auto word = [&](int i) { return i < words ? __ldg(row + i) : 0u; };
  const uint32_t a = word(w), b = word(w + 1), c = word(w + 2);
  return __funnelshift_r(a, b, sh) | static_cast<unsigned long long>(__funnelshift_r(b, c, sh)) << 32;
}

// Does a 16-byte granule hold a non-finite value (bf16: NaN or infinity; e4m3: NaN)?
template <bool kFp8>
__device__ __forceinline__ bool granule_nonfinite(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kFp8) {
      // a byte is NaN iff its low 7 bits are all set: adding 1 to them carries into bit 7
      bad |= (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
    } else {
      bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    }
  }
  return bad;
}

__device__ __forceinline__ int page_of(const Params& p, int vseq, int pg) {
  return __ldg(p.page_table + (size_t)(vseq / p.NQT) * p.max_pages + pg);
}
__device__ __forceinline__ int row_of_page(const Params& p, int page) {
  // an out-of-range page reads as zeros (coordinates outside the tensor) and is masked
  return (page >= 0 && page < p.num_pages) ? page * kPage : -2 * kPage;
}
__device__ __forceinline__ int page_row(const Params& p, int vseq, int pg) {
  return row_of_page(p, page_of(p, vseq, pg));
}

// Sixteen bf16 (times alpha, a power of two) as their hi and lo e4m3 terms, 16 bytes each.  Cut in two
// rather than hi rounded and the rest taken from its code: two conversions a pair instead of four, 253
// against 262 us for 32 sequences of 300 keys and 32 x 128 rows.  Values too small for two exact terms
// come out to 2^-9, 2^-16 of their row's largest.
__device__ __forceinline__ void split16(const uint4& w0, const uint4& w1, float alpha, uint4& hi, uint4& lo) {
  const uint32_t in[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  const uint64_t a2 = ptx::f2(alpha, alpha);
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = ptx::mul2(ptx::f2(__uint_as_float(in[2 * i] << 16), __uint_as_float(in[2 * i] & 0xffff0000u)), a2);
    const uint64_t y =
        ptx::mul2(ptx::f2(__uint_as_float(in[2 * i + 1] << 16), __uint_as_float(in[2 * i + 1] & 0xffff0000u)), a2);
    ptx::cut_e4m3x4(x, y, h[i], l[i]);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Two terms hold a weight P'' to 2^-8 of itself down to 2^-6, and to 2^-14 below (split_e4m3_e5m2x4): the 64
// keys of a page lose at most 2^-8 more, and at most 2^-3 of 64 times the page's largest P''.  That is
// nothing beside a largest weight of 2^5, but thousands of keys far below a dominating one would lose
// much of what they hold together.  So each row counts its pages by what they may lose (f8_steps, in
// units of 2^-8) and sums the pages' largest weights (f8_mass, in units of 2^5), both relative to its
// reference m.  Once there are more than kF8StepsPerMass of the one to the other, m falls to kF8FallTo above the
// maximum of the next page that lies low (the accumulator, in fp32, is scaled up), and the count starts
// again: between two falls at most 2^-9 of the sum of the pages' largest weights is lost.  m falls by 16
// bits at most at a time, and then only a mass as much larger lets it fall again, so O stays below
// 2^90; and it does not fall where the sum of p = P'' / ks is huge because the key scales are tiny.
// A fall costs what a rise does.  With kF8FallTo of 4 the scores of normal queries and keys hardly ever
// cause one (64 ragged sequences of up to 16384 keys: 255 us, as without falls; 261 with 0, as many rises
// follow); with scores of four times the spread 275 to 280 us instead of 265.
constexpr float kF8StepsPerMass = 16.f, kF8FallTo = 4.f;

constexpr int kQNonFinite = 127;  // q_exp of a row with a NaN or an infinity: all its terms are NaN

// The factor 2^k of a row's terms.
__device__ __forceinline__ float q_factor(int k) {
  return k == kQNonFinite ? __int_as_float(0x7fc00000) : __int_as_float((k + 127) << 23);
}

// Granule i of row r in a chunk of the query area (128 rows of 128 bytes, 128B-swizzled).
__device__ __forceinline__ uint4* q_granule(unsigned char* base, int r, int chunk, int i) {
  return reinterpret_cast<uint4*>(base + chunk * kQChunk + r * 128 + ((i ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t larger(uint32_t mx, const uint4& w) {  // magnitudes as integers, two a word
  return __vmaxu2(__vmaxu2(__vmaxu2(mx, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu),
                  __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}

// The largest exponent field (0 .. 255) of row r's bf16 values in chunks 0 .. n - 1.
__device__ __forceinline__ int q_field(unsigned char* base, int r, int n) {
  uint32_t mx = 0;
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = larger(mx, *q_granule(base, r, c, i));
  }
  return static_cast<int>(max(mx & 0xffffu, mx >> 16) >> 7);
}

// The same over whole query rows row0 + lane (lane < rows), read from memory by one warp, eight rows at a
// time: the next segment's, while this one's pages are under way.
__device__ __forceinline__ int q_field_ahead(const Params& p, size_t row0, int rows) {
  const int lane = threadIdx.x & 31;
  int field = 0;
#pragma unroll 1
  for (int b = 0; b < rows; b += 8) {
    uint4 w[8][2], rope[2];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q_latent + (row0 + b + i) * kDl) + lane;
      w[i][0] = b + i < rows ? __ldg(src) : zero;
      w[i][1] = b + i < rows ? __ldg(src + 32) : zero;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // rope: a row's 128 bytes in eight lanes
      const int at = b + 4 * i + (lane >> 3);
      rope[i] = at < rows ? __ldg(reinterpret_cast<const uint4*>(p.q_rope + (row0 + at) * 64) + (lane & 7)) : zero;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t mx = larger(larger(0, w[i][0]), w[i][1]);
      if ((lane >> 3) == (i & 3)) mx = larger(mx, rope[i >> 2]);
      mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
      if (lane == b + i) field = static_cast<int>(mx >> 7);
    }
  }
  return field;
}

// The power of two that a row with this largest field is scaled by (field 255: NaN or infinity).
__device__ __forceinline__ int q_exponent(int field) {
  return field == 255 ? kQNonFinite : min(max(134 - field, -120), 120);
}

// Row r's raw chunks 0 and 1 (64 columns of bf16 each) at p0, then those at p1, become a hi and a lo
// chunk; 0 where the row is not live.
__device__ __forceinline__ void q_turn(unsigned char* p0, unsigned char* p1, int r, float f, bool live) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    unsigned char* base = c ? p1 : p0;
    uint4 raw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) raw[i] = live ? *q_granule(base, r, i >> 3, i & 7) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint4 h, l;
      split16(raw[2 * i], raw[2 * i + 1], f, h, l);
      *q_granule(base, r, 0, i) = h;
      *q_granule(base, r, 1, i) = l;
    }
  }
}

// The same for the rope chunk: 64 columns, hi and lo in one chunk.
__device__ __forceinline__ void q_turn_rope(unsigned char* base, int r, float f, bool live) {
  uint4 raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) raw[i] = live ? *q_granule(base, r, 4, i) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 h, l;
    split16(raw[2 * i], raw[2 * i + 1], f, h, l);
    *q_granule(base, r, 4, i) = h;
    *q_granule(base, r, 4, 4 + i) = l;
  }
}

// Tree: an item without keys (a query tile of padding, an empty sequence) is in no work unit's range.
// Unit u writes O = 0 and LSE = -inf for the items u, u + G, u + 2G, ... that are empty, each half its
// columns, by its warps 2 and 3, which have the least to do.
__device__ __forceinline__ void empty_items(const Params& p, int unit, int half, int TH) {
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 2;
  for (int v = unit; v < p.B * p.NQT; v += p.G) {
    if (decode_plan::item_len<true>(p, v) > 0) continue;
    const int b = v / p.NQT, row0 = (v % p.NQT) * kRows, rows = min(kRows, TH - row0);
    uint4* o = reinterpret_cast<uint4*>(p.out + ((size_t)b * TH + row0) * kDl + half * 256) + lane;
    for (int i = w; i < rows; i += 2)
      if (MLA_STORE_OK(o + i * (kDl / 8), p.out, p.out_bytes, p.err)) o[i * (kDl / 8)] = make_uint4(0, 0, 0, 0);
    if (half) continue;
    if (p.few && threadIdx.x == 64) p.deferred[1 + v] = make_int4(v, 0, 0, 0);
    for (int i = row0 + w * 32 + lane; i < row0 + rows; i += 64) {
      float* lp = p.lse + ((size_t)b * p.H + i % p.H) * p.T + i / p.H;
      if (MLA_STORE_OK(lp, p.lse, p.lse_bytes, p.err)) *lp = -INFINITY;
    }
  }
}

// Tree: warps 2 and 3 take non-finite values out of the pages that hold drafted keys, and what lies
// behind a sequence's end out of its last page: a weight of zero times such a value would reach every
// row.  Scores need no such care, a key's are its own column, so only the value columns of this half
// are zeroed, and for fp8 the MMA thread issues the scores meanwhile (it tells nobody of them before
// `zeroed`; what they read of a row that is being zeroed is a column that nobody uses).
// A drafted key's flag, on the other hand, stands for its whole row.  It is found ahead of the page's
// copy, from memory: after the copy, an item's last page took 4 us longer than its others (bf16; 32
// sequences of 300 keys and 32 x 128 rows: 247 us against 195).
template <bool kFp8, typename B>
__device__ __forceinline__ void prepare_pages(const Params& p, B& bars, SegmentsOf<true> segs, unsigned char* sm, int half) {
  constexpr int kGranules = kDc * (kFp8 ? 1 : 2) / 16;  // of a row
  constexpr int kLoads = 8 * kGranules / 32;            // eight rows (contiguous) by a warp
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 2;
  // a warp has the rows 16 j + 8 w .. + 7 of a page; bit and lane 8 j + i: row 16 j + 8 w + i
  const int mine = (lane >> 3) * 16 + w * 8 + (lane & 7);
  int seq, L, lo, hi, g = 0, nseg = 0, n_zero = 0;
  while (segs.next(seq, L, lo, hi)) {
    ++nseg;
    const int clean = max(L - drafted(p, seq), 0);
    if constexpr (!kFp8) {
      for (int pg = lo + (int)threadIdx.x - 64; pg < hi && seq % p.NQT == 0; pg += 64) {
        const int page = page_of(p, seq, pg);
        if (page < 0 || page >= p.num_pages) latch_error(p.err, kErrBadPage);
      }
    }
    for (int pg = max(lo, clean / kPage); pg < hi; ++pg) {
      const int gg = g + pg - lo, first = max(clean - pg * kPage, 0), valid = min(kPage, L - pg * kPage);
      const int page = page_of(p, seq, pg);
      uint32_t flagged = 0;
      if (page >= 0 && page < p.num_pages) {
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          const int r0 = 16 * j + 8 * w;
          if (r0 + 8 <= first || r0 >= valid) continue;
          const uint4* src = reinterpret_cast<const uint4*>(p.cache_bytes) + ((size_t)page * kPage + r0) * kGranules;
          uint4 v[kLoads];
          uint32_t rows = 0;
#pragma unroll
          for (int x = 0; x < kLoads; ++x) v[x] = __ldcg(src + lane + 32 * x);
#pragma unroll
          for (int x = 0; x < kLoads; ++x)
            if (granule_nonfinite<kFp8>(v[x])) rows |= 1u << ((lane + 32 * x) / kGranules);
          flagged |= __reduce_or_sync(0xffffffffu, rows) << (8 * j);
        }
      }
      flagged &= __ballot_sync(0xffffffffu, mine >= first && mine < valid);
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bars.zero_go, n_zero++ & 1, &bars.abort_flag, p.err, kItemWait))) return;
      bars.key_nan[gg & 1][mine] = flagged >> lane & 1;
      const uint32_t zero = flagged | __ballot_sync(0xffffffffu, mine >= valid);
      // (whole rows of a chunk, so the swizzle is immaterial)
      unsigned char* values = kFp8 ? sm + kOffStage + (gg + 2 * nseg) % kF8Stages * kF8Page + 2 * half * kPageChunk
                                   : sm + kOffVPart + (gg + 2 * nseg) % kVSlots * kVPartBytes;
      for (int i = 0; i < 32; ++i)
        if ((zero >> i & 1) && lane < (kFp8 ? 16 : 32))
          *reinterpret_cast<uint4*>(values + (lane >> 3) * kPageChunk + ((i >> 3) * 16 + w * 8 + (i & 7)) * 128 +
                                    (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.zeroed);
    }
    g += hi - lo;
  }
}

// Warpgroup 2 of the tree over an fp8 cache makes the query terms of every segment: raw rows by TMA,
// turned in place into terms by one thread a row (128 columns: 256 bytes of bf16 become 128 of hi and
// 128 of lo).  Latent 0..255 comes through two entries of the page ring ahead of the segment's pages
// and is copied on to TMEM by the MMA thread, the rest stays in the query area, which is free when the
// previous segment has its last scores.  A row's power of two needs all its columns: it is found ahead,
// from memory, while the previous segment's pages are under way.  Only the first segment, which no
// other work covers, finds it from both parts in shared memory, and warpgroup 1, which has no scores
// yet, turns its latent 0..255.
template <typename B>
__device__ __forceinline__ void prepare_queries(const Params& p, B& bars, SegmentsOf<true> segs, unsigned char* sm, int TH) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  volatile int* abort_flag = &bars.abort_flag;
  unsigned char* qa = sm + kOffQhi;
  int seq, L, lo, hi, g = 0, nseg = 0;
  auto wait = [&](uint64_t* bar, int phase) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, phase & 1, abort_flag, p.err, kItemWait)) != 0;
  };
  auto done = [&](uint64_t* bar) {
    ptx::fence_proxy_async();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
  };
  auto rows_of = [&](int v) { return min(p.TQ, TH - (v % p.NQT) * kRows); };
  const int r = (warp & 3) * 32 + lane;
  int field = 0;  // of this thread's row in the segment at hand
  while (segs.next(seq, L, lo, hi)) {
    const bool live = r < rows_of(seq);
    if (nseg == 0) {
      if (!wait(&bars.f8.q_raw, 0)) return;
      if (live) field = q_field(qa, r, 5);
      bars.f8.q_exp[0][r] = static_cast<signed char>(field);
      done(&bars.f8.q0_sync);
      if (!wait(&bars.f8.q0_sync, 0)) return;
      field = max(field, static_cast<int>(static_cast<unsigned char>(bars.f8.q_exp[1][r])));
    }
    const int k = q_exponent(field);
    const float f = q_factor(k);
    if (nseg > 0) {
      const int e = g + 2 * nseg;  // ring entries of latent 0..127 and (e + 1) 128..255
      unsigned char *e0 = sm + kOffStage + (e % kF8Stages) * kF8Page,
                    *e1 = sm + kOffStage + ((e + 1) % kF8Stages) * kF8Page;
      if (!wait(&bars.f8.q_lo_raw, nseg)) return;
      q_turn(e0, e1, r, f, live);
      done(&bars.q_lo_full);
      if (!wait(&bars.f8.q_raw, nseg)) return;
      bars.f8.q_exp[nseg & 1][r] = static_cast<signed char>(k);
    }
    q_turn(qa, qa + 2 * kQChunk, r, f, live);
    q_turn_rope(qa, r, f, live);
    done(&bars.q_hi_full);
    ++nseg;
    g += hi - lo;
    SegmentsOf<true> nx = segs;
    int s2, L2, lo2, hi2;
    if (nx.next(s2, L2, lo2, hi2)) {
      const size_t row0 = (size_t)(s2 / p.NQT) * TH + (s2 % p.NQT) * kRows + (warp & 3) * 32;
      field = q_field_ahead(p, row0, min(32, rows_of(s2) - (warp & 3) * 32));
    }
  }
}

template <bool kFp8, bool kTree>
__global__ void __launch_bounds__(kThreadsOf<kFp8>, 1)
    decode_split_kernel(const __grid_constant__ CUtensorMap tm_cache,
                        const __grid_constant__ CUtensorMap tm_page,
                        const __grid_constant__ CUtensorMap tm_c4,
                        const __grid_constant__ CUtensorMap tm_c5,
                        const __grid_constant__ CUtensorMap tm_qlat,
                        const __grid_constant__ CUtensorMap tm_qrope, const Params p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ Bars<kFp8, kTree> bars;
  constexpr bool kF8 = kFp8 && kTree;       // e4m3 operands throughout
  constexpr bool kWiden = kFp8 && !kTree;   // e4m3 pages widened to bf16
  if (kF8 && sm != smem_raw) {  // allocated without the slack of the others (never taken: it is 1024-aligned)
    if (threadIdx.x == 0) latch_error(p.err, kErrBounds);
    wait_for_stream();  // (as at the end)
    return;
  }
  constexpr int kThreads = kThreadsOf<kFp8>;
  // fp8: with fewer than 128 query rows per tile, softmax warps whose 32 rows are all padding
  // of the M = 128 MMA (never stored) widen pages instead: warps 4 .. 4 + n_soft - 1 run the
  // softmax, warps 4 + n_soft .. 7 join the preparation warps (2-3 and 8-11)
  const int n_soft = kWiden ? (p.TQ + 31) / 32 : kRows / 32;
  const int n_prep = kPrepOf<kFp8> + (kWiden ? 32 * (kRows / 32 - n_soft) : 0);
  // readiness parts of a page stage: fp8 three groups of three widened chunks; bf16 the
  // score-only part, then the value part
  constexpr int kParts = kF8 ? 1 : kFp8 ? 3 : 2;
  // the first sequence's Q latent 0..255 (four 16 KB chunks) is staged where pages 1 (fp8)
  // or 1 and 2 (bf16: value slots 1 and 2) land
  auto q_stage_off = [&](int c) -> int {
    if constexpr (kFp8) return kOffStage + kStageBytes + c * kQChunk;
    return kOffVPart + (1 + (c >> 1)) * kVPartBytes + (c & 1) * kQChunk;
  };
  // Tree: every sequence's Q latent 0..255 takes two entries of a ring ahead of its pages (fp8: whole
  // pages; bf16: value parts), so that it is there when the sequence before has its last scores
  constexpr int kRing = kF8 ? kF8Stages : kVSlots;
  auto ring_full = [&](int entry) -> uint64_t* {
    if constexpr (kF8) return &bars.f8.full[entry % kRing];
    else return &bars.vpart_full[entry % kRing];
  };
  auto ring_empty = [&](int entry) -> uint64_t* {
    if constexpr (kF8) return &bars.f8.empty[entry % kRing];
    else return &bars.vpart_empty[entry % kRing];
  };
  auto ring_off = [&](int entry) {
    return kF8 ? kOffStage + entry % kRing * kF8Page : kOffVPart + entry % kRing * kVPartBytes;
  };
  const int warp = threadIdx.x >> 5;
  const int unit = blockIdx.x >> 1, half = blockIdx.x & 1;
  const int TH = p.T * p.H, TQ = p.TQ;
  // first Q row of virtual sequence v: its sequence's rows, then 128 per query tile
  auto q_row0 = [&](int v) { return (v / p.NQT) * TH + (v % p.NQT) * kRows; };
  // bf16: keys of sequence v up to here go from the copy straight to the MMA; a page that reaches
  // further (past the sequence's end, or into its drafted keys) passes the preparation warps
  auto clean_keys = [&](int v, int len) { return kTree ? max(len - drafted(p, v), 0) : len; };

  if (threadIdx.x == 0) {
    // the descriptors are fetched while the barriers are set up and the plan is made: a TMA
    // instruction whose map is not cached waits for that fetch
    ptx::prefetch_tensormap(&tm_qlat);
    ptx::prefetch_tensormap(&tm_qrope);
    if (kFp8 || p.page_box) ptx::prefetch_tensormap(&tm_page);
    if constexpr (kF8) {
      ptx::prefetch_tensormap(&tm_c4);
      for (int s = 0; s < kF8Stages; ++s) {
        ptx::mbar_init(&bars.f8.full[s], 1);
        ptx::mbar_init(&bars.f8.empty[s], 1);
      }
      ptx::mbar_init(&bars.f8.q_lo_raw, 1);
      ptx::mbar_init(&bars.f8.q_raw, 1);
      ptx::mbar_init(&bars.f8.q0_sync, 8);
    }
    if (!kFp8 && p.page_box) {
      ptx::prefetch_tensormap(&tm_c4);
      ptx::prefetch_tensormap(&tm_c5);
    }
    ptx::prefetch_tensormap(&tm_cache);
    bars.abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars.stage_full[s], 1);
      for (int k = 0; k < 3; ++k) ptx::mbar_init(&bars.stage_ready[s][k], n_prep / 32);
      ptx::mbar_init(&bars.stage_empty[s], 1);
    }
    ptx::mbar_init(&bars.spart_full, 1);
    ptx::mbar_init(&bars.spart_empty, 1);
    for (int v = 0; v < kVSlots; ++v) {
      ptx::mbar_init(&bars.vpart_full[v], 1);
      ptx::mbar_init(&bars.vpart_empty[v], 1);
    }
    ptx::mbar_init(&bars.zero_go, 1);
    ptx::mbar_init(&bars.zeroed, kTree ? 2 : n_prep / 32);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars.s_full[i], 1);
      ptx::mbar_init(&bars.p_full[i], n_soft);  // one arrival per softmax warp
    }
    ptx::mbar_init(&bars.o_done, 1);
    ptx::mbar_init(&bars.seg_done, 1);
    ptx::mbar_init(&bars.q_free, 1);
    ptx::mbar_init(&bars.q_lo_full, kF8 ? 4 : 1);  // kF8: a warpgroup's warps (first segment: 1, later ones: 2)
    ptx::mbar_init(&bars.q_cp_done, 1);
    ptx::mbar_init(&bars.q_hi_full, kF8 ? 4 : 1);
    ptx::mbar_init(&bars.q0_copied, 1);
    ptx::mbar_init(&bars.conv_sync, n_prep / 32);  // one arrival per preparation warp
    ptx::mbar_init(&bars.part_done, n_soft);
    ptx::mbar_init(&bars.merge_go, 1);
    ptx::mbar_init(&bars.dec_go, 1);
    ptx::mbar_init(&bars.merge_full, 1);
    ptx::fence_barrier_init();
  }
  if (kTree && p.few) wait_for_stream();
  // the plan's length loads go out first; the other warps set up meanwhile
  if (warp == 3) make_plan<kTree>(p, unit, &bars.plan);
  // Q rows T*H..127 are never loaded: keep them zero (finite scores in the padded rows)
  for (int i = threadIdx.x; i < 5 * kQChunk / 16; i += kThreads)
    reinterpret_cast<uint4*>(sm + kOffQhi)[i] = make_uint4(0, 0, 0, 0);
  ptx::fence_proxy_async();
  if (warp == 2) ptx::tmem_alloc(&bars.tmem_base, 512);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort_flag;
  using Segments = SegmentsOf<kTree>;
  Segments segs;
  segs.init(p, bars.plan);
  int seq, L, lo, hi;

  if (warp < 4 || warp >= 8 || warp >= 4 + n_soft) {
   if constexpr (kF8) ptx::regs_dec<kF8RegsLow>();
   if (warp == 0) {
    // -------------------------------------------------------------- TMA producer
    // One lane issues Q, the pages in order (fp8: whole pages; bf16: the value part as soon
    // as its ring slot frees, then the score-only part once the previous page's scores are
    // done with that slot) and the L2 warming.  Copies are served in issue order, so the
    // value part, which goes out about a page earlier, never waits behind a score-only part.
    if ((threadIdx.x & 31) == 0) {
      int g = 0, nseg = 0;
      [[maybe_unused]] int n_ring = 0, n_q = 0, n_s = 0;  // tree: ring entries, queries in them, score-only parts issued
      bool ok = true;
      while (ok && segs.next(seq, L, lo, hi)) {
        // the first page's table entry is read before Q is issued, so its latency overlaps
        // the Q copies instead of delaying the page's own
        const int page_first = page_of(p, seq, lo);
        if constexpr (kTree) {
          // Q latent 0..255 as two ring entries, the rest into the Q area once the previous segment's
          // last scores are done (fp8: raw rows, which warps 8-11 turn into terms)
          uint64_t *lo_bar = &bars.q_lo_full, *hi_bar = &bars.q_hi_full;
          if constexpr (kF8) {
            lo_bar = &bars.f8.q_lo_raw;
            hi_bar = &bars.f8.q_raw;
          }
          // (after one page the ring may have room while that segment's are still on their way)
          if (n_q > 0 && !(ok = ptx::mbar_wait(lo_bar, (n_q - 1) & 1, abort_flag, p.err))) break;
          for (int e = 0; e < 2; ++e, ++n_ring) {
            if (!(ok = ptx::mbar_wait(ring_empty(n_ring), ((n_ring / kRing) & 1) ^ 1, abort_flag, p.err))) break;
            ptx::mbar_arrive(ring_full(n_ring));  // nobody waits for this phase
            if (e == 0) ptx::mbar_arrive_expect_tx(lo_bar, 4 * TQ * 128), ++n_q;
            for (int c = 0; c < 2; ++c)
              ptx::tma_load_2d(sm + ring_off(n_ring) + c * kQChunk, &tm_qlat, lo_bar, e * 128 + c * 64, q_row0(seq));
          }
          if (!ok) break;
          if (nseg > 0 && !(ok = ptx::mbar_wait(&bars.q_free, (nseg - 1) & 1, abort_flag, p.err))) break;
          ptx::mbar_arrive_expect_tx(hi_bar, 5 * TQ * 128);
          for (int c = 0; c < 4; ++c)
            ptx::tma_load_2d(sm + kOffQhi + c * kQChunk, &tm_qlat, hi_bar, 256 + c * 64, q_row0(seq));
          ptx::tma_load_2d(sm + kOffQhi + 4 * kQChunk, &tm_qrope, hi_bar, 0, q_row0(seq));
          ++nseg;
        } else {
          if (nseg == 0) {
            // first sequence: Q latent 0..255 staged in the (still unused) second page
            // stage, the rest of Q straight into the Q area, all at once
            ptx::mbar_arrive_expect_tx(&bars.q_lo_full, 4 * TQ * 128);
            for (int c = 0; c < 4; ++c)
              ptx::tma_load_2d(sm + q_stage_off(c), &tm_qlat, &bars.q_lo_full, c * 64, q_row0(seq));
            ptx::mbar_arrive_expect_tx(&bars.q_hi_full, 5 * TQ * 128);
            for (int c = 0; c < 4; ++c)
              ptx::tma_load_2d(sm + kOffQhi + c * kQChunk, &tm_qlat, &bars.q_hi_full, 256 + c * 64, q_row0(seq));
            ptx::tma_load_2d(sm + kOffQhi + 4 * kQChunk, &tm_qrope, &bars.q_hi_full, 0, q_row0(seq));
          } else {
            // Q latent 0..255 into the Q area once the previous sequence's last S is done
            if (!(ok = ptx::mbar_wait(&bars.q_free, (nseg - 1) & 1, abort_flag, p.err))) break;
            ptx::mbar_arrive_expect_tx(&bars.q_lo_full, 4 * TQ * 128);
            for (int c = 0; c < 4; ++c)
              ptx::tma_load_2d(sm + kOffQhi + c * kQChunk, &tm_qlat, &bars.q_lo_full, c * 64, q_row0(seq));
          }
          ++nseg;
        }
        // warm L2 with the next segment's Q (read when this one's pages are done) once this
        // segment's first page is issued: finding the next segment reads the lengths again
        auto warm_next_q = [&]() {
          Segments nx = segs;
          int s2, L2, lo2, hi2;
          if (nx.next(s2, L2, lo2, hi2)) {
            const int r0 = q_row0(s2), rows = min(TQ, p.B * TH - r0);
            if (rows > 0) {
              ptx::bulk_prefetch(p.q_latent + (size_t)r0 * kDl, rows * kDl * 2);
              ptx::bulk_prefetch(p.q_rope + (size_t)r0 * 64, rows * 128);
            }
          }
        };
        for (int pg = lo; pg < hi; ++pg, ++g) {
          const int s = g % kStages;
          if (kWiden && !(ok = ptx::mbar_wait(&bars.stage_empty[s], ((g / kStages) & 1) ^ 1, abort_flag, p.err)))
            break;
          // the first sequence's staged Q stays in place until it is copied to TMEM
          if (kWiden && g == 1 && !(ok = ptx::mbar_wait(&bars.q0_copied, 0, abort_flag, p.err))) break;
          const int y = pg == lo ? row_of_page(p, page_first) : page_row(p, seq, pg);
          if constexpr (kF8) {
            if (!(ok = ptx::mbar_wait(ring_empty(n_ring), ((n_ring / kRing) & 1) ^ 1, abort_flag, p.err))) break;
            unsigned char* dst = sm + ring_off(n_ring);
            uint64_t* full = ring_full(n_ring++);
            ptx::mbar_arrive_expect_tx(full, kF8Page);
            if (p.page_box) {
              ptx::tma_load_3d(dst, &tm_page, full, 0, y, 0);
            } else {
              for (int c = 0; c < 4; ++c)
                ptx::tma_load_2d(dst + c * kPageChunk, &tm_cache, full, c * 128, y);
            }
            ptx::tma_load_2d(dst + 4 * kPageChunk, &tm_c4, full, 512, y);
          } else if constexpr (kFp8) {
            unsigned char* dst = sm + kOffStage + s * kStageBytes + kRawOffset;
            ptx::mbar_arrive_expect_tx(&bars.stage_full[s], 9 * kRawChunk);
            if (p.page_box) {
              ptx::tma_load_3d(dst, &tm_page, &bars.stage_full[s], 0, y, 0);
            } else {
              for (int c = 0; c < 9; ++c)
                ptx::tma_load_2d(dst + c * kRawChunk, &tm_cache, &bars.stage_full[s], c * 64, y);
            }
          } else {
            // The value part first: its slot (the page three back has had its PV) frees about
            // a page before the score-only slot does, so it goes out then and lands before the
            // score k-steps reach it, instead of queueing behind this page's score-only part.
            // Own latent chunks 4 half .. 4 half + 3 (value slots 1 and 2 first hold the first
            // sequence's staged Q).
            const int v = kTree ? n_ring : g;
            if (!(ok = ptx::mbar_wait(ring_empty(v), ((v / kVSlots) & 1) ^ 1, abort_flag, p.err))) break;
            if (!kTree && (g == 1 || g == 2) && !(ok = ptx::mbar_wait(&bars.q0_copied, 0, abort_flag, p.err))) break;
            unsigned char* dst = sm + ring_off(v);
            uint64_t* full = ring_full(v);
            ptx::mbar_arrive_expect_tx(full, kVPartBytes);
            if (p.page_box) {
              ptx::tma_load_3d(dst, &tm_c4, full, 0, y, 4 * half);
            } else {
              for (int c = 0; c < 4; ++c)
                ptx::tma_load_2d(dst + c * kPageChunk, &tm_cache, full, (4 * half + c) * 64, y);
            }
            ++n_ring;
            // then the score-only chunks (chunk_idx order: half 0 takes 4..8, half 1 0..3 and
            // 8), once the previous page's score k-steps over them are done
            if (!(ok = ptx::mbar_wait(&bars.spart_empty, (g & 1) ^ 1, abort_flag, p.err))) break;
            dst = sm + kOffSPart;
            ptx::mbar_arrive_expect_tx(&bars.spart_full, kSPartBytes);
            if (p.page_box && half == 0) {
              ptx::tma_load_3d(dst, &tm_c5, &bars.spart_full, 0, y, 4);
            } else if (p.page_box) {
              ptx::tma_load_3d(dst, &tm_c4, &bars.spart_full, 0, y, 0);
              ptx::tma_load_2d(dst + 4 * kPageChunk, &tm_cache, &bars.spart_full, 512, y);
            } else {
              for (int i = 0; i < 5; ++i)
                ptx::tma_load_2d(dst + i * kPageChunk, &tm_cache, &bars.spart_full,
                                 (half == 0 ? 4 + i : (i < 4 ? i : 8)) * 64, y);
            }
            ++n_s;
          }
          if (pg == lo) warm_next_q();
          // warm L2 with the pages ahead (after this page's own load has been issued)
          for (int a = (pg == lo ? lo + 1 : pg + kPrefetchAhead); a <= min(hi - 1, pg + kPrefetchAhead); ++a) {
            const int ya = page_row(p, seq, a);
            if (ya < 0) continue;
            // the page is 72 KB (bf16; 36 KB fp8) of contiguous bytes: one linear prefetch
            // reads it in address order
            constexpr uint32_t kPageBytes = kPage * kDc * (kFp8 ? 1 : 2);
            ptx::bulk_prefetch(p.cache_bytes + (size_t)ya * (kDc * (kFp8 ? 1 : 2)), kPageBytes);
          }
        }
      }
      if (kTree) {  // copies that after an abort nobody may wait for land before the CTA leaves
        for (int v = max(0, n_ring - kRing); v < n_ring; ++v) ptx::mbar_wait_drain(ring_full(v), (v / kRing) & 1);
        if (!kF8 && n_s > 0) ptx::mbar_wait_drain(&bars.spart_full, (n_s - 1) & 1);
        uint64_t *lo_bar = &bars.q_lo_full, *hi_bar = &bars.q_hi_full;
        if constexpr (kF8) {
          lo_bar = &bars.f8.q_lo_raw;
          hi_bar = &bars.f8.q_raw;
        }
        if (n_q > 0) ptx::mbar_wait_drain(lo_bar, (n_q - 1) & 1);
        if (nseg > 0) ptx::mbar_wait_drain(hi_bar, (nseg - 1) & 1);
      }
    }
   } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    if (ptx::elect_one()) {
      constexpr uint32_t kIdS = ptx::make_idesc(1, kRows, kPage, 0, 0);
      constexpr uint32_t kIdPV = ptx::make_idesc(1, kRows, 256, 0, 1);
      const uint32_t qhi = ptx::smem_u32(sm + kOffQhi);
      const uint32_t stage0 = ptx::smem_u32(sm + kOffStage);
      const uint32_t o_tm = tmem + 256;
      int g = 0, nseg = 0;
      int n_zeroed = 0;  // bf16: partial pages zeroed so far
      bool ok = true;
      const uint32_t smb = ptx::smem_u32(sm);
      // Operand descriptors, built once (k-step j of a chunk is 32 bytes further, i.e. 2 in
      // the start-address field; a chunk 8 KB, i.e. 512): B = the page chunks (fp8: stage 0 /
      // 1 in chunk order; bf16: the score-only slot, value slot 0 / 1 / 2), A = the shared-
      // memory Q chunks.  This keeps the issue loop at an add or two per MMA: the MMA thread
      // shares its SM sub-partition with a softmax warp.
      const uint64_t b0 = ptx::sw128_desc(smb + (kFp8 ? kOffStage : kOffSPart), 16, 1024);
      const uint64_t b1 = ptx::sw128_desc(smb + (kFp8 ? kOffStage + kStageBytes : kOffVPart), 16, 1024);
      const uint64_t b2 = ptx::sw128_desc(smb + kOffVPart + kVPartBytes, 16, 1024);
      const uint64_t b3 = ptx::sw128_desc(smb + kOffVPart + 2 * kVPartBytes, 16, 1024);
      const uint64_t qd = ptx::sw128_desc(qhi, 16, 1024);
      // the ring entry of this segment's page gg (tree: two entries of Q precede a segment's pages)
      auto entry = [&](int gg) { return kTree ? gg + 2 * (nseg + 1) : gg; };
      // k-step k (a compile-time constant at every call) of S into d, B from chunk base bc
      auto mma_k = [&](uint32_t d, uint64_t bc, int k, bool acc) {
        const uint64_t db = bc + 2 * (k & 3);
        if (k < 16)  // latent 0..255: A from TMEM
          ptx::mma_bf16_ts(d, tmem + k * 8, db, kIdS, acc ? 1u : 0u);
        else         // latent 256..511 + rope: A from shared memory (16 KB per Q chunk)
          ptx::mma_bf16_ss(d, qd + 1024 * ((k - 16) >> 2) + 2 * ((k - 16) & 3), db, kIdS, acc ? 1u : 0u);
      };
      // part `part` of S(gg): fp8 k-steps 12 part .. 12 part + 11; bf16 the k-steps of the
      // score-only chunks (part 0), then those of the value chunks (part 1).  The first MMA
      // of S(gg) starts the accumulator.
      auto issue_s = [&](int gg, int part) {
        const uint32_t d = tmem + 128 + (gg & 1) * 64;
        if constexpr (kF8) {
          // 18 k-steps of 32 columns, the query's hi term and its lo term
          constexpr uint32_t kIdS8 = ptx::make_idesc(0, kRows, kPage, 0, 0);
          const uint64_t st = b0 + entry(gg) % kF8Stages * (kF8Page / 16);
          const uint64_t rp = ptx::smem_desc(smb + ring_off(entry(gg)) + 4 * kPageChunk, 16, 512, ptx::kSwz64);
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // latent 0..255: A from TMEM
            const uint64_t db = st + 512 * (j >> 2) + 2 * (j & 3);
            const uint32_t qa = tmem + (j >> 2) * 64 + (j & 3) * 8;
            ptx::mma_f8_ts(d, qa, db, kIdS8, j > 0 ? 1u : 0u);
            ptx::mma_f8_ts(d, qa + 32, db, kIdS8, 1u);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // latent 256..511: A from shared memory
            const uint64_t db = st + 512 * (2 + (j >> 2)) + 2 * (j & 3);
            const uint64_t da = qd + 2048 * (j >> 2) + 2 * (j & 3);
            ptx::mma_f8_ss(d, da, db, kIdS8, 1u);
            ptx::mma_f8_ss(d, da + 1024, db, kIdS8, 1u);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // rope
            ptx::mma_f8_ss(d, qd + 4096 + 2 * j, rp + 2 * j, kIdS8, 1u);
            ptx::mma_f8_ss(d, qd + 4096 + 4 + 2 * j, rp + 2 * j, kIdS8, 1u);
          }
        } else if constexpr (kFp8) {
          const uint64_t st = (gg % kStages) ? b1 : b0;
          if (part == 0) {
#pragma unroll
            for (int k = 0; k < 12; ++k) mma_k(d, st + 512 * (k >> 2), k, k > 0);
          } else if (part == 1) {
#pragma unroll
            for (int k = 12; k < 24; ++k) mma_k(d, st + 512 * (k >> 2), k, true);
          } else {
#pragma unroll
            for (int k = 24; k < 36; ++k) mma_k(d, st + 512 * (k >> 2), k, true);
          }
        } else if (part == 0) {
          if (half == 0) {
#pragma unroll
            for (int k = 16; k < 36; ++k) mma_k(d, b0 + 512 * chunk_idx(k >> 2, 0), k, k > 16);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) mma_k(d, b0 + 512 * chunk_idx(k >> 2, 1), k, k > 0);
#pragma unroll
            for (int k = 32; k < 36; ++k) mma_k(d, b0 + 512 * chunk_idx(k >> 2, 1), k, true);
          }
        } else {
          const int v = entry(gg) % kVSlots;
          const uint64_t vb = v == 0 ? b1 : v == 1 ? b2 : b3;
          if (half == 0) {
#pragma unroll
            for (int k = 0; k < 16; ++k) mma_k(d, vb + 512 * (k >> 2), k, true);
          } else {
#pragma unroll
            for (int k = 16; k < 32; ++k) mma_k(d, vb + 512 * ((k >> 2) - 4), k, true);
          }
        }
      };
      // PV: B = this half's 256 latent columns (four chunks 8 KB apart), 16 keys per k-step
      auto issue_pv = [&](int gg, bool first) {
        uint32_t st;
        if constexpr (kF8) {
          // two 128-column chunks 8 KB apart, 32 keys per k-step; P'' hi (e4m3) in 16 TMEM columns, lo
          // (e5m2) in 16 more
          constexpr uint32_t kIdPV8 = ptx::make_idesc(0, kRows, 256, 0, 1);
          constexpr uint32_t kIdPV8Lo = ptx::make_idesc2(1, 0, kRows, 256, 0, 1);
          const uint64_t vd8 = ptx::sw128_desc(smb + ring_off(entry(gg)) + 2 * half * kPageChunk, kPageChunk, 1024);
          const uint32_t pa8 = tmem + 128 + (gg & 1) * 64;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            ptx::mma_f8_ts(o_tm, pa8 + k * 8, vd8 + 256 * k, kIdPV8, (!first || k > 0) ? 1u : 0u);
            ptx::mma_f8_ts(o_tm, pa8 + 16 + k * 8, vd8 + 256 * k, kIdPV8Lo, 1u);
          }
          return;
        }
        if constexpr (kFp8) st = kOffStage + (gg % kStages) * kStageBytes + 4 * half * kPageChunk;
        else st = ring_off(entry(gg));
        const uint64_t vd = ptx::sw128_desc(smb + st, kPageChunk, 1024);
        const uint32_t pa = tmem + 128 + (gg & 1) * 64;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::mma_bf16_ts(o_tm, pa + k * 8, vd + 128 * k, kIdPV, (!first || k > 0) ? 1u : 0u);
      };
      while (ok && segs.next(seq, L, lo, hi)) {
        // Q latent 0..255: staged in the Q area by the producer, copied into TMEM columns
        // 0..127 (lane = query row); then latent 256..511 + rope over the staging copy
        if (!(ok = ptx::mbar_wait(&bars.q_lo_full, nseg & 1, abort_flag, p.err))) break;
        ptx::tc_fence_after();
        // the first sequence's Q latent 0..255 was staged in the second page stage; tree: every one's
        // in two ring entries, which the copies free
        const int e0 = entry(g) - 2;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t qc = kTree ? smb + ring_off(e0 + (k >> 3)) + ((k >> 2) & 1) * kQChunk
                            : nseg == 0 ? smb + q_stage_off(k >> 2) : qhi + (k >> 2) * kQChunk;
          ptx::tmem_cp_128x256b(tmem + k * 8, ptx::sw128_desc(qc + (k & 3) * 32, 16, 1024));
        }
        if constexpr (kTree) {
          ptx::mma_commit(ring_empty(e0));
          ptx::mma_commit(ring_empty(e0 + 1));
        } else {
          ptx::mma_commit(&bars.q_cp_done);
          if (nseg == 0) ptx::mma_commit(&bars.q0_copied);
        }
        if (!kTree && nseg > 0) {  // the rest of Q over the staging copy (the producer loaded the first)
          if (!(ok = ptx::mbar_wait(&bars.q_cp_done, nseg & 1, abort_flag, p.err))) break;
          ptx::mbar_arrive_expect_tx(&bars.q_hi_full, 5 * TQ * 128);
          for (int c = 0; c < 4; ++c)
            ptx::tma_load_2d(sm + kOffQhi + c * kQChunk, &tm_qlat, &bars.q_hi_full, 256 + c * 64, q_row0(seq));
          ptx::tma_load_2d(sm + kOffQhi + 4 * kQChunk, &tm_qrope, &bars.q_hi_full, 0, q_row0(seq));
        }
        if (!(ok = ptx::mbar_wait(&bars.q_hi_full, nseg & 1, abort_flag, p.err))) break;
        ptx::tc_fence_after();
        const int g_end = g + (hi - lo), g_first = g;
        const int clean = clean_keys(seq, L);
        int gs = g, gp = g;  // next page whose S / whose PV is to be issued
        int sp = 0;          // next part of S(gs)
        bool zero_asked = false;  // bf16: the partial page gs was handed to the preparation warps
        long long t0 = clock64();
        bool s_held = false;      // kF8: S(gs) is issued, its page not prepared yet
        auto s_issued = [&](int& page) {
          ptx::mma_commit(&bars.s_full[page & 1]);
          ++page;
          if (page == g_end) ptx::mma_commit(&bars.q_free);  // Q no longer read
        };
        while (gp < g_end) {
          bool progress = false;
          // PV first: it releases the page stage for the next load
          if (gp < gs && ptx::mbar_test_wait(&bars.p_full[gp & 1], (gp >> 1) & 1)) {
            ptx::tc_fence_after();
            issue_pv(gp, gp == g_first);
            ptx::mma_commit(&bars.o_done);
            // fp8: the whole stage; bf16: the value part (the score-only part was released
            // after the scores)
            ptx::mma_commit(kWiden ? &bars.stage_empty[gp % kStages] : ring_empty(entry(gp)));
            ++gp;
            progress = true;
          }
          // S(gs) may run at most one page ahead of the oldest unissued PV (two S buffers).
          // A full bf16 page needs no preparation: its parts are ready when they land.  A page
          // that ends its sequence part-way goes to the preparation warps once both parts have
          // landed (tree: the value part, which the scores' second part then waits for; fp8: the
          // page, with the scores issued meanwhile) and comes back with the rows past the end zeroed.
          bool can = false;
          if (gs < g_end && gs <= gp + 1) {
            const bool whole = (lo + (gs - g_first) + 1) * kPage <= clean;
            if constexpr (kF8) {
              if (s_held) {
                // the scores of a page that is prepared are out; their readers may go on once it is
                if (ptx::mbar_test_wait(&bars.zeroed, n_zeroed & 1)) {
                  ++n_zeroed;
                  s_held = false;
                  s_issued(gs);
                  progress = true;
                }
              } else {
                can = ptx::mbar_test_wait(ring_full(entry(gs)), (entry(gs) / kRing) & 1);
                if (can && !whole) ptx::mbar_arrive(&bars.zero_go);
              }
            } else if constexpr (kFp8) {
              can = ptx::mbar_test_wait(&bars.stage_ready[gs % kStages][sp], (gs / kStages) & 1);
            } else if (whole) {
              can = sp == 0 ? ptx::mbar_test_wait(&bars.spart_full, gs & 1)
                            : ptx::mbar_test_wait(ring_full(entry(gs)), (entry(gs) / kVSlots) & 1);
            } else if (kTree) {
              // prepared from its value part on, which lands about a page ahead of the score-only part
              if (!zero_asked && ptx::mbar_test_wait(ring_full(entry(gs)), (entry(gs) / kVSlots) & 1)) {
                ptx::mbar_arrive(&bars.zero_go);
                zero_asked = progress = true;
              }
              can = sp == 0 ? ptx::mbar_test_wait(&bars.spart_full, gs & 1)
                            : zero_asked && ptx::mbar_test_wait(&bars.zeroed, n_zeroed & 1);
              if (can && sp == 1) {
                zero_asked = false;
                ++n_zeroed;
              }
            } else if (sp == 1) {
              can = true;  // zeroed before its part 0
            } else if (!zero_asked) {
              if (ptx::mbar_test_wait(&bars.spart_full, gs & 1) &&
                  ptx::mbar_test_wait(ring_full(entry(gs)), (entry(gs) / kVSlots) & 1)) {
                ptx::mbar_arrive(&bars.zero_go);
                zero_asked = true;
                progress = true;
              }
            } else if (ptx::mbar_test_wait(&bars.zeroed, n_zeroed & 1)) {
              can = true;
              zero_asked = false;
              ++n_zeroed;
            }
          }
          if (can) {
            ptx::tc_fence_after();
            issue_s(gs, sp);
            if (!kFp8 && sp == 0) ptx::mma_commit(&bars.spart_empty);
            if (sp + 1 < kParts) {
              ++sp;
            } else if (kF8 && (lo + (gs - g_first) + 1) * kPage > clean) {
              s_held = true;
            } else {
              sp = 0;
              s_issued(gs);
            }
            progress = true;
          }
          if (progress) {
            t0 = clock64();
          } else if (*abort_flag) {
            ok = false;
            break;
          } else if (clock64() - t0 > 1000000000LL) {
            latch_error(p.err, kErrTimeout);
            *abort_flag = 1;
            ok = false;
            break;
          }
        }
        if (ok) ptx::mma_commit(&bars.seg_done);  // the segment's last PV product is complete
        g = g_end;
        ++nseg;
      }
      if (kTree && !ok) {  // after an abort: every MMA issued completes before the CTA frees its TMEM
        ptx::mma_commit(&bars.stage_empty[0]);  // (a barrier that only the widening kernel uses)
        ptx::mbar_wait_drain(&bars.stage_empty[0], 0);
      }
    }
   } else if constexpr (kF8) {
    if (warp < 4) {
      empty_items(p, unit, half, TH);
      prepare_pages<true>(p, bars, segs, sm, half);
    } else {
      prepare_queries(p, bars, segs, sm, TH);
    }
   } else if constexpr (kTree) {
    empty_items(p, unit, half, TH);
    prepare_pages<false>(p, bars, segs, sm, half);
   } else {
    // -------------------------------------------------------------- stage preparation
    // 0 .. n_prep - 1: warps 2-3, then 8-11, then the softmax warps that joined
    const int tid = warp < 4 ? threadIdx.x - 64
                  : warp >= 8 ? threadIdx.x - 192
                              : kPrepOf<kFp8> + threadIdx.x - 32 * (4 + n_soft);
    const int row = tid & (kPage - 1);  // the page row whose scale (fp8) this thread stages
    int g = 0, n_zero = 0;
    bool ok = true;
    while (ok && segs.next(seq, L, lo, hi)) {
      const int clean = clean_keys(seq, L);
      for (int pg = lo; pg < hi; ++pg, ++g) {
        const int s = g % kStages;
        unsigned char* st = sm + kOffStage + s * kStageBytes;
        const int valid = min(kPage, L - pg * kPage);  // rows holding tokens of this sequence
        const int page = __ldg(p.page_table + (size_t)(seq / p.NQT) * p.max_pages + pg);
        const bool bad = page < 0 || page >= p.num_pages;
        if (bad && tid == 0 && seq % p.NQT == 0) latch_error(p.err, kErrBadPage);
        const bool live = !bad && row < valid;
        auto live_row = [&](int rr) { return !bad && rr < valid; };
        float ksc = 0.f;
        if constexpr (kFp8) ksc = live && tid < kPage ? __ldg(p.kv_scale + (size_t)page * kPage + row) : 0.f;
        if constexpr (!kFp8) {
          // A page that ends its sequence part-way: once the MMA thread has seen both of its
          // parts land it hands the page over (zero_go); rows valid..63 of its nine chunks
          // are zeroed (16-byte granules; whole rows, so the swizzle is immaterial) and handed
          // back (zeroed).  Full pages go straight from the copy to the MMA.
          if ((pg + 1) * kPage > clean) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.zero_go, n_zero & 1, abort_flag, p.err, kItemWait));
            if (!ok) break;
            const int nrow = kPage - valid;
            for (int part = 0; part < 2; ++part) {
              const int nch = part == 0 ? 5 : 4;
              unsigned char* base = sm + (part == 0 ? kOffSPart : kOffVPart + (g % kVSlots) * kVPartBytes);
              for (int e = tid; e < nrow * nch * 8; e += n_prep) {
                const int rw = valid + e / (nch * 8), rem = e % (nch * 8), c = rem >> 3, gr = rem & 7;
                *reinterpret_cast<uint4*>(base + c * kPageChunk + rw * 128 + gr * 16) = make_uint4(0, 0, 0, 0);
              }
            }
            ptx::fence_proxy_async();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bars.zeroed);
            ++n_zero;
          }
        } else {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.stage_full[s], (g / kStages) & 1, abort_flag, p.err));
          if (!ok) break;
          if (tid < kPage) bars.kscale[s][row] = ksc;
          // Widen in place, in three lockstep steps of three chunks (four 16-byte granules
          // per thread per step).  bf16 chunk c (bytes [8c, 8c+8) KB) overlaps raw chunks 2c-9
          // and 2c-8 (raw chunk c' sits at [36 + 4c', 40 + 4c') KB), which are at most the
          // step's own chunks 3k..3k+2 or earlier ones: after every thread has read its raw
          // granules of the step (bounded mbarrier), the step's writes only destroy bytes that
          // were already read, and never those of a later step.
#pragma unroll 1
          for (int k = 0; k < 3 && ok; ++k) {
            // the step's 3 chunks are 768 granules of 16 raw bytes (64 rows x 4 per chunk);
            // thread tid takes granules tid + n_prep q (at most four: n_prep >= 192), so a warp
            // reads 512 contiguous bytes
            uint4 raw[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int G = tid + n_prep * q, c = 3 * k + (G >> 8), gi = G & 255;
              raw[q] = (G < 768 && live_row(gi >> 2))
                           ? *reinterpret_cast<const uint4*>(st + kRawOffset + c * kRawChunk + gi * 16)
                           : make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bars.conv_sync);
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.conv_sync, (3 * g + k) & 1, abort_flag, p.err));
            if (!ok) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int G = tid + n_prep * q, c = 3 * k + (G >> 8), gi = G & 255;
              if (G >= 768) continue;
              const int rw = gi >> 2, quarter = gi & 3;  // 16 columns 16 quarter .. of row rw
              const uint32_t words[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
              uint32_t w[8];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                w[2 * x] = ptx::e4m3x2_to_bf16x2(words[x]);
                w[2 * x + 1] = ptx::e4m3x2_to_bf16x2(words[x] >> 16);
              }
              unsigned char* dst = st + c * kPageChunk + rw * 128;
              *reinterpret_cast<uint4*>(dst + (((2 * quarter) ^ (rw & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(dst + (((2 * quarter + 1) ^ (rw & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
            }
            // chunks 3k..3k+2 are ready for the score MMA (the next steps write above them)
            ptx::fence_proxy_async();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bars.stage_ready[s][k]);
          }
          if (!ok) break;
        }
      }
    }
   }
  } else {
    // -------------------------------------------------------------- softmax / epilogue
    if constexpr (kF8) ptx::regs_inc<kF8RegsHigh>();
    const int r = threadIdx.x - 128;  // query row == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int g = 0, n_epi = 0, n_dec = 0, n_part = 0, n_bulk = 0, n_bulk_issued = 0;
    bool ok = true;
    // a sequence with no keys is in no work unit's range: unit u writes O = 0 and LSE = -inf for
    // such sequences u, u + G, u + 2G, ...  (tree: empty_items)
    if (!kTree && half == 0) {
      for (int b = unit; b < p.B; b += p.G) {
        if (clamp_len(__ldg(p.cache_lens + b), p.max_pages) > 0) continue;
        uint4* o = reinterpret_cast<uint4*>(p.out + (size_t)b * TH * kDl);
        for (int i = r; i < TH * (kDl / 8); i += 32 * n_soft)
          if (MLA_STORE_OK(o + i, p.out, p.out_bytes, p.err)) o[i] = make_uint4(0, 0, 0, 0);
        for (int i = r; i < TH; i += 32 * n_soft) {
          float* lp = p.lse + ((size_t)b * p.H + i % p.H) * p.T + i / p.H;
          if (MLA_STORE_OK(lp, p.lse, p.lse_bytes, p.err)) *lp = -INFINITY;
        }
      }
    }
    if constexpr (kF8) {
      // The first segment's query terms of latent 0..255 (warpgroup 2 makes the others).  A row's two
      // largest fields change hands through q_exp, whose first entry then holds the row's power of two.
      Segments first = segs;
      if (first.next(seq, L, lo, hi)) {
        unsigned char *e0 = sm + kOffStage, *e1 = e0 + kF8Page;
        const bool live = r < min(p.TQ, TH - (seq % p.NQT) * kRows);
        int mine = 0;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.f8.q_lo_raw, 0, abort_flag, p.err));
        if (ok) {
          if (live) mine = max(q_field(e0, r, 2), q_field(e1, r, 2));
          bars.f8.q_exp[1][r] = static_cast<signed char>(mine);
          ptx::fence_proxy_async();
          __syncwarp();
          if ((r & 31) == 0) ptx::mbar_arrive(&bars.f8.q0_sync);
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.f8.q0_sync, 0, abort_flag, p.err));
        }
        if (ok) {
          const int k = q_exponent(max(mine, static_cast<int>(static_cast<unsigned char>(bars.f8.q_exp[0][r]))));
          bars.f8.q_exp[0][r] = static_cast<signed char>(k);
          q_turn(e0, e1, r, q_factor(k), live);
          ptx::fence_proxy_async();
          __syncwarp();
          if ((r & 31) == 0) ptx::mbar_arrive(&bars.q_lo_full);
        }
      }
    }
    while (ok && segs.next(seq, L, lo, hi)) {
      const int gr = (seq % p.NQT) * kRows + r;  // row within the sequence's T*H rows
      const int t_row = gr / p.H;
      const int last_visible = p.causal ? (L - p.T + t_row) : (L - 1);  // keys <= this are visible
      const int n_new = kTree ? drafted(p, seq) : 0;
      const int first_new = L - n_new;  // tree: the first drafted key (negative if L < n_new)
      const bool pad_row = kTree && t_row >= n_new;
      const uint32_t* mask_row =
          kTree ? p.tree_mask + (seq / p.NQT) * p.mask_stride + (long long)t_row * p.mask_words : nullptr;
      float m = -INFINITY, l = 0.f, lr = 0.f;  // exact row sum (LSE) and bf16-rounded (PV)
      const uint32_t o_addr = tmem + lane_off + 256;
      // kF8: each lane has the scales of keys 2 lane and 2 lane + 1 of the next page on their way, and
      // the page-table entry of the one after
      float f8_scale = 0.f;  // softmax scale in the exponent over the row's power of two
      float f8_mass = 0.f, f8_steps = 0.f;  // see kF8StepsPerMass
      int tab[2] = {-1, -1};
      float2 ks_next = make_float2(0.f, 0.f);
      auto entry = [&](int pg) {
        return pg < hi ? __ldg(p.page_table + (size_t)(seq / p.NQT) * p.max_pages + pg) : -1;
      };
      auto scales = [&](int page) {
        return page >= 0 && page < p.num_pages
                   ? __ldg(reinterpret_cast<const float2*>(p.kv_scale + (size_t)page * kPage) + (r & 31))
                   : make_float2(0.f, 0.f);
      };
      if constexpr (kF8) {
        tab[0] = entry(lo);
        tab[1] = entry(lo + 1);
        ks_next = scales(tab[0]);
      }
      for (int pg = lo; pg < hi; ++pg, ++g) {
        const bool tree_page = kTree && (pg + 1) * kPage > first_new;
        unsigned long long vis = ~0ull;  // tree: bit x says whether this row sees key pg * 64 + x
        if (tree_page) {
          const int off = pg * kPage - first_new;  // drafted index of the page's first key, > -64
          if (pad_row)
            vis = 0;
          else if (off >= 0)
            vis = mask_bits(mask_row, p.mask_words, off);
          else
            vis = mask_bits(mask_row, p.mask_words, 0) << -off | ((1ull << -off) - 1);
          if (L - pg * kPage < kPage) vis &= (1ull << (L - pg * kPage)) - 1;
        }
        int page8 = -1;
        uint32_t nan_keys[2] = {0, 0};
        if constexpr (kF8) {
          page8 = tab[0];
          const int key = pg * kPage + 2 * (r & 31);
          float2 k2 = make_float2(key < L ? ks_next.x : 0.f, key + 1 < L ? ks_next.y : 0.f);
          // log2 of the scale, floored (a scale of 0 gives weights of 0); a drafted key whose scale is
          // not finite is flagged
          float2 l2 = make_float2(fmaxf(__log2f(fabsf(k2.x)), -100.f), fmaxf(__log2f(fabsf(k2.y)), -100.f));
          if (tree_page) {
            const bool bad0 = !(fabsf(k2.x) < INFINITY), bad1 = !(fabsf(k2.y) < INFINITY);
            if (bad0) k2.x = l2.x = 0.f;
            if (bad1) k2.y = l2.y = 0.f;
            const uint32_t even = __ballot_sync(0xffffffffu, bad0), odd = __ballot_sync(0xffffffffu, bad1);
            nan_keys[0] = nan_keys[1] = 0;
            if (even | odd) {  // keys 2 lane, 2 lane + 1 of each lane, as bits of the keys
              for (int x = 0; x < 32; ++x) nan_keys[x >> 4] |= ((even >> x & 1) | (odd >> x & 1) << 1) << (2 * x & 31);
            }
          }
          __syncwarp();  // the warp has read the page before's
          *reinterpret_cast<float2*>(&bars.f8.ks[warp - 4][2 * (r & 31)]) = k2;
          *reinterpret_cast<float2*>(&bars.f8.lk[warp - 4][2 * (r & 31)]) = l2;
          __syncwarp();
          tab[0] = tab[1];
          tab[1] = entry(pg + 2);
          ks_next = scales(tab[0]);
        }
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.s_full[g & 1], (g >> 1) & 1, abort_flag, p.err));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t s_addr = tmem + lane_off + 128 + (g & 1) * 64;
        float s[64];
        {
          uint32_t* su = reinterpret_cast<uint32_t*>(s);
          ptx::tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(su));
          ptx::tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(su + 32));
          ptx::tmem_ld_wait();
        }
        const int page = kF8 ? page8 : __ldg(p.page_table + (size_t)(seq / p.NQT) * p.max_pages + pg);
        const bool bad = page < 0 || page >= p.num_pages;
        if constexpr (kF8) {
          if (bad && r == 0 && seq % p.NQT == 0) latch_error(p.err, kErrBadPage);
          if (pg == lo)  // written before this segment's first scores were issued
            f8_scale = p.scale_log2 * __int_as_float((127 - bars.f8.q_exp[n_epi & 1][r]) << 23);
        }
        const int key0 = pg * kPage;
        const int lim = bad ? -1 : min(last_visible, L - 1);  // visible keys: key0+x <= lim
        // unscaled scores (fp8: times the key's scale), two keys per packed instruction; the
        // softmax scale is applied in the exponent argument
        // (kF8: scaled scores, in the exponent's units)
        const float* ks;
        if constexpr (kF8) ks = bars.f8.ks[warp - 4];
        else ks = bars.kscale[kFp8 ? g % kStages : 0];
        uint64_t s2[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          s2[x] = ptx::f2(s[2 * x], s[2 * x + 1]);
          if constexpr (kF8)
            s2[x] = ptx::mul2(ptx::mul2(s2[x], *reinterpret_cast<const uint64_t*>(ks + 2 * x)), ptx::f2(f8_scale, f8_scale));
          else if constexpr (kFp8) s2[x] = ptx::mul2(s2[x], ptx::f2(ks[2 * x], ks[2 * x + 1]));
        }
        if constexpr (kTree) {
          if (bad) vis = 0;
          if (tree_page || bad) {
            if (tree_page && !bad) {
              // keys whose row (or scale) is not finite, hardly ever any: NaN for who sees them
              const unsigned char* kn = bars.key_nan[g & 1];
              const uint32_t f0 = __ballot_sync(0xffffffffu, kn[r & 31] != 0) | nan_keys[0];
              const uint32_t f1 = __ballot_sync(0xffffffffu, kn[32 + (r & 31)] != 0) | nan_keys[1];
              if (f0 | f1) {
                const float nan = __int_as_float(0x7fc00000);
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                  const uint32_t f = x < 16 ? f0 >> (2 * x) : f1 >> (2 * x - 32);
                  s2[x] = ptx::f2(f & 1 ? nan : ptx::f2_lo(s2[x]), f & 2 ? nan : ptx::f2_hi(s2[x]));
                }
              }
            }
            const uint32_t v0 = static_cast<uint32_t>(vis), v1 = static_cast<uint32_t>(vis >> 32);
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const uint32_t v = x < 16 ? v0 : v1;
              s2[x] = ptx::f2(v & (1u << (2 * x & 31)) ? ptx::f2_lo(s2[x]) : -INFINITY,
                              v & (2u << (2 * x & 31)) ? ptx::f2_hi(s2[x]) : -INFINITY);
            }
          }
        } else if (key0 + kPage - 1 > lim) {  // a partial page (or a bad one): mask invisible keys
#pragma unroll
          for (int x = 0; x < 32; ++x)
            s2[x] = ptx::f2(key0 + 2 * x <= lim ? ptx::f2_lo(s2[x]) : -INFINITY,
                            key0 + 2 * x + 1 <= lim ? ptx::f2_hi(s2[x]) : -INFINITY);
        }
        // kF8: the weights P'' = p ks are what has to fit the two terms, so the maximum is that of their
        // exponents, and it is mapped to 2^5: they lie in (0, 2^8]
        auto exponents = [&](int x) {
          if constexpr (kF8) return ptx::add2(s2[x], *reinterpret_cast<const uint64_t*>(&bars.f8.lk[warp - 4][2 * x]));
          else return s2[x];
        };
        constexpr float kTop = kF8 ? 5.f : 0.f;
        const uint64_t e0 = exponents(0), e1 = exponents(1);
        float mx4[4] = {ptx::f2_lo(e0), ptx::f2_hi(e0), ptx::f2_lo(e1), ptx::f2_hi(e1)};
#pragma unroll
        for (int x = 2; x < 32; ++x) {
          const uint64_t ex = exponents(x);
          mx4[x & 3] = ptx::fmax3(mx4[x & 3], ptx::f2_lo(ex), ptx::f2_hi(ex));
        }
        // tile maximum in the exponent domain (the scale is positive; -inf stays -inf)
        const float mx = kF8 ? ptx::fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) - kTop
                             : ptx::fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) * p.scale_log2;
        float m_use = m;
        if (pg == lo) {
          m_use = mx;
          if constexpr (kF8) f8_mass = f8_steps = 0.f;
        } else {
          // (a tree's rows past the last token hold whatever lay in the ring: they ask for nothing)
          const bool asks = !kTree || (r < TQ && gr < TH);
          const bool grow = asks && mx > m + (8.0f - kTop);
          const bool fall = kF8 && asks && mx < m - (kF8FallTo + 3.f) && mx > m - 20.f && l < 0x1p80f &&
                            f8_steps > kF8StepsPerMass * f8_mass;
          if (__any_sync(0xffffffffu, grow || fall)) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.o_done, (g - 1) & 1, abort_flag, p.err));
            if (!ok) break;
            ptx::tc_fence_after();
            if (grow) m_use = mx;
            if (fall) m_use = mx + kF8FallTo;
            const float alpha = grow || fall ? ptx::ex2(m - m_use) : 1.f;  // m = -inf gives 0
            if constexpr (kF8) {
              f8_mass *= alpha;
              f8_steps = fall ? 0.f : f8_steps * alpha;
            }
            uint32_t v[2][32];
#pragma unroll 1
            for (int c = 0; c < 8; c += 2) {
              ptx::tmem_ld32(o_addr + c * 32, v[0]);
              ptx::tmem_ld32(o_addr + (c + 1) * 32, v[1]);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                v[0][x] = __float_as_uint(__uint_as_float(v[0][x]) * alpha);
                v[1][x] = __float_as_uint(__uint_as_float(v[1][x]) * alpha);
              }
              ptx::tmem_st32(o_addr + c * 32, v[0]);
              ptx::tmem_st32(o_addr + (c + 1) * 32, v[1]);
            }
            l *= alpha;
            lr *= alpha;
          }
        }
        m = m_use;
        const float neg_m = (m == -INFINITY) ? 0.f : -m;
        const uint64_t sc2 = ptx::f2(p.scale_log2, p.scale_log2), nm2 = ptx::f2(neg_m, neg_m);
        uint64_t ps2[2] = {ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f)};
        float pr[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[32];
        if constexpr (kF8) {
#pragma unroll
          for (int x = 0; x < 32; x += 2) {  // four keys: one word of hi codes, one of lo codes
            uint32_t w16[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint64_t a2 = ptx::add2(s2[x + y], nm2);
              const uint64_t pp = ptx::f2(ptx::ex2(ptx::f2_lo(a2)), ptx::ex2(ptx::f2_hi(a2)));
              ps2[y] = ptx::add2(ps2[y], pp);
              const uint64_t ab = ptx::mul2(pp, *reinterpret_cast<const uint64_t*>(ks + 2 * (x + y)));
              w16[y] = ptx::pack_f16x2(ptx::f2_lo(ab), ptx::f2_hi(ab));
            }
            ptx::split_e4m3_e5m2x4(w16[0], w16[1], pk[x / 2], pk[16 + x / 2]);
          }
        }
#pragma unroll
        for (int x = 0; x < (kF8 ? 0 : 32); ++x) {
          const uint64_t a2 = ptx::fma2(s2[x], sc2, nm2);
          const uint64_t pp = ptx::f2(ptx::ex2(ptx::f2_lo(a2)), ptx::ex2(ptx::f2_hi(a2)));
          ps2[x & 1] = ptx::add2(ps2[x & 1], pp);
          if constexpr (kFp8) {
            const uint64_t ab = ptx::mul2(pp, ptx::f2(ks[2 * x], ks[2 * x + 1]));  // P' = p ks
            pk[x] = ptx::pack_bf16x2(ptx::f2_lo(ab), ptx::f2_hi(ab));
          } else {
            // O is normalised by the sum of the bf16-rounded values the PV product uses
            // (exact for a dominant key); the LSE uses the exact sum
            const uint32_t w = ptx::pack_bf16x2(ptx::f2_lo(pp), ptx::f2_hi(pp));
            pk[x] = w;
            ptx::add_bf16x2(pr[2 * (x & 1)], pr[2 * (x & 1) + 1], w);
          }
        }
        const uint64_t ps_all = ptx::add2(ps2[0], ps2[1]);
        const float psum = ptx::f2_lo(ps_all) + ptx::f2_hi(ps_all);
        l += psum;
        lr += kFp8 ? psum : (pr[0] + pr[1]) + (pr[2] + pr[3]);
        ptx::tmem_st32(s_addr, pk);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bars.p_full[g & 1]);
        if constexpr (kF8) {
          const float w = mx == -INFINITY ? 0.f : ptx::ex2(mx - m);
          f8_mass += w;
          f8_steps += fminf(1.f, 65536.f * w);
        }
      }
      if (!ok) break;
      // epilogue of the segment: partial (O_half / l, LSE) into slot unit + seq, once the
      // segment's last PV product is complete.  That is signalled once per segment: the
      // per-page o_done cannot be used here, since a warp that ran ahead of a slower one may
      // arrive while PV(g-2) is still pending and one parity bit cannot tell that phase from
      // the one after PV(g-1).  seg_done of the next segment needs this warp's P, so it is
      // never more than one phase ahead.
      bool last_seg;
      auto look_ahead = [&]() {
        Segments nx = segs;
        int s2, L2, lo2, hi2;
        last_seg = !nx.next(s2, L2, lo2, hi2);
      };
      if constexpr (kTree) look_ahead();  // while the last PV product is on its way
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.seg_done, n_epi & 1, abort_flag, p.err));
      if (!ok) break;
      ptx::tc_fence_after();
      const size_t slot = (size_t)unit + seq;
      if (pad_row) l = lr = 0.f;
      // (tree: a NaN sum stays one, and a row without keys is zero whatever its accumulator holds)
      const float inv = (kTree ? lr != 0.f : lr > 0.f) ? 1.f / lr : 0.f;
      const float lse_own = (kTree ? l != 0.f : l > 0.f) ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
      auto own_o = [&](uint32_t v) {
        const float o = __uint_as_float(v) * inv;
        return kTree && lr == 0.f ? 0.f : o;
      };
      const bool row_live = r < TQ && gr < TH;
      const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;  // tree: rows in whole sectors
      // The work units that cover this virtual sequence write their partials of this column
      // half into slots c + seq, c_first <= c <= c_first + nsplit - 1; this one is k_own.
      const int n_pages = pages_of(L, kPage);
      const int c_first = segs.flat0 / bars.plan.chunk;
      const int nsplit = (segs.flat0 + n_pages - 1) / bars.plan.chunk - c_first + 1;
      const int k_own = unit - c_first;
      // (a tree's other items are merged by the kernel behind this one)
      const bool deferred = kTree && nsplit > (p.few ? 1 : kFusedSplits);
      if (kTree && p.few && half == 0 && k_own == 0 && r == 0) p.deferred[1 + seq] = make_int4(seq, c_first, nsplit, 0);
      // Merge path.  A split that finds every other split of this (sequence, column half)
      // counted in (always so for a sequence with one split) merges at once, its own share
      // read from the accumulator.  Otherwise it writes its partial (O_half / l, LSE), makes
      // it visible device-wide and counts itself in; the split that completes the count
      // merges: O = sum_c exp(lse_c - lse) O_c with lse = ln sum_c exp(lse_c).
      // After the unit's last segment nothing more is loaded and every MMA is complete: Q's
      // area takes the staged bf16 output rows, the page stages a bulk copy of the other
      // split's partial when the sequence has exactly two (one TMA transfer instead of
      // rounds of dependent L2 loads per thread).
      if constexpr (!kTree) look_ahead();
      // (a tree's item in one split needs no decision: it merges)
      const bool decide = !kTree || nsplit > 1;
      if (r == 0 && decide) {
        int fast = 1, bulk = 0;
        if (deferred) {
          fast = 0;
          if (!p.few && half == 0 && k_own == 1) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // zeroed before
            p.deferred[1 + atomicAdd(&p.deferred[0].x, 1)] = make_int4(seq, c_first, nsplit, 0);
          }
        } else if (nsplit > 1) {
          // the counters were zeroed by the kernel this one was launched behind
          asm volatile("griddepcontrol.wait;" ::: "memory");
          fast = ptx::ld_acquire_gpu(p.counters + (size_t)seq * 2 + half) == nsplit - 1;
          if (fast && nsplit == 2 && last_seg) {
            const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                                ((size_t)(c_first + seq + (1 - k_own)) * 128 + half * 64) * TQ;
            ptx::fence_proxy_async_global();
            ptx::mbar_arrive_expect_tx(&bars.merge_full, 1024u * TQ);
            ptx::bulk_load(sm + kOffStage, src, 1024u * TQ, &bars.merge_full);
            bulk = 1;
            ++n_bulk_issued;
          }
        }
        bars.merge_fast = fast;
        bars.merge_bulk = bulk;
        ptx::mbar_arrive(&bars.dec_go);
      }
      if (decide) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.dec_go, n_dec++ & 1, abort_flag, p.err));
      ++n_epi;
      if (!ok) break;
      // The accumulator is intact until the next segment's first PV product, which waits for
      // this epilogue: a split that merges always takes its own share from it.
      bool own_in_tmem = !decide || *reinterpret_cast<volatile int*>(&bars.merge_fast) != 0;
      bool bulk = decide && *reinterpret_cast<volatile int*>(&bars.merge_bulk) != 0;
      bool merge = own_in_tmem;
      if (!own_in_tmem) {
        // partial layout [slot][column quad (128)][row (T*H)][4]: the 32 rows of a warp store
        // one quad as 512 contiguous bytes; kept in L2 ahead of the cache lines streaming past,
        // since the merge reads it back, possibly at the end of the launch
        const uint64_t keep = ptx::l2_policy_evict_last();
        float4* dst = reinterpret_cast<float4*>(p.part_o) + (slot * 128 + half * 64) * TQ + r;
#pragma unroll 1
        for (int c = 0; c < 8; c += 2) {
          uint32_t v[2][32];
          ptx::tmem_ld32(o_addr + c * 32, v[0]);
          ptx::tmem_ld32(o_addr + (c + 1) * 32, v[1]);
          ptx::tmem_ld_wait();
          if (row_live) {
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                float4* d4 = dst + (size_t)((c + h2) * 8 + x) * TQ;
                if (MLA_STORE_OK(d4, p.part_o, p.part_o_bytes, p.err))
                  ptx::st_l2_hint(d4,
                                  make_float4(own_o(v[h2][4 * x]), own_o(v[h2][4 * x + 1]), own_o(v[h2][4 * x + 2]),
                                              own_o(v[h2][4 * x + 3])),
                                  keep);
              }
          }
        }
        float* plp = p.part_lse + ((size_t)half * p.n_slots + slot) * TQ + r;
        if (row_live && MLA_STORE_OK(plp, p.part_lse, p.part_lse_bytes, p.err)) *plp = lse_own;
      }
      if (!own_in_tmem && !deferred) {
        __threadfence();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bars.part_done);
        if (r == 0) {
          bool go = ptx::mbar_wait(&bars.part_done, n_part & 1, abort_flag, p.err);
          if (go) {
            __threadfence();
            int* cnt = p.counters + (size_t)seq * 2 + half;
            const int done = MLA_STORE_OK(cnt, p.counters, p.counters_bytes, p.err) ? atomicAdd(cnt, 1) + 1 : 0;
            __threadfence();
            bars.merge_last = done == nsplit ? 1 : 0;
            if (done == nsplit && nsplit == 2 && last_seg) {
              const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                                  ((size_t)(c_first + seq + (1 - k_own)) * 128 + half * 64) * TQ;
              ptx::fence_proxy_async_global();
              ptx::mbar_arrive_expect_tx(&bars.merge_full, 1024u * TQ);
              ptx::bulk_load(sm + kOffStage, src, 1024u * TQ, &bars.merge_full);
              bars.merge_bulk = 1;
              ++n_bulk_issued;
            }
          } else {
            bars.merge_last = 0;
          }
          ptx::mbar_arrive(&bars.merge_go);
        }
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.merge_go, n_part & 1, abort_flag, p.err));
        ++n_part;
        if (!ok) break;
        merge = *reinterpret_cast<volatile int*>(&bars.merge_last) != 0;
        bulk = *reinterpret_cast<volatile int*>(&bars.merge_bulk) != 0;
        own_in_tmem = merge;
      }
      if (kTree && !decide) {
        // One split: the rows go out from the accumulator.  A thread stores its own row, whole 32-byte
        // sectors at a time: half sectors took 1.2 us a round of 64 columns, most of an epilogue of 8 us.
        uint4* orow = reinterpret_cast<uint4*>(p.out + ((size_t)(seq / p.NQT) * TH + gr) * kDl + half * 256);
#pragma unroll 1
        for (int c = 0; c < 256; c += 64) {
          uint32_t v[2][32];
          ptx::tmem_ld32(o_addr + c, v[0]);
          ptx::tmem_ld32(o_addr + c + 32, v[1]);
          ptx::tmem_ld_wait();
          if (!row_live) continue;
#pragma unroll
          for (int j = 0; j < 64; j += 16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = ptx::pack_bf16x2(own_o(v[j >> 5][(j & 31) + 2 * i]), own_o(v[j >> 5][(j & 31) + 2 * i + 1]));
            uint4* at = orow + (c + j) / 8;
            if (!MLA_STORE_OK(at + 1, p.out, p.out_bytes, p.err)) continue;  // (the later of the two)
            if (wide) {
              ptx::st_v8(at, w);
            } else {
              at[0] = make_uint4(w[0], w[1], w[2], w[3]);
              at[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
        float* lp = p.lse + ((size_t)(seq / p.NQT) * p.H + gr % p.H) * p.T + gr / p.H;
        if (half == 0 && row_live && MLA_STORE_OK(lp, p.lse, p.lse_bytes, p.err)) *lp = lse_own;
      } else if (merge) {
        // Every lane of a warp runs this block (the accumulator loads are warp-collective:
        // a lane that skipped them would stall its warp for good); global memory is touched
        // for the live rows only.  This thread's row: weights of the splits from their LSEs
        // (read through L2: they were written by other SMs during this launch).  The first
        // kLseRegs LSEs are loaded together and kept; any further split's is read again
        // where it is used.
        const float* lsp = p.part_lse + ((size_t)half * p.n_slots + c_first + seq) * TQ + r;
        auto lse_of = [&](int k) -> float {
          if (own_in_tmem && k == k_own) return lse_own;
          return row_live ? ptx::ld_l2(lsp + (size_t)k * TQ) : -INFINITY;
        };
        constexpr int kLseRegs = 4;
        float lse_r[kLseRegs];
#pragma unroll
        for (int k = 0; k < kLseRegs; ++k) lse_r[k] = k < nsplit ? lse_of(k) : -INFINITY;
        float mxl = -INFINITY;
#pragma unroll
        for (int k = 0; k < kLseRegs; ++k) mxl = fmaxf(mxl, lse_r[k]);
        for (int k = kLseRegs; k < nsplit; ++k) mxl = fmaxf(mxl, lse_of(k));
        auto wraw = [&](float ls) {
          if (kTree && ls != ls) return ls;
          return (mxl == -INFINITY || ls == -INFINITY) ? 0.f : __expf(ls - mxl);
        };
        float wsum = 0.f;
#pragma unroll
        for (int k = 0; k < kLseRegs; ++k) wsum += wraw(lse_r[k]);
        for (int k = kLseRegs; k < nsplit; ++k) wsum += wraw(lse_of(k));
        const float winv = (kTree ? wsum != 0.f : wsum > 0.f) ? 1.f / wsum : 0.f;
        float w_r[kLseRegs];
#pragma unroll
        for (int k = 0; k < kLseRegs; ++k) w_r[k] = wraw(lse_r[k]) * winv;
        const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                            ((size_t)(c_first + seq) * 128 + half * 64) * TQ + r;
        const size_t slot_stride = (size_t)128 * TQ;
        uint4* orow = reinterpret_cast<uint4*>(
            p.out + ((size_t)(seq / p.NQT) * TH + gr) * kDl + half * 256);
        // After the unit's last segment the bf16 rows are staged in Q's area, 512 bytes per
        // row with 16-byte chunk c of row r at chunk c ^ (r mod 32), and each warp then stores
        // its 32 rows as one 512-byte run per instruction.  Earlier segments store straight
        // from the row's thread.
        const bool staged = last_seg;
        unsigned char* stage_out = sm + kOffQhi;
        // the bulk-copied partial of the other split: [quad][row][4] floats from the stages
        const float4* part_sm = reinterpret_cast<const float4*>(sm + kOffStage) + r;
        if (bulk) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars.merge_full, n_bulk & 1, abort_flag, p.err));
          ++n_bulk;
          if (!ok) break;
        }
        // Sixteen column quads (64 columns) per round: 16 independent 16-byte loads of a
        // split's partial in flight.  The splits are summed in split order, each as weight x
        // (O_c / l_c) in fp32, the own share formed from the accumulator exactly as its stored
        // partial would be: the result does not depend on which split merges.
#pragma unroll 1
        for (int q = 0; q < 64; q += 16) {
          float4 acc[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int k = 0; k < nsplit; ++k) {
            const float w = k == 0 ? w_r[0] : k == 1 ? w_r[1] : k == 2 ? w_r[2] : k == 3 ? w_r[3]
                                                                                 : wraw(lse_of(k)) * winv;
            float4 x[16];
            if (own_in_tmem && k == k_own) {
              uint32_t v[2][32];
              ptx::tmem_ld32(o_addr + q * 4, v[0]);
              ptx::tmem_ld32(o_addr + q * 4 + 32, v[1]);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[j] = make_float4(own_o(v[j >> 3][4 * (j & 7)]), own_o(v[j >> 3][4 * (j & 7) + 1]),
                                   own_o(v[j >> 3][4 * (j & 7) + 2]), own_o(v[j >> 3][4 * (j & 7) + 3]));
            } else if (bulk) {  // the other split of two, copied into shared memory
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[j] = row_live ? part_sm[(size_t)(q + j) * TQ] : make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
              const float4* b = src + (size_t)k * slot_stride;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[j] = row_live ? ptx::ld_l2(b + (size_t)(q + j) * TQ) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              acc[j].x = fmaf(w, x[j].x, acc[j].x);
              acc[j].y = fmaf(w, x[j].y, acc[j].y);
              acc[j].z = fmaf(w, x[j].z, acc[j].z);
              acc[j].w = fmaf(w, x[j].w, acc[j].w);
            }
          }
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            uint32_t w[8];  // 16 columns: 16-byte chunks ch and ch + 1 of the row's 512 bytes
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[2 * i] = ptx::pack_bf16x2(acc[j + i].x, acc[j + i].y);
              w[2 * i + 1] = ptx::pack_bf16x2(acc[j + i].z, acc[j + i].w);
            }
            const int ch = (q + j) >> 1;
            if (kTree && wide && !staged) {
              if (row_live && MLA_STORE_OK(orow + ch + 1, p.out, p.out_bytes, p.err)) ptx::st_v8(orow + ch, w);
              continue;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 x = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
              if (staged)
                *reinterpret_cast<uint4*>(stage_out + r * 512 + (((ch + i) ^ (r & 31)) << 4)) = x;
              else if (row_live && MLA_STORE_OK(orow + ch + i, p.out, p.out_bytes, p.err))
                orow[ch + i] = x;
            }
          }
        }
        if (staged) {
          __syncwarp();
          const int lane = threadIdx.x & 31;
          const int r_base = r - lane;  // the warp's 32 rows
#pragma unroll 4
          for (int i = 0; i < 32; ++i) {
            const int rr = r_base + i, grr = (seq % p.NQT) * kRows + rr;
            uint4* od = reinterpret_cast<uint4*>(p.out + ((size_t)(seq / p.NQT) * TH + grr) * kDl + half * 256) + lane;
            if (rr < TQ && grr < TH && MLA_STORE_OK(od, p.out, p.out_bytes, p.err))
              *od = *reinterpret_cast<const uint4*>(stage_out + rr * 512 + ((lane ^ (rr & 31)) << 4));
          }
        }
        float* lp = p.lse + ((size_t)(seq / p.NQT) * p.H + gr % p.H) * p.T + gr / p.H;
        if (half == 0 && row_live && MLA_STORE_OK(lp, p.lse, p.lse_bytes, p.err))
          *lp = (kTree ? wsum != 0.f : wsum > 0.f) ? mxl + logf(wsum) : -INFINITY;
      }
      // the accumulator was read: the next segment's first PV product may overwrite it
      ptx::tc_fence_before();
    }
    // after an abort: a bulk copy issued but never waited for lands before the CTA exits
    if (r == 0 && n_bulk_issued > n_bulk) ptx::mbar_wait_drain(&bars.merge_full, n_bulk & 1);
  }
  // Kernels behind this one may be its programmatic dependents, which wait for this one alone: it ends
  // after the zeroing kernel has, also where no item was split and so nobody waited for that above.
  if (threadIdx.x == 0) wait_for_stream();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Merges the tree items that no split merges (see kFusedSplits), all over the GPU: the split
// kernel lists them (Params::deferred), the blocks here share the list's slices of 32 rows and 16
// column quads.  Left to the split that finishes last, the merge reads every partial through one SM,
// about 4 us a split: one sequence of 1000 keys and 128 rows, in 16 splits, took 68 us, 50 of them
// there.  The splits are weighed and summed in split order, as in the split kernel's own merge.
constexpr int kMergeThreads = 256, kMergeRows = 32, kMergeQuads = 16;  // two quads a thread
constexpr int kMergeSlices = (kRows / kMergeRows) * (128 / kMergeQuads);
constexpr int kMergeBlocks = 304;

// One thread's part of a slice: row r of the item (gr of its sequence's), column quads q and q + 1, of
// nsplit splits from the item's first on, eight of them in flight; the first eight log-sum-exps stay
// in registers.
__device__ __forceinline__ void merge_row(const Params& p, int item, int c_first, int nsplit, int r, int gr, int q) {
  constexpr int kBatch = 8;
  const float* lsp = p.part_lse + ((size_t)(q / 64) * p.n_slots + c_first + item) * p.TQ + r;
  float first[kBatch], mx = -INFINITY, sum = 0.f;
  auto lse_of = [&](int k) { return k < nsplit ? ptx::ld_l2(lsp + (size_t)k * p.TQ) : -INFINITY; };
  auto weight = [&](float ls) { return ls != ls ? ls : ls == -INFINITY ? 0.f : __expf(ls - mx); };
#pragma unroll
  for (int k = 0; k < kBatch; ++k) first[k] = lse_of(k);
#pragma unroll
  for (int k = 0; k < kBatch; ++k) mx = fmaxf(mx, first[k]);
  for (int k0 = kBatch; k0 < nsplit; k0 += kBatch) {
    float ls[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) ls[k] = lse_of(k0 + k);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) mx = fmaxf(mx, ls[k]);
  }
#pragma unroll
  for (int k = 0; k < kBatch; ++k) sum += weight(first[k]);
  for (int k0 = kBatch; k0 < nsplit; k0 += kBatch) {
    float ls[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) ls[k] = lse_of(k0 + k);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) sum += weight(ls[k]);
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const float4* src = reinterpret_cast<const float4*>(p.part_o) + ((size_t)(c_first + item) * 128 + q) * p.TQ + r;
  const size_t slot_stride = (size_t)128 * p.TQ;
  float4 acc[2] = {};
  for (int k0 = 0; k0 < nsplit; k0 += kBatch) {
    float4 x[kBatch][2];
    float ls[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      ls[k] = k0 == 0 ? first[k] : lse_of(k0 + k);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        x[k][j] = k0 + k < nsplit ? ptx::ld_l2(src + (k0 + k) * slot_stride + (size_t)j * p.TQ)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = weight(ls[k]) * inv;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[j].x = fmaf(w, x[k][j].x, acc[j].x);
        acc[j].y = fmaf(w, x[k][j].y, acc[j].y);
        acc[j].z = fmaf(w, x[k][j].z, acc[j].z);
        acc[j].w = fmaf(w, x[k][j].w, acc[j].w);
      }
    }
  }
  uint4* o = reinterpret_cast<uint4*>(p.out + ((size_t)(item / p.NQT) * p.T * p.H + gr) * kDl + q * 4);
  if (MLA_STORE_OK(o, p.out, p.out_bytes, p.err))
    *o = make_uint4(ptx::pack_bf16x2(acc[0].x, acc[0].y), ptx::pack_bf16x2(acc[0].z, acc[0].w),
                    ptx::pack_bf16x2(acc[1].x, acc[1].y), ptx::pack_bf16x2(acc[1].z, acc[1].w));
  float* lp = p.lse + ((size_t)(item / p.NQT) * p.H + gr % p.H) * p.T + gr / p.H;
  if (q == 0 && MLA_STORE_OK(lp, p.lse, p.lse_bytes, p.err)) *lp = sum != 0.f ? mx + logf(sum) : -INFINITY;
}

__global__ void __launch_bounds__(kMergeThreads, 2) tree_merge_kernel(const Params p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_stream();  // the split kernel is done, and with it the zeroing
  const int listed = p.few ? p.B * p.NQT : min(__ldcg(&p.deferred[0].x), p.G);
  const int work = listed * kMergeSlices;
  for (int w = blockIdx.x; w < work; w += gridDim.x) {
    const int4 d = __ldcg(reinterpret_cast<const int4*>(p.deferred + 1) + w / kMergeSlices);
    const int item = d.x, c_first = d.y, nsplit = d.z, slice = w % kMergeSlices;
    // (an entry that a split kernel that gave up left unwritten may hold anything)
    if (nsplit < 2 || nsplit > p.G || c_first < 0 || c_first > p.G - nsplit) continue;
    if (item < 0 || item >= p.B * p.NQT || (p.few && item != w / kMergeSlices)) continue;
    const int r = (slice & 3) * kMergeRows + lane, gr = (item % p.NQT) * kRows + r;
    if (r >= p.TQ || gr >= p.T * p.H) continue;
    const int q = (slice >> 2) * kMergeQuads + 2 * warp;
    merge_row(p, item, c_first, nsplit, r, gr, q);
  }
}

// Zeroes the split counters of a decode call; the split kernel is launched behind it as a
// programmatic dependent and waits for it where it first touches a counter, or else before it ends.
__global__ void __launch_bounds__(256) zero_counters_kernel(int* __restrict__ c, int n,
                                                               int4* __restrict__ deferred) {
  // (A tree's zeroing is itself a programmatic dependent.  It lets the split kernel, which reads its
  // inputs without waiting, start only once the work ahead is complete.)
  if (deferred) wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (deferred && blockIdx.x == 0 && threadIdx.x == 0) deferred[0] = make_int4(0, 0, 0, 0);
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) c[i] = 0;
}

}  // namespace sm103_decode

// ---------------------------------------------------------------- host side

// Makes the driver load every decode kernel on the current device (under lazy module loading
// a kernel's module is otherwise loaded, and its device memory allocated, at its first launch).
cudaError_t load_decode_t_kernels();
cudaError_t load_decode_kernels() {
  using namespace sm103_decode;
  cudaFuncAttributes fa;
  cudaError_t e = load_decode_t_kernels();
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncGetAttributes(&fa, decode_split_kernel<false, false>)) != cudaSuccess) return e;
  if ((e = cudaFuncGetAttributes(&fa, decode_split_kernel<true, false>)) != cudaSuccess) return e;
  return cudaFuncGetAttributes(&fa, zero_counters_kernel);
}

cudaError_t encode_tensor_map_swz(CUtensorMap* map, CUtensorMapDataType dt, int rank,
                                  const void* ptr, const uint64_t* dims, const uint64_t* strides,
                                  const uint32_t* box, bool swizzle128);
cudaError_t encode_tensor_map_swizzle(CUtensorMap* map, CUtensorMapDataType dt, int rank,
                                      const void* ptr, const uint64_t* dims, const uint64_t* strides,
                                      const uint32_t* box, CUtensorMapSwizzle swizzle);

cudaError_t launch_decode_sm103(const void* q_latent, const void* q_rope, const void* kv_cache,
                                const float* kv_scale, const int* page_table,
                                const int* cache_lens, int B, int H, int T, int max_pages,
                                int num_pages, float softmax_scale, int causal, bool fp8,
                                const void* tree_mask, long long mask_stride, const int* new_lens,
                                float* part_o, float* part_lse, int* counters, void* out,
                                float* lse, int G, unsigned int* err, cudaStream_t stream) {
  using namespace sm103_decode;
  CUtensorMap tm;
  // the cache as a 2-D tensor [num_pages * 64 rows, 576 columns]; boxes of 64 x 64
  // (the tree over an fp8 cache: 128 columns, swizzled as operands, and the rope columns on their own)
  const bool f8 = fp8 && tree_mask;
  uint64_t dims[2] = {(uint64_t)kDc, (uint64_t)num_pages * kPage};
  uint64_t strides[1] = {(uint64_t)kDc * (fp8 ? 1 : 2)};
  uint32_t box[2] = {f8 ? 128u : 64u, kPage};
  cudaError_t e = encode_tensor_map_swz(
      &tm, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kv_cache,
      dims, strides, box, /*swizzle128=*/!fp8 || f8);
  if (e != cudaSuccess) return e;
  // the list of deferred items in a slot of one row (2048 bytes)
  if (tree_mask && (G + 1) * sizeof(int4) > kDl * sizeof(float)) return cudaErrorNotSupported;
  // The same bytes as a 3-D tensor (64 columns of a chunk, row, chunk of 64 columns): a box
  // of 64 x 64 x n is n consecutive 64-column chunks of a page, landing chunk-major exactly as
  // n 2-D boxes do (one TMA instruction instead of n): fp8 pages take one box of nine chunks,
  // bf16 page parts boxes of four and five.  The chunk stride is smaller than the row stride
  // (an overlapping view); should the driver refuse that, the 2-D boxes are used.
  CUtensorMap tm_page = tm, tm_c4 = tm, tm_c5 = tm;
  uint64_t pdims[3] = {64, (uint64_t)num_pages * kPage, 9};
  uint64_t pstrides[2] = {(uint64_t)kDc * (fp8 ? 1 : 2), (uint64_t)(fp8 ? 64 : 128)};
  const CUtensorMapDataType pdt = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto enc3 = [&](CUtensorMap* m, uint32_t nchunks) {
    uint32_t pbox[3] = {64, (uint32_t)kPage, nchunks};
    return encode_tensor_map_swz(m, pdt, 3, kv_cache, pdims, pstrides, pbox, /*swizzle128=*/!fp8) == cudaSuccess;
  };
  bool page_box;
  if (f8) {
    const uint64_t d3[3] = {128, (uint64_t)num_pages * kPage, 4}, s3[2] = {(uint64_t)kDc, 128};
    const uint32_t b3[3] = {128, (uint32_t)kPage, 4}, br[2] = {64, (uint32_t)kPage};
    page_box = encode_tensor_map_swz(&tm_page, pdt, 3, kv_cache, d3, s3, b3, true) == cudaSuccess;
    if (!page_box) tm_page = tm;
    if ((e = encode_tensor_map_swizzle(&tm_c4, pdt, 2, kv_cache, dims, strides, br, CU_TENSOR_MAP_SWIZZLE_64B)) != cudaSuccess)
      return e;
  } else {
    page_box = enc3(&tm_page, 9) && (fp8 || (enc3(&tm_c4, 4) && enc3(&tm_c5, 5)));
    if (!page_box) tm_page = tm_c4 = tm_c5 = tm;
  }
  // Q as 2-D tensors [B*T*H rows, 512 | 64 columns]; boxes of 64 columns x T*H rows
  // (one sequence), 128B-swizzled like the operand tiles
  const int TH = T * H;
  CUtensorMap tm_qlat, tm_qrope;
  uint64_t qdims[2] = {(uint64_t)kDl, (uint64_t)B * TH};
  uint64_t qstrides[1] = {(uint64_t)kDl * 2};
  const int TQ = TH < 128 ? TH : 128;
  uint32_t qbox[2] = {64, (uint32_t)TQ};
  e = encode_tensor_map_swz(&tm_qlat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q_latent, qdims, qstrides, qbox, true);
  if (e != cudaSuccess) return e;
  qdims[0] = 64;
  qstrides[0] = 128;
  e = encode_tensor_map_swz(&tm_qrope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q_rope, qdims, qstrides, qbox, true);
  if (e != cudaSuccess) return e;
  Params p;
  p.q_latent = static_cast<const uint16_t*>(q_latent);
  p.q_rope = static_cast<const uint16_t*>(q_rope);
  p.kv_scale = kv_scale;
  p.cache_bytes = static_cast<const unsigned char*>(kv_cache);
  p.page_table = page_table;
  p.cache_lens = cache_lens;
  p.part_o = part_o;
  p.part_lse = part_lse;
  p.counters = counters;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.err = err;
  p.B = B;
  p.H = H;
  p.T = T;
  p.NQT = (TH + 127) / 128;
  p.TQ = TQ;
  p.n_slots = G + B * p.NQT;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.causal = causal;
  p.G = G;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.tree_mask = static_cast<const uint32_t*>(tree_mask);
  p.mask_stride = mask_stride;
  p.mask_words = (T + 31) / 32;
  p.new_lens = new_lens;
  p.deferred = reinterpret_cast<int4*>(part_o + (size_t)(p.n_slots - 1) * TQ * kDl);
  p.few = tree_mask && 2 * B * p.NQT <= G && B * p.NQT < 2048 / 16;  // the entries fit any slot
  p.page_box = page_box ? 1 : 0;
  // one flat page charged per work item (its Q load, epilogue and merge; measured against
  // 0, 2 and 4 on uniform and ragged batches: the same time for 64 sequences of 4096 keys,
  // up to 7 % less where sequences split over several units or end mid-unit)
  if (tree_mask) p.item_cost = fp8 ? kF8ItemCost : kTreeItemCost;  // at most, the plan adapts them
  else p.item_cost = 1;
  const size_t out_full = (size_t)B * T * H * kDl * 2;
  p.out_bytes = out_full - std::min(out_full, testing_out_shrink());
  p.lse_bytes = (size_t)B * H * T * sizeof(float);
  p.part_o_bytes = (size_t)(reinterpret_cast<char*>(part_lse) - reinterpret_cast<char*>(part_o));
  p.part_lse_bytes = (size_t)(reinterpret_cast<char*>(counters) - reinterpret_cast<char*>(part_lse));
  p.counters_bytes = (size_t)2 * B * p.NQT * sizeof(int);
  // the split counters of the merge start at zero on every call
  const long long n_cnt = 2LL * B * p.NQT;
  if (n_cnt > 0x7fffffffLL) return cudaErrorInvalidValue;
  // same shared-memory carveout as the split kernel, so the SMs are not reconfigured between
  // the two launches
  static int carveout_set = 0;
  if (!__atomic_load_n(&carveout_set, __ATOMIC_ACQUIRE)) {
    if ((e = cudaFuncSetAttribute(zero_counters_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                  cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
      return e;
    __atomic_store_n(&carveout_set, 1, __ATOMIC_RELEASE);
  }
  const int zero_blocks = (int)std::min<long long>((n_cnt + 2047) / 2048, 1024);
  if (p.few) {
    // no counter is used
  } else if (tree_mask) {
    if ((e = launch_dependent(zero_counters_kernel, zero_blocks, 256, stream, counters, (int)n_cnt, p.deferred)) != cudaSuccess)
      return e;
  } else {
    zero_counters_kernel<<<zero_blocks, 256, 0, stream>>>(counters, (int)n_cnt, nullptr);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  auto go = [&](auto kern) -> cudaError_t {
    static unsigned long long smem_set[4] = {0, 0, 0, 0};
    const int smem = f8 ? kSmemBytes : kSmemAlloc;
    const cudaError_t e2 = smem_attr_once(kern, smem, &smem_set[(fp8 ? 1 : 0) + (tree_mask ? 2 : 0)]);
    if (e2 != cudaSuccess) return e2;
    // programmatic dependent of the zeroing kernel: the prologue (barriers, TMEM, plan, first
    // loads) overlaps it (Params::few: of the work ahead)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * G);
    cfg.blockDim = dim3(fp8 ? kThreadsOf<true> : kThreadsOf<false>);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tm, tm_page, tm_c4, tm_c5, tm_qlat, tm_qrope, p);
  };
  if (tree_mask) {
    if (fp8) {
      // the register split between its warpgroups draws on what the launch holds
      static int regs = 0;
      if (!__atomic_load_n(&regs, __ATOMIC_ACQUIRE)) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, decode_split_kernel<true, true>)) != cudaSuccess) return e;
        __atomic_store_n(&regs, fa.numRegs, __ATOMIC_RELEASE);
      }
      if (regs < kF8RegsLaunch) return cudaErrorInvalidDeviceFunction;
    }
    if ((e = fp8 ? go(decode_split_kernel<true, true>) : go(decode_split_kernel<false, true>)) != cudaSuccess) return e;
    return launch_dependent(tree_merge_kernel, kMergeBlocks, kMergeThreads, stream, p);
  }
  return fp8 ? go(decode_split_kernel<true, false>) : go(decode_split_kernel<false, false>);
}

}  // namespace mla
