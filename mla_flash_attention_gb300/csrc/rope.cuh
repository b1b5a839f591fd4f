// Position rotation shared by the head norms and the cache append.
//
// Frequency i of a 64-wide rope part turns by turns[i] * 2^-64 turns a position, turns[i] an
// unsigned 64-bit integer.  The phase of position p is the product p * turns[i] mod 2^64: whole
// turns fall off the top exactly, so the angle of a far position is as good as that of a near
// one (a product p * inv_freq in fp32 is off by up to 2^-25 p radians).  The phase error is
// p * 2^-65 turns from the rounding of turns[i] and 2^-32 turns from the 32 bits kept here.
// With several axes (time, height, width) a token has a position on each and turns is a table
// [axes][32]; the phase is the sum over the axes, as exact mod 2^64 as each term.  A pair that one
// axis turns has zeros in the other rows, so any assignment of pairs to axes is a table, and no index
// of an axis has to be read or checked.
#pragma once

#include "common.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace rope {

constexpr int kDr = 64, kFreqs = kDr / 2;
constexpr int kMaxAxes = 4;

// The phase of position `pos` (any int32, negative ones included) on one axis.
__device__ __forceinline__ unsigned long long phase(int pos, unsigned long long turns) {
  return static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
}

// cos and sin of a phase.  The angle lies in [-pi, pi), where the fast sine and cosine are within
// 2^-21 of the true ones: results are rounded to 8 bits or fewer, and the accurate functions took a
// quarter of the append's instructions.
__device__ __forceinline__ void cos_sin(unsigned long long phase, float& c, float& s) {
  // the top 32 bits, as a signed fraction of a turn in [-1/2, 1/2): times 2 pi 2^-32
  const float angle = static_cast<float>(static_cast<int>(phase >> 32)) * 1.4629180792671596e-9f;
  s = __sinf(angle);
  c = __cosf(angle);
}

// Eight consecutive bf16 as floats, and back (round to nearest even).
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                    ptx::pack_bf16x2(x[6], x[7]));
}

// The rotation of a 64-wide part spread over 8 lanes, lane j = lane & 7 holding columns
// 8j .. 8j + 7.  cos / sin of frequency f live in lane f of the warp.  kPairs: columns
// (2i, 2i + 1) turn together, else (i, i + 32).  kBack: by the opposite angle (the transpose,
// which takes a gradient back through the rotation).  All 32 lanes call it.
template <bool kPairs, bool kBack>
__device__ __forceinline__ void rotate8(float (&x)[8], float c_lane, float s_lane, int lane) {
  const int j = lane & 7;
  if constexpr (kPairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = __shfl_sync(0xffffffffu, c_lane, 4 * j + i);
      float s = __shfl_sync(0xffffffffu, s_lane, 4 * j + i);
      if (kBack) s = -s;
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c - b * s;
      x[2 * i + 1] = b * c + a * s;
    }
  } else {
    // lanes 0..3 hold the first of each pair, lanes 4..7 the second
    const bool second = (j & 4) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = __shfl_sync(0xffffffffu, c_lane, (8 * j + i) & 31);
      float s = __shfl_sync(0xffffffffu, s_lane, (8 * j + i) & 31);
      if (kBack) s = -s;
      const float other = __shfl_xor_sync(0xffffffffu, x[i], 4);
      x[i] = x[i] * c + (second ? other * s : -(other * s));
    }
  }
}

}  // namespace rope
}  // namespace mla
