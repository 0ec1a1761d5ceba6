// The rotation of 64 dimensions by a position's 32 angles, rounded once, and the
// loads and roundings of 16-byte pieces around it (the appends and the rotation
// of queries).
#pragma once

#include "indexer_common.h"

namespace pmqa {
namespace {

constexpr int kRope = IDX_ROPE_DIM;        // 64 rotated dimensions
constexpr int kHalfRope = kRope / 2;       // 32 angles

// The rotation of [tokens][heads] rows: workgroups of 32 heads of a token, and launches
// of up to kSlabTokens tokens.  (A grid is counted in threads, below 2^32: 2^24 tokens
// of one head in one launch have 2^32, a slab of 128 heads has 2^31.)
constexpr int kRotateThreads = 256;
constexpr int kHeadsPerWg = kRotateThreads / 8;
constexpr int kSlabTokens = 1 << 21;
inline int chunks_of(int32_t heads) { return (heads + kHeadsPerWg - 1) / kHeadsPerWg; }
inline uint32_t rotate_workgroups(int32_t tokens, int32_t heads) {
  return static_cast<uint32_t>(tokens) * chunks_of(heads);
}

struct F32Row {
  float v[8];
};

// Eight consecutive elements as float32 (exact for all three types).
template <int DT>
__device__ __forceinline__ F32Row load8(const char* p) {
  F32Row r;
  if constexpr (DT == IDX_FP32) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = a[i], r.v[4 + i] = b[i];
  } else {
    const i32x4 raw = *reinterpret_cast<const i32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = static_cast<uint32_t>(raw[i]);
      if constexpr (DT == IDX_BF16) {
        r.v[2 * i] = __uint_as_float(w << 16);
        r.v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
      } else {
        r.v[2 * i] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w)));
        r.v[2 * i + 1] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
      }
    }
  }
  return r;
}

// a c - b s (or, with s negated, b c + a s with the roles exchanged) in float64:
// two exact products and one rounding.
__device__ __forceinline__ double turn(float a, float c, float b, float s) {
  return static_cast<double>(a) * c - static_cast<double>(b) * s;
}

// The same rounded to odd: the nearest value, or its neighbour on the other side
// of the exact one where that is inexact and the nearest one's last bit is clear.
// A rounding to at most 51 bits of it is that of the exact value.  `lost`, what
// the sum's rounding took away, is exact.
__device__ __forceinline__ double turn_odd(float a, float c, float b, float s) {
  const double p = static_cast<double>(a) * c, q = -static_cast<double>(b) * s;
  const double sum = p + q, part = sum - p;
  const double lost = (p - (sum - part)) + (q - part);
  uint64_t bits = __builtin_bit_cast(uint64_t, sum);
  if ((lost < 0.0 || lost > 0.0) && !(bits & 1)) bits += (lost > 0.0) == (sum > 0.0) ? 1 : -1;  // (not for NaN)
  return __builtin_bit_cast(double, bits);
}

// Whether y (float64, within half a step of its last bit) may round otherwise
// than the exact value does when it is rounded to TO, by way of float32 f for the
// 16-bit types: where y, or f, lies half-way between two values of TO.  Below
// the smallest normal value half-way lies elsewhere; there, always.  (One random
// value in 2^29, 2^16 and 2^13.)
template <int TO>
__device__ __forceinline__ bool on_border(double y, float f) {
  const uint32_t bits = __float_as_uint(f);
  if constexpr (TO == IDX_BF16) return (bits & 0xFFFFu) == 0x8000u;  // (its subnormals are float32's)
  if constexpr (TO == IDX_FP16) return (bits & 0x1FFFu) == 0x1000u || (fabsf(f) < 0x1p-14f && f != 0.0f);
  return (static_cast<uint32_t>(__builtin_bit_cast(uint64_t, y)) & 0x1FFFFFFFu) == 0x10000000u ||
         (fabsf(f) < 0x1p-126f && y != 0.0);
}

// float32 of x: rounded to nearest, or, if it is rounded to 16 bits next, to odd.
template <int TO>
__device__ __forceinline__ float narrow(double x) {
  const float f = static_cast<float>(x);
  if constexpr (TO == IDX_FP32) return f;
  uint32_t bits = __float_as_uint(f);
  const double back = f;
  if ((back < x || back > x) && !(bits & 1)) bits += fabs(back) < fabs(x) ? 1 : -1;
  return __uint_as_float(bits);
}

// a c - b s as a float32 value whose rounding to TO is the rounding of the exact
// one.  (Without the branch, 8192 latent rows 5.5 -> 8.3 us; with one branch for
// the eight values of a lane, whose factors all stay in registers for it, 6.2.)
template <int TO>
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
  const double y = turn(a, c, b, s);
  const float f = static_cast<float>(y);
  if (__builtin_expect(on_border<TO>(y, f), false)) return narrow<TO>(turn_odd(a, c, b, s));
  return f;
}

// What dimensions 8 piece .. 8 piece + 7 of the 64 are turned by: eight angles
// from 8 (piece % 4), or, interleaved, four from 4 piece.  The second half of
// the pairs (i, i + 32) turns the other way.
struct Factors {
  float c[8], s[8];
};
__device__ __forceinline__ Factors factors_of(int piece, bool interleaved, const float* __restrict__ table) {
  Factors f;
  const int first = interleaved ? 4 * piece : 8 * (piece & 3), more = interleaved ? 0 : 4;
  const float sign = interleaved || piece < 4 ? 1.0f : -1.0f;
  const f32x4 c0 = *reinterpret_cast<const f32x4*>(table + first);
  const f32x4 c1 = *reinterpret_cast<const f32x4*>(table + first + more);
  const f32x4 s0 = *reinterpret_cast<const f32x4*>(table + kHalfRope + first);
  const f32x4 s1 = *reinterpret_cast<const f32x4*>(table + kHalfRope + first + more);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.c[i] = c0[i], f.c[4 + i] = c1[i];
    f.s[i] = sign * s0[i], f.s[4 + i] = sign * s1[i];
  }
  return f;
}

// Rotates eight of the 64 dimensions (x) in place, for rounding to TO; `partner`
// holds the same elements of the other half (unused when interleaved).
template <int TO>
__device__ __forceinline__ void turn8(F32Row& x, const F32Row& partner, bool interleaved, const Factors& f) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x.v[2 * i], b = x.v[2 * i + 1];
      x.v[2 * i] = turned<TO>(a, f.c[i], b, f.s[i]);
      x.v[2 * i + 1] = turned<TO>(b, f.c[i], a, -f.s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] = turned<TO>(x.v[i], f.c[i], partner.v[i], f.s[i]);
  }
}

template <int TO>
__device__ __forceinline__ void rotate8(F32Row& x, const F32Row& partner, int piece, bool interleaved,
                                        const float* __restrict__ table) {
  turn8<TO>(x, partner, interleaved, factors_of(piece, interleaved, table));
}

// Round to nearest even in the row's type.
template <int DT>
__device__ __forceinline__ uint32_t bits16(float x) {
  if constexpr (DT == IDX_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  return f16_bits_rn(x);
}

template <int DT>
__device__ __forceinline__ i32x4 pack16(const F32Row& x) {
  i32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = static_cast<int>(bits16<DT>(x.v[2 * i]) | (bits16<DT>(x.v[2 * i + 1]) << 16));
  return y;
}

// Eight float32 values of magnitudes up to 448, or NaN, as E4M3FN codes, nearest
// even.
__device__ __forceinline__ int2 e4m3_codes(const float (&x)[8]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return make_int2(lo, hi);
}

}  // namespace
}  // namespace pmqa
