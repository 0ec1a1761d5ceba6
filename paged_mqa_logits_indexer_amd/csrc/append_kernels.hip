// Appending rows to the paged caches, with the position rotation on the way
// (gfx950).
//
// A token at position p turns each pair (a, b) of its 64 rotated dimensions
// by that position's angle: (a, b) -> (a c - b s, b c + a s), the 32 cosines
// and 32 sines of p read from a table row.  The pairs are (i, i + 32), or
// (2i, 2i + 1) with `interleaved`.  The products of two 24-bit values are
// exact in float64, so the rotation is computed there, and where the result
// comes to lie on a rounding border, what was lost on the way decides: a rotated
// value is rounded once, and a code or a 16-bit value comes out as the definition
// says.  Float64 costs nothing here (all three kernels only move bytes).
//
//   index_k_append        FP8: scale = max|y| / 448 (float32), E4M3 codes of
//                         y / scale, nearest even; a token with a NaN or an
//                         infinity gets codes 0 and the scale NaN (its logits
//                         are NaN, which the top-k never selects)
//   index_k_append_mxfp4  per 32 dimensions a power of two, floor(log2 max|y|)
//                         - 2, and E2M1 codes, nearest even, saturating at 6;
//                         a block with a NaN or an infinity gets codes 0 and
//                         the E8M0 code 255 (NaN)
//   latent_append         512 dimensions as they are, 64 rotated, 16 bits each
//
// Every lane moves 16-byte pieces and no lane waits for another token's, so
// the kernels are bound by memory (and, for a few tokens, by one dependent
// load chain: slot and position, then the table row).  Measured (medians of 25
// under the kernel trace): 8192 latent rows 6.8 us (21 MB, 3.1 TB/s), 8191 MXFP4
// keys 4.8 us, 8 FP8 keys 2.5 us.
#include "indexer_common.h"
#include "launches.h"

namespace pmqa {
namespace {

constexpr int kRope = IDX_ROPE_DIM;        // 64 rotated dimensions
constexpr int kHalfRope = kRope / 2;       // 32 angles
constexpr int kThreads = 256;
constexpr int kLanesPerKey = kDim / 8;     // 16 lanes of 8 dimensions each
constexpr int kKeysPerWg = kThreads / kLanesPerKey;
constexpr int kRowPieces = IDX_LATENT_ROW * 2 / 16;    // 72 16-byte pieces of a latent row
constexpr int kLatentPieces = IDX_LATENT_DIM * 2 / 16;  // the first 64 are copied as they are

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

// Rotates dimensions 8 piece .. 8 piece + 7 of the 64 (x) in place, for rounding
// to TO; `partner` holds the same elements of the other half (unused when
// interleaved).
template <int TO>
__device__ __forceinline__ void rotate8(F32Row& x, const F32Row& partner, int piece, bool interleaved,
                                        const float* __restrict__ table) {
  if (interleaved) {
    const f32x4 c = *reinterpret_cast<const f32x4*>(table + 4 * piece);
    const f32x4 s = *reinterpret_cast<const f32x4*>(table + kHalfRope + 4 * piece);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x.v[2 * i], b = x.v[2 * i + 1];
      x.v[2 * i] = turned<TO>(a, c[i], b, s[i]);
      x.v[2 * i + 1] = turned<TO>(b, c[i], a, -s[i]);
    }
  } else {
    const float* ct = table + 8 * (piece & 3);
    const float sign = piece < 4 ? 1.0f : -1.0f;
    const f32x4 c0 = reinterpret_cast<const f32x4*>(ct)[0], c1 = reinterpret_cast<const f32x4*>(ct)[1];
    const f32x4 s0 = reinterpret_cast<const f32x4*>(ct + kHalfRope)[0];
    const f32x4 s1 = reinterpret_cast<const f32x4*>(ct + kHalfRope)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.v[i] = turned<TO>(x.v[i], c0[i], partner.v[i], sign * s0[i]);
      x.v[4 + i] = turned<TO>(x.v[4 + i], c1[i], partner.v[4 + i], sign * s1[i]);
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Largest |x| as bits: integers order as the floats do, and infinities and
// NaNs come out at 0x7F800000 or above.
__device__ __forceinline__ uint32_t amax_bits(const F32Row& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x.v[i]));
  return m;
}

// E2M1 code of z (|z| exact): thresholds between the values 0, .5, 1, 1.5, 2,
// 3, 4, 6; a tie belongs to the even code.
__device__ __forceinline__ uint32_t e2m1_code(float z) {
  const float m = fabsf(z);
  const uint32_t code = (m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) + (m >= 3.5f) + (m > 5.0f);
  return code | (__float_as_uint(z) >> 31 << 3);
}

// 16 lanes per key, 8 dimensions per lane; lanes 0-7 of a key hold the
// rotated half.  DT: element type of k.
template <int DT, bool MX>
__global__ __launch_bounds__(kThreads) void index_k_append_kernel(
    const char* __restrict__ k, int64_t k_stride, const int32_t* __restrict__ positions,
    const int32_t* __restrict__ slots, const float* __restrict__ rope, int max_positions, int interleaved,
    int tokens, int total_slots, uint8_t* __restrict__ pages, float* __restrict__ k_scales) {
  constexpr int kBytes = DT == IDX_FP32 ? 4 : 2;
  const int token = blockIdx.x * kKeysPerWg + static_cast<int>(threadIdx.x) / kLanesPerKey;
  const int piece = threadIdx.x % kLanesPerKey;
  if (token >= tokens) return;  // whole keys: the 16 lanes of a key leave together
  const int slot = slots[token];
  int pos = positions[token];
  if (slot < 0 || slot >= total_slots) return;
  pos = max(0, min(pos, max_positions - 1));
  const char* row = k + static_cast<int64_t>(token) * k_stride * kBytes;
  F32Row x = load8<DT>(row + piece * 8 * kBytes);
  if (piece < kRope / 8) {
    const F32Row other = load8<DT>(row + (piece ^ 4) * 8 * kBytes);
    rotate8<IDX_FP32>(x, other, piece, interleaved != 0, rope + static_cast<int64_t>(pos) * kRope);
  }
  uint32_t amax = amax_bits(x);
  amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 1)));
  amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 2)));
  if constexpr (MX) {
    // four lanes are one block of 32 dimensions
    const bool finite = amax < 0x7F800000u;
    const int code = finite ? max(static_cast<int>(amax >> 23) - 2, 0) : 255;
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - min(code, 252)) << 23);  // 2^-(code - 127), exact
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) packed |= (finite ? e2m1_code(x.v[i] * inv) : 0u) << (4 * i);
    uint8_t* out = pages + static_cast<int64_t>(slot) * (kDim / 2 + 4);
    reinterpret_cast<uint32_t*>(out)[piece] = packed;
    if ((piece & 3) == 0) out[kDim / 2 + piece / 4] = static_cast<uint8_t>(code);
  } else {
    amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 4)));
    amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 8)));
    const bool finite = amax < 0x7F800000u;
    const float scale = __uint_as_float(amax) / 448.0f;
    // a token of zeros (or of values so small that the scale is zero) keeps
    // scale 0 and codes of the values themselves, which all round to 0
    const float by = scale > 0.0f ? scale : 1.0f;
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = finite ? fminf(fmaxf(x.v[i] / by, -448.0f), 448.0f) : 0.0f;
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
    reinterpret_cast<int2*>(pages + static_cast<int64_t>(slot) * kDim)[piece] = make_int2(lo, hi);
    if (piece == 0) k_scales[slot] = finite ? scale : __uint_as_float(0x7FC00000u);
  }
}

// Round to nearest even in the row's type.
template <int DT>
__device__ __forceinline__ uint32_t bits16(float x) {
  if constexpr (DT == IDX_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  return f16_bits_rn(x);
}

// One thread per 16-byte piece: 64 pieces of a row are copied, 8 rotated.
template <int DT>
__global__ __launch_bounds__(kThreads) void latent_append_kernel(
    const char* __restrict__ kv, int64_t kv_stride, const int32_t* __restrict__ positions,
    const int32_t* __restrict__ slots, const float* __restrict__ rope, int max_positions, int interleaved,
    int tokens, int total_slots, char* __restrict__ pages) {
  const uint32_t at = blockIdx.x * kThreads + threadIdx.x;
  const int token = at / kRowPieces, piece = at % kRowPieces;
  if (token >= tokens) return;
  const int slot = slots[token];
  if (slot < 0 || slot >= total_slots) return;
  const char* row = kv + static_cast<int64_t>(token) * kv_stride * 2;
  char* out = pages + static_cast<int64_t>(slot) * (IDX_LATENT_ROW * 2) + piece * 16;
  if (piece < kLatentPieces) {
    *reinterpret_cast<i32x4*>(out) = *reinterpret_cast<const i32x4*>(row + piece * 16);
    return;
  }
  const int pos = max(0, min(positions[token], max_positions - 1));
  const int rotated = piece - kLatentPieces;
  F32Row x = load8<DT>(row + piece * 16);
  const F32Row other = load8<DT>(row + (piece ^ 4) * 16);
  rotate8<DT>(x, other, rotated, interleaved != 0, rope + static_cast<int64_t>(pos) * kRope);
  i32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = static_cast<int>(bits16<DT>(x.v[2 * i]) | (bits16<DT>(x.v[2 * i + 1]) << 16));
  *reinterpret_cast<i32x4*>(out) = y;
}

template <int DT>
void launch_index(const AppendArgs& a, hipStream_t stream, LaunchEvents ev) {
  const dim3 grid((a.tokens + kKeysPerWg - 1) / kKeysPerWg);
  const char* k = static_cast<const char*>(a.rows);
  const int total = a.num_pages * kPage;
  if (a.k_scales)
    launch_kernel(index_k_append_kernel<DT, false>, grid, dim3(kThreads), stream, ev.start, ev.stop, k, a.row_stride,
                  a.positions, a.slots, a.rope, a.max_positions, a.interleaved, a.tokens, total,
                  static_cast<uint8_t*>(a.pages), a.k_scales);
  else
    launch_kernel(index_k_append_kernel<DT, true>, grid, dim3(kThreads), stream, ev.start, ev.stop, k, a.row_stride,
                  a.positions, a.slots, a.rope, a.max_positions, a.interleaved, a.tokens, total,
                  static_cast<uint8_t*>(a.pages), a.k_scales);
}

template <int DT>
void launch_latent(const AppendArgs& a, hipStream_t stream, LaunchEvents ev) {
  const int64_t pieces = static_cast<int64_t>(a.tokens) * kRowPieces;
  launch_kernel(latent_append_kernel<DT>, dim3(static_cast<uint32_t>((pieces + kThreads - 1) / kThreads)),
                dim3(kThreads), stream, ev.start, ev.stop, static_cast<const char*>(a.rows), a.row_stride, a.positions,
                a.slots, a.rope, a.max_positions, a.interleaved, a.tokens, a.num_pages * kPage,
                static_cast<char*>(a.pages));
}

}  // namespace

hipError_t launch_index_k_append(const AppendArgs& a, hipStream_t stream, LaunchEvents ev) {
  if (a.dtype == IDX_BF16) launch_index<IDX_BF16>(a, stream, ev);
  else if (a.dtype == IDX_FP16) launch_index<IDX_FP16>(a, stream, ev);
  else launch_index<IDX_FP32>(a, stream, ev);
  return hipGetLastError();
}

hipError_t launch_latent_append(const AppendArgs& a, hipStream_t stream, LaunchEvents ev) {
  if (a.dtype == IDX_BF16) launch_latent<IDX_BF16>(a, stream, ev);
  else launch_latent<IDX_FP16>(a, stream, ev);
  return hipGetLastError();
}

}  // namespace pmqa
