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
//   latent_append_mxfp4   512 dimensions as E2M1 codes, nearest even, with a power
//                         of two per 32 (as above), 64 rotated, 16 bits each
//
// Every lane moves 16-byte pieces and no lane waits for another token's, so
// the kernels are bound by memory (and, for a few tokens, by one dependent
// load chain: slot and position, then the table row).  Measured (medians of 25
// under the kernel trace): 8192 latent rows 6.8 us (21 MB, 3.1 TB/s), 8191 into 4-bit
// rows 6.0 us (15 MB), 8191 MXFP4 keys 4.8 us, 8 FP8 keys 2.5 us.
#include "indexer_common.h"
#include "launches.h"
#include "rotary.h"

namespace pmqa {
namespace {

constexpr int kThreads = 256;
constexpr int kLanesPerKey = kDim / 8;     // 16 lanes of 8 dimensions each
constexpr int kKeysPerWg = kThreads / kLanesPerKey;
constexpr int kRowPieces = IDX_LATENT_ROW * 2 / 16;    // 72 16-byte pieces of a latent row
constexpr int kLatentPieces = IDX_LATENT_DIM * 2 / 16;  // the first 64 are copied as they are, or become codes
constexpr int kPacked = IDX_LATENT_DIM / 2 + IDX_LATENT_DIM / 32;  // codes and power bytes of a 4-bit row

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

// E8M0 byte of a block from its largest |x| (as bits): floor(log2 max|x|) - 2, and
// 255 with a NaN or an infinity in the block.
__device__ __forceinline__ int block_power(uint32_t amax) {
  return amax < 0x7F800000u ? max(static_cast<int>(amax >> 23) - 2, 0) : 255;
}

// Eight codes under that byte.
__device__ __forceinline__ uint32_t e2m1_codes(const F32Row& x, int code) {
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - min(code, 252)) << 23);  // 2^-(code - 127), exact
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) packed |= (code < 255 ? e2m1_code(x.v[i] * inv) : 0u) << (4 * i);
  return packed;
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
    const int code = block_power(amax);
    uint8_t* out = pages + static_cast<int64_t>(slot) * (kDim / 2 + 4);
    reinterpret_cast<uint32_t*>(out)[piece] = e2m1_codes(x, code);
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
    reinterpret_cast<int2*>(pages + static_cast<int64_t>(slot) * kDim)[piece] = e4m3_codes(c);
    if (piece == 0) k_scales[slot] = finite ? scale : __uint_as_float(0x7FC00000u);
  }
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
  *reinterpret_cast<i32x4*>(out) = pack16<DT>(x);
}

// e2m1_codes by the conversion instruction, two values at a time (nearest even, to
// +-6 at most; it takes the power of two from its operand's exponent): with the
// comparisons of e2m1_code, which 32 values of a thread's own make its whole time,
// 8191 rows 10.8 us instead of 6.0.
__device__ __forceinline__ uint32_t packed_e2m1(const F32Row& x, int code) {
  const float power = __uint_as_float(static_cast<uint32_t>(code) << 23);
  uint32_t y = 0;
  y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x.v[0], x.v[1], power, 0);
  y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x.v[2], x.v[3], power, 1);
  y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x.v[4], x.v[5], power, 2);
  y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x.v[6], x.v[7], power, 3);
  return code < 255 ? y : 0u;
}

// 32 threads per token: 16 take a block of 32 dimensions each, its largest magnitude
// and codes in their own registers, 8 an eighth of the rotated part.
constexpr int kPackThreads = 32;
template <int DT>
__global__ __launch_bounds__(kThreads) void latent_append_mxfp4_kernel(
    const char* __restrict__ kv, int64_t kv_stride, const int32_t* __restrict__ positions,
    const int32_t* __restrict__ slots, const float* __restrict__ rope, int max_positions, int interleaved,
    int tokens, int total_slots, char* __restrict__ pages) {
  const int token = blockIdx.x * (kThreads / kPackThreads) + static_cast<int>(threadIdx.x) / kPackThreads;
  const int part = threadIdx.x % kPackThreads;
  if (token >= tokens) return;
  const char* row = kv + static_cast<int64_t>(token) * kv_stride * 2;
  const int slot = slots[token];
  const bool here = slot >= 0 && slot < total_slots;
  char* out = pages + static_cast<int64_t>(slot) * IDX_LATENT_MXFP4_ROW;
  if (part < IDX_LATENT_DIM / 32) {
    F32Row x[4];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = load8<DT>(row + part * 64 + i * 16);
      amax = max(amax, amax_bits(x[i]));
    }
    const int code = block_power(amax);
    i32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = static_cast<int>(packed_e2m1(x[i], code));
    if (!here) return;
    reinterpret_cast<i32x4*>(out)[part] = y;
    out[IDX_LATENT_DIM / 2 + part] = static_cast<char>(code);
  } else if (part < IDX_LATENT_DIM / 32 + kRope / 8) {
    const int piece = part - IDX_LATENT_DIM / 32;
    const int pos = max(0, min(positions[token], max_positions - 1));
    F32Row x = load8<DT>(row + kLatentPieces * 16 + piece * 16);
    const F32Row other = load8<DT>(row + kLatentPieces * 16 + (piece ^ 4) * 16);
    rotate8<DT>(x, other, piece, interleaved != 0, rope + static_cast<int64_t>(pos) * kRope);
    if (here) reinterpret_cast<i32x4*>(out + kPacked)[piece] = pack16<DT>(x);
  }
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
void launch_latent(const AppendArgs& a, bool mxfp4, hipStream_t stream, LaunchEvents ev) {
  const int64_t pieces = static_cast<int64_t>(a.tokens) * (mxfp4 ? kPackThreads : kRowPieces);
  launch_kernel(mxfp4 ? latent_append_mxfp4_kernel<DT> : latent_append_kernel<DT>,
                dim3(static_cast<uint32_t>((pieces + kThreads - 1) / kThreads)),
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

hipError_t launch_latent_append(const AppendArgs& a, bool mxfp4, hipStream_t stream, LaunchEvents ev) {
  if (a.dtype == IDX_BF16) launch_latent<IDX_BF16>(a, mxfp4, stream, ev);
  else launch_latent<IDX_FP16>(a, mxfp4, stream, ev);
  return hipGetLastError();
}

}  // namespace pmqa
