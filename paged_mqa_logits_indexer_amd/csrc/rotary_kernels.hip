// Rotation of queries by positions of one or several axes, and the composition of
// several axes' angles into one table row per token (gfx950).
//
// Angle i of a token (i < 32) is that of the position on axis a(i): text has one
// axis, images and video have time, height and width, each with angles of its own.
// Two bits per angle give its axis.  All layers of a model turn by the same angles,
// so axis_rotations gathers them once a step, [tokens][64], and the appends take
// that table with position t for token t; the queries' kernels gather for
// themselves, once per token and thread, and turn several heads with it.
//
//   rotate_queries        64 dimensions of every (row, head), 16 bits in and out,
//                         from and to strided places
//   rotate_index_queries  the first 64 of 128 dimensions; all of them to E4M3 codes,
//                         clamped to +-448, which indexer_logits reads
//
// Each value is rounded once (rotary.h).  Bound by memory.
#include "indexer_common.h"
#include "launches.h"
#include "rotary.h"

namespace pmqa {
namespace {

constexpr int kThreads = 256;

// Positions of one token on up to four axes, clamped into the table.
struct AxisPositions {
  int at[4];
};
__device__ __forceinline__ AxisPositions axis_positions(const RotaryArgs& a, int token) {
  AxisPositions p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int axis = min(i, a.axes - 1);
    p.at[i] = max(0, min(a.positions[static_cast<int64_t>(axis) * a.tokens + token], a.max_positions - 1));
  }
  return p;
}

// Table row that angle i is read from.
__device__ __forceinline__ const float* angle_row(const RotaryArgs& a, const AxisPositions& p, int i) {
  const int axis = static_cast<int>(a.axis_map >> (2 * i)) & 3;
  const int at = axis == 0 ? p.at[0] : axis == 1 ? p.at[1] : axis == 2 ? p.at[2] : p.at[3];
  return a.rope + static_cast<int64_t>(at) * kRope;
}

// factors_of for positions on several axes.
__device__ __forceinline__ Factors gather_factors(const RotaryArgs& a, int token, int piece) {
  const AxisPositions p = axis_positions(a, token);
  if (a.axes == 1) return factors_of(piece, a.interleaved != 0, a.rope + static_cast<int64_t>(p.at[0]) * kRope);
  Factors f;
  const int first = a.interleaved ? 4 * piece : 8 * (piece & 3);
  const float sign = a.interleaved || piece < 4 ? 1.0f : -1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int angle = first + (a.interleaved ? i & 3 : i);
    const float* row = angle_row(a, p, angle);
    f.c[i] = row[angle];
    f.s[i] = sign * row[kHalfRope + angle];
  }
  return f;
}

// 16 threads per token, four values each.
__global__ __launch_bounds__(kThreads) void axis_rotations_kernel(RotaryArgs a) {
  const uint32_t at = blockIdx.x * kThreads + threadIdx.x;
  const int token = at / 16, part = at % 16;
  if (token >= a.tokens) return;
  const AxisPositions p = axis_positions(a, token);
  f32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int column = 4 * part + i;
    y[i] = angle_row(a, p, column % kHalfRope)[column];
  }
  static_cast<f32x4*>(a.out)[at] = y;
}

// Clamped to the codes' range (a comparison with NaN fails: it passes through).
__device__ __forceinline__ int2 clamped_codes(F32Row x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x.v[i] = x.v[i] > 448.0f ? 448.0f : x.v[i] < -448.0f ? -448.0f : x.v[i];
  return e4m3_codes(x.v);
}

// 8 threads per (token, head), each with 8 rotated dimensions and, of an index query,
// 8 of the others (the rotation, in float64, then keeps whole waves busy: with 16
// threads, of which half rotate, 4001 rows of 32 heads 17.8 us instead of 13.7).  A
// thread asks for AT heads before it turns the first, so that the chain position,
// table row, factors stands beside them (4096 rows of 128 heads 45 -> 33 us).
template <int DT, bool INDEX, int AT>
__global__ __launch_bounds__(kThreads) void rotate_kernel(RotaryArgs a, int chunks) {
  constexpr int kBytes = DT == IDX_FP32 ? 4 : 2, kPiece = 8 * kBytes;
  constexpr int kPieces = 8, kHeadsPerPass = kThreads / kPieces;
  const int token = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int piece = threadIdx.x % kPieces;
  const char* in = static_cast<const char*>(a.x) + static_cast<int64_t>(token) * a.x_token_stride * kBytes + piece * kPiece;
  F32Row x[AT], other[AT], plain[INDEX ? AT : 1];
  const int head0 = chunk * AT * kHeadsPerPass + static_cast<int>(threadIdx.x) / kPieces;
#pragma unroll
  for (int k = 0; k < AT; ++k) {
    const int head = head0 + k * kHeadsPerPass;
    if (head >= a.heads) continue;
    const char* row = in + head * a.x_head_stride * kBytes;
    x[k] = load8<DT>(row);
    if (!a.interleaved) other[k] = load8<DT>(row + ((piece ^ 4) - piece) * kPiece);
    if constexpr (INDEX) plain[k] = load8<DT>(row + kPieces * kPiece);
  }
  const Factors f = gather_factors(a, token, piece);
#pragma unroll
  for (int k = 0; k < AT; ++k) {
    const int head = head0 + k * kHeadsPerPass;
    if (head >= a.heads) continue;
    turn8<INDEX ? IDX_FP32 : DT>(x[k], other[k], a.interleaved != 0, f);
    if constexpr (INDEX) {
      int2* out = static_cast<int2*>(a.out) + (static_cast<int64_t>(token) * a.heads + head) * (2 * kPieces) + piece;
      out[0] = clamped_codes(x[k]);
      out[kPieces] = clamped_codes(plain[k]);
    } else {
      // (in place: a row's 8 threads are of one wave, which has read its rows by now)
      char* out = static_cast<char*>(a.out) +
                  (static_cast<int64_t>(token) * a.out_token_stride + head * a.out_head_stride) * kBytes;
      reinterpret_cast<i32x4*>(out)[piece] = pack16<DT>(x[k]);
    }
  }
}

template <int DT, bool INDEX, int AT>
void launch_at(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  constexpr int kHeads = AT * kThreads / 8;
  const int chunks = (a.heads + kHeads - 1) / kHeads;
  launch_kernel(rotate_kernel<DT, INDEX, AT>, dim3(static_cast<uint32_t>(a.tokens) * chunks), dim3(kThreads), stream,
                ev.start, ev.stop, a, chunks);
}

template <int DT, bool INDEX>
void launch_rotate(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  if constexpr (!INDEX) {
    if (a.tokens >= 1024 && a.heads > kThreads / 8) return launch_at<DT, INDEX, 4>(a, stream, ev);
  }
  launch_at<DT, INDEX, 1>(a, stream, ev);
}

}  // namespace

hipError_t launch_axis_rotations(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  const int64_t threads = static_cast<int64_t>(a.tokens) * 16;
  launch_kernel(axis_rotations_kernel, dim3(static_cast<uint32_t>((threads + kThreads - 1) / kThreads)), dim3(kThreads),
                stream, ev.start, ev.stop, a);
  return hipGetLastError();
}

hipError_t launch_rotate_queries(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  if (a.dtype == IDX_BF16) launch_rotate<IDX_BF16, false>(a, stream, ev);
  else launch_rotate<IDX_FP16, false>(a, stream, ev);
  return hipGetLastError();
}

hipError_t launch_rotate_index_queries(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  if (a.dtype == IDX_BF16) launch_rotate<IDX_BF16, true>(a, stream, ev);
  else if (a.dtype == IDX_FP16) launch_rotate<IDX_FP16, true>(a, stream, ev);
  else launch_rotate<IDX_FP32, true>(a, stream, ev);
  return hipGetLastError();
}

}  // namespace pmqa
