// Rotation of queries by positions of one or several axes, and the composition of
// several axes' angles into one table row per token (gfx950).
//
// Angle i of a token (i < 32) is that of the position on axis a(i): text has one
// axis, images and video have time, height and width, each with angles of its own.
// Two bits per angle give its axis.  All layers of a model turn by the same angles,
// so axis_rotations gathers them once a step, [tokens][64], and the appends take
// that table with position t for token t; the queries' kernels gather for
// themselves, once per token and workgroup.
//
//   rotate_queries        64 dimensions of every (row, head), 16 bits in and out,
//                         from and to strided places
//   rotate_index_queries  the first 64 of 128 dimensions; all of them to E4M3 codes,
//                         clamped to +-448, which indexer_logits reads
//
// Each value is rounded once (rotary.h).  Bound by memory: 4096 rows of 128 heads on
// three axes, 384 and 1152 bytes apart, move 134 MB in 29 us under the kernel trace (4.6
// TB/s; calls 30.5 us, on one axis 29.8).
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
    p.at[i] = max(0, min(a.positions[axis * a.position_stride + token], a.max_positions - 1));
  }
  return p;
}

// Table row that angle i is read from.
__device__ __forceinline__ const float* angle_row(const RotaryArgs& a, const AxisPositions& p, int i) {
  const int axis = static_cast<int>(a.axis_map >> (2 * i)) & 3;
  const int at = axis == 0 ? p.at[0] : axis == 1 ? p.at[1] : axis == 2 ? p.at[2] : p.at[3];
  return a.rope + static_cast<int64_t>(at) * kRope;
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

// A workgroup per 32 heads of a token, 8 threads per head, each with 8 rotated
// dimensions and, of an index query, 8 of the others (with 16 threads, of which half
// rotate in float64, 4001 rows of 32 heads took 1.3 times as long when it was tried).
// The angles are read from the table, or, on several axes, gathered in LDS by 64
// threads (each thread its own: half as long again, 4096 rows of 128 heads, likewise).
// The queries are asked for first, beside the chain position, table row, angles.  What
// is written goes past the caches, which it would only fill (30.5 us a call with it,
// 30.3 without: the rows of one call alone do not show it).
template <int DT, bool INDEX>
__global__ __launch_bounds__(kRotateThreads) void rotate_kernel(RotaryArgs a, int chunks) {
  constexpr int kBytes = DT == IDX_FP32 ? 4 : 2, kPiece = 8 * kBytes, kPieces = kRope / 8;
  __shared__ __attribute__((aligned(16))) float s_row[kRope];
  const int token = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int piece = threadIdx.x % kPieces, head = chunk * kHeadsPerWg + static_cast<int>(threadIdx.x) / kPieces;
  const bool here = head < a.heads;
  const char* row = static_cast<const char*>(a.x) +
                    (static_cast<int64_t>(token) * a.x_token_stride + head * a.x_head_stride) * kBytes;
  F32Row x{}, other{}, plain{};
  if (here) {
    x = load8<DT>(row + piece * kPiece);
    if (!a.interleaved) other = load8<DT>(row + (piece ^ 4) * kPiece);
    if constexpr (INDEX) plain = load8<DT>(row + (piece + kPieces) * kPiece);
  }
  const AxisPositions p = axis_positions(a, token);
  const float* table = a.rope + static_cast<int64_t>(p.at[0]) * kRope;
  if (a.axes > 1) {
    if (threadIdx.x < kRope) s_row[threadIdx.x] = angle_row(a, p, threadIdx.x % kHalfRope)[threadIdx.x];
    __syncthreads();
    table = s_row;
  }
  if (!here) return;
  turn8<INDEX ? IDX_FP32 : DT>(x, other, a.interleaved != 0, factors_of(piece, a.interleaved != 0, table));
  if constexpr (INDEX) {
    int2* out = static_cast<int2*>(a.out) + (static_cast<int64_t>(token) * a.heads + head) * (2 * kPieces) + piece;
    out[0] = clamped_codes(x);
    out[kPieces] = clamped_codes(plain);
  } else {
    // (in place: a row's 8 threads are of one wave, which has read the row by now)
    char* out = static_cast<char*>(a.out) +
                (static_cast<int64_t>(token) * a.out_token_stride + head * a.out_head_stride) * kBytes;
    __builtin_nontemporal_store(pack16<DT>(x), reinterpret_cast<i32x4*>(out) + piece);
  }
}

// One launch, or one for each slab of tokens.
template <int DT, bool INDEX>
hipError_t launch_rotate(RotaryArgs a, hipStream_t stream, LaunchEvents ev) {
  constexpr int kBytes = DT == IDX_FP32 ? 4 : 2;
  const int32_t all = a.tokens;
  for (int32_t first = 0; first < all; first += a.tokens) {
    a.tokens = all - first < kSlabTokens ? all - first : kSlabTokens;
    const bool last = first + a.tokens == all;
    launch_kernel(rotate_kernel<DT, INDEX>, dim3(rotate_workgroups(a.tokens, a.heads)), dim3(kRotateThreads), stream,
                  first == 0 ? ev.start : nullptr, last ? ev.stop : nullptr, a, chunks_of(a.heads));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || last) return e;
    a.positions += a.tokens;
    a.x = static_cast<const char*>(a.x) + a.tokens * a.x_token_stride * kBytes;
    a.out = static_cast<char*>(a.out) + a.tokens * a.out_token_stride * (INDEX ? 1 : kBytes);
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_axis_rotations(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  const int64_t threads = static_cast<int64_t>(a.tokens) * 16;
  launch_kernel(axis_rotations_kernel, dim3(static_cast<uint32_t>((threads + kThreads - 1) / kThreads)), dim3(kThreads),
                stream, ev.start, ev.stop, a);
  return hipGetLastError();
}

hipError_t launch_rotate_queries(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  return a.dtype == IDX_BF16 ? launch_rotate<IDX_BF16, false>(a, stream, ev)
                             : launch_rotate<IDX_FP16, false>(a, stream, ev);
}

hipError_t launch_rotate_index_queries(const RotaryArgs& a, hipStream_t stream, LaunchEvents ev) {
  if (a.dtype == IDX_BF16) return launch_rotate<IDX_BF16, true>(a, stream, ev);
  if (a.dtype == IDX_FP16) return launch_rotate<IDX_FP16, true>(a, stream, ev);
  return launch_rotate<IDX_FP32, true>(a, stream, ev);
}

}  // namespace pmqa
