// Attention over the paged latent cache (gfx950): over a request's pages, over
// pages that a batch shares, and over the keys that the top-k selected.
//
// All heads of a row read the same cache row per key (576 values: 512 latent,
// which are also the value vector, and 64 rotated), so a tile of M (row, head)
// pairs against 64 keys is one matrix product S = K Q^T, an online softmax
// per pair, and a second product O^T += V^T P^T on the same keys.
//
//   z_s = scale q . k_s,  c tanh(z / c),  - slope_h |pos_r - s|
//   m = max z, p_s = exp(z_s - m), l = sum p_s, o = sum p_s k_s[0:512]
//   out = o / l, lse = m + log l;  a row without keys: 0 and -inf
//
// Both products run transposed, keys on the MFMA's rows and pairs on its
// columns: a lane then holds four consecutive keys of ONE pair, which is at
// once the layout the second product takes P in (no exchange through LDS) and
// one in which the softmax of a pair needs two lane exchanges.  The value
// operand V^T comes from the same LDS tile with the transposing 64-bit reads.
//
// Work: the (pair tile, 64-key tile) list of the whole batch is cut into equal
// contiguous shares, one per persistent workgroup (one per CU), whatever the
// requests' lengths.  A share that covers all keys of a pair tile writes its
// output; the pieces of a pair tile that several workgroups share go to the
// workspace as (o, m, l) in float32 and a second kernel joins them, in a fixed
// order.
//
// Measured (MI355X, medians of 25 under the kernel trace): 64 requests of 1 ..
// 32768 keys with 16 heads 54 us (a K stream of 240 MB in about 35 us, the rest
// each workgroup's start and end); 1024 rows of 128 heads over 2048 listed keys
// 634 us (584 GFLOP, 920 TFLOP/s; the library's 8192^3 product reaches 1193), the
// MFMAs busy 42 % of all cycles -- a third of that case's 64-key tiles hold nothing
// but padding, which is multiplied like keys; 8 requests on 32768 shared keys
// 97 us; one request of 65 keys 9.3 us, five dependent round trips to memory.
#include "attention_tiles.h"

namespace pmqa {
namespace {

// Size of the pair tiles: the one whose estimated time is least.  A workgroup
// spends kPerTile on each of its shares of the 64-key tiles and kFixed on the
// call (start, queries, output, and the float32 pieces of pair tiles that are
// split, 2 KiB per pair and workgroup, written and joined).  Microseconds, from
// every size forced on selections of 512 and 2048 keys for 1 .. 256 rows of 32,
// 64 and 128 heads, and on 1 .. 64 requests of 256 .. 32768 keys with 16 .. 128
// heads.  Between them (16 / 32 / 64 / 128 pairs): 8 rows of 128 heads over
// 2048 keys 31 / 29 / 36 / 46 us, 64 rows 123 / 80 / 96 / 103, 256 rows 689 /
// 367 / 296 / 203; 64 heads, 256 rows 354 / 188 / 152 / 180; 16 requests of
// 8192 keys with 128 heads 112 / 85 / 103 / 121, of 32768 keys 396 / 265 / 268
// / 221.  (For whole pages the table's width stands for the lengths, which the
// host does not know; the times are of tables as wide as the requests, and in a
// wider one the choice falls on larger tiles than those would take.)  Tiles wider
// than the pairs would only idle.
constexpr double kPerTile[] = {2.2, 2.1, 3.5, 3.9}, kFixed[] = {19, 20, 32, 65};

template <int DT, int KIND, int M>
hipError_t launch(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_joined<DT, KIND, M>(attention_kernel<DT, KIND, M, false>, kAttnThreads, a, stream, ev);
}

template <int DT, int KIND>
hipError_t launch_kind(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  switch (tile_pairs<KIND>(a, kPerTile, kFixed, ScanOf256<KIND>::kItems)) {
    case 16: return launch<DT, KIND, 16>(a, stream, ev);
    case 32: return launch<DT, KIND, 32>(a, stream, ev);
    case 64: return launch<DT, KIND, 64>(a, stream, ev);
    default: return launch<DT, KIND, 128>(a, stream, ev);
  }
}

template <int KIND>
hipError_t launch_type(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return a.dtype == IDX_BF16 ? launch_kind<IDX_BF16, KIND>(a, stream, ev)
                             : launch_kind<IDX_FP16, KIND>(a, stream, ev);
}

}  // namespace

// For any size of the pair tiles that the calls may take: the queries do not
// know the keys.
size_t attention_workspace_size(int32_t rows, int32_t heads, int32_t requests) {
  if (rows <= 0 || heads <= 0 || requests <= 0) return 0;
  const int64_t together = (static_cast<int64_t>(rows) + requests - 1) / requests * heads;
  const int m = together <= 16 ? 16 : together <= 32 ? 32 : together <= 64 ? 64 : 128;
  return join_bytes(kMaxGrid) + 2 * kMaxGrid * static_cast<size_t>(piece_floats(m)) * sizeof(float);
}

size_t shared_prefix_workspace_size(int32_t rows, int32_t heads, int32_t requests) {
  if (rows <= 0 || heads <= 0 || requests <= 0) return 0;
  const int64_t per_request = (static_cast<int64_t>(rows) + requests - 1) / requests * heads;
  size_t most = 0;
  for (int m = 16; m <= 128; m *= 2) {
    const int64_t items = (static_cast<int64_t>(rows) * heads + m - 1) / m + requests * ((per_request + m - 1) / m);
    most = std::max(most, join_bytes(items) + (items + kMaxGrid) * static_cast<size_t>(piece_floats(m)) * sizeof(float));
  }
  return most;
}

hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kDense>(a, stream, ev);
}
hipError_t launch_shared_prefix_attention(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kShared>(a, stream, ev);
}
hipError_t launch_sparse_attention(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kSparse>(a, stream, ev);
}

}  // namespace pmqa
