// What the attention kernels over the latent cache have in common, whatever the
// cache's format: the softmax weights in 16 bits, the work list and its equal
// shares, and the second kernel that joins the pieces of split pair tiles.
#pragma once

#include <algorithm>
#include <climits>
#include <type_traits>

#include "indexer_common.h"
#include "launches.h"

namespace pmqa {
namespace {

constexpr int kRowDim = IDX_LATENT_ROW;            // 576
constexpr int kValDim = IDX_LATENT_DIM;            // 512
constexpr int kDimTiles = kValDim / 16;            // 32 output tiles of 16 dimensions
constexpr int kTile = 64;                          // keys per entry of the work list
constexpr float kMInit = -__FLT_MAX__;             // running maximum before any key: no finite score is below it (finite: no inf - inf)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// P is rounded to the cache's 16-bit type for the second product (an MFMA
// takes both operands in one type), by at most half a step d_s of it per key.
// The output is divided by the sum of the same rounded weights (one instruction
// adds two of them to it in float32, to 1.5 steps and with FP16 subnormals, as
// measured on a million of each type), so it is off by
// sum p_s d_s (v_s - out): what all keys' weights have in common cancels, and
// where one key outweighs the rest nothing is left (divided by the unrounded
// sum, such a row is off by up to half a step as a whole).  The log of the sum,
// and the shares of a pair's pieces, take the unrounded sum l.
//
// The running maximum m is raised only when a score passes it by enough, so that
// the accumulators are hardly ever rescaled: a first score z sets m = z - kShift,
// and a later one is let pass until it is kRaise above z (powers of two).
// BF16 has float32's exponents: with m 16 above the first score, P lies between
// 2^-16 and 1 at the row's maximum, so an accumulator never passes the sum of
// its values' magnitudes (a score let pass by 2^60 instead, with m at the first
// score, turned values above 2^68 into infinities; neither measures faster), and
// products of values down to 2^-110 are still normal.  FP16 ends at 2^16: m is 8
// below the first score, so that weights down to 2^-22 of the maximum are still
// normal, and P ends at 2^14.
template <int DT>
struct Elem;
template <>
struct Elem<IDX_BF16> {
  static constexpr float kShift = -16.0f, kRaise = 16.0f;
  static __device__ __forceinline__ f32x4 mfma32(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma_wide(s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  static __device__ __forceinline__ void mfma_acc(s16x8 a0, s16x8 a1, s16x8 b, f32x16& c0, f32x16& c1) {
    __asm__ volatile("s_nop 1\nv_mfma_f32_32x32x16_bf16 %0, %2, %4, %0\nv_mfma_f32_32x32x16_bf16 %1, %3, %4, %1"
                     : "+a"(c0), "+a"(c1)
                     : "v"(a0), "v"(a1), "v"(b));
  }
  static __device__ __forceinline__ f32x4 mfma16(s16x4 a, s16x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int round2(float x, float y) {
    return __builtin_bit_cast(int, __builtin_convertvector((f32x2{x, y}), bf16x2));
  }
  static __device__ __forceinline__ float add2(int both, float sum) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, both), bf16x2{1, 1}, sum, false);
  }
};
template <>
struct Elem<IDX_FP16> {
  static constexpr float kShift = 8.0f, kRaise = 6.0f;
  static __device__ __forceinline__ f32x4 mfma32(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  static __device__ __forceinline__ f32x16 mfma_wide(s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  static __device__ __forceinline__ void mfma_acc(s16x8 a0, s16x8 a1, s16x8 b, f32x16& c0, f32x16& c1) {
    __asm__ volatile("s_nop 1\nv_mfma_f32_32x32x16_f16 %0, %2, %4, %0\nv_mfma_f32_32x32x16_f16 %1, %3, %4, %1"
                     : "+a"(c0), "+a"(c1)
                     : "v"(a0), "v"(a1), "v"(b));
  }
  static __device__ __forceinline__ f32x4 mfma16(s16x4 a, s16x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a), __builtin_bit_cast(f16x4, b), c, 0, 0,
                                                 0);
  }
  static __device__ __forceinline__ int round2(float x, float y) {
    return __builtin_bit_cast(int, __builtin_convertvector((f32x2{x, y}), f16x2));
  }
  static __device__ __forceinline__ float add2(int both, float sum) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, both), f16x2{1, 1}, sum, false);
  }
};

// Where invalid keys are read from: a row of zeros, so that neither S nor the
// value product meets what the cache holds there (a 4-bit row is shorter).
__device__ __attribute__((aligned(128))) const uint32_t kZeroRow[IDX_LATENT_ROW / 2] = {};

// 16-byte chunks of a key's 128 bytes are exchanged by c ^ swz(key) in LDS, which
// spreads the K operand's 128-bit reads and V's transposing 64-bit reads over all
// banks (attention_tiles.h).
__device__ __forceinline__ int swz(int key) { return (((key >> 1) & 1) << 2) | (-(key >> 2) & 3); }
// Keys that are written to LDS from registers (MX) also exchange by their last bit:
// eight lanes that write the same chunk of eight keys then take all 32 banks of a
// write, where pairs of keys took the same ones.  The reads' 64 banks hold even and
// odd keys apart, so nothing changes for them.
template <bool MX>
__device__ __forceinline__ int swz_of(int key) { return MX ? swz(key) ^ (key & 1) : swz(key); }

// A value whose origin the compiler does not see: constants added to such an
// LDS address become the read's own offset instead of an addition per read.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  __asm__("" : "+v"(x));
  return x;
}

typedef __attribute__((address_space(3))) const s16x8* LdsVec8;
typedef __attribute__((address_space(3))) s16x4* LdsVec4;
__device__ __forceinline__ void lds_write(uint32_t at, s16x8 x) {
  *reinterpret_cast<__attribute__((address_space(3))) s16x8*>(at) = x;
}
__device__ __forceinline__ s16x8 lds_read(uint32_t at) { return *reinterpret_cast<LdsVec8>(at); }
__device__ __forceinline__ s16x4 lds_read_tr(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<LdsVec4>(at));
}

// Maximum and sum of a value over the lanes of a pair: l, l ^ 16, l ^ 32 and
// l ^ 48, or (WIDE) l and l ^ 32.
template <bool WIDE>
__device__ __forceinline__ float pair_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  if constexpr (WIDE) return x;
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
template <bool WIDE>
__device__ __forceinline__ float pair_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  if constexpr (WIDE) return x;
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Softmax weight of score z (powers of two) under the maximum m.  The maximum is
// that of the rounded scores, so the subtraction is not contracted with the
// multiplication that made z: from 2^31 on, what that rounds away is itself
// hundreds of powers of two.
__device__ __forceinline__ float weight(float z, float m) {
#pragma clang fp contract(off)
  return __builtin_amdgcn_exp2f(z - m);
}

// tanh(x) = 1 - 2 / (1 + e^2x): absolute error of about one float32 step of 1,
// which the cap's factor turns into that of the score; near zero, where the
// difference would lose the argument's digits, the odd series
// x - x^3/3 + 2 x^5/15 - 17 x^7/315 (the next term is below 2^-24 relative for
// |x| < 0.1).
__device__ __forceinline__ float tanh_f32(float x) {
  const float e = __builtin_amdgcn_exp2f(x * (2.0f * kLog2e));
  const float far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e);
  const float y = x * x;
  const float near = x * (1.0f + y * (-1.0f / 3.0f + y * (2.0f / 15.0f - y * (17.0f / 315.0f))));
  return fabsf(x) < 0.1f ? near : far;
}

// One pair tile of the work list: its pairs and the 64-key tiles it reads.
struct Item {
  int request;   // block-table row
  int row0;      // the first row of the request (pair p is row row0 + p / heads)
  int pair0;     // first pair, counted from row0 * heads
  int pairs;     // 1 .. M (0: no such item)
  int tile0;     // first 64-key tile
  int tiles;     // number of tiles (at least 1 when pairs > 0)
  int max_start; // largest first key and smallest end over the rows: tiles inside need no mask
  int min_end;
  int min_start; // keys that some row may see: [min_start, max_end)
  int max_end;
  int key_lo;    // keys of this item: [key_lo, key_hi) (shared: prefix and rest)
  int key_hi;
};

// KIND: what the key tiles are.
enum { kDense = 0, kShared = 1, kSparse = 2 };

__device__ __forceinline__ int clamp_len(int len, int capacity) { return max(0, min(len, capacity)); }

// Rows of request b as [r0, r1), clamped into the batch.
__device__ __forceinline__ void request_rows(const AttentionArgs& a, int b, int& r0, int& r1) {
  if (a.cu_q) {
    r0 = max(0, min(a.cu_q[b], a.rows));
    r1 = max(r0, min(a.cu_q[b + 1], a.rows));
  } else {
    r0 = b * a.next_n;
    r1 = r0 + a.next_n;
  }
}

// First item id of request b of a ragged batch: one id per M pairs of the
// rows before it plus one per request, so every request has enough ids
// (floor((x + n) / M) + 1 - floor(x / M) >= ceil(n / M)) and an id finds its
// request by bisection, without a scan.
template <int M>
__device__ __forceinline__ int ragged_base(const AttentionArgs& a, int b) {
  const int r = max(0, min(a.cu_q[b], a.rows));
  return static_cast<int>(static_cast<int64_t>(r) * a.heads / M) + b;
}

// Key range of rows [r0, r1): every lane of the caller computes it (BY = 1) or
// the lanes of a wave share the rows (BY = 64).
template <int BY>
__device__ __forceinline__ void key_range(const AttentionArgs& a, int r0, int r1, int capacity, Item& it) {
  int lo = INT_MAX, hi = 0, max_start = 0, min_end = INT_MAX;
  for (int r = r0 + (BY > 1 ? lane_id() : 0); r < r1; r += BY) {
    const int end = clamp_len(a.row_lens[r], capacity);
    const int start = a.row_starts ? max(0, a.row_starts[r]) : 0;
    max_start = max(max_start, start);
    min_end = min(min_end, end);
    if (start < end) {
      lo = min(lo, start);
      hi = max(hi, end);
    }
  }
  if constexpr (BY > 1) {
    lo = -wave_max(-lo);
    hi = wave_max(hi);
    max_start = wave_max(max_start);
    min_end = -wave_max(-min_end);
  }
  if (lo > hi) lo = hi;  // no row sees a key
  it.max_start = max(max_start, it.key_lo);
  it.min_end = min(min_end, it.key_hi);
  it.min_start = max(lo, it.key_lo);
  it.max_end = min(hi, it.key_hi);
  it.tile0 = lo / kTile;
  it.tiles = (hi + kTile - 1) / kTile - it.tile0;
}

// What the join kernel needs to know of a pair tile that several workgroups
// share: written by the workgroup that holds the tile's beginning.
struct alignas(16) JoinInfo {
  int first;      // the first workgroup with a part of it
  int pieces;     // 0: nothing to join here
  int pairs;
  int pad;
  int64_t pair0;  // first pair, counted over the whole batch
  int64_t pad2;
};

constexpr int kMaxGrid = 256;  // one persistent workgroup per CU
__host__ __device__ __forceinline__ size_t join_bytes(int64_t infos) {
  return (static_cast<size_t>(infos) * sizeof(JoinInfo) + 255) / 256 * 256;
}

// Pieces in the workspace: float o[M][512], then float2 (m, l)[M].  Dense and
// sparse: two per workgroup, for a pair tile that began before it (2 w) and one
// that ends after it (2 w + 1).  Shared: every (workgroup, item) visit is a
// piece, w + item -- consecutive over a pair tile's workgroups.
__host__ __device__ __forceinline__ int64_t piece_floats(int m) { return static_cast<int64_t>(m) * (kValDim + 2); }

// Counted selections: a byte for each row, its tiles (at most 128), where the pieces
// would begin.  No pair tile began before the first workgroup and none ends after the
// last, so two pieces are never written, the first and the last: counts take the
// place of the first, and where that is too short for them (16 pairs), the pieces go
// on behind them, up to the end of the last.
constexpr int kCountBytes = 65536;
__host__ __device__ __forceinline__ uint8_t* row_tiles(const AttentionArgs& a) {
  return static_cast<uint8_t*>(a.workspace) + join_bytes(kMaxGrid);
}
constexpr int64_t piece_bytes(int m) { return static_cast<int64_t>(m) * (kValDim + 2) * sizeof(float); }
constexpr int64_t counted_shift(int m) { return kCountBytes > piece_bytes(m) ? kCountBytes - piece_bytes(m) : 0; }
static_assert(IDX_MAX_ROWS <= kCountBytes && (IDX_CANDIDATE_CAPACITY + kTile - 1) / kTile < 256, "a byte for each row");
static_assert(counted_shift(16) <= piece_bytes(16) && counted_shift(16) % 16 == 0, "counts and pieces fit");

// Item `id` of the list.  Dense: requests' pair tiles.  Shared: first the pair
// tiles of the whole batch over the prefix pages, then the requests' pair
// tiles over what follows.  Sparse: rows' pair tiles over the selection.
// COUNTED: selections may come with the tiles of each row that hold a key
// (row_tiles); the 16-bit kernels do not look for them.
template <int KIND, int M, int BY, bool COUNTED = false>
__device__ __forceinline__ Item make_item(const AttentionArgs& a, int id) {
  const int capacity = a.max_pages * kPage;
  Item it{};
  it.key_hi = capacity;
  if constexpr (KIND == kSparse) {
    const int per_row = (a.heads + M - 1) / M;
    const int row = id / per_row, t = id - row * per_row;
    it.row0 = row;
    it.pair0 = t * M;
    it.pairs = min(M, a.heads - it.pair0);
    it.tiles = (a.k + kTile - 1) / kTile;
    if (COUNTED && a.counted) it.tiles = row_tiles(a)[row];
    if (a.cu_q) {
      // the last request that starts at or before the row
      int lo = 0, hi = a.requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.cu_q[mid] <= row) lo = mid; else hi = mid;
      }
      it.request = lo;
      if (row < a.cu_q[lo] || row >= a.cu_q[lo + 1]) it.pairs = it.tiles = 0;
    } else {
      it.request = row / a.next_n;
    }
    return it;
  } else {
    int prefix_items = 0;
    if constexpr (KIND == kShared) {
      const int64_t all = static_cast<int64_t>(a.rows) * a.heads;
      prefix_items = static_cast<int>((all + M - 1) / M);
      if (id < prefix_items) {
        const int64_t p0 = static_cast<int64_t>(id) * M;
        const int n = static_cast<int>(min(static_cast<int64_t>(M), all - p0));
        it.row0 = static_cast<int>(p0 / a.heads);
        it.key_hi = a.prefix_pages * kPage;
        it.pair0 = static_cast<int>(p0 - static_cast<int64_t>(it.row0) * a.heads);
        it.pairs = n;
        key_range<BY>(a, it.row0, it.row0 + (it.pair0 + n - 1) / a.heads + 1, capacity, it);
        const int end = min(it.tile0 + it.tiles, a.prefix_pages);
        it.tile0 = min(it.tile0, a.prefix_pages - 1);
        it.tiles = max(1, end - it.tile0);
        return it;
      }
      id -= prefix_items;
    }
    int b, t;
    if (a.cu_q) {
      int lo = 0, hi = a.requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (ragged_base<M>(a, mid) <= id) lo = mid; else hi = mid;
      }
      b = lo;
      t = id - ragged_base<M>(a, b);
    } else {
      const int per = (a.next_n * a.heads + M - 1) / M;
      b = id / per;
      t = id - b * per;
    }
    int r0, r1;
    request_rows(a, b, r0, r1);
    it.request = b;
    it.row0 = r0;
    it.pair0 = t * M;
    it.pairs = static_cast<int>(min(static_cast<int64_t>(M), static_cast<int64_t>(r1 - r0) * a.heads - static_cast<int64_t>(t) * M));
    if (t < 0 || it.pairs <= 0) {
      it.pairs = 0;
      return it;
    }
    if constexpr (KIND == kShared) it.key_lo = a.prefix_pages * kPage;
    key_range<BY>(a, r0 + it.pair0 / a.heads, r0 + (it.pair0 + it.pairs - 1) / a.heads + 1, capacity, it);
    if constexpr (KIND == kShared) {
      const int end = it.tile0 + it.tiles;
      it.tile0 = max(it.tile0, min(a.prefix_pages, a.max_pages - 1));
      it.tiles = end - it.tile0;
    }
    it.tiles = max(1, it.tiles);
    it.tile0 = min(it.tile0, a.max_pages - 1);
    return it;
  }
}

template <int KIND>
__host__ __device__ __forceinline__ int64_t item_count(const AttentionArgs& a, int m) {
  const int64_t pairs = static_cast<int64_t>(a.rows) * a.heads;
  if (KIND == kSparse) return static_cast<int64_t>(a.rows) * ((a.heads + m - 1) / m);
  const int64_t own = a.cu_q ? pairs / m + a.requests
                             : static_cast<int64_t>(a.requests) * ((static_cast<int64_t>(a.next_n) * a.heads + m - 1) / m);
  return KIND == kShared ? (pairs + m - 1) / m + own : own;
}
template <int KIND, int M>
__host__ __device__ __forceinline__ int64_t item_count(const AttentionArgs& a) {
  return item_count<KIND>(a, M);
}

// find_share adds up the list a chunk at a time, as many items as the workgroup has
// threads, and keeps the sums in LDS: a kernel takes lists of up to kChunks chunks.
// Pair tiles of a size whose list is longer are not chosen (tile_pairs).  The widest
// tiles that a call may take always fit: at most 65535 items over selections, a
// request's 4096 more over pages, and twice that with a shared prefix.
template <int KIND>
struct ScanOf256 {  // threads
  static constexpr int kThreads = 256, kChunks = KIND == kSparse ? 644 : 1056;
  static constexpr int64_t kItems = int64_t{kThreads} * kChunks;
  static_assert(kItems >= (KIND == kShared ? 2 : 1) * (IDX_MAX_ROWS + IDX_MAX_REQUESTS), "the widest tiles fit");
};
template <int KIND>
struct ScanOf512 {
  static constexpr int kThreads = 512, kChunks = KIND == kShared ? 2080 : 1056;
  static constexpr int64_t kItems = int64_t{kThreads} * kChunks;
};

// The workgroup's share [t0, t1) of the tile list and the item it starts in.
struct Share {
  int64_t t0, t1;      // units
  int64_t total;
  int64_t item_at;     // unit offset of `item`
  int item;
  int groups;          // workgroups with work
  int cost;            // units that an item counts for beside its tiles
};

// Taking up a pair tile and writing it costs about as much as kItemCost tiles
// of keys: a pair tile counts for that many more, at its beginning.  (64
// requests of 1 .. 32768 keys 162 -> 78 us against 0; 5 and 8 measure 2 and 1 us
// slower there, but the wide form writes more: 109 -> 105 and 130 -> 117 us for
// ragged extends and 8 requests on a shared prefix with 6 instead of 3.)
template <int M>
constexpr int kItemCost = M == 128 ? 6 : 3;
__device__ __forceinline__ int item_units(const Item& it, int cost) { return it.tiles ? it.tiles + cost : 0; }

// Share of workgroup w of a grid: equal parts [w, w + 1) / groups of the units,
// of as many groups as have min_units each.
__device__ __forceinline__ int64_t share_begin(int64_t total, int groups, int w) {
  return total * w / groups;
}
// The workgroup whose share holds tile t.
__device__ __forceinline__ int share_owner(int64_t total, int groups, int64_t t) {
  int w = static_cast<int>((t * groups + groups - 1) / total);
  while (w > 0 && share_begin(total, groups, w) > t) --w;
  while (w + 1 < groups && share_begin(total, groups, w + 1) <= t) ++w;
  return w;
}

// min_units 0 (sparse lists of few rows): every item is cut into grid / items
// equal parts, so that a workgroup has one of them, and items cost nothing.
// COST: what an item counts for beside its tiles.
template <int KIND, int M, int THREADS, int COST = kItemCost<M>, bool COUNTED = false>
__device__ Share find_share(const AttentionArgs& a, int w, int grid, int min_units, int* s_scan, int64_t* s_res) {
  Share s;
  const int items = static_cast<int>(item_count<KIND, M>(a));
  const int tid = threadIdx.x;
  s.cost = COST;
  if constexpr (KIND == kSparse) {
    if (!a.cu_q && !(COUNTED && a.counted)) {
      if (min_units == 0) s.cost = 0;
      const int n = (a.k + kTile - 1) / kTile + s.cost;
      s.total = static_cast<int64_t>(items) * n;
      s.groups = min_units == 0
                     ? grid
                     : static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), s.total / min_units)));
      s.t0 = w < s.groups ? share_begin(s.total, s.groups, w) : 0;
      s.t1 = w < s.groups ? share_begin(s.total, s.groups, w + 1) : 0;
      s.item = static_cast<int>(s.t0 / n);
      s.item_at = static_cast<int64_t>(s.item) * n;
      return s;
    }
  }
  if (items <= kWave) {
    // few items: every wave by itself, an item per lane
    const int n = lane_id() < items ? item_units(make_item<KIND, M, 1, COUNTED>(a, lane_id()), COST) : 0;
    const int upto = wave_inclusive_scan(n);
    s.total = __builtin_amdgcn_readlane(upto, kWave - 1);
    s.groups = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), s.total / min_units)));
    s.t0 = w < s.groups ? share_begin(s.total, s.groups, w) : 0;
    s.t1 = w < s.groups ? share_begin(s.total, s.groups, w + 1) : 0;
    s.item = first_lane(__ballot(upto > s.t0));
    s.item_at = __builtin_amdgcn_readlane(upto, s.item) - __builtin_amdgcn_readlane(n, s.item);
    return s;
  }
  // Tiles per chunk of THREADS items, then their sum, then the chunk that holds t0
  // is walked again.  s_scan: a counter per wave, then the chunk sums.
  const int chunks = (items + THREADS - 1) / THREADS;
  int* s_wave = s_scan;
  int* s_chunk = s_scan + THREADS / kWave;
  int n = 0;
  for (int c = 0; c < chunks; ++c) {
    const int id = c * THREADS + tid;
    n = id < items ? item_units(make_item<KIND, M, 1, COUNTED>(a, id), COST) : 0;
    const int sum = wave_sum(n);
    if (lane_id() == 0) s_wave[tid / kWave] = sum;
    __syncthreads();
    if (tid == 0) {
      int all = 0;
#pragma unroll
      for (int i = 0; i < THREADS / kWave; ++i) all += s_wave[i];
      s_chunk[c] = all;
    }
    __syncthreads();
  }
  int64_t total = 0;
  for (int c = 0; c < chunks; ++c) total += s_chunk[c];
  s.total = total;
  s.groups = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), total / min_units)));
  if (w >= s.groups || total == 0) {
    s.t0 = s.t1 = 0;
    s.item = 0;
    s.item_at = 0;
    return s;
  }
  s.t0 = share_begin(total, s.groups, w);
  s.t1 = share_begin(total, s.groups, w + 1);
  int64_t at = 0;
  int c = 0;
  while (c + 1 < chunks && at + s_chunk[c] <= s.t0) at += s_chunk[c++];
  const int id = c * THREADS + tid;
  if (c + 1 < chunks) n = id < items ? item_units(make_item<KIND, M, 1, COUNTED>(a, id), COST) : 0;
  const int upto = wave_inclusive_scan(n);
  if (lane_id() == kWave - 1) s_wave[tid / kWave] = upto;
  __syncthreads();
  int64_t before = at + upto - n;
  for (int i = 0; i < tid / kWave; ++i) before += s_wave[i];
  if (n > 0 && before <= s.t0 && s.t0 < before + n) {
    s_res[0] = id;
    s_res[1] = before;
  }
  __syncthreads();
  s.item = static_cast<int>(s_res[0]);
  s.item_at = s_res[1];
  return s;
}

// What masks and the bias need to know of a pair; read when they do (the wide
// form has no registers to keep it in).
struct alignas(16) PairInfo {
  int start, end;  // keys that its row sees
  int pos;
  float slope;     // in powers of two
};

// Joins the pieces of pairs.  One wave per pair; lanes hold 8 dimensions each.
struct JoinArgs {
  const JoinInfo* info;
  const float* pieces;
  void* out;
  float* lse;
};

struct Joined {
  f32x4 o0, o1;
  float m, l;
};

constexpr int kAtOnce = 8;  // pieces whose loads are in flight together

// Adds n pieces: 64 at a time, first their maxima and sums (one lane each),
// then their rows, whose loads do not wait for one another.
template <class At>
__device__ __forceinline__ void join_list(Joined& j, int n, int M, int local, At at) {
  const int lane = lane_id();
  for (int i0 = 0; i0 < n; i0 += kWave) {
    float2 ml = make_float2(kMInit, 0.0f);
    if (i0 + lane < n) ml = reinterpret_cast<const float2*>(at(i0 + lane) + M * kValDim)[local];
    float top = ml.x;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    top = fmaxf(top, j.m);
    const float mine = __builtin_amdgcn_exp2f(j.m - top), part = __builtin_amdgcn_exp2f(ml.x - top);
    float sum = ml.y * part;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) sum += __shfl_xor(sum, d);
    j.l = j.l * mine + sum;
    j.m = top;
    j.o0 *= mine;
    j.o1 *= mine;
    const int some = min(n - i0, kWave);
    // (every lane: piece 0 for those past the end, with weight 0)
    for (int i = 0; i < some; i += kAtOnce) {
      f32x4 a[kAtOnce], b[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const f32x4* o = reinterpret_cast<const f32x4*>(at(i0 + min(i + k, some - 1)) +
                                                        static_cast<int64_t>(local) * kValDim + lane * 8);
        a[k] = o[0];
        b[k] = o[1];
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float by = i + k < some ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(part), i + k)) : 0.0f;
        j.o0 += a[k] * by;
        j.o1 += b[k] * by;
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void write_joined(const Joined& j, int64_t pair, void* out, float* lse) {
  using E = Elem<DT>;
  const float inv = j.l == 0.0f ? 0.0f : 1.0f / j.l;
  const i32x4 r = {E::round2(j.o0[0] * inv, j.o0[1] * inv), E::round2(j.o0[2] * inv, j.o0[3] * inv),
                   E::round2(j.o1[0] * inv, j.o1[1] * inv), E::round2(j.o1[2] * inv, j.o1[3] * inv)};
  *reinterpret_cast<i32x4*>(static_cast<short*>(out) + pair * kValDim + lane_id() * 8) = r;
  if (lse && lane_id() == 0) lse[pair] = (j.m + __log2f(j.l)) * kLn2;
}

// Dense and sparse: block (x, w) joins pairs of the pair tile that workgroup w
// began and others went on with: pairs 4 x .. 4 x + 3, one wave each, or (SPREAD)
// pair x, its pieces dealt to the four waves -- few pairs have many pieces each,
// and the loads of a wave are one round trip per kAtOnce pieces.  (Pairs on x:
// blocks are dealt to the 8 XCDs in turn, and the workgroups that begin a tile
// are often every eighth; with them on x all work fell on one XCD, 16 instead
// of 6 us for 8 rows over 2048 keys.)
template <int DT, bool SPREAD>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a, int M) {
  __shared__ f32x4 s_o[SPREAD ? 4 : 1][2][kWave];
  __shared__ float2 s_ml[4];
  const JoinInfo info = a.info[blockIdx.y];
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int local = SPREAD ? blockIdx.x : blockIdx.x * 4 + wave;
  if (info.pieces == 0 || local >= info.pairs) return;
  constexpr int kBy = SPREAD ? 4 : 1;
  const int skip = SPREAD ? wave : 0;
  Joined j{{0, 0, 0, 0}, {0, 0, 0, 0}, kMInit, 0.0f};
  join_list(j, (info.pieces - skip + kBy - 1) / kBy, M, local, [&](int i) {
    const int piece = i * kBy + skip;
    return a.pieces + static_cast<int64_t>(piece == 0 ? 2 * info.first + 1 : 2 * (info.first + piece)) * piece_floats(M);
  });
  if constexpr (SPREAD) {
    s_o[wave][0][lane] = j.o0;
    s_o[wave][1][lane] = j.o1;
    if (lane == 0) s_ml[wave] = make_float2(j.m, j.l);
    __syncthreads();
    if (wave) return;
    for (int k = 1; k < 4; ++k) {
      const float2 ml = s_ml[k];
      const float top = fmaxf(j.m, ml.x);
      const float mine = __builtin_amdgcn_exp2f(j.m - top), theirs = __builtin_amdgcn_exp2f(ml.x - top);
      j.o0 = j.o0 * mine + s_o[k][0][lane] * theirs;
      j.o1 = j.o1 * mine + s_o[k][1][lane] * theirs;
      j.l = j.l * mine + ml.y * theirs;
      j.m = top;
    }
  }
  write_joined<DT>(j, info.pair0 + local, a.out, a.lse);
}

// Shared: every pair has pieces of its prefix item and of its request's item.
template <int DT>
__global__ __launch_bounds__(256) void join_shared_kernel(JoinArgs a, int M, int64_t pairs, int heads, int next_n) {
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (pair >= pairs) return;
  const int prefix_items = static_cast<int>((pairs + M - 1) / M);
  const int of_request = next_n * heads;
  const int b = static_cast<int>(pair / of_request), in = static_cast<int>(pair - static_cast<int64_t>(b) * of_request);
  const int items[2] = {static_cast<int>(pair / M), prefix_items + b * ((of_request + M - 1) / M) + in / M};
  const int locals[2] = {static_cast<int>(pair % M), in % M};
  Joined j{{0, 0, 0, 0}, {0, 0, 0, 0}, kMInit, 0.0f};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const JoinInfo info = a.info[items[k]];
    join_list(j, info.pieces, M, locals[k], [&](int i) {
      return a.pieces + (static_cast<int64_t>(info.first) + i + items[k]) * piece_floats(M);
    });
  }
  write_joined<DT>(j, pair, a.out, a.lse);
}

constexpr int kMinTiles = 2;   // smallest part of an item that is cut into equal ones
template <int M>
constexpr int kMinUnits = kItemCost<M> + 2;  // smallest share: below, the join costs more than the split saves

// Pairs that one request (sparse: one row; shared: the batch, for the prefix)
// brings together.
template <int KIND>
int64_t pairs_together(const AttentionArgs& a) {
  if (KIND == kSparse) return a.heads;
  if (KIND == kShared) return static_cast<int64_t>(a.rows) * a.heads;
  return (static_cast<int64_t>(a.rows) + a.requests - 1) / a.requests * a.heads;
}

// Size of the pair tiles: the one whose estimated time is least, from what a
// workgroup spends on each 64-key tile and on the call (16 / 32 / 64 / 128 pairs).
// Tiles wider than the pairs would only idle.  narrowest: the longest list of the
// kernel for 16 pairs.
template <int KIND>
int tile_pairs(const AttentionArgs& a, const double (&per_tile)[4], const double (&fixed)[4], int64_t narrowest) {
  constexpr int kSizes[] = {16, 32, 64, 128};
  const int64_t together = pairs_together<KIND>(a);
  int best = 16;
  double least = 1e300;
  for (int i = 0; i < 4; ++i) {
    const int m = kSizes[i];
    if (i > 0 && together <= m / 2) break;
    if (item_count<KIND>(a, m) > (i == 0 ? narrowest : ScanOf256<KIND>::kItems)) continue;
    const int64_t pairs = static_cast<int64_t>(a.rows) * a.heads;
    double tiles;
    if (KIND == kSparse) {
      tiles = static_cast<double>(a.rows) * ((a.heads + m - 1) / m) * ((a.k + kTile - 1) / kTile);
    } else {
      const double own = a.cu_q ? static_cast<double>(pairs / m + a.requests)
                                : static_cast<double>(a.requests) * ((static_cast<int64_t>(a.next_n) * a.heads + m - 1) / m);
      tiles = KIND == kShared ? static_cast<double>((pairs + m - 1) / m) * a.prefix_pages + own * (a.max_pages - a.prefix_pages)
                              : own * a.max_pages;
    }
    const double t = tiles / kMaxGrid * per_tile[i] + fixed[i];
    if (t < least) {
      least = t;
      best = m;
    }
  }
  return best;
}

// One attention kernel over shares of the work list, and the join of what it split.
template <int DT, int KIND, int M, int COST = kItemCost<M>>
hipError_t launch_joined(void (*kernel)(AttentionArgs, int, JoinInfo*, float*), int threads, const AttentionArgs& a,
                         hipStream_t stream, LaunchEvents ev) {
  const int64_t items = item_count<KIND, M>(a);
  const int64_t tiles = KIND == kSparse ? (a.k + kTile - 1) / kTile : a.max_pages;
  int grid = static_cast<int>(
      std::max(int64_t{1}, std::min(int64_t{kMaxGrid}, items * (tiles + COST) / kMinUnits<M>)));
  // One item of a few tiles stays whole and needs no join, also where it counts for more
  // than the smallest share: one request of 65 keys 12.2 us in two parts, 10.5 in one.
  // (64 such requests on 64 workgroups 21.2 us, on 121 16.4.)
  if (items == 1) grid = static_cast<int>(std::min<int64_t>(grid, std::max<int64_t>(1, tiles / kMinTiles)));
  int min_units = kMinUnits<M>;
  if (KIND == kSparse && !a.cu_q && !a.counted && items <= kMaxGrid / 2) {  // parts of one item each
    grid = static_cast<int>(items * std::min<int64_t>(kMaxGrid / items, std::max<int64_t>(1, tiles / kMinTiles)));
    min_units = 0;
  }
  JoinInfo* info = static_cast<JoinInfo*>(a.workspace);
  float* pieces = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                           join_bytes(KIND == kShared ? items : kMaxGrid) +
                                           (a.counted ? counted_shift(M) : 0));
  const bool joins = KIND == kShared || grid > 1;
  launch_kernel(kernel, dim3(grid), dim3(threads), stream, ev.start, joins ? nullptr : ev.stop, a, min_units, info,
                pieces);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !joins) return e;
  const JoinArgs j{info, pieces, a.out, a.lse};
  if constexpr (KIND == kShared) {
    const int64_t pairs = static_cast<int64_t>(a.rows) * a.heads;
    launch_kernel(join_shared_kernel<DT>, dim3(static_cast<uint32_t>((pairs + 3) / 4)), dim3(256), stream, nullptr,
                  ev.stop, j, M, pairs, a.heads, a.next_n);
  } else {
    // (at 16 pairs, 14 -> 7 us where requests of up to 32768 keys have up to 35
    // pieces; at 32 pairs and 8 pieces 6 -> 7 us)
    if (M == 16)
      launch_kernel(join_kernel<DT, true>, dim3(M, grid), dim3(256), stream, nullptr, ev.stop, j, M);
    else
      launch_kernel(join_kernel<DT, false>, dim3(M / 4, grid), dim3(256), stream, nullptr, ev.stop, j, M);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace pmqa
