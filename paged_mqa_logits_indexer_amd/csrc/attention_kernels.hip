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
#include <algorithm>
#include <climits>
#include <type_traits>

#include "indexer_common.h"
#include "launches.h"

namespace pmqa {
namespace {

constexpr int kRowDim = IDX_LATENT_ROW;            // 576
constexpr int kValDim = IDX_LATENT_DIM;            // 512
constexpr int kRowBytes = kRowDim * 2;             // 1152
constexpr int kKSteps = kRowDim / 32;              // 18 MFMA steps of S
constexpr int kDimTiles = kValDim / 16;            // 32 output tiles of 16 dimensions
constexpr int kTile = 64;                          // keys per entry of the work list
constexpr int kOctBytes = 8 * kRowBytes;           // 8 keys in LDS: 9216
constexpr int kBlkBytes = 2 * kOctBytes;           // 16 keys
constexpr int kRingBytes = 2 * kTile * kRowBytes;  // 147456: 128 keys in all slots together
constexpr int kWindow = 2048;                      // sparse: keys whose cache rows are resolved at a time
constexpr int kAttnThreads = 256;
constexpr int kScanChunks = 1056;                  // work-list chunks of 256 pair tiles
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

// mfma_acc: the 256 accumulators of a wide wave take exactly the accumulation
// registers, the queries and everything else the 256 vector registers; written
// out, the instruction leaves the compiler no other choice (left to itself it
// moves operands between the two files at every step).  The two wait states
// cover an operand that a vector instruction has just written (they pass while
// the MFMA before is still running); before vector instructions read an
// accumulator, settle() lets the last MFMA finish.
__device__ __forceinline__ void settle(f32x16& c) { __asm__ volatile("s_nop 15\ns_nop 7" : "+a"(c)); }

// No instruction: keeps an accumulator in its registers where control flow
// joins (a value that every reader takes from the accumulation registers is
// not moved out of them).
__device__ __forceinline__ void pin(f32x16& c) { __asm__ volatile("" : "+a"(c)); }

// Where invalid keys are read from: a row of zeros, so that neither S nor the
// value product meets what the cache holds there.
__device__ __attribute__((aligned(128))) const uint32_t kZeroRow[kRowBytes / 4] = {};

// LDS image of 8 keys (9 KiB): nine 1 KiB pieces, each holding 128 bytes of
// every key -- what one direct-to-LDS load of 64 x 16 bytes writes.  Within
// its 128 bytes a key's 16-byte chunks are exchanged by c ^ swz(key), which
// spreads every kind of read over all 64 banks: the 128-bit reads of the K
// operand (served 16 lanes at a time, in groups 0-3, 12-15, 20-23, 24-27 and
// 4-7, 8-11, 16-19, 28-31 of each half wave) for 16 keys by 4 chunks and for 32
// keys by 2, and the transposing 64-bit reads of V (half a wave at a time) for
// 8 keys by 2 chunks and for 4 keys by 4.  Measured: 245 and 226 bytes a clock
// and CU, against 125 for the first with the chunks exchanged by bits 1-3 of
// the key.
__device__ __forceinline__ int swz(int key) { return (((key >> 1) & 1) << 2) | (-(key >> 2) & 3); }
__device__ __forceinline__ int key_offset(int key) { return (key >> 3) * kOctBytes + (key & 7) * 128; }

// Issues 8 keys into LDS: lane l reads 16-byte pieces of key l / 8 from `at`.
// The instruction's offset advances both the source and the LDS address by
// 128; M0 supplies the rest of the 1 KiB step.  Written in assembly so that
// the compiler does not drain the loads in flight before every LDS access of
// the other slots; the caller waits (vmcnt) before the barrier that publishes
// the keys.
constexpr int kOctLoads = 9;
template <int J>
__device__ __forceinline__ void load_piece(const char* at, uint32_t lds) {
  __asm__ volatile(
      "s_add_u32 m0, %0, %2\n"
      "s_nop 0\n"
      "global_load_lds_dwordx4 %1, off offset:%3"
      :
      : "s"(lds), "v"(at), "n"(J * 896), "n"(J * 128)
      : "memory", "m0", "scc");
}
__device__ __forceinline__ void load_octet(const char* at, uint32_t lds) {
  load_piece<0>(at, lds);
  load_piece<1>(at, lds);
  load_piece<2>(at, lds);
  load_piece<3>(at, lds);
  load_piece<4>(at, lds);
  load_piece<5>(at, lds);
  load_piece<6>(at, lds);
  load_piece<7>(at, lds);
  load_piece<8>(at, lds);
}

// Waits until at most LEFT vector memory operations of this wave are
// outstanding, then for the other waves; LDS accesses on both sides keep their
// sides.
template <int LEFT>
__device__ __forceinline__ void wait_and_barrier() {
  __asm__ volatile("" ::: "memory");
  // lgkmcnt(0), vmcnt(LEFT): the counter's two fields
  __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | ((LEFT >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

// A value whose origin the compiler does not see: constants added to such an
// LDS address become the read's own offset instead of an addition per read.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  __asm__("" : "+v"(x));
  return x;
}

typedef __attribute__((address_space(3))) const s16x8* LdsVec8;
typedef __attribute__((address_space(3))) s16x4* LdsVec4;
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

// Item `id` of the list.  Dense: requests' pair tiles.  Shared: first the pair
// tiles of the whole batch over the prefix pages, then the requests' pair
// tiles over what follows.  Sparse: rows' pair tiles over the selection.
template <int KIND, int M, int BY>
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

template <int KIND, int M>
__host__ __device__ __forceinline__ int64_t item_count(const AttentionArgs& a) {
  const int64_t pairs = static_cast<int64_t>(a.rows) * a.heads;
  if (KIND == kSparse) return static_cast<int64_t>(a.rows) * ((a.heads + M - 1) / M);
  const int64_t own = a.cu_q ? pairs / M + a.requests
                             : static_cast<int64_t>(a.requests) * ((static_cast<int64_t>(a.next_n) * a.heads + M - 1) / M);
  return KIND == kShared ? (pairs + M - 1) / M + own : own;
}

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
template <int M>
__device__ __forceinline__ int item_units(const Item& it) { return it.tiles ? it.tiles + kItemCost<M> : 0; }

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
template <int KIND, int M>
__device__ Share find_share(const AttentionArgs& a, int w, int grid, int min_units, int* s_scan, int64_t* s_res) {
  Share s;
  const int items = static_cast<int>(item_count<KIND, M>(a));
  const int tid = threadIdx.x;
  s.cost = kItemCost<M>;
  if constexpr (KIND == kSparse) {
    if (!a.cu_q) {
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
    const int n = lane_id() < items ? item_units<M>(make_item<KIND, M, 1>(a, lane_id())) : 0;
    const int upto = wave_inclusive_scan(n);
    s.total = __builtin_amdgcn_readlane(upto, kWave - 1);
    s.groups = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), s.total / min_units)));
    s.t0 = w < s.groups ? share_begin(s.total, s.groups, w) : 0;
    s.t1 = w < s.groups ? share_begin(s.total, s.groups, w + 1) : 0;
    s.item = first_lane(__ballot(upto > s.t0));
    s.item_at = __builtin_amdgcn_readlane(upto, s.item) - __builtin_amdgcn_readlane(n, s.item);
    return s;
  }
  // Tiles per chunk of 256 items, then their sum, then the chunk that holds t0
  // is walked again.  s_scan: a counter per wave, then the chunk sums.
  const int chunks = (items + kAttnThreads - 1) / kAttnThreads;
  int* s_wave = s_scan;
  int* s_chunk = s_scan + kAttnThreads / kWave;
  int n = 0;
  for (int c = 0; c < chunks; ++c) {
    const int id = c * kAttnThreads + tid;
    n = id < items ? item_units<M>(make_item<KIND, M, 1>(a, id)) : 0;
    const int sum = wave_sum(n);
    if (lane_id() == 0) s_wave[tid / kWave] = sum;
    __syncthreads();
    if (tid == 0) s_chunk[c] = s_wave[0] + s_wave[1] + s_wave[2] + s_wave[3];
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
  const int id = c * kAttnThreads + tid;
  if (c + 1 < chunks) n = id < items ? item_units<M>(make_item<KIND, M, 1>(a, id)) : 0;
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

// Pieces in the workspace: float o[M][512], then float2 (m, l)[M].  Dense and
// sparse: two per workgroup, for a pair tile that began before it (2 w) and one
// that ends after it (2 w + 1).  Shared: every (workgroup, item) visit is a
// piece, w + item -- consecutive over a pair tile's workgroups.
__host__ __device__ __forceinline__ int64_t piece_floats(int m) { return static_cast<int64_t>(m) * (kValDim + 2); }

// How a workgroup of four waves divides a pair tile of M pairs and a step of
// keys.  Narrow (M <= 64): 16 pairs per wave, 64 keys per step in 2 slots, and
// where fewer than four waves cover the pairs the others take other keys of
// the same pairs (streams, joined at the end); their time is the K stream's.
// Wide (M = 128): 32 pairs per wave, so that each LDS operand feeds twice the
// arithmetic, and 32 keys per step in 4 slots: the value product of a step runs
// after the next step's scores, between whose MFMAs its weights are computed,
// and two steps of loads are ahead.  (1024 rows of 128 heads over 2048 selected
// keys, calls in a row on the same card: 624 us, with 64-pair tiles of the narrow
// form 793.)
template <int M>
struct Shape {
  static constexpr bool kWide = M == 128;
  static constexpr int kWavePairs = kWide ? 32 : 16;
  static constexpr int kGroups = M / kWavePairs;      // waves that cover the pairs
  static constexpr int kStreams = 4 / kGroups;
  static constexpr int kKeys = kWide ? 32 : 64;       // keys of a step
  static constexpr int kSlots = 128 / kKeys;
  static constexpr int kSlotBytes = kKeys * kRowBytes;
  static constexpr int kDistance = kWide ? 2 : 1;     // steps that are loaded ahead
  static constexpr int kOctets = kKeys / 32;          // octets that each wave loads per step
  static constexpr int kBlocks = kWide ? 2 : kKeys / 16 / kStreams;  // 16-key blocks of a step per wave
};

// What masks and the bias need to know of a pair; read when they do (the wide
// form has no registers to keep it in).
struct alignas(16) PairInfo {
  int start, end;  // keys that its row sees
  int pos;
  float slope;     // in powers of two
};

template <int DT, int KIND, int M>
__global__ __launch_bounds__(kAttnThreads, 1) void attention_kernel(AttentionArgs a, int min_units, JoinInfo* join,
                                                                    float* pieces) {
  using E = Elem<DT>;
  using S = Shape<M>;
  constexpr int kStepsPerTile = kTile / S::kKeys;
  constexpr int ST = S::kBlocks;
  __shared__ __attribute__((aligned(1024))) char s_keys[kRingBytes];
  __shared__ int s_rows[KIND == kSparse ? kWindow : 1];       // sparse: cache row of each listed key, -1: none
  __shared__ uint32_t s_live[S::kSlots][4];                   // sparse: bits of the keys that are there
  __shared__ float2 s_ml[4][S::kWavePairs];
  __shared__ PairInfo s_pair[S::kWavePairs * S::kGroups];
  __shared__ int64_t s_res[2];
  __shared__ int s_scan[KIND == kSparse ? 8 + 640 : kAttnThreads / kWave + kScanChunks];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grid = gridDim.x;
  // consecutive shares on one XCD (workgroups are dealt to the 8 XCDs in turn)
  const int w = (grid & 7) ? static_cast<int>(blockIdx.x)
                           : static_cast<int>(blockIdx.x & 7) * (grid >> 3) + static_cast<int>(blockIdx.x >> 3);
  const Share share = find_share<KIND, M>(a, w, grid, min_units, s_scan, s_res);
  if (KIND != kShared && tid == 0) join[w].pieces = 0;
  if (share.t0 >= share.t1) return;

  const uint32_t ring = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)s_keys));
  const int pg = wave / S::kStreams, ts = wave % S::kStreams;
  const int n16 = lane & 15, g4 = lane >> 4, half = lane >> 5;
  const int col = lane & (S::kWavePairs - 1);  // this lane's pair of the wave's
  // places of this lane in a step's keys: K operand and transposed V operand
  uint32_t k_at, v_at;
  if constexpr (S::kWide) {
    const int key = lane & 31, vkey = 4 * half + (n16 >> 2);
    k_at = key_offset(key) + (half ^ swz(key)) * 16;
    v_at = key_offset(vkey) + (((2 * (g4 & 1) + ((lane & 3) >> 1)) ^ swz(vkey)) * 16) + (lane & 1) * 8;
  } else {
    const int vkey = 4 * g4 + (n16 >> 2);
    k_at = key_offset(n16) + (g4 ^ swz(n16)) * 16;
    v_at = key_offset(vkey) + (((n16 >> 1) & 1) ^ swz(vkey)) * 16 + (n16 & 1) * 8;
  }
  const int capacity = a.max_pages * kPage;
  const char* cache = static_cast<const char*>(a.cache);
  const float to_log2 = a.scale * kLog2e;
  // wide: the factor is applied where the maximum is taken, unless the score is
  // changed before (or the factor turns the order round)
  const bool prescale = a.softcap > 0.0f || a.slopes || !(to_log2 > 0.0f);
  const float z_scale = prescale ? 1.0f : to_log2;

  const int items = static_cast<int>(item_count<KIND, M>(a));
  int64_t at = share.t0;
  int64_t item_at = share.item_at;
  int item = share.item;
  for (; at < share.t1 && item < items; ++item) {
    const Item it = make_item<KIND, M, kWave>(a, item);
    const int64_t tiles_at = item_at + (it.tiles ? share.cost : 0);
    item_at = tiles_at + it.tiles;
    const int lo = static_cast<int>(max(int64_t{0}, at - tiles_at));
    const int hi = static_cast<int>(min(static_cast<int64_t>(it.tiles), share.t1 - tiles_at));
    at = item_at;
    if (lo >= hi) continue;  // no pairs, or another workgroup's keys
    const bool whole = lo == 0 && hi == it.tiles && KIND != kShared;
    const int32_t* table = a.block_table + static_cast<int64_t>(it.request) * a.max_pages;
    const int step0 = lo * kStepsPerTile, step_end = hi * kStepsPerTile;

    // ---- loading
    int page_window = -1, window_page = 0;  // dense: page ids of 64 tiles, one per lane
    int row_window = -1;                    // sparse: window of keys in s_rows
    // sparse: cache rows of kWindow listed keys, two dependent loads for AT of
    // them per thread at a time (all at the beginning, one by one where a list
    // longer than the window goes on between two steps: there the loop's
    // registers have no room for more)
    auto resolve = [&](int window, auto many) {
      constexpr int AT = decltype(many)::value;
      row_window = window;
      const int32_t* list = a.indices + static_cast<int64_t>(it.row0) * a.k + window * kWindow;
      const int n = min(kWindow, a.k - window * kWindow);
#pragma unroll 1
      for (int i0 = tid; i0 < kWindow; i0 += AT * kAttnThreads) {
        int tok[AT], page[AT];
#pragma unroll
        for (int i = 0; i < AT; ++i) tok[i] = i0 + i * kAttnThreads < n ? list[i0 + i * kAttnThreads] : -1;
#pragma unroll
        for (int i = 0; i < AT; ++i) {
          if (tok[i] >= capacity) tok[i] = -1;
          page[i] = tok[i] >= 0 ? table[tok[i] / kPage] : 0;
        }
#pragma unroll
        for (int i = 0; i < AT; ++i)
          s_rows[i0 + i * kAttnThreads] =
              tok[i] >= 0 ? max(0, min(page[i], a.num_pages - 1)) * kPage + (tok[i] & (kPage - 1)) : -1;
      }
    };
    const char* zero = reinterpret_cast<const char*>(kZeroRow);
    const char* from[S::kOctets];  // next loads: this lane's source ...
    uint32_t to[S::kOctets];       // ... and the wave's place in the ring
    // (the wide form also loads the two steps after the last, from the row of
    // zeros: it then has no branch between its MFMAs)
    auto locate = [&](int step) {
      const int slot = (step - step0) & (S::kSlots - 1);
      const bool any = step < step_end;
      int page = 0;
      const int key0 = step * S::kKeys + wave * (8 * S::kOctets);  // this wave's first key of the item's list
      if constexpr (KIND == kSparse) {
        if (any && key0 / kWindow != row_window) {  // the same for all waves: a window is whole steps
          lds_barrier();
          resolve(key0 / kWindow, std::integral_constant<int, 1>{});
          lds_barrier();
        }
      } else {
        const int tile = it.tile0 + min(key0 / kTile, it.tiles - 1);
        if ((tile >> 6) != page_window) {
          page_window = tile >> 6;
          window_page = table[min(page_window * 64 + lane, a.max_pages - 1)];
          __asm__ volatile("" : "+v"(window_page));  // waited for here, not in the steps that only read it
        }
        page = max(0, min(__builtin_amdgcn_readlane(window_page, tile & 63), a.num_pages - 1));
      }
      uint32_t live_bits = 0;
#pragma unroll
      for (int o = 0; o < S::kOctets; ++o) {
        const int key = key0 + 8 * o + (lane >> 3);
        int row;
        bool live;
        if constexpr (KIND == kSparse) {
          row = s_rows[key & (kWindow - 1)];
          live = any && row >= 0;
          const uint64_t mask = __ballot(live);
#pragma unroll
          for (int i = 0; i < 8; ++i) live_bits |= static_cast<uint32_t>(mask >> (8 * i) & 1) << (8 * o + i);
        } else {
          // keys that no row of the pair tile sees are not read
          const int tok = it.tile0 * kTile + key;
          row = page * kPage + (key & (kPage - 1));
          live = any && tok >= it.min_start && tok < it.max_end;
        }
        from[o] = (live ? cache + static_cast<int64_t>(row) * kRowBytes : zero) +
                  (((lane & 7) ^ swz((8 * ((wave * S::kOctets + o) & 1)) + (lane >> 3))) * 16);
        to[o] = ring + slot * S::kSlotBytes + (wave * S::kOctets + o) * kOctBytes;
      }
      if (KIND == kSparse && lane == 0) s_live[slot][wave] = live_bits;
    };
    auto load_one = [&](int j) {  // wide: j is a constant of the unrolled loop
      switch (j) {
        case 0: return load_piece<0>(from[0], to[0]);
        case 1: return load_piece<1>(from[0], to[0]);
        case 2: return load_piece<2>(from[0], to[0]);
        case 3: return load_piece<3>(from[0], to[0]);
        case 4: return load_piece<4>(from[0], to[0]);
        case 5: return load_piece<5>(from[0], to[0]);
        case 6: return load_piece<6>(from[0], to[0]);
        case 7: return load_piece<7>(from[0], to[0]);
        case 8: return load_piece<8>(from[0], to[0]);
      }
    };
    auto issue = [&](int step) {
      locate(step);
#pragma unroll
      for (int o = 0; o < S::kOctets; ++o) load_octet(from[o], to[o]);
    };

    // ---- the queries come through the ring as well (whole 128-byte pieces; the
    // operand layout's own addresses would take a quarter of each line), in
    // the last slots, beside the first keys where there is room
    constexpr int kQ = S::kWide ? 36 : kKSteps;
    const uint32_t q_ring = ring + kRingBytes - M * kRowBytes;
    const int64_t pair_base = static_cast<int64_t>(it.row0) * a.heads + it.pair0;  // over the whole batch
    lds_barrier();  // the previous item's epilogue has left the ring
    if constexpr (KIND != kSparse) {  // asked for together with what the pairs need to know
      page_window = (it.tile0 + lo) >> 6;
      window_page = table[min(page_window * 64 + lane, a.max_pages - 1)];
    }
    for (int local = tid; local < M; local += kAttnThreads) {
      const int pair = it.pair0 + min(local, it.pairs - 1);
      const int row = it.row0 + pair / a.heads;
      PairInfo info{0, capacity, 0, 0.0f};
      if constexpr (KIND != kSparse) {
        info.end = clamp_len(a.row_lens[row], capacity);
        if (a.row_starts) info.start = max(0, a.row_starts[row]);
      }
      if (a.slopes) {
        info.slope = a.slopes[pair % a.heads] * kLog2e;
        info.pos = a.row_positions ? a.row_positions[row] : info.end - 1;
      }
      info.start = max(info.start, it.key_lo);
      info.end = min(info.end, it.key_hi);
      s_pair[local] = info;
    }
    if constexpr (KIND == kSparse) {
      resolve(step0 * S::kKeys / kWindow, std::integral_constant<int, kWindow / kAttnThreads>{});
      lds_barrier();
    }
    if constexpr (KIND != kSparse) __asm__ volatile("" : "+v"(window_page));
    for (int o = wave; o < M / 8; o += 4) {
      const int pair = 8 * o + (lane >> 3);
      const char* from = (pair < it.pairs ? static_cast<const char*>(a.q) + (pair_base + pair) * kRowBytes : zero) +
                         (((lane & 7) ^ swz(pair & 15)) * 16);
      load_octet(from, q_ring + o * kOctBytes);
    }
    // narrow: slot 0 holds step0's keys, slot 1 the queries
    if constexpr (!S::kWide) issue(step0);
    wait_and_barrier<0>();
    s16x8 q[kQ];
    // wide: recomputed for every item (as 36 addresses kept over the items they go
    // to scratch memory, one reload behind the other: 4 % of the call at 1024 rows
    // as above)
    uint32_t q_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q_at[i] = opaque(q_ring + pg * 32 * kRowBytes + (k_at ^ (i * 32)));
#pragma unroll
    for (int ks = 0; ks < kQ; ++ks) {
      if constexpr (S::kWide)
        q[ks] = lds_read(q_at[ks & 3] + (ks >> 2) * 1024);
      else
        q[ks] = lds_read(q_ring + pg * 16 * kRowBytes + (k_at ^ ((ks & 1) * 64)) + (ks >> 1) * 1024);
    }
    lds_barrier();
    if constexpr (S::kWide) {
#pragma unroll
      for (int d = 0; d < S::kDistance; ++d) issue(step0 + d);
    }

    // accumulators: dimensions on the rows, pairs on the columns
    using Acc = std::conditional_t<S::kWide, f32x16, f32x4>;
    constexpr int kAccs = S::kWide ? kValDim / 32 : kDimTiles;
    constexpr int kScores = ST * (S::kWide ? 8 : 4);  // scores of this lane per step
    Acc acc[kAccs];
#pragma unroll
    for (int d = 0; d < kAccs; ++d) acc[d] = Acc{};
    float m = kMInit, l = 0.0f, l_kept = 0.0f;  // l_kept: of the rounded weights
    // wide: scores of the step before (of none before the first: weights of zero)
    // and its weights
    float z_before[kScores];
    i32x4 p_wide[2];
#pragma unroll
    for (int i = 0; i < kScores; ++i) z_before[i] = -__builtin_inff();
    auto weigh = [&](int i, float& sum) {  // scores 2 i and 2 i + 1
      const float e0 = weight(z_before[2 * i], m), e1 = weight(z_before[2 * i + 1], m);
      sum += e0 + e1;
      int both = E::round2(e0, e1);
      __asm__ volatile("" : "+v"(both), "+v"(sum));  // computed here, between the MFMAs, and not where it is used
      p_wide[i / 4][i % 4] = both;
    };

    // (wide) the rounded weights into their sum, in the eight dimension tiles of
    // the value product that no maximum is taken in
    auto keep = [&](int i, float& kept) {
      kept = E::add2(p_wide[i / 4][i % 4], kept);
      __asm__ volatile("" : "+v"(kept));
    };

    // the value product of one step (wide), V^T P^T on the keys at `base`; each
    // of the 16 dimension tiles is followed by a piece of other work, and the
    // operands are read two tiles ahead (four, or the first ones before the
    // scores: 118 -> 130 us for 8 requests on 32768 shared keys; there are no
    // registers for them)
    auto value_wide = [&](uint32_t base, auto&& between) {
      if constexpr (S::kWide) {
        constexpr int kRing = 4;
        s16x8 v[kRing][2];
        uint32_t at[4];  // even and odd dimension tile, first and second half of 16 keys
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = opaque(base + (v_at ^ ((i & 1) * 64) ^ ((i >> 1) * 32)));
        auto read = [&](int d) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            v[d % kRing][kk] =
                __builtin_shufflevector(lds_read_tr(at[d & 1] + (2 * kk) * kOctBytes + (d >> 1) * 1024),
                                        lds_read_tr(at[2 + (d & 1)] + (2 * kk + 1) * kOctBytes + (d >> 1) * 1024), 0, 1,
                                        2, 3, 4, 5, 6, 7);
        };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < kRing - 2; ++d) read(d);
#pragma unroll
        for (int d = 0; d < kAccs; d += 2) {
          if (d + kRing - 2 < kAccs) read(d + kRing - 2);
          __builtin_amdgcn_sched_barrier(0);
          E::mfma_acc(v[d % kRing][0], v[(d + 1) % kRing][0], __builtin_bit_cast(s16x8, p_wide[0]), acc[d],
                      acc[d + 1]);
          between(d);
          __builtin_amdgcn_sched_barrier(0);
          if (d + kRing - 1 < kAccs) read(d + kRing - 1);
          __builtin_amdgcn_sched_barrier(0);
          E::mfma_acc(v[d % kRing][1], v[(d + 1) % kRing][1], __builtin_bit_cast(s16x8, p_wide[1]), acc[d],
                      acc[d + 1]);
          between(d + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };

    // One step.  Returns whether the accumulators of a wide wave have to take a
    // raised maximum; they do outside the step, so that inside it nothing but
    // the MFMAs touches them.
    float by = 1.0f;
    auto do_step = [&](int step) -> bool {
      // the step's keys are in their slot, and every wave has left the slot
      // that the next issue fills
      if constexpr (S::kWide) {
        wait_and_barrier<S::kOctets * kOctLoads>();  // all but the next step's
      } else {
        wait_and_barrier<0>();
        if (step + S::kDistance < step_end) issue(step + S::kDistance);
      }
      const int slot = (step - step0) & (S::kSlots - 1);
      const uint32_t base = ring + slot * S::kSlotBytes + (S::kWide ? 0 : ts * ST * kBlkBytes);

      // ---- S = K Q^T
      float z[kScores];
      if constexpr (S::kWide) {
        // Between the MFMAs: the loads of the step after next and the weights
        // of the step before.
        f32x16 s0 = {};
        float sum = 0.0f;
        constexpr int kRing = 6;  // operands: 4 read ahead
        s16x8 kk[kRing];
        uint32_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = opaque(base + (k_at ^ (i * 32)));
        auto read = [&](int ks) { kk[ks % kRing] = lds_read(at[ks & 3] + (ks >> 2) * 1024); };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < kRing - 2; ++ks) read(ks);
        __builtin_amdgcn_sched_barrier(0);
        locate(step + S::kDistance);  // while they come
#pragma unroll
        for (int ks = 0; ks < kQ; ks += 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ks + kRing - 2 + i < kQ) read(ks + kRing - 2 + i);
          __builtin_amdgcn_sched_barrier(0);
          s0 = E::mfma_wide(kk[ks % kRing], q[ks], s0);
          s0 = E::mfma_wide(kk[(ks + 1) % kRing], q[ks + 1], s0);
          if (ks / 2 < kOctLoads)
            load_one(ks / 2);
          else if (ks / 2 - kOctLoads < 8)
            weigh(ks / 2 - kOctLoads, sum);
          __builtin_amdgcn_sched_barrier(0);
        }
        l += sum;
#pragma unroll
        for (int i = 0; i < kScores; ++i) z[i] = s0[i];
      } else {
        constexpr int kChains = ST == 1 ? 2 : 1;
        constexpr int kReads = kKSteps * ST, kRing = 8;
        f32x4 s[ST][kChains] = {};
        s16x8 kk[kRing];
        const uint32_t at[2] = {opaque(base + k_at), opaque(base + (k_at ^ 64))};
        auto read = [&](int r) {
          const int ks = r / ST, st = r % ST;
          kk[r % kRing] = lds_read(at[ks & 1] + st * kBlkBytes + (ks >> 1) * 1024);
        };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < kRing - 2; ++r) read(r);
#pragma unroll
        for (int r = 0; r < kReads; ++r) {
          if (r % 2 == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (r + kRing - 2 + i < kReads) read(r + kRing - 2 + i);
            __builtin_amdgcn_sched_barrier(0);
          }
          const int ks = r / ST, st = r % ST;
          s[st][ks % kChains] = E::mfma32(kk[r % kRing], q[ks], s[st][ks % kChains]);
          if (r % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < kScores; ++i) {
          z[i] = s[i / 4][0][i % 4];
          if constexpr (kChains == 2) z[i] += s[i / 4][1][i % 4];
        }
      }

      // ---- scores in powers of two, masked keys at -inf.  Score i is key
      // key_of(i) of the wave's part of the step.
      auto key_of = [&](int i) {
        return S::kWide ? 8 * (i >> 2) + 4 * half + (i & 3) : ts * ST * 16 + 16 * (i >> 2) + 4 * g4 + (i & 3);
      };
      const int step_key = step * S::kKeys;  // of the item's list
      if (a.softcap > 0.0f) {
        const float in = a.scale / a.softcap, cap = a.softcap * kLog2e;
        // (z - z: 0, and NaN where z is not finite, which tanh would hide)
#pragma unroll
        for (int i = 0; i < kScores; ++i) z[i] = __builtin_fmaf(cap, tanh_f32(z[i] * in), z[i] - z[i]);
      } else if (!S::kWide || prescale) {
#pragma unroll
        for (int i = 0; i < kScores; ++i) z[i] *= to_log2;
      }
      if (a.slopes) {
        const PairInfo info = s_pair[pg * S::kWavePairs + col];
        const int32_t* list = KIND == kSparse ? a.indices + static_cast<int64_t>(it.row0) * a.k : nullptr;
#pragma unroll
        for (int i = 0; i < kScores; ++i) {
          const int c = step_key + key_of(i);
          const int tok = KIND == kSparse ? list[min(c, a.k - 1)] : it.tile0 * kTile + c;
          z[i] -= info.slope * fabsf(static_cast<float>(info.pos - tok));
        }
      }
      bool mixed = false;  // some key that was read is hidden from some row
      if constexpr (KIND == kSparse) {
        uint32_t live[2];
        if constexpr (S::kWide) {
          live[0] = s_live[slot][0] | s_live[slot][1] << 8 | s_live[slot][2] << 16 | s_live[slot][3] << 24;
          live[1] = ~0u;
        } else {
          live[0] = s_live[slot][0] | s_live[slot][1] << 16;
          live[1] = s_live[slot][2] | s_live[slot][3] << 16;
        }
        if (__builtin_amdgcn_readfirstlane(live[0] & live[1]) != -1) {
#pragma unroll
          for (int i = 0; i < kScores; ++i) {
            const int c = key_of(i);
            const uint32_t word = S::kWide || c < 32 ? live[0] : live[1];
            z[i] = (word >> (c & 31)) & 1 ? z[i] : -__builtin_inff();
          }
        }
      } else {
        const int first = it.tile0 * kTile + step_key;
        mixed = max(first, it.min_start) < it.max_start || min(first + S::kKeys, it.max_end) > it.min_end;
        if (first < it.max_start || first + S::kKeys > it.min_end) {
          const PairInfo info = s_pair[pg * S::kWavePairs + col];
#pragma unroll
          for (int i = 0; i < kScores; ++i) {
            const int tok = first + key_of(i);
            z[i] = tok >= info.start && tok < info.end ? z[i] : -__builtin_inff();
          }
        }
      }

      // A key that some rows of the pair tile see and others do not may hold an
      // infinity or a NaN; a weight of zero would not take it out of the
      // product.  Rows that see it get their NaN from S, also under a cap; a
      // score of -inf leaves the key a weight of zero.
      auto clear_nonfinite = [&] {
        __syncthreads();
        for (int i = tid; i < S::kSlotBytes / 16; i += kAttnThreads) {
          s16x8* v = reinterpret_cast<s16x8*>(s_keys + slot * S::kSlotBytes) + i;
          s16x8 x = *v;
          constexpr int kExp = DT == IDX_BF16 ? 0x7F80 : 0x7C00;
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = (x[j] & kExp) == kExp ? 0 : x[j];
          *v = x;
        }
        __syncthreads();
      };
      if constexpr (KIND != kSparse) {
        if (mixed) clear_nonfinite();
      }

      if constexpr (S::kWide) {
        // ---- the step before: O^T += V^T P^T, with this step's maximum between
        // its MFMAs; then the accumulators take it.  (The first step has none
        // before it: weights of zero on its own keys, which every row of the
        // pair tile sees or whose non-finite values have been cleared.)
        float mx = -__builtin_inff(), kept = 0.0f;
        value_wide(step > step0 ? ring + ((step - step0 - 1) & (S::kSlots - 1)) * S::kSlotBytes : base, [&](int d) {
          if (d < 8) {
            z[2 * d] *= z_scale;
            z[2 * d + 1] *= z_scale;
            mx = fmaxf(mx, fmaxf(z[2 * d], z[2 * d + 1]));
          } else {
            keep(d - 8, kept);
          }
        });
        mx = pair_max<true>(mx) - E::kShift;
        const float raised = mx > m + E::kRaise ? mx : m;
        const bool any_raised = step > step0 && __ballot(raised != m) != 0;  // nothing to rescale in the first step
        by = __builtin_amdgcn_exp2f(m - raised);
        m = raised;
        l *= by;
        l_kept = (l_kept + kept) * by;
#pragma unroll
        for (int i = 0; i < kScores; ++i) z_before[i] = z[i];
        return any_raised;
      } else {
        // ---- running maximum: raised where a score passes it by kRaise
        float mx = z[0];
#pragma unroll
        for (int i = 1; i < kScores; ++i) mx = fmaxf(mx, z[i]);
        mx = pair_max<false>(mx) - E::kShift;
        const float raised = mx > m + E::kRaise ? mx : m;
        const bool any_raised = step > step0 && __ballot(raised != m) != 0;  // nothing to rescale in the first step
        by = __builtin_amdgcn_exp2f(m - raised);
        m = raised;
        if (any_raised) {
          l *= by;
          l_kept *= by;
#pragma unroll
          for (int d = 0; d < kAccs; ++d) acc[d] *= by;
        }
        s16x4 p[ST];
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = weight(z[st * 4 + i], m);
          l += (e[0] + e[1]) + (e[2] + e[3]);
          const int2 both = make_int2(E::round2(e[0], e[1]), E::round2(e[2], e[3]));
          l_kept += E::add2(both.x, E::add2(both.y, 0.0f));
          p[st] = __builtin_bit_cast(s16x4, both);
        }
        // ---- O^T += V^T P^T
        if constexpr (!S::kWide) {
          constexpr int kRing = ST == 1 ? 10 : ST == 2 ? 6 : 4;
          s16x4 v[kRing][ST];
          uint32_t at[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) at[i] = opaque(base + (v_at ^ (i * 32)));
          auto read = [&](int d) {
#pragma unroll
            for (int st = 0; st < ST; ++st)
              v[d % kRing][st] = lds_read_tr(at[d & 3] + (d >> 2) * 1024 + st * kBlkBytes);
          };
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int d = 0; d < kRing - 2; ++d) read(d);
#pragma unroll
          for (int d = 0; d < kAccs; ++d) {
            if (d % 2 == 0) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (d + kRing - 2 + i < kAccs) read(d + kRing - 2 + i);
              __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (ST == 1) {
              acc[d] = E::mfma16(v[d % kRing][0], p[0], acc[d]);
            } else {
#pragma unroll
              for (int st = 0; st < ST; st += 2)
                acc[d] = E::mfma32(__builtin_shufflevector(v[d % kRing][st], v[d % kRing][st + 1], 0, 1, 2, 3, 4, 5, 6, 7),
                                   __builtin_shufflevector(p[st], p[st + 1], 0, 1, 2, 3, 4, 5, 6, 7), acc[d]);
            }
            if (d % 2 == 1) __builtin_amdgcn_sched_barrier(0);
          }
        }
        return false;
      }
    };
    if constexpr (S::kWide) {
      for (int step = step0; step < step_end;) {
#pragma unroll
        for (int d = 0; d < kAccs; ++d) pin(acc[d]);
        bool raise;
        do {
          raise = do_step(step);
          ++step;
        } while (!raise && step < step_end);
        if (raise) {
#pragma unroll
          for (int d = 0; d < kAccs; ++d) {  // one at a time: there are registers for one
            settle(acc[d]);
            acc[d] *= by;
            pin(acc[d]);
          }
        }
#pragma unroll
        for (int d = 0; d < kAccs; ++d) pin(acc[d]);
      }
#pragma unroll
      for (int d = 0; d < kAccs; ++d) pin(acc[d]);
#pragma unroll
      for (int i = 0; i < 8; ++i) weigh(i, l);
      value_wide(ring + ((step_end - step0 - 1) & (S::kSlots - 1)) * S::kSlotBytes, [&](int d) {
        if (d < 8) keep(d, l_kept);
      });
    } else {
      for (int step = step0; step < step_end; ++step) do_step(step);
    }

    // ---- the streams' parts of each pair become one, through LDS, and leave as
    // whole rows
    float factor = 1.0f;  // of this lane's part of its pair
    {
      const float sum = pair_sum<S::kWide>(l), kept = pair_sum<S::kWide>(l_kept);
      if (lane < S::kWavePairs) s_ml[wave][lane] = make_float2(m, sum);
      if (kept > 0.0f) factor = sum / kept;  // (no key, or NaN, otherwise)
    }
    wait_and_barrier<0>();  // every wave has left the ring, its last loads have ended, and s_ml is complete
    float* piece = nullptr;
    if (!whole) {
      const int64_t id = KIND == kShared ? static_cast<int64_t>(w) + item : (lo == 0 ? 2 * w + 1 : 2 * w);
      piece = pieces + id * piece_floats(M);
    }
    {
      const int first = pg * S::kStreams;
      float top = kMInit, sum = 0.0f;
#pragma unroll
      for (int k = 0; k < S::kStreams; ++k) top = fmaxf(top, s_ml[first + k][col].x);
#pragma unroll
      for (int k = 0; k < S::kStreams; ++k) {
        const float2 ml = s_ml[first + k][col];
        sum += ml.y * __builtin_amdgcn_exp2f(ml.x - top);
      }
      factor *= __builtin_amdgcn_exp2f(m - top);
      const int local = pg * S::kWavePairs + col;
      if (whole) {
        factor = sum == 0.0f ? 0.0f : factor / sum;
        if (a.lse && ts == 0 && lane < S::kWavePairs && local < it.pairs)
          a.lse[pair_base + local] = (top + __log2f(sum)) * kLn2;
      } else if (ts == 0 && lane < S::kWavePairs && local < it.pairs) {
        reinterpret_cast<float2*>(piece + M * kValDim)[local] = make_float2(top, sum);
      }
    }
    // 64 (narrow) or 128 (wide) rows of accumulators; the pad of 4 floats
    // spreads the pairs over all banks
    constexpr int kChunks = S::kWide ? 2 : 1, kChunkDims = kValDim / kChunks, kStride = kChunkDims + 4;
    float* s_o = reinterpret_cast<float*>(s_keys);
    float* mine = s_o + (wave * S::kWavePairs + col) * kStride;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (c) lds_barrier();  // stores to memory go on meanwhile
      if constexpr (S::kWide) {
#pragma unroll
        for (int d = 8 * c; d < 8 * c + 8; ++d) {
          settle(acc[d]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(mine + (d & 7) * 32 + 8 * i + 4 * half) =
                f32x4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]} * factor;
        }
      } else {
#pragma unroll
        for (int d = 0; d < kAccs; ++d) {
          if constexpr (!S::kWide) *reinterpret_cast<f32x4*>(mine + d * 16 + 4 * g4) = acc[d] * factor;
        }
      }
      lds_barrier();
      constexpr int kPerRow = kChunkDims / 4, kRows = kAttnThreads / kPerRow;  // rows at a time
      const int dim = tid % kPerRow * 4;
#pragma unroll 4
      for (int local = tid / kPerRow; local < it.pairs; local += kRows) {
        const float* parts = s_o + (local / S::kWavePairs * S::kStreams * S::kWavePairs + local % S::kWavePairs) * kStride + dim;
        f32x4 o = *reinterpret_cast<const f32x4*>(parts);
#pragma unroll
        for (int k = 1; k < S::kStreams; ++k) o += *reinterpret_cast<const f32x4*>(parts + k * S::kWavePairs * kStride);
        if (whole) {
          const int2 r = make_int2(E::round2(o[0], o[1]), E::round2(o[2], o[3]));
          *reinterpret_cast<int2*>(static_cast<short*>(a.out) + (pair_base + local) * kValDim + c * kChunkDims + dim) = r;
        } else {
          *reinterpret_cast<f32x4*>(piece + static_cast<int64_t>(local) * kValDim + c * kChunkDims + dim) = o;
        }
      }
    }
    if (!whole && lo == 0 && tid == 0) {
      const int last = share_owner(share.total, share.groups, item_at - 1);
      JoinInfo j;
      j.pair0 = pair_base;
      j.pairs = it.pairs;
      j.pieces = last - w + 1;
      j.first = w;
      j.pad = 0;
      j.pad2 = 0;
      join[KIND == kShared ? item : w] = j;
    }
  }
}

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

constexpr int kMaxGrid = 256;  // one persistent workgroup per CU
constexpr int kMinTiles = 2;   // smallest part of an item that is cut into equal ones
template <int M>
constexpr int kMinUnits = kItemCost<M> + 2;  // smallest share: below, the join costs more than the split saves

size_t join_bytes(int64_t infos) { return (static_cast<size_t>(infos) * sizeof(JoinInfo) + 255) / 256 * 256; }

// Pairs that one request (sparse: one row; shared: the batch, for the prefix)
// brings together.
template <int KIND>
int64_t pairs_together(const AttentionArgs& a) {
  if (KIND == kSparse) return a.heads;
  if (KIND == kShared) return static_cast<int64_t>(a.rows) * a.heads;
  return (static_cast<int64_t>(a.rows) + a.requests - 1) / a.requests * a.heads;
}

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
template <int KIND>
int tile_pairs(const AttentionArgs& a) {
  constexpr int kSizes[] = {16, 32, 64, 128};
  constexpr double kPerTile[] = {2.2, 2.1, 3.5, 3.9}, kFixed[] = {19, 20, 32, 65};
  const int64_t together = pairs_together<KIND>(a);
  int best = 16;
  double least = 1e300;
  for (int i = 0; i < 4; ++i) {
    const int m = kSizes[i];
    if (i > 0 && together <= m / 2) break;
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
    const double t = tiles / kMaxGrid * kPerTile[i] + kFixed[i];
    if (t < least) {
      least = t;
      best = m;
    }
  }
  return best;
}

template <int DT, int KIND, int M>
hipError_t launch(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  const int64_t items = item_count<KIND, M>(a);
  const int64_t tiles = KIND == kSparse ? (a.k + kTile - 1) / kTile : a.max_pages;
  int grid = static_cast<int>(
      std::max(int64_t{1}, std::min(int64_t{kMaxGrid}, items * (tiles + kItemCost<M>) / kMinUnits<M>)));
  int min_units = kMinUnits<M>;
  if (KIND == kSparse && !a.cu_q && items <= kMaxGrid / 2) {  // parts of one item each
    grid = static_cast<int>(items * std::min<int64_t>(kMaxGrid / items, std::max<int64_t>(1, tiles / kMinTiles)));
    min_units = 0;
  }
  JoinInfo* info = static_cast<JoinInfo*>(a.workspace);
  float* pieces = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                           join_bytes(KIND == kShared ? items : kMaxGrid));
  const bool joins = KIND == kShared || grid > 1;
  launch_kernel(attention_kernel<DT, KIND, M>, dim3(grid), dim3(kAttnThreads), stream, ev.start,
                joins ? nullptr : ev.stop, a, min_units, info, pieces);
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

template <int DT, int KIND>
hipError_t launch_kind(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  switch (tile_pairs<KIND>(a)) {
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
