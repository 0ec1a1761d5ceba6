// Attention over the latent cache in 4 bits (gfx950): a request's pages, pages that a
// batch shares, and the keys that the top-k selected.
//
// A key is 400 bytes: 512 latent values, E2M1 codes under a power of two per 32
// dimensions, and 64 rotated ones in 16 bits.  A code times its power of two is
// exact in the queries' 16-bit type, so the keys are turned into that type on the
// way (two values an instruction) and everything behind is the 16-bit attention: the
// same work list, products, softmax and joins (attention_common.h), with the same
// results as over a cache of the values.
//
// Tiles of 32 pairs and more go through the kernel of the 16-bit cache, with keys
// that pass through registers on their way to LDS (attention_tiles.h).  For 16 pairs,
// whose time is the K stream's, there is one with eight waves of two a SIMD, each
// with 16 keys of its own at a time: they come from memory in the layout the first
// product takes them in -- a lane's 16 bytes are one block of 32 dimensions, one
// power of two -- and go from there through LDS, where the second product reads them
// transposed.  No wave waits for another before the output.  (The 32-pair form of the
// other kernel, on 16 heads: 1 request of 2048 keys 21 instead of 18 us, 16 of 32768
// keys 88 instead of 49.)
//
// Measured (MI355X; kernels, medians under the kernel trace): 64 requests of 1 .. 32768
// keys with 16 heads, capped and biased, 34 us (85 MB of keys; over 16 bits 54), one
// request of 65 keys 10.5.  Calls of the C entry points, in turn with those over 16 bits
// (in brackets): 64 requests of 32768 keys 168 us (839 MB, 5.0 TB/s, partly from the
// last-level cache; 401), 16 requests of 32768 keys with 128 heads 185 us (790 TFLOP/s;
// 186), 512 rows of 128 heads over 2048 listed keys 317 us (922 TFLOP/s; 306), a third
// of the places empty 238 (287), one request of 65 keys 10.8 (9.6).  With few heads the K
// stream bounds it, with many the MFMAs and what stands between them, as over 16 bits;
// unpacking is 0 to 5 % of the wide form's time.
#include "attention_tiles.h"

namespace pmqa {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kRow4 = IDX_LATENT_MXFP4_ROW;

// Infinities and NaN to zero.
template <int DT>
__device__ __forceinline__ s16x8 finite_or_zero(s16x8 x) {
  constexpr int kExp = DT == IDX_BF16 ? 0x7F80 : 0x7C00;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (x[j] & kExp) == kExp ? 0 : x[j];
  return x;
}

// What taking up and writing a pair tile counts for in tiles, whose time here is short.
// Calls of 16 heads with 3, as in the other kernel, 6, 8, 9 and 12: 64 requests of 1 ..
// 32768 keys 41.1 / 34.1 / 33.7 / 33.7 / 34.1 us, of 64 keys 18.7 / 13.2 / 13.4 / 12.7 /
// 13.7, of 512 keys 25.4 / 23.0 / 22.8 / 23.1 / 24.2, 256 of 1 .. 4096 keys 38.4 / 36.4 /
// 36.2 / 37.7 / 38.8, 4 of 8192 keys 20.3 / 20.0 / 20.3 / 20.2 / 20.2; selections that are
// counted (600 rows, 900 of 2048 places) 84.3 / 83.3 / 82.9 / 83.3 / 83.6, and ragged
// (200 rows, 2048 places) 62.1 / 61.2 / 62.2 / 62.2 / 62.2.
constexpr int kOwnCost = 8;
constexpr int kOwnKeys = 16;                 // keys that a wave takes at a time
constexpr int kOwnOctet = 8 * 1024;              // LDS image of 8 keys: their values alone
constexpr int kOwnImage = 2 * kOwnOctet;
constexpr int kQueryAt = kWaves * kOwnImage;     // behind the waves' images: the queries
constexpr int kOwnRing = kQueryAt + 16 * kRowDim * 2;

template <int DT, int KIND>
__global__ __launch_bounds__(kThreads, 2) void own_keys_kernel(AttentionArgs a, int min_units, JoinInfo* join,
                                                               float* pieces) {
  using E = Elem<DT>;
  constexpr int M = 16;
  constexpr int kBlocksPerTile = kTile / kOwnKeys;
  static_assert(ScanOf512<KIND>::kThreads == kThreads, "chunks of the work list");
  __shared__ __attribute__((aligned(1024))) char s_ring[kOwnRing];
  __shared__ float2 s_ml[kWaves][16];
  __shared__ PairInfo s_pair[M];
  __shared__ int64_t s_res[2];
  __shared__ int s_scan[kWaves + ScanOf512<KIND>::kChunks];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grid = gridDim.x;
  // consecutive shares on one XCD (workgroups are dealt to the 8 XCDs in turn)
  const int w = (grid & 7) ? static_cast<int>(blockIdx.x)
                           : static_cast<int>(blockIdx.x & 7) * (grid >> 3) + static_cast<int>(blockIdx.x >> 3);
  const Share share = find_share<KIND, M, kThreads, kOwnCost, true>(a, w, grid, min_units, s_scan, s_res);
  if (KIND != kShared && tid == 0) join[w].pieces = 0;
  if (share.t0 >= share.t1) return;

  const int n16 = lane & 15, g4 = lane >> 4;
  const int capacity = a.max_pages * kPage;
  const char* cache = static_cast<const char*>(a.cache);
  const char* zero = reinterpret_cast<const char*>(kZeroRow);
  const float to_log2 = a.scale * kLog2e;
  // this lane's places in its wave's image: where it writes its key, and where the
  // transposed operand is
  char* image = s_ring + wave * kOwnImage;
  const char* s_query = s_ring + kQueryAt + lane * 16;
  auto place = [](int key) { return (key >> 3) * kOwnOctet + (key & 7) * 128; };
  const int vkey = 4 * g4 + (n16 >> 2);
  const uint32_t k_at = place(n16) + (g4 >> 1) * 1024 + (((g4 & 1) * 4) ^ swz_of<true>(n16)) * 16;
  const uint32_t v_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)image)) +
                        place(vkey) + (((n16 >> 1) & 1) ^ swz_of<true>(vkey)) * 16 + (n16 & 1) * 8;

  const int items = static_cast<int>(item_count<KIND, M>(a));
  int64_t at = share.t0;
  int64_t item_at = share.item_at;
  int item = share.item;
  for (; at < share.t1 && item < items; ++item) {
    const Item it = make_item<KIND, M, kWave, true>(a, item);
    const int64_t tiles_at = item_at + (it.tiles ? share.cost : 0);
    item_at = tiles_at + it.tiles;
    const int lo = static_cast<int>(max(int64_t{0}, at - tiles_at));
    const int hi = static_cast<int>(min(static_cast<int64_t>(it.tiles), share.t1 - tiles_at));
    at = item_at;
    if (lo >= hi) continue;  // no pairs, or another workgroup's keys
    const bool whole = lo == 0 && hi == it.tiles && KIND != kShared;
    const int32_t* table = a.block_table + static_cast<int64_t>(it.request) * a.max_pages;
    const int64_t pair_base = static_cast<int64_t>(it.row0) * a.heads + it.pair0;  // over the whole batch
    const int block0 = lo * kBlocksPerTile + wave, block_end = hi * kBlocksPerTile;

    // ---- where a block's keys are
    int page_window = -1, window_page = 0;  // dense: page ids of 64 tiles, one per lane
    // sparse: the lane's key of a block (-1: none), a block ahead of its page, which is one ahead of the key's bytes
    auto token_of = [&](int block) -> int {
      const int c = block * kOwnKeys + n16;
      if (block >= block_end || c >= a.k) return -1;
      const int tok = a.indices[static_cast<int64_t>(it.row0) * a.k + c];
      return tok < capacity ? tok : -1;
    };
    auto page_of = [&](int tok) -> int { return tok >= 0 ? table[tok / kPage] : 0; };
    int token_next = -1, page_next = 0, token_after = -1;
    uint32_t live_next = 0xFFFF;  // of the block that was asked for last
    auto row_of = [&](int block) -> const char* {
      int64_t row;
      bool live;
      if constexpr (KIND == kSparse) {
        live = token_next >= 0;
        row = static_cast<int64_t>(max(0, min(page_next, a.num_pages - 1))) * kPage + (token_next & (kPage - 1));
        live_next = static_cast<uint32_t>(__ballot(live)) & 0xFFFF;
        token_next = token_after;
        page_next = page_of(token_next);
        token_after = token_of(block + 2 * kWaves);
      } else {
        const int tile = it.tile0 + block / kBlocksPerTile;
        if ((tile >> 6) != page_window) {
          page_window = tile >> 6;
          window_page = table[min(page_window * 64 + lane, a.max_pages - 1)];
        }
        const int page = max(0, min(__builtin_amdgcn_readlane(window_page, tile & 63), a.num_pages - 1));
        const int tok = it.tile0 * kTile + block * kOwnKeys + n16;
        row = static_cast<int64_t>(page) * kPage + (tok & (kPage - 1));
        live = tok >= it.min_start && tok < it.max_end;  // keys that no row of the pair tile sees are not read
      }
      return live ? cache + row * kRow4 : zero;
    };

    // ---- a block's bytes: blocks g4, 4 + g4, .. of 32 dimensions of key n16, all its
    // powers of two, and 8 of every 32 rotated dimensions
    i32x4 codes[4], powers, rotated[2];
    auto load_block = [&](int block) {
      const i32x4* p = reinterpret_cast<const i32x4*>(row_of(block));
#pragma unroll
      for (int j = 0; j < 4; ++j) codes[j] = p[4 * j + g4];
      powers = p[kPowersAt / 16];
#pragma unroll
      for (int j = 0; j < 2; ++j) rotated[j] = p[kRotatedAt / 16 + 4 * j + g4];
    };

    // ---- what the pairs need to know, their queries, the first keys
    lds_barrier();  // the previous item's epilogue has left the ring
    for (int local = tid; local < M; local += kThreads) {
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
      token_next = token_of(block0);
      token_after = token_of(block0 + kWaves);
      page_next = page_of(token_next);
    }
    if (block0 < block_end) load_block(block0);
    // the queries as the first product takes them, one operand behind the other, in
    // the order in which the keys' blocks come
    for (int c = tid; c < 16 * (kRowDim / 8); c += kThreads) {
      const int pair = c / (kRowDim / 8), piece = c % (kRowDim / 8);  // 8 dimensions
      const char* from = static_cast<const char*>(a.q) + (pair_base + pair) * (kRowDim * 2);
      const i32x4 x = *reinterpret_cast<const i32x4*>((pair < it.pairs ? from : zero) + piece * 16);
      const int block = piece >> 2;
      const int step = piece < 64 ? (block >> 2) * 4 + (piece & 3) : 16 + ((piece - 64) >> 2);
      const int group = piece < 64 ? block & 3 : piece & 3;
      *reinterpret_cast<i32x4*>(s_ring + kQueryAt + step * 1024 + (group * 16 + pair) * 16) = x;
    }
    lds_barrier();

    // accumulators: dimensions on the rows, pairs on the columns
    f32x4 acc[kDimTiles];
#pragma unroll
    for (int d = 0; d < kDimTiles; ++d) acc[d] = f32x4{0, 0, 0, 0};
    float m = kMInit, l = 0.0f, l_kept = 0.0f;  // l_kept: of the rounded weights

    for (int block = block0; block < block_end; block += kWaves) {
      const int block_key = block * kOwnKeys;         // of the item's list
      const int first = it.tile0 * kTile + block_key;  // dense: its first key
      bool mixed = false, masked = false;  // some key that was read is hidden from some row; some key is
      if constexpr (KIND != kSparse) {
        mixed = max(first, it.min_start) < it.max_start || min(first + kOwnKeys, it.max_end) > it.min_end;
        masked = first < it.max_start || first + kOwnKeys > it.min_end;
      }
      // ---- S = K Q^T
      f32x4 s[2] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float power = __uint_as_float((static_cast<uint32_t>(powers[j]) >> (8 * g4) & 255u) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const s16x8 x = dequant8<DT>(static_cast<uint32_t>(codes[j][i]), power);
          s[i & 1] = E::mfma32(x, *reinterpret_cast<const s16x8*>(s_query + (4 * j + i) * 1024), s[i & 1]);
          *reinterpret_cast<s16x8*>(image + (k_at ^ (i * 16)) + j * 2048) = x;
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        s[j] = E::mfma32(__builtin_bit_cast(s16x8, rotated[j]),
                         *reinterpret_cast<const s16x8*>(s_query + (16 + j) * 1024), s[j]);
      if (mixed) {  // (a row that sees a NaN has it from the score; others must not meet it)
#pragma unroll 1
        for (int i = 0; i < kOwnImage / 1024; ++i) {
          s16x8* v = reinterpret_cast<s16x8*>(image + i * 1024) + lane;
          *v = finite_or_zero<DT>(*v);
        }
      }
      const uint32_t live = live_next;  // sparse: bits of the block's keys
      if (block + kWaves < block_end) load_block(block + kWaves);
      float z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = s[0][i] + s[1][i];

      // ---- scores in powers of two, masked keys at -inf.  Score i is key
      // 4 g4 + i of the block.
      if (a.softcap > 0.0f) {
        const float in = a.scale / a.softcap, cap = a.softcap * kLog2e;
        // (z - z: 0, and NaN where z is not finite, which tanh would hide)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __builtin_fmaf(cap, tanh_f32(z[i] * in), z[i] - z[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] *= to_log2;
      }
      if (a.slopes) {
        const PairInfo info = s_pair[n16];
        const int32_t* list = KIND == kSparse ? a.indices + static_cast<int64_t>(it.row0) * a.k : nullptr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = block_key + 4 * g4 + i;
          const int tok = KIND == kSparse ? list[min(c, a.k - 1)] : it.tile0 * kTile + c;
          z[i] -= info.slope * fabsf(static_cast<float>(info.pos - tok));
        }
      }
      if constexpr (KIND == kSparse) {
        if (live != 0xFFFF) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = live >> (4 * g4 + i) & 1 ? z[i] : -__builtin_inff();
        }
      } else if (masked) {
        const PairInfo info = s_pair[n16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = first + 4 * g4 + i;
          z[i] = tok >= info.start && tok < info.end ? z[i] : -__builtin_inff();
        }
      }

      // ---- running maximum: raised where a score passes it by kRaise
      const float mx = pair_max<false>(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]))) - E::kShift;
      const float raised = mx > m + E::kRaise ? mx : m;
      const bool any_raised = block > block0 && __ballot(raised != m) != 0;  // nothing to rescale in the first block
      const float by = __builtin_amdgcn_exp2f(m - raised);
      m = raised;
      if (any_raised) {
        l *= by;
        l_kept *= by;
#pragma unroll
        for (int d = 0; d < kDimTiles; ++d) acc[d] *= by;
      }
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = weight(z[i], m);
      l += (e[0] + e[1]) + (e[2] + e[3]);
      const int2 both = make_int2(E::round2(e[0], e[1]), E::round2(e[2], e[3]));
      l_kept += E::add2(both.x, E::add2(both.y, 0.0f));
      const s16x4 p = __builtin_bit_cast(s16x4, both);
      // ---- O^T += V^T P^T
      // (the image is this wave's alone: its LDS accesses stay in order)
      __asm__ volatile("" ::: "memory");
#pragma unroll
      for (int d = 0; d < kDimTiles; ++d)
        acc[d] = E::mfma16(lds_read_tr((v_at ^ ((d & 3) * 32)) + (d >> 2) * 1024), p, acc[d]);
      __asm__ volatile("" ::: "memory");
    }

    // ---- the waves' parts of each pair become one, through LDS, and leave as
    // whole rows
    float factor = 1.0f;  // of this lane's part of its pair
    {
      const float sum = pair_sum<false>(l), kept = pair_sum<false>(l_kept);
      if (lane < 16) s_ml[wave][lane] = make_float2(m, sum);
      if (kept > 0.0f) factor = sum / kept;  // (no key, or NaN, otherwise)
    }
    lds_barrier();  // every wave has left the ring, and s_ml is complete
    float* piece = nullptr;
    if (!whole) {
      const int64_t id = KIND == kShared ? static_cast<int64_t>(w) + item : (lo == 0 ? 2 * w + 1 : 2 * w);
      piece = pieces + id * piece_floats(M);
    }
    {
      float top = kMInit, sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) top = fmaxf(top, s_ml[k][n16].x);
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        const float2 ml = s_ml[k][n16];
        sum += ml.y * __builtin_amdgcn_exp2f(ml.x - top);
      }
      factor *= __builtin_amdgcn_exp2f(m - top);
      if (whole) factor = sum == 0.0f ? 0.0f : factor / sum;
      if (tid < it.pairs) {
        if (!whole) reinterpret_cast<float2*>(piece + M * kValDim)[tid] = make_float2(top, sum);
        else if (a.lse) a.lse[pair_base + tid] = (top + __log2f(sum)) * kLn2;
      }
    }
    // 128 rows of accumulators, half of their dimensions at a time; the pad of 4
    // floats spreads the pairs over all banks
    constexpr int kChunkDims = kValDim / 2, kStride = kChunkDims + 4;
    static_assert(kWaves * 16 * kStride * 4 <= kOwnRing, "the output's exchange fits the ring");
    float* s_o = reinterpret_cast<float*>(s_ring);
    float* mine = s_o + (wave * 16 + n16) * kStride;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (c) lds_barrier();  // stores to memory go on meanwhile
#pragma unroll
      for (int d = 0; d < 16; ++d) *reinterpret_cast<f32x4*>(mine + d * 16 + 4 * g4) = acc[16 * c + d] * factor;
      lds_barrier();
      constexpr int kPerRow = kChunkDims / 4, kRows = kThreads / kPerRow;  // rows at a time
      const int dim = tid % kPerRow * 4;
#pragma unroll 4
      for (int local = tid / kPerRow; local < it.pairs; local += kRows) {
        const float* parts = s_o + local * kStride + dim;
        f32x4 o = *reinterpret_cast<const f32x4*>(parts);
#pragma unroll
        for (int k = 1; k < kWaves; ++k) o += *reinterpret_cast<const f32x4*>(parts + k * 16 * kStride);
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

// Microseconds of a workgroup per 64-key tile, and of a call, over pages and over
// selections (whose keys each pair tile gathers for itself), from every size forced on
// selections of 512 and 2048 keys for 1 .. 256 rows of 32, 64 and 128 heads, and on 1
// .. 64 requests of 512 .. 32768 keys with 16 .. 128 heads (the entries for 16 pairs with
// an item's cost of 3, before it was 8).  Between them (16 / 32 / 64 / 128 pairs, the
// cost 8): 64 rows of 32 heads over 2048 keys 43 / 42 / 50 / 63 us, 256 rows of 64 heads
// 177 / 160 / 119 / 161, of 128 heads 338 / 310 / 230 / 169; 16 requests of 32768 keys
// with 32 heads 79 / 90 / 120 / 160, with 64 heads 143 / 154 / 124 / 171, with 128 heads
// 262 / 291 / 221 / 190.
constexpr double kPerTile[2][4] = {{0.95, 2.1, 3.1, 4.8}, {1.35, 2.4, 3.45, 5.0}};
constexpr double kFixed[2][4] = {{19, 22, 27, 47}, {17, 18, 24, 45}};

// Tiles of a row's list up to the last one that holds a key (at least one): a wave per
// row, from the end.
__global__ __launch_bounds__(256) void count_tiles_kernel(const int32_t* __restrict__ indices, int rows, int k,
                                                          int capacity, uint8_t* __restrict__ tiles) {
  const int row = blockIdx.x * 4 + static_cast<int>(threadIdx.x) / kWave, lane = lane_id();
  if (row >= rows) return;
  const int32_t* list = indices + static_cast<int64_t>(row) * k;
  constexpr int kAt = 16;  // loads in flight
  int last = 0;
  for (int end = k; end > 0 && last == 0; end -= kAt * kWave) {
    int tok[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int c = end - (i + 1) * kWave + lane;
      tok[i] = c >= 0 ? list[c] : -1;
    }
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const uint64_t live = __ballot(tok[i] >= 0 && tok[i] < capacity);
      if (live && last == 0) last = end - i * kWave - static_cast<int>(__builtin_clzll(live));
    }
  }
  if (lane == 0) tiles[row] = static_cast<uint8_t>(max(1, (last + kTile - 1) / kTile));
}

// Selections of rows that see fewer keys than the list has places end in padding: with
// enough tiles for a workgroup, those behind a row's last key are counted out before
// the list is shared.  (512 rows of 128 heads, 2048 places, a third of the tiles empty:
// 239 us, with all of them 327; none empty: 317 and 312.  1024 rows of 16 heads: 139 and
// 177; 300 of 704 places, 200 keys: 35 and 43, none empty: 47 and 43.)
constexpr int kCountFrom = 4 * kMaxGrid;

template <int DT, int KIND, int M>
hipError_t launch(AttentionArgs a, hipStream_t stream, LaunchEvents ev) {
  if constexpr (KIND == kSparse) {
    const int64_t tiles = (a.k + kTile - 1) / kTile, items = item_count<KIND, M>(a);
    if (tiles > 1 && items * tiles >= kCountFrom && (a.cu_q || items > kMaxGrid / 2)) {
      launch_kernel(count_tiles_kernel, dim3((a.rows + 3) / 4), dim3(256), stream, ev.start, nullptr, a.indices, a.rows,
                    a.k, a.max_pages * kPage, row_tiles(a));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      a.counted = 1;
      ev.start = nullptr;
    }
  }
  if constexpr (M == 16) return launch_joined<DT, KIND, M, kOwnCost>(own_keys_kernel<DT, KIND>, kThreads, a, stream, ev);
  else return launch_joined<DT, KIND, M>(attention_kernel<DT, KIND, M, true>, kAttnThreads, a, stream, ev);
}

template <int DT, int KIND>
hipError_t launch_kind(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  switch (tile_pairs<KIND>(a, kPerTile[KIND == kSparse], kFixed[KIND == kSparse], ScanOf512<KIND>::kItems)) {
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

hipError_t launch_paged_attention_mxfp4(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kDense>(a, stream, ev);
}
hipError_t launch_shared_prefix_attention_mxfp4(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kShared>(a, stream, ev);
}
hipError_t launch_sparse_attention_mxfp4(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kSparse>(a, stream, ev);
}

}  // namespace pmqa
