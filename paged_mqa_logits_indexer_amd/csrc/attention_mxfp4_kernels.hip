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
// Eight waves of 16 pairs each, 128 accumulators a wave, two waves a SIMD.
//   16 pairs    each wave has 16 keys of its own at a time.  They come from memory in
//               the layout the first product takes them in -- a lane's 16 bytes are
//               one block of 32 dimensions, one power of two -- and go from there
//               through LDS, where the second product reads them transposed.  No wave
//               waits for another before the output.
//   more        the waves share 64 keys: each turns 8 of them into the LDS image while
//               all work on the 64 before.
#include "attention_common.h"

namespace pmqa {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kRow4 = IDX_LATENT_MXFP4_ROW;
constexpr int kScaleAt = kValDim / 2;                 // 16 power bytes
constexpr int kRotatedAt = kScaleAt + kValDim / 32;   // 64 values of 16 bits

// Eight codes under one power of two (as a float32 whose exponent is the E8M0 byte;
// 255, an exponent of ones, gives NaN), exact: beyond the type's range they become
// infinities, below it they are rounded.
template <int DT>
__device__ __forceinline__ s16x8 dequant8(uint32_t codes, float power) {
  i32x4 x;
  if constexpr (DT == IDX_BF16) {
    x[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, power, 0));
    x[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, power, 1));
    x[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, power, 2));
    x[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, power, 3));
  } else {
    x[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, power, 0));
    x[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, power, 1));
    x[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, power, 2));
    x[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, power, 3));
  }
  return __builtin_bit_cast(s16x8, x);
}

// Infinities and NaN to zero.
template <int DT>
__device__ __forceinline__ s16x8 finite_or_zero(s16x8 x) {
  constexpr int kExp = DT == IDX_BF16 ? 0x7F80 : 0x7C00;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (x[j] & kExp) == kExp ? 0 : x[j];
  return x;
}

template <int M>
struct Form {
  static constexpr bool kOwn = M == 16;             // every wave has keys of its own
  static constexpr int kGroups = M / 16;            // waves that cover the pairs
  static constexpr int kStreams = kWaves / kGroups;
  static constexpr int kUnitKeys = kOwn ? 16 : 64;  // keys of a unit: a wave's block, or a step of all
  static constexpr int kBlocks = kOwn ? 1 : 4 / kStreams;           // 16-key blocks of a unit per wave
  static constexpr int kOctBytes = kOwn ? 8 * 1024 : 9 * 1024;  // 8 keys in LDS: their values, or all of them
  static constexpr int kSlotBytes = kUnitKeys / 8 * kOctBytes;
  static constexpr int kQueryBytes = kOwn ? 16 * kRowDim * 2 : 0;
  static constexpr int kRingBytes = (kOwn ? kWaves : 2) * kSlotBytes + kQueryBytes;
};

template <int DT, int KIND, int M>
__global__ __launch_bounds__(kThreads, 2) void attention_mxfp4_kernel(AttentionArgs a, int min_units, JoinInfo* join,
                                                                      float* pieces) {
  using E = Elem<DT>;
  using F = Form<M>;
  constexpr int ST = F::kBlocks;
  constexpr int kScores = 4 * ST;
  constexpr int kUnitsPerTile = kTile / F::kUnitKeys;
  constexpr int kUnitStep = F::kOwn ? kWaves : 1;
  // (work lists: at most 2^16 rows of 8 pair tiles and a request's more, twice that with a shared prefix)
  constexpr int kScan = kWaves + (KIND == kShared ? 2080 : 1056);
  __shared__ __attribute__((aligned(1024))) char s_ring[F::kRingBytes];
  __shared__ float2 s_ml[kWaves][16];
  __shared__ PairInfo s_pair[M];
  __shared__ int64_t s_res[2];
  __shared__ uint64_t s_live[2];  // sparse, shared keys: bits of the keys that are there
  __shared__ int s_scan[kScan];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grid = gridDim.x;
  // consecutive shares on one XCD (workgroups are dealt to the 8 XCDs in turn)
  const int w = (grid & 7) ? static_cast<int>(blockIdx.x)
                           : static_cast<int>(blockIdx.x & 7) * (grid >> 3) + static_cast<int>(blockIdx.x >> 3);
  const Share share = find_share<KIND, M, kThreads>(a, w, grid, min_units, s_scan, s_res);
  if (KIND != kShared && tid == 0) join[w].pieces = 0;
  if (share.t0 >= share.t1) return;

  const int pg = wave / F::kStreams, ts = wave % F::kStreams;
  const int n16 = lane & 15, g4 = lane >> 4;
  const int load_key = F::kOwn ? n16 : wave * 8 + (lane >> 3);  // the key of a unit that this lane loads
  const int c8 = lane & 7;
  const int capacity = a.max_pages * kPage;
  const char* cache = static_cast<const char*>(a.cache);
  const char* zero = reinterpret_cast<const char*>(kZeroRow);
  const float to_log2 = a.scale * kLog2e;
  const uint32_t ring = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)s_ring));
  auto key_offset = [](int key) { return (key >> 3) * F::kOctBytes + (key & 7) * 128; };
  const int vkey = 4 * g4 + (n16 >> 2);
  const uint32_t k_at = key_offset(n16) + (g4 ^ swz(n16)) * 16;
  const uint32_t v_at = key_offset(vkey) + (((n16 >> 1) & 1) ^ swz(vkey)) * 16 + (n16 & 1) * 8;

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
    const int64_t pair_base = static_cast<int64_t>(it.row0) * a.heads + it.pair0;  // over the whole batch
    const int unit0 = lo * kUnitsPerTile + (F::kOwn ? wave : 0), unit_end = hi * kUnitsPerTile;

    // ---- where a unit's keys are
    int page_window = -1, window_page = 0;  // dense: page ids of 64 tiles, one per lane
    // sparse: the lane's key of the unit (-1: none), two loads ahead of its page
    auto token_of = [&](int unit) -> int {
      const int c = unit * F::kUnitKeys + load_key;
      if (unit >= unit_end || c >= a.k) return -1;
      const int tok = a.indices[static_cast<int64_t>(it.row0) * a.k + c];
      return tok < capacity ? tok : -1;
    };
    auto page_of = [&](int tok) -> int { return tok >= 0 ? table[tok / kPage] : 0; };
    int token_next = -1, page_next = 0, token_after = -1;
    uint64_t live_next = ~0ull;  // of the unit that was asked for last, by lane
    auto row_of = [&](int unit) -> const char* {
      int64_t row;
      bool live;
      if constexpr (KIND == kSparse) {
        live = token_next >= 0;
        row = static_cast<int64_t>(max(0, min(page_next, a.num_pages - 1))) * kPage + (token_next & (kPage - 1));
        live_next = __ballot(live);
        token_next = token_after;
        page_next = page_of(token_next);
        token_after = token_of(unit + 2 * kUnitStep);
      } else {
        const int tile = it.tile0 + unit / kUnitsPerTile;
        if ((tile >> 6) != page_window) {
          page_window = tile >> 6;
          window_page = table[min(page_window * 64 + lane, a.max_pages - 1)];
        }
        const int page = max(0, min(__builtin_amdgcn_readlane(window_page, tile & 63), a.num_pages - 1));
        const int tok = it.tile0 * kTile + unit * F::kUnitKeys + load_key;
        row = static_cast<int64_t>(page) * kPage + (tok & (kPage - 1));
        live = tok >= it.min_start && tok < it.max_end;  // keys that no row of the pair tile sees are not read
      }
      return live ? cache + row * kRow4 : zero;
    };

    // ---- a unit's bytes
    i32x4 codes[F::kOwn ? 4 : 2], rotated[F::kOwn ? 2 : 1], powers;
    auto load_unit = [&](int unit) {
      const char* row = row_of(unit);
      const i32x4* p = reinterpret_cast<const i32x4*>(row);
      if constexpr (F::kOwn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) codes[j] = p[4 * j + g4];
        powers = p[kScaleAt / 16];
#pragma unroll
        for (int j = 0; j < 2; ++j) rotated[j] = p[kRotatedAt / 16 + 4 * j + g4];
      } else {
        codes[0] = p[c8];
        codes[1] = p[8 + c8];
        powers[0] = reinterpret_cast<const uint8_t*>(row)[kScaleAt + c8];
        powers[1] = reinterpret_cast<const uint8_t*>(row)[kScaleAt + 8 + c8];
        rotated[0] = p[kRotatedAt / 16 + c8];
      }
    };
    auto store_unit = [&](int slot) {  // shared keys: 8 of them into the image
      if constexpr (!F::kOwn) {
        char* to = s_ring + slot * F::kSlotBytes + key_offset(load_key);
        const int sw = swz(lane >> 3 | (wave & 1) << 3);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float power = __uint_as_float(static_cast<uint32_t>(powers[h]) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<s16x8*>(to + (4 * h + (c8 >> 1)) * 1024 + ((((c8 & 1) * 4 + i) ^ sw) * 16)) =
                dequant8<DT>(static_cast<uint32_t>(codes[h][i]), power);
        }
        *reinterpret_cast<i32x4*>(to + 8 * 1024 + (c8 ^ sw) * 16) = rotated[0];
        if constexpr (KIND == kSparse) {
          uint32_t bits = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) bits |= static_cast<uint32_t>(live_next >> (8 * i) & 1) << i;
          if (lane == 0) reinterpret_cast<uint8_t*>(s_live + slot)[wave] = static_cast<uint8_t>(bits);
        }
      }
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
      token_next = token_of(unit0);
      token_after = token_of(unit0 + kUnitStep);
      page_next = page_of(token_next);
    }
    if (unit0 < unit_end) load_unit(unit0);
    // own keys: the queries as the first product takes them, one operand behind the
    // other, in the order in which the keys' blocks come; shared keys: in registers
    const char* queries = static_cast<const char*>(a.q);
    char* s_query = s_ring + (F::kOwn ? kWaves : 2) * F::kSlotBytes;
    s16x8 q[F::kOwn ? 1 : 18];
    if constexpr (F::kOwn) {
      for (int c = tid; c < 16 * (kRowDim / 8); c += kThreads) {
        const int pair = c / (kRowDim / 8), piece = c % (kRowDim / 8);  // 8 dimensions
        const i32x4 x = pair < it.pairs ? *reinterpret_cast<const i32x4*>(queries + (pair_base + pair) * (kRowDim * 2) + piece * 16)
                                        : i32x4{0, 0, 0, 0};
        const int block = piece >> 2;
        const int step = piece < 64 ? (block >> 2) * 4 + (piece & 3) : 16 + ((piece - 64) >> 2);
        const int group = piece < 64 ? block & 3 : piece & 3;
        *reinterpret_cast<i32x4*>(s_query + step * 1024 + (group * 16 + pair) * 16) = x;
      }
    } else {
      const int pair = pg * 16 + n16;
      const char* from = pair < it.pairs ? queries + (pair_base + pair) * (kRowDim * 2) : zero;
#pragma unroll
      for (int ks = 0; ks < 18; ++ks) q[ks] = *reinterpret_cast<const s16x8*>(from + ks * 64 + g4 * 16);
      store_unit(0);
      if (unit0 + 1 < unit_end) load_unit(unit0 + 1);
    }
    lds_barrier();

    // accumulators: dimensions on the rows, pairs on the columns
    f32x4 acc[kDimTiles];
#pragma unroll
    for (int d = 0; d < kDimTiles; ++d) acc[d] = f32x4{0, 0, 0, 0};
    float m = kMInit, l = 0.0f, l_kept = 0.0f;  // l_kept: of the rounded weights

    for (int unit = unit0; unit < unit_end; unit += kUnitStep) {
      const int slot = F::kOwn ? wave : (unit - unit0) & 1;
      const uint32_t base = ring + slot * F::kSlotBytes + ts * (F::kOwn ? 0 : ST * 2 * F::kOctBytes);
      const int unit_key = unit * F::kUnitKeys;           // of the item's list
      const int first = it.tile0 * kTile + unit_key;      // dense: its first key
      bool mixed = false, masked = false;  // some key that was read is hidden from some row; some key is
      if constexpr (KIND != kSparse) {
        mixed = max(first, it.min_start) < it.max_start || min(first + F::kUnitKeys, it.max_end) > it.min_end;
        masked = first < it.max_start || first + F::kUnitKeys > it.min_end;
      }
      uint64_t live = ~0ull;  // sparse: bits of the unit's keys
      float z[kScores];
      // ---- S = K Q^T
      if constexpr (F::kOwn) {
        f32x4 s[2] = {};
        const uint32_t to = key_offset(n16) + (g4 >> 1) * 1024 + (((g4 & 1) * 4) ^ swz(n16)) * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float power = __uint_as_float((static_cast<uint32_t>(powers[j]) >> (8 * g4) & 255u) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const s16x8 x = dequant8<DT>(static_cast<uint32_t>(codes[j][i]), power);
            const s16x8 query = *reinterpret_cast<const s16x8*>(s_query + (4 * j + i) * 1024 + lane * 16);
            s[i & 1] = E::mfma32(x, query, s[i & 1]);
            // (a row that sees a NaN has it from the score; others must not meet it)
            *reinterpret_cast<s16x8*>(s_ring + slot * F::kSlotBytes + (to ^ (i * 16)) + j * 2048) =
                mixed ? finite_or_zero<DT>(x) : x;
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          s[j] = E::mfma32(__builtin_bit_cast(s16x8, rotated[j]),
                           *reinterpret_cast<const s16x8*>(s_query + (16 + j) * 1024 + lane * 16), s[j]);
        if constexpr (KIND == kSparse) live = live_next;
        if (unit + kUnitStep < unit_end) load_unit(unit + kUnitStep);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = s[0][i] + s[1][i];
      } else {
        // the unit's keys are in their slot, and every wave has left the other one
        lds_barrier();
        if (unit + 1 < unit_end) {
          store_unit(slot ^ 1);
          if (unit + 2 < unit_end) load_unit(unit + 2);
        }
        if constexpr (KIND == kSparse) live = s_live[slot];
        f32x4 s[ST] = {};
#pragma unroll
        for (int ks = 0; ks < 18; ++ks)
#pragma unroll
          for (int st = 0; st < ST; ++st)
            s[st] = E::mfma32(lds_read(base + (k_at ^ ((ks & 1) * 64)) + (ks >> 1) * 1024 + st * 2 * F::kOctBytes),
                              q[ks], s[st]);
#pragma unroll
        for (int i = 0; i < kScores; ++i) z[i] = s[i / 4][i % 4];
      }

      // ---- scores in powers of two, masked keys at -inf.  Score i is key key_of(i)
      // of the unit.
      auto key_of = [&](int i) { return (F::kOwn ? 0 : ts * ST * 16) + 16 * (i >> 2) + 4 * g4 + (i & 3); };
      if (a.softcap > 0.0f) {
        const float in = a.scale / a.softcap, cap = a.softcap * kLog2e;
        // (z - z: 0, and NaN where z is not finite, which tanh would hide)
#pragma unroll
        for (int i = 0; i < kScores; ++i) z[i] = __builtin_fmaf(cap, tanh_f32(z[i] * in), z[i] - z[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kScores; ++i) z[i] *= to_log2;
      }
      if (a.slopes) {
        const PairInfo info = s_pair[pg * 16 + n16];
        const int32_t* list = KIND == kSparse ? a.indices + static_cast<int64_t>(it.row0) * a.k : nullptr;
#pragma unroll
        for (int i = 0; i < kScores; ++i) {
          const int c = unit_key + key_of(i);
          const int tok = KIND == kSparse ? list[min(c, a.k - 1)] : it.tile0 * kTile + c;
          z[i] -= info.slope * fabsf(static_cast<float>(info.pos - tok));
        }
      }
      if constexpr (KIND == kSparse) {
        constexpr uint64_t kAll = F::kOwn ? 0xFFFFull : ~0ull;
        if ((live & kAll) != kAll) {
#pragma unroll
          for (int i = 0; i < kScores; ++i) z[i] = live >> key_of(i) & 1 ? z[i] : -__builtin_inff();
        }
      } else if (masked) {
        const PairInfo info = s_pair[pg * 16 + n16];
#pragma unroll
        for (int i = 0; i < kScores; ++i) {
          const int tok = first + key_of(i);
          z[i] = tok >= info.start && tok < info.end ? z[i] : -__builtin_inff();
        }
      }
      if constexpr (KIND != kSparse && !F::kOwn) {
        if (mixed) {  // (the same for all waves)
          lds_barrier();
          for (int i = tid; i < F::kSlotBytes / 16; i += kThreads) {
            s16x8* v = reinterpret_cast<s16x8*>(s_ring + slot * F::kSlotBytes) + i;
            *v = finite_or_zero<DT>(*v);
          }
          lds_barrier();
        }
      }

      // ---- running maximum: raised where a score passes it by kRaise
      float mx = z[0];
#pragma unroll
      for (int i = 1; i < kScores; ++i) mx = fmaxf(mx, z[i]);
      mx = pair_max<false>(mx) - E::kShift;
      const float raised = mx > m + E::kRaise ? mx : m;
      const bool any_raised = unit > unit0 && __ballot(raised != m) != 0;  // nothing to rescale in the first unit
      const float by = __builtin_amdgcn_exp2f(m - raised);
      m = raised;
      if (any_raised) {
        l *= by;
        l_kept *= by;
#pragma unroll
        for (int d = 0; d < kDimTiles; ++d) acc[d] *= by;
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
      __asm__ volatile("" ::: "memory");
#pragma unroll
      for (int d = 0; d < kDimTiles; ++d) {
        const uint32_t from = base + (v_at ^ ((d & 3) * 32)) + (d >> 2) * 1024;
        if constexpr (ST == 1) {
          acc[d] = E::mfma16(lds_read_tr(from), p[0], acc[d]);
        } else {
#pragma unroll
          for (int st = 0; st < ST; st += 2)
            acc[d] = E::mfma32(__builtin_shufflevector(lds_read_tr(from + st * 2 * F::kOctBytes),
                                                       lds_read_tr(from + (st + 1) * 2 * F::kOctBytes), 0, 1, 2, 3, 4,
                                                       5, 6, 7),
                               __builtin_shufflevector(p[st], p[st + 1], 0, 1, 2, 3, 4, 5, 6, 7), acc[d]);
        }
      }
      __asm__ volatile("" ::: "memory");
    }

    // ---- the streams' parts of each pair become one, through LDS, and leave as
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
      const int first = pg * F::kStreams;
      float top = kMInit, sum = 0.0f;
#pragma unroll
      for (int k = 0; k < F::kStreams; ++k) top = fmaxf(top, s_ml[first + k][n16].x);
#pragma unroll
      for (int k = 0; k < F::kStreams; ++k) {
        const float2 ml = s_ml[first + k][n16];
        sum += ml.y * __builtin_amdgcn_exp2f(ml.x - top);
      }
      factor *= __builtin_amdgcn_exp2f(m - top);
      const int local = pg * 16 + n16;
      if (whole) {
        factor = sum == 0.0f ? 0.0f : factor / sum;
        if (a.lse && ts == 0 && lane < 16 && local < it.pairs)
          a.lse[pair_base + local] = (top + __log2f(sum)) * kLn2;
      } else if (ts == 0 && lane < 16 && local < it.pairs) {
        reinterpret_cast<float2*>(piece + M * kValDim)[local] = make_float2(top, sum);
      }
    }
    // 128 rows of accumulators, half of their dimensions at a time; the pad of 4
    // floats spreads the pairs over all banks
    constexpr int kChunkDims = kValDim / 2, kStride = kChunkDims + 4;
    static_assert(kWaves * 16 * kStride * 4 <= F::kRingBytes, "the output's exchange fits the ring");
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
        const float* parts = s_o + (local / 16 * F::kStreams * 16 + local % 16) * kStride + dim;
        f32x4 o = *reinterpret_cast<const f32x4*>(parts);
#pragma unroll
        for (int k = 1; k < F::kStreams; ++k) o += *reinterpret_cast<const f32x4*>(parts + k * 16 * kStride);
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

// Microseconds of a workgroup per 64-key tile, and of a call.
constexpr double kPerTile[] = {1.5, 1.8, 2.5, 4.0}, kFixed[] = {15, 18, 24, 35};

template <int DT, int KIND>
hipError_t launch_kind(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  switch (tile_pairs<KIND>(a, kPerTile, kFixed)) {
    case 16: return launch_joined<DT, KIND, 16>(attention_mxfp4_kernel<DT, KIND, 16>, kThreads, a, stream, ev);
    case 32: return launch_joined<DT, KIND, 32>(attention_mxfp4_kernel<DT, KIND, 32>, kThreads, a, stream, ev);
    case 64: return launch_joined<DT, KIND, 64>(attention_mxfp4_kernel<DT, KIND, 64>, kThreads, a, stream, ev);
    default: return launch_joined<DT, KIND, 128>(attention_mxfp4_kernel<DT, KIND, 128>, kThreads, a, stream, ev);
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
