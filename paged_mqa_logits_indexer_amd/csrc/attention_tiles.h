// The attention kernel whose pair tiles share their keys between the waves of a
// workgroup, over 16-bit rows (MX false) and over 4-bit ones.
#pragma once

#include "attention_common.h"

namespace pmqa {
namespace {

constexpr int kRowBytes = kRowDim * 2;             // 1152
constexpr int kKSteps = kRowDim / 32;              // 18 MFMA steps of S
constexpr int kOctBytes = 8 * kRowBytes;           // 8 keys in LDS: 9216
constexpr int kBlkBytes = 2 * kOctBytes;           // 16 keys
constexpr int kRingBytes = 2 * kTile * kRowBytes;  // 147456: 128 keys in all slots together
constexpr int kWindow = 2048;                      // sparse: keys whose cache rows are resolved at a time
constexpr int kAttnThreads = 256;

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
__device__ __forceinline__ int key_offset(int key) { return (key >> 3) * kOctBytes + (key & 7) * 128; }

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

// Eight E2M1 codes under one power of two (as a float32 whose exponent is the E8M0
// byte; 255, an exponent of ones, gives NaN), exact: beyond the type's range they
// become infinities, below it they are rounded.
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

// MX: what a lane holds of a 4-bit key (lane % 8 of an octet) between memory and
// LDS: two blocks of 32 codes, their powers of two, and 8 of the rotated part.
constexpr int kPowersAt = kValDim / 2;               // 16 power bytes behind the codes
constexpr int kRotatedAt = kPowersAt + kValDim / 32;
struct Packed {
  i32x4 codes[2], rotated;
  uint32_t power[2];
};
__device__ __forceinline__ uint32_t lds_read_byte(uint32_t at) {
  return *reinterpret_cast<__attribute__((address_space(3))) const uint8_t*>(at);
}
template <int LEFT>
__device__ __forceinline__ void wait_loads() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LEFT & 15) | ((LEFT >> 4) << 14));  // vmcnt(LEFT) alone
  __asm__ volatile("" ::: "memory");
}
constexpr int kPackedParts = 5;  // loads of it
// MX, wide: the keys come by direct loads, three steps ahead, and wait in LDS until
// they are unpacked; the image then needs three slots instead of four.  A wave's 8
// keys are four pieces of 128 bytes of each: two of codes, one that begins with the
// powers, and the rotated part (bytes 272 .. 383 are loaded twice: four whole
// instructions instead of three and an eighth of one).
constexpr int kStageAt = 3 * 32 * kRowBytes, kStageBytes = 4 * 1024, kStageLoads = 4;
static_assert(kStageAt + 4 * 2 * kStageBytes <= kRingBytes, "two steps of packed keys behind the image");
template <int J>
__device__ __forceinline__ void load_stage(const char* at, uint32_t lds) {
  constexpr int kFrom = J < 3 ? J * 128 : kRotatedAt;
  __asm__ volatile(
      "s_add_u32 m0, %0, %2\n"
      "s_nop 0\n"
      "global_load_lds_dwordx4 %1, off offset:%3"
      :
      : "s"(lds), "v"(at), "n"(J * 1024 - kFrom), "n"(kFrom)
      : "memory", "m0", "scc");
}
__device__ __forceinline__ void load_packed(Packed& x, const char* row, int part) {
  const int c8 = lane_id() >> 3;
  switch (part) {
    case 0: x.codes[0] = *reinterpret_cast<const i32x4*>(row + c8 * 16); break;
    case 1: x.power[0] = static_cast<uint8_t>(row[kPowersAt + c8]); break;
    case 2: x.codes[1] = *reinterpret_cast<const i32x4*>(row + 128 + c8 * 16); break;
    case 3: x.power[1] = static_cast<uint8_t>(row[kPowersAt + 8 + c8]); break;
    case 4: x.rotated = *reinterpret_cast<const i32x4*>(row + kRotatedAt + c8 * 16); break;
  }
}

template <int DT, int KIND, int M, bool MX>
__global__ __launch_bounds__(kAttnThreads, 1) void attention_kernel(AttentionArgs a, int min_units, JoinInfo* join,
                                                                    float* pieces) {
  using E = Elem<DT>;
  using S = Shape<M>;
  constexpr int kStepsPerTile = kTile / S::kKeys;
  constexpr int ST = S::kBlocks;
  constexpr bool kStaged = MX && S::kWide;
  constexpr int kAhead = kStaged ? 3 : S::kDistance;  // steps that are loaded ahead
  __shared__ __attribute__((aligned(1024))) char s_keys[kRingBytes];
  __shared__ int s_rows[KIND == kSparse ? kWindow : 1];       // sparse: cache row of each listed key, -1: none
  __shared__ uint32_t s_live[S::kSlots][4];                   // sparse: bits of the keys that are there
  __shared__ float2 s_ml[4][S::kWavePairs];
  __shared__ PairInfo s_pair[S::kWavePairs * S::kGroups];
  __shared__ int64_t s_res[2];
  static_assert(ScanOf256<KIND>::kThreads == kAttnThreads, "chunks of the work list");
  __shared__ int s_scan[kAttnThreads / kWave + ScanOf256<KIND>::kChunks];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grid = gridDim.x;
  // consecutive shares on one XCD (workgroups are dealt to the 8 XCDs in turn)
  const int w = (grid & 7) ? static_cast<int>(blockIdx.x)
                           : static_cast<int>(blockIdx.x & 7) * (grid >> 3) + static_cast<int>(blockIdx.x >> 3);
  const Share share = find_share<KIND, M, kAttnThreads, kItemCost<M>, MX>(a, w, grid, min_units, s_scan, s_res);
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
    k_at = key_offset(key) + (half ^ swz_of<MX>(key)) * 16;
    v_at = key_offset(vkey) + (((2 * (g4 & 1) + ((lane & 3) >> 1)) ^ swz_of<MX>(vkey)) * 16) + (lane & 1) * 8;
  } else {
    const int vkey = 4 * g4 + (n16 >> 2);
    k_at = key_offset(n16) + (g4 ^ swz_of<MX>(n16)) * 16;
    v_at = key_offset(vkey) + (((n16 >> 1) & 1) ^ swz_of<MX>(vkey)) * 16 + (n16 & 1) * 8;
  }
  // MX: where this lane's first chunk of codes goes in a slot
  uint32_t pack_at = 0;
  if constexpr (MX) {
    const int key = wave * (8 * S::kOctets) + (lane & 7), c = lane >> 3;
    pack_at = key_offset(key) + (c >> 1) * 1024 + (((c & 1) * 4) ^ swz_of<MX>(key & 15)) * 16;
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
    const Item it = make_item<KIND, M, kWave, MX>(a, item);
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
    // MX: the keys between memory and LDS, and which of them are there
    Packed packed[MX ? S::kOctets : 1];
    uint32_t packed_live = 0;
    // (the wide form also loads the steps after the last, from the row of zeros: it
    // then has no branch between its MFMAs)
    auto slot_base = [&](int step) {
      return kStaged ? (step - step0) % 3 * S::kSlotBytes : ((step - step0) & (S::kSlots - 1)) * S::kSlotBytes;
    };
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
        const int key = key0 + 8 * o + (MX && !kStaged ? lane & 7 : lane >> 3);
        int row;
        bool live;
        if constexpr (KIND == kSparse) {
          row = s_rows[key & (kWindow - 1)];
          live = any && row >= 0;
          const uint64_t mask = __ballot(live);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            live_bits |= static_cast<uint32_t>(mask >> (MX && !kStaged ? i : 8 * i) & 1) << (8 * o + i);
        } else {
          // keys that no row of the pair tile sees are not read
          const int tok = it.tile0 * kTile + key;
          row = page * kPage + (key & (kPage - 1));
          live = any && tok >= it.min_start && tok < it.max_end;
        }
        from[o] = live ? cache + static_cast<int64_t>(row) * (MX ? IDX_LATENT_MXFP4_ROW : kRowBytes) : zero;
        if constexpr (kStaged) from[o] += ((lane & 7) ^ (lane >> 3)) * 16;
        if constexpr (!MX) {
          from[o] += ((lane & 7) ^ swz((8 * ((wave * S::kOctets + o) & 1)) + (lane >> 3))) * 16;
          to[o] = ring + slot * S::kSlotBytes + (wave * S::kOctets + o) * kOctBytes;
        }
      }
      if constexpr (MX && !S::kWide) packed_live = live_bits;  // (of the two slots, this one is still in use)
      else if (KIND == kSparse && lane == 0) s_live[slot][wave] = live_bits;
    };
    // MX: one of the nine 16-byte pieces of this lane's part of an octet into the image,
    // whose place for the step's codes is pack_base(step).  (The second octet's keys
    // exchange their chunks by bit 1 more than the first's.)
    auto pack_base = [&](int step) { return opaque(ring + slot_base(step) + pack_at); };
    auto stage_of = [&](int step) { return ring + kStageAt + (wave * 2 + ((step - step0) & 1)) * kStageBytes; };
    auto load_staged = [&](int step, int j) {  // j is a constant of the unrolled loop
      const uint32_t to = stage_of(step);
      switch (j) {
        case 0: return load_stage<0>(from[0], to);
        case 1: return load_stage<1>(from[0], to);
        case 2: return load_stage<2>(from[0], to);
        case 3: return load_stage<3>(from[0], to);
      }
    };
    // (a key's 16-byte chunks are exchanged by its number, the first one of the third
    // piece holds its powers)
    auto read_staged = [&](uint32_t stage, int part) {
      const uint32_t key = stage + (lane & 7) * 128, c = lane >> 3;
      const uint32_t at = key + (c ^ (lane & 7)) * 16, power = key + 2048 + (lane & 7) * 16 + c;
      if (part == 0) packed[0].codes[0] = __builtin_bit_cast(i32x4, lds_read(at)), packed[0].power[0] = lds_read_byte(power);
      if (part == 1)
        packed[0].codes[1] = __builtin_bit_cast(i32x4, lds_read(at + 1024)), packed[0].power[1] = lds_read_byte(power + 8);
      if (part == 2) packed[0].rotated = __builtin_bit_cast(i32x4, lds_read(at + 3 * 1024));
    };
    auto unpack = [&](uint32_t base, int step, int o, int j) {
      if (j < 8) {
        const float power = __uint_as_float(packed[o].power[j >> 2] << 23);
        lds_write((base ^ (((j & 3) ^ 2 * o) * 16)) + o * kOctBytes + (j >> 2) * 4096,
                  dequant8<DT>(static_cast<uint32_t>(packed[o].codes[j >> 2][j & 3]), power));
      } else {
        // from chunk 4 (c8 & 1) of piece c8 / 2 to chunk c8 of piece 8
        const uint32_t c = (opaque(tid) & 63) >> 3;
        lds_write((base ^ ((c ^ (c & 1) * 4 ^ 2 * o) * 16)) + o * kOctBytes + (8 - (c >> 1)) * 1024,
                  __builtin_bit_cast(s16x8, packed[o].rotated));
        if (KIND == kSparse && !S::kWide && o == S::kOctets - 1 && lane == 0)
          s_live[(step - step0) & (S::kSlots - 1)][wave] = packed_live;
      }
    };
    auto unpack_all = [&](int step) {
      const uint32_t base = pack_base(step);
#pragma unroll
      for (int o = 0; o < S::kOctets; ++o)
#pragma unroll
        for (int j = 0; j < 9; ++j) unpack(base, step, o, j);
    };
    auto fetch_all = [&](int step) {
      locate(step);
      if constexpr (kStaged) {
#pragma unroll
        for (int j = 0; j < kStageLoads; ++j) load_staged(step, j);
        return;
      }
#pragma unroll
      for (int o = 0; o < S::kOctets; ++o)
#pragma unroll
        for (int j = 0; j < kPackedParts; ++j) load_packed(packed[o], from[o], j);
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
                         (((lane & 7) ^ swz_of<MX>(pair & 15)) * 16);
      load_octet(from, q_ring + o * kOctBytes);
    }
    // narrow: slot 0 holds step0's keys, slot 1 the queries
    if constexpr (MX && !kStaged) fetch_all(step0);
    else if constexpr (!S::kWide) issue(step0);
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
    if constexpr (kStaged) {
      fetch_all(step0);
      fetch_all(step0 + 1);
      wait_loads<kStageLoads>();
#pragma unroll
      for (int j = 0; j < 3; ++j) read_staged(stage_of(step0), j);
      unpack_all(step0);
      fetch_all(step0 + 2);
    } else if constexpr (MX) {
      unpack_all(step0);
      if (step0 + 1 < step_end) fetch_all(step0 + 1);
    } else if constexpr (S::kWide) {
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
      if constexpr (kStaged) {
        wait_and_barrier<kStageLoads>();  // all but the loads of the step after next
      } else if constexpr (MX) {
        lds_barrier();
        if (step + 1 < step_end) unpack_all(step + 1);
        if (step + 2 < step_end) fetch_all(step + 2);
      } else if constexpr (S::kWide) {
        wait_and_barrier<S::kOctets * kOctLoads>();  // all but the next step's
      } else {
        wait_and_barrier<0>();
        if (step + S::kDistance < step_end) issue(step + S::kDistance);
      }
      const int slot = (step - step0) & (S::kSlots - 1);
      const uint32_t base = ring + slot_base(step) + (S::kWide ? 0 : ts * ST * kBlkBytes);

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
        if constexpr (kStaged) read_staged(stage_of(step + 1), 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!MX || KIND == kSparse) locate(step + kAhead);  // while they come
        const uint32_t image = MX ? pack_base(step + 1) : 0;
#pragma unroll
        for (int ks = 0; ks < kQ; ks += 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ks + kRing - 2 + i < kQ) read(ks + kRing - 2 + i);
          __builtin_amdgcn_sched_barrier(0);
          s0 = E::mfma_wide(kk[ks % kRing], q[ks], s0);
          s0 = E::mfma_wide(kk[(ks + 1) % kRing], q[ks + 1], s0);
          if (ks / 2 < kOctLoads) {
            if constexpr (MX) {
              unpack(image, step + 1, 0, ks / 2);
              if (ks / 2 == 1 || ks / 2 == 5) read_staged(stage_of(step + 1), ks / 2 == 1 ? 1 : 2);
              if (KIND != kSparse && ks / 2 == kOctLoads - 1) locate(step + kAhead);
            } else {
              load_one(ks / 2);
            }
          } else if (ks / 2 - kOctLoads < 8) {
            weigh(ks / 2 - kOctLoads, sum);
            if (kStaged && ks / 2 - kOctLoads < kStageLoads) load_staged(step + kAhead, ks / 2 - kOctLoads);
          }
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
          s16x8* v = reinterpret_cast<s16x8*>(s_keys + slot_base(step)) + i;
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
        value_wide(step > step0 ? ring + slot_base(step - 1) : base, [&](int d) {
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
      value_wide(ring + slot_base(step_end - 1), [&](int d) {
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

}  // namespace
}  // namespace pmqa
