// The 16-bit matrix-product tile shared by the output head's kernels
// (k_head.hip): C[m][n] += sum_k A[m][k] B[k][n] over a TM x TN tile of one
// workgroup of WM x WN waves, on v_mfma_f32_16x16x32_{bf16,f16} (fp32 sums).
//
// An operand comes from memory in one of two orders:
//   kRows  k runs along the memory row (weights or hidden states as the
//          logits read them).  LDS tile: [row][64 k], 128-byte rows of 8
//          16-byte chunks; a lane's operand (8 consecutive k of one row) is
//          one 16-byte LDS read.
//   kCols  k runs down the memory rows (the gradients contract over tokens
//          or vocabulary, the row index of every array).  LDS tile: [64 k][T
//          columns]; gfx950's transposing LDS read (ds_read_b64_tr_b16) hands
//          each lane 4 consecutive k of one column, so no transposed copy of
//          anything is ever written.
// Tiles go from memory to LDS directly (buffer_load ... lds, 16 bytes a
// lane), one or two steps of 64 k ahead; rows past the end of a buffer read
// zeros.  The direct load writes lane l at base + 16 l, so swizzles are made by
// permuting which chunk a lane fetches:
//   kRows  chunk c of row r lies in slot c ^ f(r).  A 16-byte read serves 16
//          lanes at a time from 64 banks (two rows): f takes 8 values over the
//          16 rows that one operand read touches.
//   kCols  the 32-byte unit u of row k lies at u ^ F(k), F = (k % 4) + 4 (k / 8
//          % 2): the 8 rows that half a transposing read touches lie on
//          disjoint banks.
#pragma once

#include "sbl_internal.h"

namespace sbl {
namespace head {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// The two 16-bit types.
struct Bf16 {
  static __device__ __forceinline__ v4f mma(v8s a, v8s b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, v2b{(__bf16)a, (__bf16)b});
  }
  // what rounding a and b to `v` = pack2(a, b) left, rounded itself
  static __device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t v) {
    const v2b x = __builtin_bit_cast(v2b, v);
    return pack2(a - (float)x[0], b - (float)x[1]);
  }
};
struct Fp16 {
  static __device__ __forceinline__ v4f mma(v8s a, v8s b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, v2h{(_Float16)a, (_Float16)b});
  }
  static __device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t v) {
    const v2h x = __builtin_bit_cast(v2h, v);
    return pack2(a - (float)x[0], b - (float)x[1]);
  }
};

constexpr int kBK = 64;                   // k per step
constexpr uint32_t kFar = 0x80000000u;    // a buffer offset beyond every buffer: reads zeros

enum Order { kRows, kCols };

constexpr int kNt = 2;                    // cache-policy bit "nt" of a buffer load: read once

template <int kPolicy>
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, 0, 0, kPolicy);
}

// Where one wave's share of an operand tile comes from: the byte offset of
// each of its 1 KB pieces (piece q = wave + waves * p), per lane.  The pieces
// are a fixed distance apart, except when rows are picked from a list (kList).
// kPerm (kRows only): rows are read in the order of the logits' row operand, below.
// kPanel (kRows only): the memory is panels of 256 k, [panel][row][256], with
// zeros from klen to the end of its panel.
template <Order O, int T, int WAVES, bool kPerm, bool kList = false, bool kPanel = false, int kPolicy = 0>
struct Source {
  static constexpr int kPieces = T * kBK * 2 / 1024 / WAVES;
  static_assert(T * kBK * 2 % (1024 * WAVES) == 0 && WAVES % 4 == 0, "whole pieces");
  static_assert(O == kRows || T == 256 || T == 128, "LDS rows of 512 or 256 bytes");
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t off[kList ? kPieces : 1];
  uint32_t apart;                          // bytes from piece to piece
  uint32_t step;                           // bytes per 64 k
  int chunk;                               // kRows: first k of this lane's chunk
  uint32_t panel;                          // kPanel: bytes per panel
  int first;                               // kPanel: step 0's place, in steps from the first panel

  __device__ __forceinline__ int first_chunk(int wave, int lane) const {
    // f of row 8q + lane / 8 (q % 4 = wave % 4): see Reader
    const int r8 = lane >> 3;
    const int f = kPerm ? ((r8 >> 1) & 1) | ((wave & 3) << 1) : (r8 >> 1) | ((wave & 1) << 2);
    return ((lane & 7) ^ f) * 8;
  }
  // kRows: tile row r at byte r * pitch
  __device__ __forceinline__ void init_rows(__amdgpu_buffer_rsrc_t rs, int wave, int lane, uint32_t pitch) {
    static_assert(O == kRows && !kList, "");
    rsrc = rs;
    step = kBK * 2;
    apart = 8 * WAVES * pitch;
    chunk = first_chunk(wave, lane);
    off[0] = (uint32_t)(8 * wave + (lane >> 3)) * pitch + 2u * chunk;
  }
  // kRows: tile row r at byte row_off(r), or kFar
  template <class F>
  __device__ __forceinline__ void init_list(__amdgpu_buffer_rsrc_t rs, int wave, int lane, F row_off) {
    static_assert(O == kRows && kList, "");
    rsrc = rs;
    step = kBK * 2;
    apart = 0;
    chunk = first_chunk(wave, lane);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) off[p] = row_off(8 * (wave + WAVES * p) + (lane >> 3)) + 2u * chunk;
  }
  // kCols: memory rows of `pitch` bytes, the tile's columns start at byte `col`
  __device__ __forceinline__ void init_cols(__amdgpu_buffer_rsrc_t rs, int wave, int lane, uint32_t pitch,
                                            uint32_t col) {
    static_assert(O == kCols, "");
    rsrc = rs;
    step = kBK * pitch;
    constexpr int kRowLanes = T / 8, kPer = 64 / kRowLanes;     // lanes per memory row, rows per piece
    const int k = kPer * wave + lane / kRowLanes, c = lane % kRowLanes;
    apart = kPer * WAVES * pitch;
    static_assert(!kList && (O != kCols || kPer * WAVES % 16 == 0), "F repeats every 16 k");
    off[0] = (uint32_t)k * pitch + col + 16u * (c ^ (2 * unit_of(k)));
  }
  static __device__ __forceinline__ int unit_of(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }
  // piece p of step ks into `lds`; k at or past klen read zeros (an offset with
  // the top bit set is beyond every buffer, kFar rows stay so)
  __device__ __forceinline__ void piece(uint8_t* lds, int wave, int p, int ks, int klen) const {
    const bool ok = O == kRows && !kPanel ? ks * kBK + chunk < klen : ks * kBK < klen;
    const uint32_t at = kPanel ? (uint32_t)((first + ks) >> 2) * panel + (uint32_t)((first + ks) & 3) * (kBK * 2)
                               : (uint32_t)ks * step;
    const uint32_t o = kList ? off[kList ? p : 0] + at : off[0] + (at + p * apart);
    dma16<kPolicy>(rsrc, lds + 1024 * (wave + WAVES * p), o | (ok ? 0u : kFar));
  }
  __device__ __forceinline__ void fetch(uint8_t* lds, int wave, int ks, int klen) const {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) piece(lds, wave, p, ks, klen);
  }
};

// Reads operands of 16-row (16-column) tiles from an LDS tile of T rows
// (columns); `base`, a multiple of 32, is the wave's first one in it.
// kPerm: row r of the MFMA operand of tile i is tile row
//   32 (i / 2) + 8 (r / 4) + 4 (i % 2) + r % 4,
// so that a lane's results of tiles 2j and 2j + 1 are 8 consecutive rows.
template <Order O, int T, bool kPerm>
struct Reader {
  int addr;

  __device__ __forceinline__ void init(int base, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (O == kRows) {
      const int row = base + (kPerm ? 8 * (r >> 2) + (r & 3) : r);
      const int f = kPerm ? ((r >> 1) & 1) | ((r >> 2) << 1) : (r >> 1);
      addr = row * 128 + 16 * (g ^ f);
    } else {
      const int k = 8 * g + (r >> 2), F = (r >> 2) | ((g & 1) << 2);
      addr = k * (T * 2) + 32 * ((base / 16) ^ F) + 8 * (r & 3);
    }
  }
  // keeps the few address variants from being kept in registers across steps
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(addr)); }
  // operand of tile i for the 32 k of half kk
  __device__ __forceinline__ v8s get(const uint8_t* lds, int i, int kk) const {
    if constexpr (O == kRows) {
      const int d = kPerm ? 32 * (i >> 1) + 4 * (i & 1) : 16 * i;
      return *reinterpret_cast<const v8s*>(lds + (addr ^ (64 * kk)) + d * 128);
    } else {
      typedef __attribute__((address_space(3))) v4s* lp;
      const uint8_t* p = lds + (addr ^ (32 * i)) + kk * 32 * (T * 2);
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)p);
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p + 4 * (T * 2)));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// s_waitcnt vmcnt(n), n < 64 (expcnt and lgkmcnt: no wait)
template <int n>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

// XCD-aware order: workgroups go to the 8 XCDs in turn, so XCD x takes the
// x-th contiguous run of tiles, whose operands then share its L2.
__device__ __forceinline__ int xcd_tile(int b, int n) {
  const int x = b & 7, per = n >> 3, rem = n & 7;
  return x * per + (x < rem ? x : rem) + (b >> 3);
}

__device__ __forceinline__ void wave_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// LDS stages are arrays of their own, picked by compile-time indexes, so that
// the compiler can tell a stage being filled from one being read: otherwise it
// waits for every direct load before the next LDS read.
template <class E, Order OA, Order OB, int TM, int TN, int WM, int WN, bool kPerm, bool kListB = false,
          bool kPanelB = false, int kPolicyA = 0>
struct Tile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kMT = TM / WM / 16, kNT = TN / WN / 16;
  static constexpr int kBytesA = TM * kBK * 2, kStageBytes = (TM + TN) * kBK * 2;
  Source<OA, TM, kWaves, kPerm, false, false, kPolicyA> sa;
  Source<OB, TN, kWaves, false, kListB, kPanelB> sb;
  v4f acc[kMT][kNT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int j = 0; j < kNT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  // The products of STEPS steps that lie in LDS, step by step: A at `la`, B at `lb`.
  template <int STEPS>
  __device__ __forceinline__ void products(const uint8_t* la, const uint8_t* lb, int wave, int lane) {
    Reader<OA, TM, kPerm> ra;
    Reader<OB, TN, false> rb;
    ra.init(wave / WN * (TM / WM), lane);
    rb.init(wave % WN * (TN / WN), lane);
    clear();
#pragma unroll
    for (int kk = 0; kk < 2 * STEPS; ++kk) {
      v8s b[kNT];
#pragma unroll
      for (int j = 0; j < kNT; ++j) b[j] = rb.get(lb + kk / 2 * (TN * kBK * 2), j, kk & 1);
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        const v8s a = ra.get(la + kk / 2 * kBytesA, i, kk & 1);
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[i][j] = E::mma(a, b[j], acc[i][j]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // Narrow tiles (bound by memory): STAGES - 1 steps in flight, two
  // workgroups per CU.
  template <int STAGES>
  __device__ __forceinline__ void run(uint8_t* const (&st)[STAGES], int wave, int lane, int klen) {
    Reader<OA, TM, kPerm> ra;
    Reader<OB, TN, false> rb;
    ra.init(wave / WN * (TM / WM), lane);
    rb.init(wave % WN * (TN / WN), lane);
    clear();
    const int steps = (klen + kBK - 1) / kBK;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      sa.fetch(st[s], wave, s, klen);
      sb.fetch(st[s] + kBytesA, wave, s, klen);
    }
    // Step ks was fetched STAGES - 1 steps ago (steps past the end fetch zeros,
    // so the count is exact); after the barrier every wave's part has landed,
    // and every wave has read the stage refilled next.
    auto step = [&](int ks, int u) {
      wait_vm<(STAGES - 2) * (decltype(sa)::kPieces + decltype(sb)::kPieces)>();
      wave_barrier();
      uint8_t* next = st[(u + STAGES - 1) % STAGES];
      sa.fetch(next, wave, ks + STAGES - 1, klen);
      sb.fetch(next + kBytesA, wave, ks + STAGES - 1, klen);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        v8s b[kNT];
#pragma unroll
        for (int j = 0; j < kNT; ++j) b[j] = rb.get(st[u] + kBytesA, j, kk);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
          const v8s a = ra.get(st[u], i, kk);
#pragma unroll
          for (int j = 0; j < kNT; ++j) acc[i][j] = E::mma(a, b[j], acc[i][j]);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    // whole turns of the stages, then the rest (no path leads from a skipped
    // step to another: the compiler would wait for every load there)
    int k0 = 0;
    // few sums per lane: kept in two levels, so that a long k rounds no more than a short one
    constexpr bool kTwoLevels = kMT * kNT <= 8;
    v4f done[kTwoLevels ? kMT : 1][kTwoLevels ? kNT : 1];
    auto carry = [&](bool first) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
          if constexpr (kTwoLevels) done[i][j] = first ? v4f{0.f, 0.f, 0.f, 0.f} : done[i][j] + acc[i][j];
          if (!first) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        }
    };
    if constexpr (kTwoLevels) carry(true);
    for (; k0 + STAGES <= steps; k0 += STAGES) {
      if constexpr (kTwoLevels)
        if (k0 % (4 * STAGES) == 0 && k0 > 0) carry(false);
#pragma unroll
      for (int u = 0; u < STAGES; ++u) step(k0 + u, u);
    }
    if (k0 < steps) step(k0, 0);
    if constexpr (STAGES > 2) {
      if (k0 + 1 < steps) step(k0 + 1, 1);
    }
    if constexpr (kTwoLevels) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[i][j] += done[i][j];
    }
    wait_vm<0>();                          // every direct load has landed before the workgroup can leave
  }

  // 256 x 256 on 8 waves of 128 x 64, two per SIMD: half of a wave's registers
  // hold the sums, most of the rest two sets of operands.  A step's 64 k are
  // two halves of 32 MFMAs; while the MFMAs of one half run, the operands of
  // the next are read, so a wave never waits for what it has just asked for:
  //   half 0   reads the operands of half 1; then (barrier: everyone has read
  //            this stage) refilling this stage with step ks + 2 begins
  //   half 1   (wait: step ks + 1 has landed everywhere) reads that step's
  //            half 0; the refill goes on
  // The 8 loads of a refill are spread over the 10 groups of 4 MFMAs that may
  // send them (kSlots).  Sent closer together they hold up the waves: logits of
  // 2048 x 32000 x 3200 take 4% longer with one per group from the first, 14%
  // with all in the first four groups.  Measured there: 304 us, 1380 TFLOP/s; the
  // matrix pipe is busy 70% of the cycles at the 1.86 GHz that the card's power
  // leaves, without an LDS bank conflict, and memory is read at 1.3 TB/s.
  // start() fetches step 0; what a caller loads between the two comes with it.
  __device__ __forceinline__ void start(uint8_t* const (&st)[2], int wave, int klen) {
    sa.fetch(st[0], wave, 0, klen);
    sb.fetch(st[0] + kBytesA, wave, 0, klen);
  }
  __device__ __forceinline__ void run_wide(uint8_t* const (&st)[2], int wave, int lane, int klen) {
    static_assert(TM == 256 && TN == 256 && WM == 2 && WN == 4, "eight waves of 128 x 64");
    Reader<OA, TM, kPerm> ra;
    Reader<OB, TN, false> rb;
    ra.init(wave / WN * (TM / WM), lane);
    rb.init(wave % WN * (TN / WN), lane);
    clear();
    const int steps = (klen + kBK - 1) / kBK;
    sa.fetch(st[1], wave, 1, klen);
    sb.fetch(st[1] + kBytesA, wave, 1, klen);
    wait_vm<8>();
    wave_barrier();
    v8s a[2][kMT], b[2][kNT];
#pragma unroll
    for (int j = 0; j < kNT; ++j) b[0][j] = rb.get(st[0] + kBytesA, j, 0);
#pragma unroll
    for (int i = 0; i < kMT; ++i) a[0][i] = ra.get(st[0], i, 0);
    // The 4 MFMAs of row tile i on operand set f.  With both operands down the
    // k axis (twice the LDS reads) a wave that has its operands goes first:
    // 5% there, and 1 to 2% the other way with fewer reads.
    constexpr bool kFirst = OA == kCols && OB == kCols;
    auto mma4 = [&](int f, int i) {
      if constexpr (kFirst) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int j = 0; j < kNT; ++j) acc[i][j] = E::mma(a[f][i], b[f][j], acc[i][j]);
      if constexpr (kFirst) __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
    };
    // two of the next 12 operands
    auto load2 = [&](int f, int n, uint8_t* from, int kk) {
#pragma unroll
      for (int q = 2 * n; q < 2 * n + 2; ++q) {
        constexpr int kOrder[12] = {0,4,5,1,6,7,2,8,9,3,10,11};   // 0 to 3: column tiles, 4 on: row tiles
        if (kOrder[q] < 4)
          b[f][kOrder[q] & 3] = rb.get(from + kBytesA, kOrder[q] & 3, kk);
        else
          a[f][kOrder[q] - 4] = ra.get(from, kOrder[q] - 4, kk);
      }
    };
    // load q of a refill goes before group kSlots[q] of the step's 16, 2 of them
    // before the wait
    constexpr int kSlots[8] = {6, 7, 9, 11, 12, 13, 14, 15};
    auto send = [&](int group, int ks, int u) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (kSlots[q] == group) {
          if (q < 4)
            sa.piece(st[u], wave, q, ks + 2, klen);
          else
            sb.piece(st[u] + kBytesA, wave, q - 4, ks + 2, klen);
        }
    };
    auto step = [&](int ks, int u) {
      ra.pin();
      rb.pin();
#pragma unroll
      for (int n = 0; n < 6; ++n) {
        load2(1, n, st[u], 1);
        mma4(0, n);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      wave_barrier();
#pragma unroll
      for (int n = 6; n < 8; ++n) {
        send(n, ks, u);
        mma4(0, n);
      }
      wait_vm<2>();
      wave_barrier();
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n < 6) load2(0, n, st[u ^ 1], 0);
        send(8 + n, ks, u);
        mma4(1, n);
      }
    };
    // an odd last step is paired with one of zeros: a branch around it costs
    // the loop its register allocation
    for (int ks = 0; ks < steps; ks += 2) {
      step(ks, 0);
      step(ks + 1, 1);
    }
    wait_vm<0>();                          // every direct load has landed before the workgroup can leave
  }
};

}  // namespace head
}  // namespace sbl
