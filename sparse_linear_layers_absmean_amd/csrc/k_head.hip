// Matrix products of the output head's losses: logits that are used where
// they are made and never stored, and the two gradients.
//
//   z[t][v] = sum_d h[t][d] w[v][d]
//   forward   per token: max of z and sum of 2^((z - max) scale) over each
//             tile's ids, joined later, and z at the token's listed ids
//   backward  dz[t][v] = coef[t] 2^(z scale - lse2[t]) - sub at the listed ids,
//             rounded once to 16 bits, a range of the vocabulary at a time;
//             dw = dz^T h, dh = dz w
//
// dz is rounded because the two products that read it run on the 16-bit matrix
// instructions: held in two 16-bit parts, as up to 64 tokens where the products
// cost nothing, both would run twice (at 2048 x 32000 x 3200 they are 690 to 720 of
// 1040 us).  The rounding is as large as the outputs' own: against 64 bits the
// BF16 gradients there are off by 1.9e-3 of their norm (cross entropy) and 2.3e-3
// (distillation), with dz in 32 bits by 1.7e-3.
//
// The logits are computed again in the backward: keeping them would take
// tokens x vocabulary values (1 GB at 4096 x 128256 in 16 bits).
#include "sbl_head.h"
#include "sbl_head_tile.h"

namespace sbl {
namespace head {

namespace {

// The lane number computed anew: epilogues use it so that nothing derived from
// the thread index occupies a register during the products.
__device__ __forceinline__ int lane_again() { return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0)); }

// The logit gradients of a range, in panels of 256 ids: [panel][rows][256].  A
// 256 x 256 tile is one run of 128 KB, wherever it is written or read, and rows
// are 512 bytes apart (rows of the whole range, 64 or 128 KB apart, would touch
// a page each).
__device__ __forceinline__ uint16_t* dz_at(uint16_t* dz, int rows, int t, int v) {
  return dz + ((int64_t)(v >> 8) * rows + t) * 256 + (v & 255);
}

// ---------------------------------------------------------------- logits
// Rows of the tile (MFMA rows) are vocabulary entries, columns are tokens: a
// lane holds one token's logits of 4 consecutive ids per 16-row tile, and with
// the permuted row order 8 consecutive ids per pair of tiles, so softmax
// statistics reduce over registers and two lane exchanges, and the gradient
// leaves as 16-byte stores.  Many tokens: bound by the matrix pipe (2048 x 32000 x
// 3200 forward 304 us; backward 330 to 340, the rest its stores of 131 MB).  Few:
// by reading w (64 x 32000 x 1536 20 us, 4.9 TB/s; 1 x 32000 x 3200 34 us, 6.0).
template <class E, int TM, int TN, int WM, int WN, bool kBackward, int kPolicy, class St>
__device__ __forceinline__ void logits_tile(const LogitsArgs& a, int tile, const St& st) {
  using T = Tile<E, kRows, kRows, TM, TN, WM, WN, true, !kBackward, false, kPolicy>;
  __shared__ int32_t row_of[kBackward ? 1 : TN];   // original row of each of the tile's tokens, -1: none
  __shared__ float2 stat[kBackward ? 1 : WM][kBackward ? 1 : TN];
  constexpr int kHits = TN <= 64 ? 512 : 1024;
  __shared__ uint32_t hit_at[kHits];       // listed ids in this tile: id less vt0, token less t0, entry; 8 bits each
  __shared__ float hit_sub[kBackward ? kHits : 1];
  __shared__ int hit_count;
  const int count = a.hdr ? a.hdr->count : a.m_tok;
  const int nvt = (a.n_vocab + TM - 1) / TM, ntt = (a.m_tok + TN - 1) / TN;
  // groups of kGroup vocabulary tiles x every token tile
  constexpr int kGroup = 4;
  const int group = tile / (kGroup * ntt), in_group = tile % (kGroup * ntt);
  const int gv = nvt - group * kGroup < kGroup ? nvt - group * kGroup : kGroup;
  const int vt = group * kGroup + in_group % gv, tt = in_group / gv;
  const int t0 = tt * TN;
  // few tokens, backward: rows without a token are written too, as zeros
  const int half = kBackward ? a.half : 0;
  if (t0 >= count && half == 0) return;
  const int64_t vt0 = (int64_t)vt * TM;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int lane = tid & 63;
  T tl;
  const int64_t wrows = a.n_vocab - vt0 < TM ? a.n_vocab - vt0 : TM;
  tl.sa.init_rows(make_rsrc(a.w + vt0 * a.k, wrows * a.k * 2), wave, lane, 2 * a.k);
  if constexpr (kBackward) {
    const int left = count > t0 ? count - t0 : 0;
    tl.sb.init_rows(make_rsrc(a.h + (int64_t)t0 * a.k, (int64_t)left * a.k * 2), wave, lane, 2 * a.k);
  } else {
    for (int i = tid; i < TN; i += T::kThreads) {
      const int t = t0 + i;
      row_of[i] = t < count ? (a.rows ? a.rows[t] : t) : -1;
    }
    __syncthreads();
    tl.sb.init_list(make_rsrc(a.h, ((a.h_rows - 1) * a.h_stride + a.k) * 2), wave, lane, [&](int r) {
      const int row = row_of[r];
      return row < 0 ? kFar : (uint32_t)((int64_t)row * a.h_stride * 2);
    });
  }
  if constexpr (TN == 256) tl.start(st, wave, a.k);
  // Backward: what the end needs is loaded now.  There, a load would wait for
  // the stores before it (the memory counter counts both, in order).
  constexpr int kMT = T::kMT, kNT = T::kNT, kRowsW = TM / WM, kColsW = TN / WN;
  const int wm = wave / WN, wn = wave % WN;
  float lse2[kNT], coef[kNT];
  if constexpr (kBackward) {
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
      const int t = t0 + wn * kColsW + 16 * j + (lane & 15);
      lse2[j] = t < count ? a.lse2[t] : 0.f;
      coef[j] = t < count ? a.coef[t] : 0.f;
    }
  }
  // The listed ids that fall into this tile, found by all threads.  Their order
  // does not matter: each has a place of its own to go to.
  if (tid == 0) hit_count = 0;
  __syncthreads();
  auto found_one = [&](int tok, int ent) {
    const int n = atomicAdd(&hit_count, 1);
    if (n < kHits) hit_at[n] = (uint32_t)tok << 8 | (uint32_t)ent << 16;
  };
  auto id_of = [&](int tok, int ent) -> int64_t {   // less the range's first id
    if constexpr (kBackward)
      return (int64_t)a.index32[(int64_t)(t0 + tok) * a.top + ent] - a.v0;
    else
      return a.index[(int64_t)row_of[tok] * a.top + ent];
  };
  if (a.near) {
    // 8 entries' 256-id blocks in 16 bytes, 4 loads of a thread at a time
    constexpr int kBatch = 4;
    const int per_row = (a.top + 7) / 8, units = TN * per_row;
    const uint32_t want = (uint32_t)((a.v0 + vt0) >> 8);
    for (int u0 = tid; u0 < units; u0 += T::kThreads * kBatch) {
      u32x4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int n = u0 + u * T::kThreads, tok = n / per_row;
        x[u] = u32x4{~0u, ~0u, ~0u, ~0u};
        if (n < units && t0 + tok < count) {
          const int64_t row = kBackward ? t0 + tok : row_of[tok];
          x[u] = reinterpret_cast<const u32x4*>(a.near)[row * per_row + n % per_row];
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int n = u0 + u * T::kThreads;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (((x[u][q >> 1] >> (16 * (q & 1))) & 0xFFFFu) == want) found_one(n / per_row, 8 * (n % per_row) + q);
      }
    }
  } else {
    constexpr int kBatch = 4;
    const int step_t = T::kThreads / a.top, step_k = T::kThreads % a.top;
    int et = tid / a.top, ek = tid % a.top;
    for (int e0 = 0; e0 < TN * a.top; e0 += T::kThreads * kBatch) {
      int64_t id[kBatch];
      int tok[kBatch], ent[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        tok[u] = et;
        ent[u] = ek;
        id[u] = et < TN && t0 + et < count ? id_of(et, ek) : -1;
        et += step_t;
        ek += step_k;
        if (ek >= a.top) {
          ek -= a.top;
          ++et;
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int64_t d = id[u] - vt0;
        if (id[u] >= 0 && d >= 0 && d < TM) found_one(tok[u], ent[u]);
      }
    }
  }
  __syncthreads();
  for (int n = tid; n < hit_count && n < kHits; n += T::kThreads) {
    const int tok = (int)(hit_at[n] >> 8 & 255), ent = (int)(hit_at[n] >> 16);
    const int64_t d = id_of(tok, ent) - vt0;     // with blocks: perhaps in the block's other tile; 255 is no row of a
    hit_at[n] |= d >= 0 && d < TM ? (uint32_t)d : 255u;     // 128-id tile
    if constexpr (kBackward) hit_sub[n] = a.sub[(int64_t)(t0 + tok) * a.top + ent];
  }
  // the other waves read the list after the products, whose first barrier waits
  // for no LDS write (and may be the only one: a single step)
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  if constexpr (TN == 256)
    tl.run_wide(st, wave, lane, a.k);
  else
    tl.template run<3>(st, wave, lane, a.k);

  lane = lane_again();
  const int r = lane & 15, g = lane >> 4;
  const int vw = (int)vt0 + wm * kRowsW;   // first id (in this range) of the wave's rows
  if (vw + kRowsW > a.n_vocab) {           // the last tile: no logit past the vocabulary
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (vw + 32 * (i >> 1) + 8 * g + 4 * (i & 1) + e >= a.n_vocab) {
#pragma unroll
          for (int j = 0; j < kNT; ++j) tl.acc[i][j][e] = -__builtin_inff();
        }
  }

#pragma unroll
  for (int j = 0; j < kNT; ++j) {
    const int tw = wn * kColsW + 16 * j + r;
    const int t = t0 + tw;
    if constexpr (!kBackward) {
      // the largest logit stays unscaled: what later cancels (it against a listed
      // logit) then cancels without a rounding of either
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, tl.acc[i][j][e]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float top = mx == -__builtin_inff() ? 0.f : mx;   // no finite logit here: a sum of zeros
      const float ref = top * a.scale, off = __builtin_fmaf(top, a.scale, -ref);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum += __builtin_amdgcn_exp2f(__builtin_fmaf(tl.acc[i][j][e], a.scale, -ref));
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      sum *= __builtin_amdgcn_exp2f(-off);                    // ref's own rounding, exactly known
      if (g == 0) stat[wm][tw] = float2{mx, sum};
    } else {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tl.acc[i][j][e] = coef[j] * __builtin_amdgcn_exp2f(__builtin_fmaf(tl.acc[i][j][e], a.scale, -lse2[j]));
      if (t < (half > 0 ? half : count)) {
        uint16_t* o = dz_at(a.dz, a.dz_rows, t, vw) + 8 * g;
#pragma unroll
        for (int i = 0; i < kMT; i += 2) {
          v4f x = tl.acc[i][j], y = tl.acc[i + 1][j];
          if (t >= count) x = y = v4f{0.f, 0.f, 0.f, 0.f};     // no token: also where the weights are not finite
          const u32x4 v = u32x4{E::pack2(x[0], x[1]), E::pack2(x[2], x[3]), E::pack2(y[0], y[1]), E::pack2(y[2], y[3])};
          *reinterpret_cast<u32x4*>(o + 16 * i) = v;
          if (half > 0)                    // what the rounding left, to rows of its own
            *reinterpret_cast<u32x4*>(o + 256 * half + 16 * i) =
                u32x4{E::rest2(x[0], x[1], v[0]), E::rest2(x[2], x[3], v[1]), E::rest2(y[0], y[1], v[2]),
                      E::rest2(y[2], y[3], v[3])};
        }
      }
    }
  }
  if constexpr (!kBackward) {
    // joins the waves' statistics: one entry per token and tile
    __syncthreads();
    for (int i = tid; i < TN; i += T::kThreads) {
      if (t0 + i >= count) break;
      float2 x = stat[0][i];
#pragma unroll
      for (int w = 1; w < WM; ++w) {
        const float2 y = stat[w][i];
        const float mx = fmaxf(x.x, y.x), ref = mx == -__builtin_inff() ? 0.f : mx;
        x.y = x.y * __builtin_amdgcn_exp2f((x.x - ref) * a.scale) + y.y * __builtin_amdgcn_exp2f((y.x - ref) * a.scale);
        x.x = mx;
      }
      a.part[(int64_t)(t0 + i) * a.np + vt] = x;
    }
  }

  // Listed ids on this wave's rows and columns, 64 at a time by ballot, then one
  // by one (a wave-uniform walk to the accumulator).  That costs with their
  // number: 2048 x 32000 x 3200 forward 345 us with one id per token, 391 with 64
  // spread evenly (140 in the fullest tile), 733 with 64 that follow 1 / (id + 10)
  // (6300), 986 with all in one block of 256 ids (16384).
  // Forward: the logit.  Backward: the lane that stored the id's gradient
  // stores it again with the listed part taken off, still from 32 bits.
  auto take = [&](int rel, int et, int ek, float sub) {
    uint64_t hits = __ballot(rel >= 0);
    while (hits) {
      const int src = __builtin_ctzll(hits);
      hits &= hits - 1;
      const int hr = __builtin_amdgcn_readlane(rel, src), ht = __builtin_amdgcn_readlane(et, src);
      const int hi = 2 * (hr >> 5) + ((hr >> 2) & 1), hj = ht >> 4, he = hr & 3;
      float val = 0.f;                     // not a switch or a tree: the compiler would put the sums in memory
#pragma unroll
      for (int j = 0; j < kNT; ++j)
        if (hj == j) {
#pragma unroll
          for (int i = 0; i < kMT; ++i)
            if (hi == i) {
              const v4f x = tl.acc[i][j];
              val = he == 0 ? x[0] : he == 1 ? x[1] : he == 2 ? x[2] : x[3];
            }
        }
      const int64_t t = t0 + wn * kColsW + ht;
      const bool mine = r == (ht & 15) && g == ((hr >> 3) & 3);
      if constexpr (!kBackward) {
        const int hk = __builtin_amdgcn_readlane(ek, src);
        if (mine) a.zlist[t * a.top + hk] = val;
      } else {
        const float hsub = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sub), src));
        if (mine) {
          uint16_t* o = dz_at(a.dz, a.dz_rows, (int)t, vw + hr);
          const uint32_t v = E::pack2(val - hsub, 0.f);
          *o = (uint16_t)v;
          if (half > 0) o[256 * half] = (uint16_t)E::rest2(val - hsub, 0.f, v);
        }
      }
    }
  };
  const int found = hit_count;             // complete, as the list is, since the products' first barrier
  if (found <= kHits) {
    for (int n0 = 0; n0 < found; n0 += 64) {
      int rel = -1, et = 0, ek = 0;
      float sub = 0.f;
      if (n0 + lane < found) {
        const uint32_t x = hit_at[n0 + lane];
        et = (int)(x >> 8 & 255) - wn * kColsW;
        ek = (int)(x >> 16);
        const int d = (int)(x & 255) - wm * kRowsW;
        if (d >= 0 && d < kRowsW && et >= 0 && et < kColsW) rel = d;
        if constexpr (kBackward) sub = hit_sub[n0 + lane];
      }
      take(rel, et, ek, sub);
    }
    return;
  }
  // more listed ids in one tile than the list holds: every entry of the wave's tokens
  for (int e0 = 0; e0 < kColsW * a.top; e0 += 64) {
    const int e = e0 + lane, et = e / a.top, ek = e % a.top, tw = wn * kColsW + et;
    int rel = -1;
    float sub = 0.f;
    if (et < kColsW && t0 + tw < count) {
      int64_t id;
      if constexpr (kBackward) {
        const int64_t slot = (int64_t)(t0 + tw) * a.top + ek;
        id = a.index32[slot] - a.v0;
        sub = a.sub[slot];
      } else {
        id = a.index[(int64_t)row_of[tw] * a.top + ek];
      }
      const int64_t d = id - vw;
      if (id >= 0 && d >= 0 && d < kRowsW) rel = (int)d;
    }
    take(rel, et, ek, sub);
  }
}

template <class E, int TM, int TN, int WM, int WN, bool kBackward, int kPolicy = 0>
__global__ __launch_bounds__(64 * WM * WN, 2) void logits_kernel(const LogitsArgs a) {
  constexpr int kStage = (TM + TN) * kBK * 2;
  __shared__ __align__(16) uint8_t lds0[kStage];
  __shared__ __align__(16) uint8_t lds1[kStage];
  const int tile = a.tile0 + xcd_tile(blockIdx.x, gridDim.x);
  if constexpr (TN == 256) {
    uint8_t* const st[2] = {lds0, lds1};
    logits_tile<E, TM, TN, WM, WN, kBackward, kPolicy>(a, tile, st);
  } else {
    __shared__ __align__(16) uint8_t lds2[kStage];
    uint8_t* const st[3] = {lds0, lds1, lds2};
    logits_tile<E, TM, TN, WM, WN, kBackward, kPolicy>(a, tile, st);
  }
}

// ---------------------------------------------------------------- gradients
// Rows of the tile are features (contiguous in memory, read down the k axis),
// so a lane's 4 consecutive results are 4 consecutive features of an output row.
// Bound by the matrix pipe from some hundred tokens on (both gradients of 2048 x
// 32000 x 3200 in 690 to 720 us, 1190 TFLOP/s at best, the pipe busy 65%): a tile of dw has few steps,
// 32 at 2048 tokens, beside the 7 us of its start and its 128 KB of stores.

template <class E, int TM, int TN, int WM, int WN, class St>
__device__ __forceinline__ void weight_grad_tile(const WeightGradArgs& a, int tile, const St& st) {
  using T = Tile<E, kCols, kCols, TM, TN, WM, WN, false>;
  const int count = a.rows > 0 ? a.rows : a.hdr->count;
  const int ndt = (a.k + TM - 1) / TM, nvt = (a.n_vocab + TN - 1) / TN;
  constexpr int kGroup = 4;
  const int group = tile / (kGroup * ndt), in_group = tile % (kGroup * ndt);
  const int gv = nvt - group * kGroup < kGroup ? nvt - group * kGroup : kGroup;
  const int vt = group * kGroup + in_group % gv, dt = in_group / gv;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int lane = threadIdx.x & 63;
  T tl;
  tl.sa.init_cols(make_rsrc(a.h, (int64_t)count * a.k * 2), wave, lane, 2 * a.k, 2 * TM * dt);
  tl.sb.init_cols(make_rsrc(a.dz + (int64_t)(vt * TN / 256) * a.m_tok * 256, (int64_t)count * 512), wave, lane, 512,
                  2 * (vt * TN % 256));
  if constexpr (TN == 256) {
    tl.start(st, wave, count);
    tl.run_wide(st, wave, lane, count);
  } else {
    tl.template run<2>(st, wave, lane, count);
  }
  lane = lane_again();
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, g = lane >> 4;
  const float down = a.hdr->down;
  // A lane holds features 4g .. 4g + 3 of a 16-feature tile.  Of two tiles, the
  // even groups of lanes give their part of the second to the odd ones for
  // those's part of the first: 8 consecutive features each, 64-byte runs per
  // store (runs of 32 bytes reach memory at 3.8 TB/s, of 64 at 6.1).
  const int d0 = dt * TM + wm * (TM / WM) + ((g & 1) ? 16 + 4 * (g - 1) : 4 * g);
#pragma unroll
  for (int j = 0; j < T::kNT; ++j) {
    const int v = vt * TN + wn * (TN / WN) + 16 * j + r;
    uint16_t* o = a.dw + (int64_t)v * a.k;
#pragma unroll
    for (int i = 0; i < T::kMT; i += 2) {
      const v4f x = tl.acc[i][j] * down, y = tl.acc[i + 1][j] * down;
      const auto lo = __builtin_amdgcn_permlane16_swap(E::pack2(x[0], x[1]), E::pack2(y[0], y[1]), false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(E::pack2(x[2], x[3]), E::pack2(y[2], y[3]), false, false);
      const int d = d0 + 16 * i;
      if (v < a.n_vocab && d < a.k) *reinterpret_cast<u32x4*>(o + d) = u32x4{lo[0], hi[0], lo[1], hi[1]};
    }
  }
}

// The shares of dh when `count` of the m_tok rows take part: the tiles that the
// others would have taken share the vocabulary instead.  They fill the grid and
// the partial sums' rows that all m_tok would (n tiles of tn rows in all).
struct Shares {
  int splits, steps, tiles;                // steps of a share; token tiles
  int64_t rows;                            // rows of a share's partial sums
};
__device__ __forceinline__ Shares hidden_shares(int splits, int range_steps, int m_tok, int tn, int count) {
  const int n = count < 1 ? 1 : count, tiles = (n + tn - 1) / tn;
  int64_t s = (int64_t)splits * ((m_tok + tn - 1) / tn) / tiles;
  const int64_t fit = (int64_t)splits * m_tok / n;
  s = s < fit ? s : fit;
  s = s < range_steps / 4 ? s : range_steps / 4;
  s = s > splits ? s : splits;
  const int steps = (int)((range_steps + s - 1) / s);
  return Shares{(range_steps + steps - 1) / steps, steps, tiles, n};
}

template <class E, int TM, int TN, int WM, int WN, class St>
__device__ __forceinline__ void hidden_grad_tile(const HiddenGradArgs& a, const Shares& sh, int tile, const St& st) {
  using T = Tile<E, kCols, kRows, TM, TN, WM, WN, false, false, true>;
  const int count = a.rows > 0 ? a.rows : a.hdr->count;
  const int ndt = (a.k + TM - 1) / TM, ntt = sh.tiles;
  // a share's tiles together: they read the same rows of w
  const int s = tile / (ndt * ntt), in = tile % (ndt * ntt);
  // groups of kGroup token tiles x every feature tile
  constexpr int kGroup = 4;
  const int group = in / (kGroup * ndt), in_group = in % (kGroup * ndt);
  const int gt = ntt - group * kGroup < kGroup ? ntt - group * kGroup : kGroup;
  const int dt = in_group / gt, t0 = (group * kGroup + in_group % gt) * TN;
  if (t0 >= count) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int lane = threadIdx.x & 63;
  const int64_t v0 = (int64_t)s * sh.steps * kBK;
  int64_t vs = a.n_vocab - v0;
  if (vs > (int64_t)sh.steps * kBK) vs = (int64_t)sh.steps * kBK;
  if (vs < 0) vs = 0;
  T tl;
  tl.sa.init_cols(make_rsrc(a.w + v0 * a.k, vs * a.k * 2), wave, lane, 2 * a.k, 2 * TM * dt);
  // rows past the last token read other rows of the panel, for columns that are not stored
  tl.sb.init_rows(make_rsrc(a.dz + (int64_t)t0 * 256, ((int64_t)(a.n_vocab + 255) / 256 * a.m_tok - t0) * 512), wave, lane,
                  512);
  tl.sb.panel = (uint32_t)a.m_tok * 512;
  tl.sb.first = s * sh.steps;
  if constexpr (TN == 256) {
    tl.start(st, wave, (int)vs);
    tl.run_wide(st, wave, lane, (int)vs);
  } else {
    tl.template run<TN == 128 && TM == 128 ? 2 : 3>(st, wave, lane, (int)vs);
  }
  lane = lane_again();
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, g = lane >> 4;
  // what earlier ranges left is loaded a column tile ahead of the stores (a
  // load waits for every store before it)
  auto at = [&](int j, int i) -> v4f* {
    const int t = t0 + wn * (TN / WN) + 16 * j + r, d = dt * TM + wm * (TM / WM) + 16 * i + 4 * g;
    return t < count && d < a.k ? reinterpret_cast<v4f*>(a.part + (s * sh.rows + t) * a.k + d) : nullptr;
  };
  constexpr int kHalf = T::kMT / 2;
  v4f old[2][kHalf];
  auto load = [&](int n) {                 // half a column tile
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      old[n & 1][i] = v4f{0.f, 0.f, 0.f, 0.f};
      const v4f* p = at(n / 2, (n & 1) * kHalf + i);
      if (p) old[n & 1][i] = *p;
    }
  };
  if (a.add) load(0);
#pragma unroll
  for (int n = 0; n < 2 * T::kNT; ++n) {
    if (a.add && n + 1 < 2 * T::kNT) load(n + 1);
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      v4f x = tl.acc[(n & 1) * kHalf + i][n / 2];
      if (a.add) x += old[n & 1][i];
      v4f* p = at(n / 2, (n & 1) * kHalf + i);
      if (p) *p = x;
    }
  }
}

__device__ __forceinline__ Shares all_rows(const HiddenGradArgs& a, int tn) {
  return Shares{a.splits, a.split_steps, (a.m_tok + tn - 1) / tn, a.m_tok};
}

// This XCD's run of n tiles (workgroups go to the 8 XCDs in turn).
__device__ __forceinline__ int xcd_share(int n, int& first) {
  const int x = blockIdx.x & 7, per = (n + 7) / 8;
  first = x * per < n ? x * per : n;
  return n - first < per ? n - first : per;
}

// More than 128 tokens: both gradients of a range in one launch (either may be
// absent), so that one's last, part empty round is filled by the other.  Each
// XCD takes a contiguous run of each kind's tiles, the hidden gradient's, the
// longer ones, first.  (Taking the two in turn costs a quarter more time:
// workgroups of one kind run in step and share operands in L2.)  Of 256 registers
// one is spilled (8 bytes of scratch per lane).
template <class E>
__global__ __launch_bounds__(512, 2) void grads_wide_kernel(const WeightGradArgs w, const HiddenGradArgs h, int n_w,
                                                            int n_h) {
  __shared__ __align__(16) uint8_t lds0[512 * kBK * 2];
  __shared__ __align__(16) uint8_t lds1[512 * kBK * 2];
  uint8_t* const st[2] = {lds0, lds1};
  const int i = blockIdx.x >> 3;
  int w0, h0;
  const int nw = xcd_share(n_w, w0), nh = xcd_share(n_h, h0);
  if (i < nh)
    hidden_grad_tile<E, 256, 256, 2, 4>(h, all_rows(h, 256), h0 + i, st);
  else if (i < nh + nw)
    weight_grad_tile<E, 256, 256, 2, 4>(w, w0 + i - nh, st);
}

// One of the gradients on smaller tiles.
template <class E>
__global__ __launch_bounds__(256, 2) void weight_grad_kernel(const WeightGradArgs a) {
  __shared__ __align__(16) uint8_t lds0[256 * kBK * 2];
  __shared__ __align__(16) uint8_t lds1[256 * kBK * 2];
  uint8_t* const st[2] = {lds0, lds1};
  weight_grad_tile<E, 128, 128, 2, 2>(a, xcd_tile(blockIdx.x, gridDim.x), st);
}

template <class E, int TM, int TN>
__global__ __launch_bounds__(TM == 256 ? 512 : 256, 2) void hidden_grad_kernel(const HiddenGradArgs a) {
  constexpr int kStage = (TM + TN) * kBK * 2;
  __shared__ __align__(16) uint8_t lds0[kStage];
  __shared__ __align__(16) uint8_t lds1[kStage];
  __shared__ __align__(16) uint8_t lds2[kStage];
  uint8_t* const st[3] = {lds0, lds1, lds2};
  const Shares sh = hidden_shares(a.splits, a.range_steps, a.m_tok, TN, a.hdr->count);
  const int n = sh.splits * sh.tiles * ((a.k + TM - 1) / TM);      // at most the grid's
  if (blockIdx.x < n) hidden_grad_tile<E, TM, TN, TM / 64, 2>(a, sh, xcd_tile(blockIdx.x, n), st);
}

// Few tokens: dw of 128 features and `run` tiles of 128 ids.  All of its k, the
// 2 kHalf token rows, lies in LDS: the hidden states for the whole run, the logit
// gradients of one tile.  The next tile's are asked for before this one's dw is
// stored, so that stores are under way all the time.
template <class E, int kHalf, int kPolicy>
__device__ __forceinline__ void weight_grad_run(const WeightGradArgs& a, int tile, int run, uint8_t* la, uint8_t* lb) {
  using T = Tile<E, kCols, kCols, 128, 128, 2, 2, false>;
  constexpr int kSteps = 2 * kHalf / kBK;
  const int ndt = (a.k + 127) / 128, nvt = (a.n_vocab + 127) / 128;
  const int dt = tile % ndt, v0 = tile / ndt * run, v1 = v0 + run < nvt ? v0 + run : nvt;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / 2, wn = wave % 2, r = lane & 15, g = lane >> 4;
  const float down = a.hdr->down;
  T tl;
  tl.sa.init_cols(make_rsrc(a.h, (int64_t)a.rows * a.k * 2), wave, lane, 2 * a.k, 256 * dt);
  auto fetch_dz = [&](int vt) {
    tl.sb.init_cols(make_rsrc(a.dz + (int64_t)(vt / 2) * a.m_tok * 256, (int64_t)a.rows * 512), wave, lane, 512,
                    256 * (vt & 1));
#pragma unroll
    for (int s = 0; s < kSteps; ++s) tl.sb.fetch(lb + s * 128 * kBK * 2, wave, s, a.rows);
  };
#pragma unroll
  for (int s = 0; s < kSteps; ++s) tl.sa.fetch(la + s * T::kBytesA, wave, s, a.rows);
  fetch_dz(v0);
  wait_vm<0>();
  wave_barrier();
  const int d0 = dt * 128 + wm * 64 + ((g & 1) ? 16 + 4 * (g - 1) : 4 * g);   // as in weight_grad_tile
  for (int vt = v0; vt < v1; ++vt) {
    tl.template products<kSteps>(la, lb, wave, lane);
    wave_barrier();                        // every wave has read this tile's gradients
    if (vt + 1 < v1) fetch_dz(vt + 1);
    const int64_t left = a.n_vocab - (int64_t)vt * 128;
    const __amdgpu_buffer_rsrc_t out = make_rsrc(a.dw + (int64_t)vt * 128 * a.k, (left < 128 ? left : 128) * a.k * 2);
    // exactly 8 stores, those past an end dropped: the wait below counts them
#pragma unroll
    for (int j = 0; j < T::kNT; ++j)
#pragma unroll
      for (int i = 0; i < T::kMT; i += 2) {
        const v4f x = tl.acc[i][j] * down, y = tl.acc[i + 1][j] * down;
        const auto lo = __builtin_amdgcn_permlane16_swap(E::pack2(x[0], x[1]), E::pack2(y[0], y[1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(E::pack2(x[2], x[3]), E::pack2(y[2], y[3]), false, false);
        const int d = d0 + 16 * i;
        const uint32_t at = (uint32_t)(wn * 64 + 16 * j + r) * (2u * a.k) + 2u * d;
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], hi[0], lo[1], hi[1]}, out, d < a.k ? at : kFar, 0, kPolicy);
      }
    if (vt + 1 < v1) {
      wait_vm<8>();                        // the next tile's gradients, asked for before the 8 stores
      wave_barrier();
    }
  }
}

// Both gradients of few tokens, bound by memory: dh by its reads of w, dw by its
// writes.  One dh tile of 2 kHalf token rows holds both parts of every logit
// gradient, so w is read once; two workgroups per CU.  Each XCD takes a contiguous
// run of dh's tiles, then one of dw's: reads and writes at the same time cost more
// than one after the other (30 x 128256 x 4096: 193 us and 283, 565 on
// alternating workgroups; 37 x 32003 x 1536 in all 90 -> 76).
template <class E, int kHalf, int kPolicy>
__global__ __launch_bounds__(256, 2) void grads_kernel(const WeightGradArgs w, const HiddenGradArgs h, int n_dw, int n_dh,
                                                       int run) {
  constexpr int kStage = (128 + 2 * kHalf) * kBK * 2;      // of dh, and at least either operand of dw
  __shared__ __align__(16) uint8_t lds0[kStage];
  __shared__ __align__(16) uint8_t lds1[kStage];
  const int i = blockIdx.x >> 3;
  int w0, h0;
  const int nw = xcd_share(n_dw, w0), nh = xcd_share(n_dh, h0);
  if (i >= nh + nw) return;
  const bool is_dw = i >= nh;
  const int tile = is_dw ? w0 + i - nh : h0 + i;
  if constexpr (kHalf == 32) {
    __shared__ __align__(16) uint8_t lds2[kStage];
    uint8_t* const st[3] = {lds0, lds1, lds2};
    if (is_dw)
      weight_grad_run<E, kHalf, kPolicy>(w, tile, run, lds0, lds1);
    else
      hidden_grad_tile<E, 128, 2 * kHalf, 2, 2>(h, all_rows(h, 2 * kHalf), tile, st);
  } else {
    uint8_t* const st[2] = {lds0, lds1};
    if (is_dw)
      weight_grad_run<E, kHalf, kPolicy>(w, tile, run, lds0, lds1);
    else
      hidden_grad_tile<E, 128, 2 * kHalf, 2, 2>(h, all_rows(h, 2 * kHalf), tile, st);
  }
}

// One workgroup per token and 256 features: 64 threads of 4 features x 4 groups
// of shares.
template <class E>
__global__ __launch_bounds__(256) void hidden_final_kernel(const float* part, const HiddenPlan plan, int range_steps,
                                                           const Header* hdr, const int32_t* rows, int32_t m_tok,
                                                           int32_t k, uint16_t* dh) {
  __shared__ v4f joined[4][64];
  const int t = blockIdx.x;
  const int count = hdr->count;
  if (t >= count) return;
  int splits = plan.splits;
  int64_t each = m_tok;
  if (plan.token_tile > 0) {
    const Shares sh = hidden_shares(splits, range_steps, m_tok, plan.token_tile, count);
    splits = sh.splits;
    each = sh.rows;
  }
  const int q = threadIdx.x >> 6, lane = threadIdx.x & 63, d = 4 * (blockIdx.y * 64 + lane);
  const bool in = d < k;
  v4f x = v4f{0.f, 0.f, 0.f, 0.f};
  if (in) {
    const float* p = part + (int64_t)t * k + d;
    const int64_t next = each * k;
#pragma unroll 4
    for (int s = q; s < splits; s += 4) x += *reinterpret_cast<const v4f*>(p + s * next);
  }
  joined[q][lane] = x;
  __syncthreads();
  if (q != 0 || !in) return;
  const float down = hdr->down;
  x = ((joined[0][lane] + joined[1][lane]) + (joined[2][lane] + joined[3][lane])) * down;
  *reinterpret_cast<uint2*>(dh + (int64_t)rows[t] * k + d) = uint2{E::pack2(x[0], x[1]), E::pack2(x[2], x[3])};
}

// ---------------------------------------------------------------- variants
// Which tiles a product runs on.  Wide tiles (256 x 256) do most per byte moved,
// but a chip of 256 CUs wants as many tiles; small ones fill it from small
// products, fit ragged sizes, and share a CU two at a time.  The cost of a
// variant, in microseconds: rounds of its workgroups (one or two per CU) times
// its steps of 64 k and what it spends before and after them.  Steps as
// measured with every CU at work: logits 256 x 256 1.5, 256 x 128 1.0, 128 x 64
// 0.75 (two per CU; 0.52 alone), 128 x 32 0.5 (0.44); so 512 x 32000 x 3200
// takes 94 us on the first and 101, 129 and 190 on the others, 559 x 1500 x
// 6264 takes 134, 101, 50 and 43.
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct LogitsTile {
  int tm, tn;
};

LogitsTile logits_variant(int64_t m_tok, int64_t n_vocab, int64_t k) {
  const struct {
    LogitsTile tile;
    int per_cu;
    float step, alone, more;
  } all[] = {{{256, 256}, 1, 1.5f, 1.5f, 5.0f},
             {{256, 128}, 1, 1.0f, 1.0f, 3.5f},
             {{128, 64}, 2, 0.75f, 0.52f, 3.0f},
             {{128, 32}, 2, 0.5f, 0.44f, 2.5f}};
  LogitsTile best = all[0].tile;
  float least = 1e30f;
  for (const auto& v : all) {
    const int64_t tiles = ceil_div(n_vocab, v.tile.tm) * ceil_div(m_tok, v.tile.tn);
    const float steps = (float)ceil_div(k, kBK);
    const float cost = tiles <= 256 ? steps * v.alone + v.more
                                    : (float)ceil_div(tiles, 256 * v.per_cu) * (steps * v.step + v.more);
    if (cost < least) {
      least = cost;
      best = v.tile;
    }
  }
  return best;
}

// The gradients of one range: tiles of dw (256 x 256 or 128 x 128), of dh
// (features x tokens), and shares of the vocabulary per dh tile.  A share's
// partial sums are written and read once more (8 bytes per value, 4.5 TB/s).
// Wide tiles of both go in one launch, whose last rounds then fill each other:
// half a tile is lost at its end, not two.  Measured at 2048 x 32000 x 3200:
// dw 362 us wide, 435 narrow; dh 433 wide, 424 on 256 x 128, 632 on 128 x 64;
// both wide together 703.  At 263 x 867 x 352: dw 11.8 and 5.5; dh 16.9, 9.1
// and 5.1.
struct GradPlan {
  bool few;                                // at most kFewTokens: grads_kernel
  bool wide_w;
  int hd, ht;                              // dh tile
  int splits;
};

GradPlan grad_plan(int64_t m_tok, int64_t n_vocab, int64_t k) {
  const int64_t steps_w = ceil_div(m_tok, kBK), steps_h = ceil_div(n_vocab, kBK);
  GradPlan p{};
  if (m_tok <= kFewTokens) {
    // two workgroups per CU or so, 4 steps each at least
    const int64_t tiles = ceil_div(k, 128);
    int64_t s = ceil_div(512, tiles);
    if (s > steps_h / 4) s = steps_h / 4;
    return GradPlan{true, false, 128, 2 * few_half(m_tok), s < 1 ? 1 : (int)s};
  }
  auto sums = [&](int64_t s) { return (float)(s * m_tok * k) * 8 / 4.5e6f; };
  const int64_t tiles_w = ceil_div(k, 256) * ceil_div(n_vocab, 256);
  const float wide_w = (float)ceil_div(tiles_w, 256) * (steps_w * 1.45f + 7);
  const float narrow_w = (float)ceil_div(ceil_div(k, 128) * ceil_div(n_vocab, 128), 512) * (steps_w * 0.95f + 3.5f);
  const struct {
    int hd, ht, slots;
    float step, more;
  } all[] = {{256, 256, 256, 1.45f, 8}, {256, 128, 256, 0.82f, 4}, {128, 64, 512, 0.65f, 4}};
  float least = 1e30f;
  for (const auto& v : all) {
    const int64_t tiles = ceil_div(k, v.hd) * ceil_div(m_tok, v.ht);
    for (int64_t s = 1; s <= 256 && (s == 1 || s * 4 <= steps_h); ++s) {
      const float each = ceil_div(steps_h, s) * v.step + v.more;
      const float alone = (float)ceil_div(tiles * s, v.slots) * each + sums(s);
      const float w = wide_w < narrow_w ? wide_w : narrow_w;
      if (alone + w + 3 < least) {         // 3: one launch more
        least = alone + w + 3;
        p = GradPlan{false, wide_w < narrow_w, v.hd, v.ht, (int)s};
      }
      if (v.ht == 256) {
        const float each_w = steps_w * 1.45f + 7, longest = each > each_w ? each : each_w;
        float both = (tiles_w * each_w + tiles * s * each) / 256 + (tiles * s < 256 ? longest : each_w) / 2;
        both = (both > longest ? both : longest) + sums(s) + 3;   // 3: the larger kernel's start
        if (both < least) {
          least = both;
          p = GradPlan{false, true, v.hd, v.ht, (int)s};
        }
      }
    }
  }
  return p;
}

// Whether an array of the weights' size is more than stays in the caches (256 MB
// in all): then what is used once goes past them.  One token's forward over 205 MB
// 42 -> 37 us; 88 MB read again and again from the cache 21 -> 27 us.  dw of 1.05 GB
// from 30 tokens 524 -> 469 us with its logits, of 98 MB 41 -> 50.
bool past_cache(int64_t n_vocab, int64_t k) { return n_vocab * k * 2 > (int64_t(128) << 20); }

// Threads of one launch stay below 2^32 (past that a grid is cut short, without an
// error); a product of more takes several.
constexpr int64_t kLaunchTiles = int64_t(1) << 22;

template <class E, bool kBackward>
hipError_t logits(LogitsArgs a, hipStream_t s) {
  const LogitsTile t = logits_variant(a.m_tok, a.n_vocab, a.k);
  const int64_t tiles = ceil_div(a.n_vocab, t.tm) * ceil_div(a.m_tok, t.tn);
  const bool once = a.m_tok <= t.tn && (kBackward ? past_cache(a.n_vocab / 2, a.k) : past_cache(a.n_vocab, a.k));
  for (int64_t first = 0; first < tiles; first += kLaunchTiles) {
    const dim3 grid((unsigned)(tiles - first < kLaunchTiles ? tiles - first : kLaunchTiles));
    a.tile0 = (int32_t)first;
    if (t.tn == 32 && once)
      logits_kernel<E, 128, 32, 4, 1, kBackward, kNt><<<grid, 256, 0, s>>>(a);
    else if (t.tn == 64 && once)
      logits_kernel<E, 128, 64, 4, 1, kBackward, kNt><<<grid, 256, 0, s>>>(a);
    else if (t.tn == 32)
      logits_kernel<E, 128, 32, 4, 1, kBackward><<<grid, 256, 0, s>>>(a);
    else if (t.tn == 64)
      logits_kernel<E, 128, 64, 4, 1, kBackward><<<grid, 256, 0, s>>>(a);
    else if (t.tn == 128)
      logits_kernel<E, 256, 128, 4, 2, kBackward><<<grid, 512, 0, s>>>(a);
    else
      logits_kernel<E, 256, 256, 2, 4, kBackward><<<grid, 512, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

constexpr int64_t kRunMax = 8;

// n_vocab of w and h is this range's; the plan is that of a whole range
template <class E>
hipError_t grads(const WeightGradArgs& w, const HiddenGradArgs& h, const GradPlan& p, hipStream_t s) {
  const int tw = p.few || !p.wide_w ? 128 : 256;
  const unsigned n_w = w.dw ? (unsigned)(ceil_div(w.k, tw) * ceil_div(w.n_vocab, tw)) : 0;
  const unsigned n_h = h.part ? (unsigned)(ceil_div(h.k, p.hd) * ceil_div(h.m_tok, p.ht) * p.splits) : 0;
  if (p.few) {
    // tiles of dw that a workgroup takes one after the other: a launch of few tiles takes them side by side
    int64_t run = n_w / 1024;
    run = run < 1 ? 1 : run > kRunMax ? kRunMax : run;
    const int64_t runs = w.dw ? ceil_div(w.k, 128) * ceil_div(ceil_div(w.n_vocab, 128), run) : 0;
    const dim3 grid((unsigned)(8 * (ceil_div(runs, 8) + ceil_div(n_h, 8))));
    // stores go past the caches only as whole 128-byte lines: parts of lines from two
    // workgroups would reach memory one by one (1 x 124987 x 2312: 508 -> 711 us)
    const bool once = past_cache(w.n_vocab, w.k) && w.k % 64 == 0;
    if (p.ht == 64 && once)
      grads_kernel<E, 32, kNt><<<grid, 256, 0, s>>>(w, h, (int)runs, (int)n_h, (int)run);
    else if (p.ht == 64)
      grads_kernel<E, 32, 0><<<grid, 256, 0, s>>>(w, h, (int)runs, (int)n_h, (int)run);
    else if (once)
      grads_kernel<E, 64, kNt><<<grid, 256, 0, s>>>(w, h, (int)runs, (int)n_h, (int)run);
    else
      grads_kernel<E, 64, 0><<<grid, 256, 0, s>>>(w, h, (int)runs, (int)n_h, (int)run);
    return hipGetLastError();
  }
  if (p.ht == 256 && (p.wide_w || n_w == 0)) {
    grads_wide_kernel<E><<<dim3(8 * ((n_w + 7) / 8 + (n_h + 7) / 8)), 512, 0, s>>>(w, h, n_w, n_h);
    return hipGetLastError();
  }
  if (n_w > 0) {
    const HiddenGradArgs none{};
    if (p.wide_w)
      grads_wide_kernel<E><<<dim3(8 * ((n_w + 7) / 8)), 512, 0, s>>>(w, none, n_w, 0);
    else
      weight_grad_kernel<E><<<dim3(n_w), 256, 0, s>>>(w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (n_h > 0) {
    const WeightGradArgs none{};
    if (p.ht == 256)
      grads_wide_kernel<E><<<dim3(8 * ((n_h + 7) / 8)), 512, 0, s>>>(none, h, 0, n_h);
    else if (p.ht == 128)
      hidden_grad_kernel<E, 256, 128><<<dim3(n_h), 512, 0, s>>>(h);
    else
      hidden_grad_kernel<E, 128, 64><<<dim3(n_h), 256, 0, s>>>(h);
  }
  return hipGetLastError();
}

}  // namespace

int64_t logits_tiles(int32_t m_tok, int32_t n_vocab, int32_t k) {
  return m_tok < 1 ? 1 : ceil_div(n_vocab, logits_variant(m_tok, n_vocab, k).tm);
}

hipError_t launch_logits(const LogitsArgs& a, bool fp16, bool backward, hipStream_t s) {
  if (fp16) return backward ? logits<Fp16, true>(a, s) : logits<Fp16, false>(a, s);
  return backward ? logits<Bf16, true>(a, s) : logits<Bf16, false>(a, s);
}

HiddenPlan hidden_plan(int32_t m_tok, int32_t n_vocab, int32_t k) {
  if (m_tok < 1) return HiddenPlan{1, 0};
  const GradPlan p = grad_plan(m_tok, n_vocab, k);
  return HiddenPlan{p.splits, p.few || p.ht == 256 ? 0 : p.ht};
}

hipError_t launch_grads(const WeightGradArgs& w, const HiddenGradArgs& h, int32_t m_tok, int32_t range, bool fp16,
                        hipStream_t s) {
  const GradPlan p = grad_plan(m_tok, range, w.k);
  return fp16 ? grads<Fp16>(w, h, p, s) : grads<Bf16>(w, h, p, s);
}

hipError_t launch_hidden_final(const float* part, const HiddenPlan& plan, int32_t range_steps, const Header* hdr,
                               const int32_t* rows, int32_t m_tok, int32_t k, uint16_t* dh, bool fp16, hipStream_t s) {
  const dim3 grid((unsigned)m_tok, (unsigned)((k + 255) / 256));
  if (fp16)
    hidden_final_kernel<Fp16><<<grid, 256, 0, s>>>(part, plan, range_steps, hdr, rows, m_tok, k, dh);
  else
    hidden_final_kernel<Bf16><<<grid, 256, 0, s>>>(part, plan, range_steps, hdr, rows, m_tok, k, dh);
  return hipGetLastError();
}

}  // namespace head
}  // namespace sbl
