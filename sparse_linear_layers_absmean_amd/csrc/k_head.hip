// Matrix products of the output head's losses: logits that are used where
// they are made and never stored, and the two gradients.
//
//   z[t][v] = sum_d h[t][d] w[v][d]
//   forward   per token: max and sum of 2^(z scale) over each 128 ids (or
//             fewer), joined later, and z at the token's listed ids
//   backward  dz[t][v] = coef[t] 2^(z scale - lse2[t]) - sub at the listed ids,
//             rounded once to 16 bits, a range of the vocabulary at a time;
//             dw = dz^T h, dh = dz w
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

// ---------------------------------------------------------------- logits
// Rows of the tile (MFMA rows) are vocabulary entries, columns are tokens: a
// lane holds one token's logits of 4 consecutive ids per 16-row tile, and with
// the permuted row order 8 consecutive ids per pair of tiles, so softmax
// statistics reduce over registers and two lane exchanges, and the gradient
// leaves as 16-byte stores.
template <class E, int TM, int TN, int WM, int WN, bool kBackward>
__global__ __launch_bounds__(64 * WM * WN, 2) void logits_kernel(const LogitsArgs a) {
  using T = Tile<E, kRows, kRows, TM, TN, WM, WN, true, false, !kBackward>;
  __shared__ __align__(16) uint8_t lds0[T::kStageBytes];
  __shared__ __align__(16) uint8_t lds1[T::kStageBytes];
  __shared__ __align__(16) uint8_t lds2[TN == 256 ? 16 : T::kStageBytes];
  __shared__ int32_t row_of[TN];           // original row of each of the tile's tokens, -1: none
  const int count = a.hdr ? a.hdr->count : a.m_tok;
  const int nvt = (a.n_vocab + TM - 1) / TM, ntt = (a.m_tok + TN - 1) / TN;
  // groups of kGroup vocabulary tiles x every token tile
  constexpr int kGroup = 4;
  const int tile = xcd_tile(blockIdx.x, gridDim.x);
  const int group = tile / (kGroup * ntt), in_group = tile % (kGroup * ntt);
  const int gv = nvt - group * kGroup < kGroup ? nvt - group * kGroup : kGroup;
  const int vt = group * kGroup + in_group % gv, tt = in_group / gv;
  const int t0 = tt * TN;
  if (t0 >= count) return;
  const int64_t vt0 = (int64_t)vt * TM;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int lane = tid & 63;
  for (int i = tid; i < TN; i += T::kThreads) {
    const int t = t0 + i;
    row_of[i] = t < count ? (a.rows ? a.rows[t] : t) : -1;
  }
  __syncthreads();

  T tl;
  const int64_t wrows = a.n_vocab - vt0 < TM ? a.n_vocab - vt0 : TM;
  tl.sa.init_rows(make_rsrc(a.w + vt0 * a.k, wrows * a.k * 2), wave, lane, 2 * a.k);
  if constexpr (kBackward)
    tl.sb.init_rows(make_rsrc(a.h + (int64_t)t0 * a.k, (int64_t)(count - t0) * a.k * 2), wave, lane, 2 * a.k);
  else
    tl.sb.init_list(make_rsrc(a.h, ((a.h_rows - 1) * a.h_stride + a.k) * 2), wave, lane, [&](int r) {
      const int row = row_of[r];
      return row < 0 ? kFar : (uint32_t)((int64_t)row * a.h_stride * 2);
    });
  if constexpr (TN == 256) {
    uint8_t* const st[2] = {lds0, lds1};
    tl.run_wide(st, wave, lane, a.k);
  } else {
    uint8_t* const st[3] = {lds0, lds1, lds2};
    tl.template run<3>(st, wave, lane, a.k);
  }

  const int wm = wave / WN, wn = wave % WN;
  lane = lane_again();
  const int r = lane & 15, g = lane >> 4;
  constexpr int kMT = T::kMT, kNT = T::kNT, kRowsW = TM / WM, kColsW = TN / WN;
  const int vw = (int)vt0 + wm * kRowsW;   // first id (in this range) of the wave's rows
  const bool tail = vw + kRowsW > a.n_vocab;
  // id of tl.acc[i][.][e] less vw
  auto id_of = [&](int i, int e) { return 32 * (i >> 1) + 8 * g + 4 * (i & 1) + e; };

#pragma unroll
  for (int j = 0; j < kNT; ++j) {
    const int tw = wn * kColsW + 16 * j + r;
    const int t = t0 + tw;
    if constexpr (!kBackward) {
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = tl.acc[i][j][e] * a.scale;
          if (tail && vw + id_of(i, e) >= a.n_vocab) x = -__builtin_inff();
          tl.acc[i][j][e] = x;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float ref = mx == -__builtin_inff() ? 0.f : mx;   // no finite logit here: a sum of zeros
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f(tl.acc[i][j][e] - ref);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0 && t < count && vw < a.n_vocab) {
        const int64_t o = (int64_t)t * a.np + vw / kRowsW;
        a.part_max[o] = mx;
        a.part_sum[o] = sum;
      }
    } else {
      const bool in = t < count;
      const float lse2 = in ? a.lse2[t] : 0.f, coef = in ? a.coef[t] : 0.f;
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = coef * __builtin_amdgcn_exp2f(__builtin_fmaf(tl.acc[i][j][e], a.scale, -lse2));
          if (tail && vw + id_of(i, e) >= a.n_vocab) p = 0.f;
          tl.acc[i][j][e] = p;
        }
      if (in) {
        uint16_t* o = a.dz + (int64_t)t * a.ldz + vw + 8 * g;
#pragma unroll
        for (int i = 0; i < kMT; i += 2) {
          const v4f x = tl.acc[i][j], y = tl.acc[i + 1][j];
          *reinterpret_cast<u32x4*>(o + 16 * i) =
              u32x4{E::pack2(x[0], x[1]), E::pack2(x[2], x[3]), E::pack2(y[0], y[1]), E::pack2(y[2], y[3])};
        }
      }
    }
  }

  // The listed ids that fall on this wave's rows and columns, 64 entries at a
  // time: the wave finds them by ballot, then takes them one by one (a
  // wave-uniform walk to the accumulator, a handful per tile).  Forward: the
  // scaled logit.  Backward: the lane that stored the id's gradient stores it
  // again with the listed part taken off, still from 32 bits.
  const int entries = kColsW * a.top;
  const int step_t = 64 / a.top, step_k = 64 % a.top;
  int et = lane / a.top, ek = lane % a.top;
  for (int e0 = 0; e0 < entries; e0 += 64) {
    const int tw = wn * kColsW + et;
    int rel = -1;
    int64_t slot = 0;
    if (et < kColsW && t0 + tw < count) {
      const int64_t t = t0 + tw;
      slot = t * a.top + ek;
      const int64_t id = kBackward ? (int64_t)a.index32[slot] - a.v0
                                   : a.index[(int64_t)row_of[tw] * a.top + ek];
      const int64_t d = id - vw;
      if (d >= 0 && d < kRowsW) rel = (int)d;
    }
    uint64_t hits = __ballot(rel >= 0);
    while (hits) {
      const int src = __builtin_ctzll(hits);
      hits &= hits - 1;
      const int hr = __builtin_amdgcn_readlane(rel, src), ht = __builtin_amdgcn_readlane(et, src);
      const int64_t hs = (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(slot >> 32), src) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)slot, src));
      const int hi = 2 * (hr >> 5) + ((hr >> 2) & 1), hj = ht >> 4, he = hr & 3;
      float val = 0.f;
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
      if (r == (ht & 15) && g == ((hr >> 3) & 3)) {
        if constexpr (!kBackward) {
          a.zlist[hs] = val;
        } else {
          const uint32_t o = E::pack2(val - a.sub[hs], 0.f);
          a.dz[(int64_t)(t0 + wn * kColsW + ht) * a.ldz + vw + hr] = (uint16_t)o;
        }
      }
    }
    et += step_t;
    ek += step_k;
    if (ek >= a.top) {
      ek -= a.top;
      ++et;
    }
  }
}

// ---------------------------------------------------------------- gradients
// Rows of the tile are features (contiguous in memory, read down the k axis),
// so a lane's 4 consecutive results are 4 consecutive features of an output row.

template <class E>
__global__ __launch_bounds__(512, 2) void weight_grad_kernel(const WeightGradArgs a) {
  using T = Tile<E, kCols, kCols, 256, 256, 2, 4, false>;
  __shared__ __align__(16) uint8_t lds0[T::kStageBytes];
  __shared__ __align__(16) uint8_t lds1[T::kStageBytes];
  const int count = a.hdr->count;
  const int ndt = (a.k + 255) / 256;
  const int nvt = (a.n_vocab + 255) / 256;
  constexpr int kGroup = 4;
  const int tile = xcd_tile(blockIdx.x, gridDim.x);
  const int group = tile / (kGroup * ndt), in_group = tile % (kGroup * ndt);
  const int gv = nvt - group * kGroup < kGroup ? nvt - group * kGroup : kGroup;
  const int vt = group * kGroup + in_group % gv, dt = in_group / gv;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int lane = tid & 63;
  T tl;
  tl.sa.init_cols(make_rsrc(a.h, (int64_t)count * a.k * 2), wave, lane, 2 * a.k, 512 * dt);
  tl.sb.init_cols(make_rsrc(a.dz, (int64_t)count * a.ldz * 2), wave, lane, 2 * a.ldz, 512 * vt);
  uint8_t* const st[2] = {lds0, lds1};
  tl.run_wide(st, wave, lane, count);
  lane = lane_again();
  const int wm = wave / 4, wn = wave % 4, r = lane & 15, g = lane >> 4;
  const float down = a.hdr->down;
#pragma unroll
  for (int j = 0; j < T::kNT; ++j) {
    const int v = vt * 256 + wn * 64 + 16 * j + r;
    if (v >= a.n_vocab) continue;
    uint16_t* o = a.dw + (int64_t)v * a.k;
#pragma unroll
    for (int i = 0; i < T::kMT; ++i) {
      const int d = dt * 256 + wm * 128 + 16 * i + 4 * g;
      const v4f x = tl.acc[i][j];
      if (d < a.k)
        *reinterpret_cast<uint2*>(o + d) = uint2{E::pack2(x[0] * down, x[1] * down), E::pack2(x[2] * down, x[3] * down)};
    }
  }
}

template <class E, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, TN == 256 ? 2 : 1) void hidden_grad_kernel(const HiddenGradArgs a) {
  using T = Tile<E, kCols, kRows, 256, TN, WM, WN, false, WM * WN == 4>;
  __shared__ __align__(16) uint8_t lds0[T::kStageBytes];
  __shared__ __align__(16) uint8_t lds1[T::kStageBytes];
  __shared__ __align__(16) uint8_t lds2[TN == 256 ? 16 : T::kStageBytes];
  const int count = a.hdr->count;
  const int ndt = (a.k + 255) / 256, ntt = (a.m_tok + TN - 1) / TN;
  const int tile = xcd_tile(blockIdx.x, gridDim.x);
  // a share's tiles together: they read the same rows of w
  const int s = tile / (ndt * ntt), in = tile % (ndt * ntt);
  const int dt = in % ndt, t0 = in / ndt * TN;
  if (t0 >= count) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int lane = tid & 63;
  const int64_t v0 = (int64_t)s * a.split_steps * kBK;
  int64_t vs = a.n_vocab - v0;
  if (vs > (int64_t)a.split_steps * kBK) vs = (int64_t)a.split_steps * kBK;
  if (vs < 0) vs = 0;
  T tl;
  tl.sa.init_cols(make_rsrc(a.w + v0 * a.k, vs * a.k * 2), wave, lane, 2 * a.k, 512 * dt);
  tl.sb.init_rows(make_rsrc(a.dz + (int64_t)t0 * a.ldz + v0, ((int64_t)(count - t0) * a.ldz - v0) * 2), wave, lane,
                  2 * a.ldz);
  if constexpr (TN == 256) {
    uint8_t* const st[2] = {lds0, lds1};
    tl.run_wide(st, wave, lane, (int)vs);
  } else {
    uint8_t* const st[3] = {lds0, lds1, lds2};
    tl.template run<3>(st, wave, lane, (int)vs);
  }
  lane = lane_again();
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < T::kNT; ++j) {
    const int t = t0 + wn * (TN / WN) + 16 * j + r;
    if (t >= count) continue;
    float* o = a.part + ((int64_t)s * a.m_tok + t) * a.k;
#pragma unroll
    for (int i = 0; i < T::kMT; ++i) {
      const int d = dt * 256 + wm * (256 / WM) + 16 * i + 4 * g;
      if (d < a.k) {
        v4f x = tl.acc[i][j];
        v4f* p = reinterpret_cast<v4f*>(o + d);
        if (a.add) x += *p;
        *p = x;
      }
    }
  }
}

template <class E>
__global__ __launch_bounds__(256) void hidden_final_kernel(const float* part, int splits, const Header* hdr,
                                                           const int32_t* rows, int32_t m_tok, int32_t k,
                                                           uint16_t* dh) {
  const int t = blockIdx.x;
  if (t >= hdr->count) return;
  const int d = 4 * (blockIdx.y * 256 + threadIdx.x);
  if (d >= k) return;
  const float down = hdr->down;
  v4f x = v4f{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) x += *reinterpret_cast<const v4f*>(part + ((int64_t)s * m_tok + t) * k + d);
  *reinterpret_cast<uint2*>(dh + (int64_t)rows[t] * k + d) =
      uint2{E::pack2(x[0] * down, x[1] * down), E::pack2(x[2] * down, x[3] * down)};
}

template <class E, bool kBackward>
hipError_t logits(const LogitsArgs& a, hipStream_t s) {
  auto grid = [&](int tm, int tn) {
    return dim3((unsigned)(((int64_t)a.n_vocab + tm - 1) / tm * ((a.m_tok + tn - 1) / tn)));
  };
  if (a.m_tok <= 32)
    logits_kernel<E, 128, 32, 4, 1, kBackward><<<grid(128, 32), 256, 0, s>>>(a);
  else if (a.m_tok <= 64)
    logits_kernel<E, 128, 64, 4, 1, kBackward><<<grid(128, 64), 256, 0, s>>>(a);
  else
    logits_kernel<E, 256, 256, 2, 4, kBackward><<<grid(256, 256), 512, 0, s>>>(a);
  return hipGetLastError();
}

template <class E>
hipError_t hidden_grad(const HiddenGradArgs& a, hipStream_t s) {
  auto grid = [&](int tn) { return dim3((unsigned)((a.k + 255) / 256 * ((a.m_tok + tn - 1) / tn) * a.splits)); };
  if (a.m_tok <= 64)
    hidden_grad_kernel<E, 64, 4, 1><<<grid(64), 256, 0, s>>>(a);
  else
    hidden_grad_kernel<E, 256, 2, 4><<<grid(256), 512, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// every variant of the logits kernel leaves one statistic per wave's rows:
// 32 ids for the narrow tiles (4 waves over 128), 128 for the wide one
int64_t logits_tiles(int32_t m_tok, int32_t n_vocab) {
  const int rows = m_tok <= 64 ? 32 : 128;
  return ((int64_t)n_vocab + rows - 1) / rows;
}

hipError_t launch_logits(const LogitsArgs& a, bool fp16, bool backward, hipStream_t s) {
  if (fp16) return backward ? logits<Fp16, true>(a, s) : logits<Fp16, false>(a, s);
  return backward ? logits<Bf16, true>(a, s) : logits<Bf16, false>(a, s);
}

hipError_t launch_weight_grad(const WeightGradArgs& a, bool fp16, hipStream_t s) {
  const dim3 grid((unsigned)((a.k + 255) / 256 * ((a.n_vocab + 255) / 256)));
  if (fp16)
    weight_grad_kernel<Fp16><<<grid, 512, 0, s>>>(a);
  else
    weight_grad_kernel<Bf16><<<grid, 512, 0, s>>>(a);
  return hipGetLastError();
}

// shares of the vocabulary per hidden-gradient tile: enough workgroups for
// every CU, at least 8 steps each
int hidden_splits(int32_t m_tok, int32_t n_vocab, int32_t k) {
  if (m_tok < 1) return 1;
  const int tn = m_tok <= 64 ? 64 : 256;
  const int64_t tiles = (int64_t)((k + 255) / 256) * ((m_tok + tn - 1) / tn);
  const int64_t steps = ((int64_t)n_vocab + kBK - 1) / kBK;
  int64_t s = tiles >= 1024 ? 1 : (1024 + tiles - 1) / tiles;
  if (s > steps / 8) s = steps / 8;
  return s < 1 ? 1 : (int)s;
}

hipError_t launch_hidden_grad(const HiddenGradArgs& a, bool fp16, hipStream_t s) {
  return fp16 ? hidden_grad<Fp16>(a, s) : hidden_grad<Bf16>(a, s);
}

hipError_t launch_hidden_final(const float* part, int splits, const Header* hdr, const int32_t* rows, int32_t m_tok,
                               int32_t k, uint16_t* dh, bool fp16, hipStream_t s) {
  const dim3 grid((unsigned)m_tok, (unsigned)((k + 1023) / 1024));
  if (fp16)
    hidden_final_kernel<Fp16><<<grid, 256, 0, s>>>(part, splits, hdr, rows, m_tok, k, dh);
  else
    hidden_final_kernel<Bf16><<<grid, 256, 0, s>>>(part, splits, hdr, rows, m_tok, k, dh);
  return hipGetLastError();
}

}  // namespace head
}  // namespace sbl
