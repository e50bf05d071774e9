// The per-token side of the output head's losses: which rows take part, the
// teacher's distribution, the joined softmax statistics and the loss, and for
// the backward each row's coefficients and a dense copy of its hidden state.
//
//   cross entropy  takes part: target >= 0
//   distillation   an entry counts when its index >= 0 and its teacher logit is
//                  not -infinity; takes part: any entry counts
// Only rows that take part are multiplied afterwards (up to 256 tokens the
// forward multiplies all: a row's products stay in its own column), so whatever
// a row that is taken out holds (NaN, infinities) reaches nothing.
#include "sbl_head.h"
#include "sbl_head_tile.h"

namespace sbl {
namespace head {

namespace {

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
  return x;
}

__device__ __forceinline__ bool counts(int64_t id, float teacher) {
  return id >= 0 && teacher != -__builtin_inff();
}

// What the logit gradients are divided by: the largest finite coefficient of any
// row; 1e-30 keeps the quotient finite when every one is zero (or next to it).
// A row whose coefficient is not finite (loss scaling that overflowed) has such
// gradients itself, and dw has, but it scales no other row.
__device__ __forceinline__ float scale_base(float top) { return fmaxf(top, 1e-30f); }
__device__ __forceinline__ float finite_size(float x) { return fabsf(x) < __builtin_inff() ? fabsf(x) : 0.f; }
__device__ __forceinline__ float row_size(const RowArgs& a, int64_t t) {
  const float g = a.dloss[t], top = finite_size(g * a.tau);
  return a.dlse ? fmaxf(top, finite_size((g + a.dlse[t]) * a.tau)) : top;
}

// Distillation: one wave per row, flag = takes part; forward: the blocks of the
// row's ids (near).  strict (backward): a row with an entry that counts and
// whose id is past the vocabulary does not (its loss is NaN, it has no gradient).
__global__ __launch_bounds__(256) void flag_kernel(const RowArgs a, bool strict) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.m_tok) return;
  bool any = false, bad = false;
  const int wide = (a.top + 7) / 8 * 8;
  for (int k = threadIdx.x & 63; k < wide; k += 64) {
    const int64_t id = k < a.top ? a.index[t * a.top + k] : -1;
    const bool here = k < a.top && counts(id, a.teacher[t * a.top + k]);
    any |= here;
    bad |= here && id >= a.n_vocab;
    if (a.near && !strict) a.near[t * wide + k] = id >= 0 && id < a.n_vocab ? (uint16_t)(id >> 8) : 0xFFFFu;
  }
  const bool in = __ballot(any) != 0 && !(strict && __ballot(bad) != 0);
  if ((threadIdx.x & 63) == 0) a.flag[t] = in;
}

// One workgroup: numbers the rows that take part, in order, and (backward)
// finds the largest coefficient.  A few microseconds at thousands of tokens.
__global__ __launch_bounds__(1024) void rows_kernel(const RowArgs a, bool backward) {
  __shared__ int32_t wave_count[16];
  __shared__ float wave_top[16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int32_t before = 0;
  float top = 0.f;
  for (int64_t t0 = 0; t0 < a.m_tok; t0 += 1024) {
    const int64_t t = t0 + tid;
    bool in = false;
    if (t < a.m_tok) in = a.target ? a.target[t] >= 0 && !(backward && a.target[t] >= a.n_vocab) : a.flag[t] != 0;
    const uint64_t m = __ballot(in);
    if (lane == 0) wave_count[wave] = __popcll(m);
    __syncthreads();
    int32_t at = before, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      at += w < wave ? wave_count[w] : 0;
      all += wave_count[w];
    }
    at += __popcll(m & ((1ull << lane) - 1));
    if (t < a.m_tok) a.pos[t] = in ? at : -1;
    if (in) {
      a.rows[at] = (int32_t)t;
      if (backward) top = fmaxf(top, row_size(a, t));
    }
    before += all;
    __syncthreads();
  }
  top = wave_max(top);
  if (lane == 0) wave_top[wave] = top;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < 16; ++w) top = fmaxf(top, wave_top[w]);
    a.hdr->count = before;
    const float amax = scale_base(top);
    a.hdr->amax = amax;
    a.hdr->down = amax / a.up;
  }
}

// The teacher's probability of this lane's entries (k = lane + 64 i) and its
// logarithm; p = 0 for entries that do not count.
constexpr int kPerLane = kMaxTop / 64;
__device__ __forceinline__ void teacher_row(const RowArgs& a, int64_t t, int lane, int64_t* id, float* p, float* logp) {
  float x[kPerLane], mx = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int k = lane + 64 * i;
    id[i] = -1;
    x[i] = -__builtin_inff();
    if (k < a.top) {
      const int64_t d = a.index[t * a.top + k];
      const float y = a.teacher[t * a.top + k];
      if (counts(d, y)) {
        id[i] = d;
        x[i] = y;
      }
    }
    mx = fmaxf(mx, x[i]);
  }
  mx = wave_max(mx);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    // the difference first: finite logits then never give inf - inf
    logp[i] = id[i] >= 0 ? (x[i] - mx) * a.inv_tau : 0.f;
    p[i] = id[i] >= 0 ? __builtin_amdgcn_exp2f(logp[i] * kLog2e) : 0.f;
    sum += p[i];
  }
  sum = wave_sum(sum);
  const float lsum = kLn2 * __builtin_amdgcn_logf(sum);
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    p[i] = id[i] >= 0 ? p[i] / sum : 0.f;
    logp[i] -= lsum;
  }
}

// Forward: joins the softmax statistics, takes the loss.  kWaves waves per row
// (one when there are rows enough to fill the chip) share the statistics; wave
// 0 does the rest.
template <int kWaves>
__global__ __launch_bounds__(256) void finish_kernel(const RowArgs a, bool compact) {
  __shared__ float2 joined[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = kWaves == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  if (t >= a.m_tok) return;                        // whole workgroups where waves share a row
  const int64_t c = compact ? a.pos[t] : t;
  const bool there = c >= 0;
  const float scale = kLog2e / a.tau;
  // what does not depend on the statistics comes first: its loads overlap theirs
  int64_t id[kPerLane];
  float p[kPerLane], logp[kPerLane], zl[kPerLane];
  bool in, bad = false;
  if (a.target) {
    const int64_t y = a.target[t];
    in = y >= 0;
    bad = y >= a.n_vocab;
    zl[0] = in && !bad && there ? a.zlist[c] : 0.f;
  } else {
    if (kWaves == 1 || wave == 0) teacher_row(a, t, lane, id, p, logp);
    bool any = false;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const bool mine = (kWaves == 1 || wave == 0) && id[i] >= 0;
      any |= mine;
      bad |= mine && id[i] >= a.n_vocab;
      zl[i] = mine && id[i] < a.n_vocab && there ? a.zlist[c * a.top + lane + 64 * i] : 0.f;
    }
    in = __ballot(any) != 0;
    bad = __ballot(bad) != 0;
  }
  // the statistics, 4 entries of a lane at a time
  float mx = -__builtin_inff(), sum = 0.f;
  if (there) {
    const float2* part = a.part + c * a.np;
    for (int i0 = kWaves == 1 ? lane : threadIdx.x; i0 < a.np; i0 += 256 * kWaves) {
      float2 x[4];
      float top = mx;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 64 * kWaves * u;
        x[u] = i < a.np ? part[i] : float2{-__builtin_inff(), 0.f};
        top = fmaxf(top, x[u].x);
      }
      const float ref = top == -__builtin_inff() ? 0.f : top;
      sum *= __builtin_amdgcn_exp2f((mx - ref) * scale);
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += x[u].y * __builtin_amdgcn_exp2f((x[u].x - ref) * scale);
      mx = top;
    }
  }
  const float own = mx;
  mx = wave_max(mx);
  sum = wave_sum(sum * __builtin_amdgcn_exp2f((own - (mx == -__builtin_inff() ? 0.f : mx)) * scale));
  if constexpr (kWaves > 1) {
    if (lane == 0) joined[wave] = float2{mx, sum};
    __syncthreads();
    if (wave > 0) return;
    float2 x = joined[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) x.x = fmaxf(x.x, joined[w].x);
    mx = x.x;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      sum += joined[w].y * __builtin_amdgcn_exp2f((joined[w].x - (mx == -__builtin_inff() ? 0.f : mx)) * scale);
  }
  if (!in) {
    if (lane == 0) {
      a.loss[t] = 0.f;
      a.lse[t] = 0.f;
    }
    return;
  }
  // the largest logit against the listed one first: what cancels is exact
  const float lsum = kLn2 * __builtin_amdgcn_logf(sum);
  float loss;
  if (a.target) {
    loss = bad ? 0.f : (mx - zl[0]) + lsum;
  } else {
    loss = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (!(p[i] == 0.f) && id[i] < a.n_vocab)             // not p > 0: a NaN teacher shows
        loss += p[i] * (logp[i] + ((mx - zl[i]) * a.inv_tau + lsum));
    loss = wave_sum(loss) * (a.tau * a.tau);
  }
  if (lane == 0) {
    a.loss[t] = bad ? __builtin_nanf("") : loss;
    a.lse[t] = mx * a.inv_tau + lsum;
  }
}

// Backward, one workgroup per original row: the row's place among those that
// take part gets its hidden state and coefficients; a row that does not take
// part gets a zero gradient.  kOwnRows: every workgroup finds its row's place
// and the scales by itself (few rows), which saves the launches before.
constexpr int kAloneRows = 1024;

template <bool kOwnRows>
__global__ __launch_bounds__(256) void gather_kernel(const RowArgs a) {
  __shared__ int32_t ids[kMaxTop];
  __shared__ float ps[kMaxTop];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  int c, pad = 0;                          // pad: the half's row that this workgroup zeroes if c < 0
  float amax;
  if constexpr (kOwnRows) {
    __shared__ int32_t before[4], all[4], here[4];
    __shared__ float tops[4];
    __shared__ int32_t any[kAloneRows], wrong[kAloneRows];
    if (!a.target) {                       // a thread per list entry
      for (int u = tid; u < a.m_tok; u += 256) any[u] = wrong[u] = 0;
      __syncthreads();
      const int entries = a.m_tok * a.top;
#pragma unroll 4
      for (int e = tid; e < entries; e += 256) {
        const int64_t id = a.index[e];
        if (!counts(id, a.teacher[e])) continue;
        any[e / a.top] = 1;
        if (id >= a.n_vocab) wrong[e / a.top] = 1;
      }
      __syncthreads();
    }
    int mine = 0, total = 0, self = 0;
    float top = 0.f;
    for (int64_t u = tid; u < a.m_tok; u += 256) {
      const bool in = a.target ? a.target[u] >= 0 && a.target[u] < a.n_vocab : any[u] && !wrong[u];
      if (!in) continue;
      top = fmaxf(top, row_size(a, u));
      ++total;
      mine += u < t;
      self |= u == t;
    }
    for (int m = 1; m < 64; m <<= 1) {
      mine += __shfl_xor(mine, m);
      total += __shfl_xor(total, m);
      self |= __shfl_xor(self, m);
    }
    top = wave_max(top);
    if ((tid & 63) == 0) {
      before[tid >> 6] = mine;
      all[tid >> 6] = total;
      here[tid >> 6] = self;
      tops[tid >> 6] = top;
    }
    __syncthreads();
    mine = before[0] + before[1] + before[2] + before[3];
    c = (here[0] | here[1] | here[2] | here[3]) ? mine : -1;
    pad = all[0] + all[1] + all[2] + all[3] + (int)(t - mine);
    amax = scale_base(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
    if (tid == 0) {
      if (c >= 0) a.rows[c] = (int32_t)t;
      if (t == 0) {
        a.hdr->count = all[0] + all[1] + all[2] + all[3];
        a.hdr->amax = amax;
        a.hdr->down = amax / a.up;
      }
    }
  } else {
    c = a.pos[t];
    amax = a.hdr->amax;
  }
  const int vecs = a.k / 8;
  if (c < 0) {
    if (kOwnRows && a.half > 0)
      for (int i = tid; i < 2 * vecs; i += 256)
        reinterpret_cast<u32x4*>(a.hc + (int64_t)(i < vecs ? pad : pad + a.half) * a.k)[i < vecs ? i : i - vecs] =
            u32x4{0, 0, 0, 0};
    if (a.dh && t < a.m_tok) {
      u32x4* o = reinterpret_cast<u32x4*>(a.dh + t * a.k);
      for (int i = tid; i < vecs; i += 256) o[i] = u32x4{0, 0, 0, 0};
    }
    return;
  }
  const u32x4* src = reinterpret_cast<const u32x4*>(a.h + t * a.h_stride);
  u32x4* dst = reinterpret_cast<u32x4*>(a.hc + (int64_t)c * a.k);
  for (int i = tid; i < vecs; i += 256) {
    dst[i] = src[i];
    if (kOwnRows && a.half > 0) dst[i + (int64_t)a.half * vecs] = src[i];
  }
  // divided by the largest finite coefficient first: equal weights give exactly 1
  const float g = a.dloss[t] * a.tau / amax * a.up;
  if (tid == 0) {
    a.lse2[c] = a.lse_in[t] * kLog2e;
    a.coef[c] = a.dlse ? (a.dloss[t] + a.dlse[t]) * a.tau / amax * a.up : g;
  }
  if (a.target) {
    if (tid == 0) {
      a.index32[c] = (int32_t)a.target[t];
      a.sub[c] = g;
    }
    return;
  }
  if (tid < 64) {
    int64_t id[kPerLane];
    float p[kPerLane], logp[kPerLane];
    teacher_row(a, t, tid, id, p, logp);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (tid + 64 * i < a.top) {
        ids[tid + 64 * i] = (int32_t)id[i];
        ps[tid + 64 * i] = p[i];
      }
  }
  __syncthreads();
  const int wide = (a.top + 7) / 8 * 8;
  // an id listed twice is subtracted once, with both probabilities
  for (int k = tid; k < a.top; k += 256) {
    const int id = ids[k];
    bool first = id >= 0;
    float sum = 0.f;
    for (int j = 0; j < a.top; ++j)
      if (ids[j] == id) {
        if (j < k) first = false;
        sum += ps[j];
      }
    a.index32[(int64_t)c * a.top + k] = first ? id : -1;
    a.sub[(int64_t)c * a.top + k] = g * sum;
    if (a.near) a.near[(int64_t)c * wide + k] = first ? (uint16_t)(id >> 8) : 0xFFFFu;
  }
  if (a.near && tid < wide - a.top) a.near[(int64_t)c * wide + a.top + tid] = 0xFFFFu;
}

// dw of no tokens: a store of 16 bytes per thread and turn, the chip filled once.
// (One of the launches that a graph may hold: no memory-set node.)
__global__ __launch_bounds__(256) void zero_kernel(u32x4* out, int64_t vecs) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * 256)
    out[i] = u32x4{0, 0, 0, 0};
}

}  // namespace

hipError_t launch_zero(uint16_t* out, int64_t values, hipStream_t s) {
  const int64_t vecs = values / 8, blocks = (vecs + 255) / 256;
  zero_kernel<<<dim3((unsigned)(blocks < 4096 ? blocks : 4096)), 256, 0, s>>>(reinterpret_cast<u32x4*>(out), vecs);
  return hipGetLastError();
}

hipError_t launch_rows(const RowArgs& a, bool backward, hipStream_t s) {
  if (!a.target) {
    flag_kernel<<<dim3((unsigned)((a.m_tok + 3) / 4)), 256, 0, s>>>(a, backward);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  rows_kernel<<<1, 1024, 0, s>>>(a, backward);
  return hipGetLastError();
}

hipError_t launch_finish(const RowArgs& a, bool compact, hipStream_t s) {
  if (a.m_tok <= 1024)
    finish_kernel<4><<<dim3((unsigned)a.m_tok), 256, 0, s>>>(a, compact);
  else
    finish_kernel<1><<<dim3((unsigned)((a.m_tok + 3) / 4)), 256, 0, s>>>(a, compact);
  return hipGetLastError();
}

// few enough list entries for every workgroup to read them all
bool gather_alone(int32_t m_tok, int32_t top) {
  return m_tok <= kFewTokens || (m_tok <= kAloneRows && m_tok * top <= 8 * 1024);
}

hipError_t launch_gather(const RowArgs& a, bool own_rows, hipStream_t s) {
  if (own_rows)
    gather_kernel<true><<<dim3((unsigned)(a.half > 0 ? a.half : a.m_tok)), 256, 0, s>>>(a);
  else
    gather_kernel<false><<<dim3((unsigned)a.m_tok), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace head
}  // namespace sbl
