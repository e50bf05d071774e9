// Layer norm and RMS norm of rows, forward (with the activation quantizer in
// the same pass) and backward (with the reduction of the weight's gradient).
//
// Forward, per row of k values:
//   mean = center * sum x / k,  var = sum (x - mean)^2 / k,
//   rstd = RN32(1 / sqrt(var + eps)),  y = RN(RN(RN32(x - mean) rstd) w) + b
//   gamma = max |y|,  xq = clamp(rint(RN(y / s)), -127, 127), s = max(gamma, 1e-5) / 128
// The sums are taken in fp64 in one pass, of the differences to the row's
// first value (with it the two sums cancel only as far as that value is from
// the mean).  Their order moves them by some 2^-50, so that mean, rstd and the
// differences, rounded to fp32, are the same numbers for any partition of a row
// but for about one row in 10^7; what follows is one rounding per step.
// Backward: xh = (x - mean) rstd, g = dy w,
//   dx = rstd (g - center * mean(g) - xh mean(g xh)),  dw = sum_t dy xh,  db = sum_t dy.
// Both are bound by memory: x (and dy) read once, the outputs written once.
// A row lies in the registers of one workgroup from its load to its store (29 of
// 227 variants, most of fp32 rows, keep 1 to 24 of 128 registers in scratch);
// workgroups go over rows, so that the next row's loads are in flight while a
// row is reduced, and the backward's column sums need no memory until the end
// (one partial row per workgroup, joined in a fixed order by a second launch).
// Measured, with a large copy at 4.9 TB/s: forward 4096 x 5120 BF16 to fp32 and int8
// 26 us, 5.7 TB/s; 16384 x 8192 BF16 108 us, 5.0, fp32 197, 5.5; backward 8192 x
// 5120 of BF16 x and fp32 dy 64 us, 5.2, and 6 for joining the parts.
#include <algorithm>

#include "sbl_actq.h"
#include "sbl_step.h"

namespace sbl {
namespace step {

namespace {

constexpr int V = 4;                             // values per thread and slot
constexpr int kMaxWaves = 16;

// What is known of the rows of an output when a kernel is compiled.  kLines:
// they are whole 128-byte lines, and many: stored past the caches (4096 x 5120
// BF16 to fp32 and int8 when the weights were held: 42 -> 32 us; rows that end
// inside a line would be slower so; loads past the caches as well: 42, an input is
// often there still).  kWhole: also exactly as many values as the threads hold.
enum Rows { kAny = 0, kLines = 1, kWhole = 2 };

// 1 / sqrt(v) to fp64's precision: v_rsq_f64 (24 bits) and two Newton steps
__device__ __forceinline__ double rsqrt64(double v) {
  double r = __builtin_amdgcn_rsq(v);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = __builtin_fma(0.5 * r, __builtin_fma(-v * r, r, 1.0), r);
  return r;
}

struct Stat {
  double mean;
  float rstd;
};
// s1, s2: sums of (x - x0) and (x - x0)^2 (not centered: x0 = 0)
__device__ __forceinline__ Stat statistics(double s1, double s2, double x0, double inv_k, double eps, int center) {
  const double e = center ? s1 * inv_k : 0.0;
  const double var = __builtin_fma(-e, e, s2 * inv_k);
  return Stat{x0 + e, (float)rsqrt64((var < 0.0 ? 0.0 : var) + eps)};   // a NaN stays one (fmax would make it 0)
}

template <int T> __device__ __forceinline__ void add_stats(const Vec<T, V>& x, int have, double x0, double& s1, double& s2) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (j < have) {
      const double e = (double)x[j] - x0;
      s1 += e;
      s2 = __builtin_fma(e, e, s2);
    }
  }
}

// Four values to four codes, as actq::q_word (sbl_actq.h) makes them, in fewer
// instructions: adding 1.5 2^23 rounds to a whole number, ties to even, whose
// low byte is the code; the quotient RN(v r) decides unless it lies within 2^-15
// of a half, where |v / s - RN(v r)| could matter, and the IEEE quotient is formed.
// Clamped first: past 127.5 every quotient gives 127.
__device__ __forceinline__ uint32_t codes(const float (&v)[V], const actq::Step& st) {
  constexpr float kWhole = 12582912.0f;
  float m[V];
  bool near = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float q = __builtin_amdgcn_fmed3f(v[j] * st.r, -127.0f, 127.0f);
    m[j] = q + kWhole;
    near = near || fabsf(q - (m[j] - kWhole)) >= 0.5f - 0x1p-15f;
  }
  if (__any(near)) {
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = __builtin_amdgcn_fmed3f(v[j] / st.s, -127.0f, 127.0f) + kWhole;
  }
  const uint32_t lo = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, m[1]), __builtin_bit_cast(uint32_t, m[0]), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, m[3]), __builtin_bit_cast(uint32_t, m[2]), 0x0c0c0400u);
  return lo | hi << 16;
}

// the row's value of one position (not centered: the mean is zero)
__device__ __forceinline__ float normal(float x, const Stat& st, float w, float b) {
  return (float)((double)x - st.mean) * st.rstd * w + b;
}

__device__ __forceinline__ void load_param(const float* p, int col, int have, float none, float (&f)[V]) {
  const Vec<kFp32, V> v = p ? load<kFp32, V>(p + col, have) : Vec<kFp32, V>{};
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = p ? v[j] : none;
}
// the same by a buffer load, without a branch: of no parameters at all it reads zeros
struct Param {
  __amdgpu_buffer_rsrc_t r;
  float none;                                    // what to add: 0, or the value that stands for a parameter that is not there
};
__device__ __forceinline__ Param param(const float* p, int k, float none) {
  return Param{make_rsrc(p, p ? (int64_t)k * 4 : 0), p ? 0.0f : none};
}
template <int W> __device__ __forceinline__ void load_param(const Param& p, int col, float (&f)[W]) {
  if constexpr (W == 4) {
    const float4 v = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(p.r, (uint32_t)col * 4u, 0, 0));
    f[0] = v.x + p.none;
    f[1] = v.y + p.none;
    f[2] = v.z + p.none;
    f[3] = v.w + p.none;
  } else {
    static_assert(W == 1, "");
    f[0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(p.r, (uint32_t)col * 4u, 0, 0)) + p.none;
  }
}

// Keeps a value where it is made: without it sums and addresses move out of
// their loop or to its end, with everything that they are made from.
__device__ __forceinline__ void pin(float& f) { asm volatile("" : "+v"(f)); }
__device__ __forceinline__ int pinned(int i) {
  asm volatile("" : "+v"(i));
  return i;
}

// Rows of at most blockDim.x * SLOTS * W values, one workgroup per row and
// then the row gridDim.x later.  Held in registers beside the row: the next row,
// and if HOLD the weights; if not they are read again for every row (from L2).
template <int TX, int TY, int SLOTS, bool HOLD, int W, int ROWS>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a) {
  constexpr bool WHOLE = ROWS == kWhole, AHEAD = SLOTS <= 4 || TX != kFp32;
  typedef typename Mem<TX>::E EX;
  typedef typename Mem<TY>::E EY;
  __shared__ double part[2][2][kMaxWaves];       // of even and odd rows: one barrier per reduction
  __shared__ float peak[2][kMaxWaves];
  const int tid = threadIdx.x, wave = tid >> 6, waves = blockDim.x >> 6;
  const int k = a.k;
  const double inv_k = 1.0 / k;
  const EX* x = static_cast<const EX*>(a.x);
  Place at[SLOTS];
  const Param pw = param(a.w, k, 1.0f), pb = param(a.b, k, 0.0f);
  float w[HOLD ? SLOTS : 1][W], b[HOLD ? SLOTS : 1][W];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    at[i] = place<W>((tid + i * (int)blockDim.x) * W, k);
    if constexpr (HOLD) {
      load_param<W>(pw, at[i].col, w[i]);
      load_param<W>(pb, at[i].col, b[i]);
    }
  }
  int64_t row = blockIdx.x;
  Vec<TX, W> next[SLOTS];
  EX next0;
  auto fetch = [&] {
    const EX* p = x + row * k;
    next0 = p[0];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) next[i] = load<TX, W>(at_col(p, at[i].col));
  };
  fetch();
  for (int p = 0;; p ^= 1) {
    const int64_t now = row, base = row * k;
    Vec<TX, W> v[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) v[i] = next[i];
    const EX e0 = a.center ? next0 : (EX)0;
    const double x0 = (double)to_f32<TX>(e0);
    // what the sums take: x0, which adds nothing, in place of the vectors past whole lines
    auto taken = [&](int i) {
      Vec<TX, W> t = v[i];
      if (ROWS == kLines && at[i].skip != 0) {
#pragma unroll
        for (int j = 0; j < W; ++j) t.e[j] = e0;
      }
      return t;
    };
    row += gridDim.x;
    if (AHEAD && row < a.m_tok) fetch();
    double s1 = 0.0, s2 = 0.0;
    if (a.center) {
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        const Vec<TX, W> t = taken(i);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          double e = (double)t[j] - x0;
          if (ROWS == kAny) e = j >= at[i].skip ? e : 0.0;
          s1 += e;
          s2 = __builtin_fma(e, e, s2);
        }
      }
      s1 = wave_sum(s1);
    } else {
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        const Vec<TX, W> t = taken(i);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float f = ROWS != kAny || j >= at[i].skip ? t[j] : 0.0f;
          s2 = __builtin_fma((double)f, (double)f, s2);
        }
      }
    }
    s2 = wave_sum(s2);
    if ((tid & 63) == 0) {
      part[p][0][wave] = s1;
      part[p][1][wave] = s2;
    }
    __syncthreads();
    s1 = part[p][0][0];
    s2 = part[p][1][0];
    for (int i = 1; i < waves; ++i) {
      s1 += part[p][0][i];
      s2 += part[p][1][i];
    }
    const Stat st = statistics(s1, s2, x0, inv_k, a.eps, a.center);
    float mx = 0.0f;
    float y[SLOTS][W];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const Place c{HOLD ? at[i].col : pinned(at[i].col), WHOLE ? 0 : at[i].skip};
      if constexpr (!HOLD) {
        forget(v[i]);
        if (i % 2 == 0) __builtin_amdgcn_sched_barrier(0);   // the weights of two slots at a time
      }
      float(&wi)[W] = w[HOLD ? i : 0];
      float(&bi)[W] = b[HOLD ? i : 0];
      if constexpr (!HOLD) {
        load_param<W>(pw, c.col, wi);
        load_param<W>(pb, c.col, bi);
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        // not centered: the mean is zero, and the difference x itself
        const float d = a.center ? (float)((double)v[i][j] - st.mean) : v[i][j];
        y[i][j] = d * st.rstd * wi[j] + bi[j];
        mx = larger(mx, fabsf(y[i][j]));         // a column seen twice does not change the largest
      }
      if (a.y) store_own<TY, W, ROWS != kAny>(static_cast<EY*>(a.y) + base, c, y[i]);
    }
    if (tid == 0) {
      if (a.mean) a.mean[now] = (float)st.mean;
      if (a.rstd) a.rstd[now] = st.rstd;
    }
    if constexpr (W == V) {                      // k % 64 == 0: no vector passes the row's end
      if (a.xq) {
        mx = wave_max(mx);
        if ((tid & 63) == 0) peak[p][wave] = mx;
        __syncthreads();
        float g = peak[p][0];
        for (int i = 1; i < waves; ++i) g = larger(g, peak[p][i]);
        const actq::Step sp = actq::make_step(g);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
          if (WHOLE || at[i].skip == 0)
            *reinterpret_cast<uint32_t*>(at_col(a.xq + base, at[i].col)) = codes(y[i], sp);
        if (tid == 0) a.gamma[now] = g;
      }
    }
    if (row >= a.m_tok) break;
    if constexpr (!AHEAD) fetch();
  }
}

// Longer rows: one workgroup per row, which reads it once for the statistics,
// once for y and once more for xq (from L2 by then).  1024 BF16 rows to fp32 and
// int8: 40000 values 118 us, 131072 473, 2 and 2.5 times the time of their bytes.
template <int TX, int TY>
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormArgs a) {
  typedef typename Mem<TX>::E EX;
  typedef typename Mem<TY>::E EY;
  __shared__ double part[2][kMaxWaves];
  __shared__ float peak[kMaxWaves];
  const int tid = threadIdx.x, wave = tid >> 6, k = a.k;
  const int64_t base = (int64_t)blockIdx.x * k;
  const EX* x = static_cast<const EX*>(a.x) + base;
  const double x0 = a.center ? (double)to_f32<TX>(x[0]) : 0.0;
  double s1 = 0.0, s2 = 0.0;
  for (int c = tid * V; c < k; c += 1024 * V) add_stats<TX>(load<TX, V>(x + c, k - c), k - c, x0, s1, s2);
  s1 = wave_sum(s1);
  s2 = wave_sum(s2);
  if ((tid & 63) == 0) {
    part[0][wave] = s1;
    part[1][wave] = s2;
  }
  __syncthreads();
  s1 = part[0][0];
  s2 = part[1][0];
  for (int i = 1; i < kMaxWaves; ++i) {
    s1 += part[0][i];
    s2 += part[1][i];
  }
  const Stat st = statistics(s1, s2, x0, 1.0 / k, a.eps, a.center);
  auto value = [&](int c, float (&y)[V]) {
    const Vec<TX, V> v = load<TX, V>(x + c, k - c);
    float w[V], b[V];
    load_param(a.w, c, k - c, 1.0f, w);
    load_param(a.b, c, k - c, 0.0f, b);
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = normal(v[j], st, w[j], b[j]);
  };
  float mx = 0.0f;
  for (int c = tid * V; c < k; c += 1024 * V) {
    float y[V];
    value(c, y);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c + j < k) mx = larger(mx, fabsf(y[j]));
    if (a.y) store<TY, V>(static_cast<EY*>(a.y) + base + c, y, k - c);
  }
  if (tid == 0) {
    if (a.mean) a.mean[blockIdx.x] = (float)st.mean;
    if (a.rstd) a.rstd[blockIdx.x] = st.rstd;
  }
  if (!a.xq) return;
  mx = wave_max(mx);
  if ((tid & 63) == 0) peak[wave] = mx;
  __syncthreads();
  float g = peak[0];
  for (int i = 1; i < kMaxWaves; ++i) g = larger(g, peak[i]);
  const actq::Step sp = actq::make_step(g);
  for (int c = tid * V; c < k; c += 1024 * V) {
    float y[V];
    value(c, y);
    *reinterpret_cast<uint32_t*>(a.xq + base + c) = codes(y, sp);
  }
  if (tid == 0) a.gamma[blockIdx.x] = g;
}

// ---------------------------------------------------------------- backward

struct Pair {
  float g, gx;                                   // sums of g and g xh
};

__device__ __forceinline__ float xhat(float x, float mean, float rstd) { return (x - mean) * rstd; }

__device__ __forceinline__ float grad(float dy, float xh, float w, float rstd, float c1, float c2) {
  return rstd * (dy * w - c1 - xh * c2);
}

// Rows of at most blockDim.x * SLOTS * W values, blockDim.x at most MOST.  Every
// thread keeps the column sums of its own columns over the workgroup's rows and, up
// to 512 threads, holds the next row beside this one and the weights.
template <int TX, int TD, int SLOTS, int W, int MOST, int ROWS>
__global__ __launch_bounds__(MOST) void norm_grad_kernel(const NormGradArgs a, float* part_w, float* part_b) {
  constexpr bool WHOLE = ROWS == kWhole, KEEP_W = SLOTS * MOST <= 2048, AHEAD = KEEP_W;
  typedef typename Mem<TX>::E EX;
  typedef typename Mem<TD>::E ED;
  __shared__ Pair part[2][kMaxWaves];
  const int tid = threadIdx.x, wave = tid >> 6, waves = blockDim.x >> 6;
  const int k = a.k;
  const float inv_k = 1.0f / k;
  const EX* x = static_cast<const EX*>(a.x);
  const ED* dy = static_cast<const ED*>(a.dy);
  Place at[SLOTS];
  const Param pw = param(a.w, k, 1.0f);
  float w[KEEP_W ? SLOTS : 1][W], sw[SLOTS][W], sb[SLOTS][W];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    at[i] = place<W>((tid + i * (int)blockDim.x) * W, k);
    if constexpr (KEEP_W) load_param<W>(pw, at[i].col, w[i]);
#pragma unroll
    for (int j = 0; j < W; ++j) sw[i][j] = sb[i][j] = 0.0f;
  }
  int64_t row = blockIdx.x;
  Vec<TX, W> nx[SLOTS];
  Vec<TD, W> nd[SLOTS];
  float nm = 0.0f, nr;
  auto fetch = [&] {
    nm = a.mean ? a.mean[row] : 0.0f;
    nr = a.rstd[row];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      nx[i] = load<TX, W>(at_col(x + row * k, at[i].col));
      nd[i] = load<TD, W>(at_col(dy + row * k, at[i].col));
    }
  };
  fetch();
  for (int p = 0;; p ^= 1) {
    const int64_t base = row * k;
    const float mean = nm, rstd = nr;
    Vec<TX, W> vx[SLOTS];
    Vec<TD, W> vd[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      vx[i] = nx[i];
      vd[i] = nd[i];
      if (ROWS == kLines && at[i].skip != 0) vd[i] = Vec<TD, W>{};   // past whole lines: adds nothing
    }
    row += gridDim.x;
    if (AHEAD && row < a.m_tok) fetch();
    auto weights = [&](int i) -> const float(&)[W] {
      float(&wi)[W] = w[KEEP_W ? i : 0];
      if constexpr (!KEEP_W) load_param<W>(pw, pinned(at[i].col), wi);
      return wi;
    };
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const float(&wi)[W] = weights(i);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float xh = xhat(vx[i][j], mean, rstd), d = vd[i][j];
        float g = d * wi[j];
        if (ROWS == kAny) g = j >= at[i].skip ? g : 0.0f;
        s1 += g;
        s2 = __builtin_fmaf(g, xh, s2);
        sw[i][j] = __builtin_fmaf(d, xh, sw[i][j]);
        sb[i][j] += d;
        if constexpr (!KEEP_W) {
          pin(sw[i][j]);
          pin(sb[i][j]);
        }
      }
    }
    if (a.dx) {
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if ((tid & 63) == 0) part[p][wave] = Pair{s1, s2};
      __syncthreads();
      s1 = part[p][0].g;
      s2 = part[p][0].gx;
      for (int i = 1; i < waves; ++i) {
        s1 += part[p][i].g;
        s2 += part[p][i].gx;
      }
      const float c1 = a.center ? s1 * inv_k : 0.0f, c2 = s2 * inv_k;
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        if constexpr (!KEEP_W) {
          forget(vx[i]);
          forget(vd[i]);
        }
        const float(&wi)[W] = weights(i);
        float d[W];
#pragma unroll
        for (int j = 0; j < W; ++j) d[j] = grad(vd[i][j], xhat(vx[i][j], mean, rstd), wi[j], rstd, c1, c2);
        store_own<TX, W, ROWS != kAny>(static_cast<EX*>(a.dx) + base,
                                       Place{KEEP_W ? at[i].col : pinned(at[i].col), WHOLE ? 0 : at[i].skip}, d);
      }
    }
    if (row >= a.m_tok) break;
    if constexpr (!AHEAD) fetch();
  }
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const Place c = WHOLE ? Place{at[i].col, 0} : at[i];
    if (part_w) store_own<kFp32, W>(part_w + (int64_t)blockIdx.x * k, c, sw[i]);
    if (part_b) store_own<kFp32, W>(part_b + (int64_t)blockIdx.x * k, c, sb[i]);
  }
}

// Longer rows: the two means of every row first (one workgroup per row), then
// every column by a thread of its own, which needs no other.  x and dy are read
// twice: 4096 x 28672 of BF16 x and fp32 dy 367 us, 1.9 times its bytes' time.
template <int TX, int TD>
__global__ __launch_bounds__(1024) void norm_grad_rows_kernel(const NormGradArgs a, float2* means) {
  __shared__ Pair part[kMaxWaves];
  const int tid = threadIdx.x, wave = tid >> 6, k = a.k;
  const int64_t row = blockIdx.x, base = row * k;
  const typename Mem<TX>::E* x = static_cast<const typename Mem<TX>::E*>(a.x) + base;
  const typename Mem<TD>::E* dy = static_cast<const typename Mem<TD>::E*>(a.dy) + base;
  const float mean = a.mean ? a.mean[row] : 0.0f, rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int c = tid * V; c < k; c += 1024 * V) {
    const Vec<TX, V> vx = load<TX, V>(x + c, k - c);
    const Vec<TD, V> vd = load<TD, V>(dy + c, k - c);
    float w[V];
    load_param(a.w, c, k - c, 1.0f, w);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float g = vd[j] * w[j];
      s1 += g;
      s2 = __builtin_fmaf(g, xhat(vx[j], mean, rstd), s2);
    }
  }
  s1 = wave_sum(s1);
  s2 = wave_sum(s2);
  if ((tid & 63) == 0) part[wave] = Pair{s1, s2};
  __syncthreads();
  if (tid != 0) return;
  s1 = s2 = 0.0f;
  for (int i = 0; i < kMaxWaves; ++i) {
    s1 += part[i].g;
    s2 += part[i].gx;
  }
  means[row] = float2{a.center ? s1 / k : 0.0f, s2 / k};
}

template <int TX, int TD>
__global__ __launch_bounds__(256) void norm_grad_columns_kernel(const NormGradArgs a, const float2* means, float* part_w,
                                                                float* part_b) {
  const int k = a.k, col = (blockIdx.x * 256 + threadIdx.x) * V, have = k - col;
  if (have <= 0) return;
  const typename Mem<TX>::E* x = static_cast<const typename Mem<TX>::E*>(a.x) + col;
  const typename Mem<TD>::E* dy = static_cast<const typename Mem<TD>::E*>(a.dy) + col;
  float w[V], sw[V] = {}, sb[V] = {};
  load_param(a.w, col, have, 1.0f, w);
  for (int64_t row = blockIdx.y; row < a.m_tok; row += gridDim.y) {
    const Vec<TX, V> vx = load<TX, V>(x + row * k, have);
    const Vec<TD, V> vd = load<TD, V>(dy + row * k, have);
    const float mean = a.mean ? a.mean[row] : 0.0f, rstd = a.rstd[row];
    const float2 c = a.dx ? means[row] : float2{0.0f, 0.0f};
    float d[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float xh = xhat(vx[j], mean, rstd);
      sw[j] = __builtin_fmaf(vd[j], xh, sw[j]);
      sb[j] += vd[j];
      d[j] = grad(vd[j], xh, w[j], rstd, c.x, c.y);
    }
    if (a.dx) store<TX, V>(static_cast<typename Mem<TX>::E*>(a.dx) + row * k + col, d, have);
  }
  if (part_w) store<kFp32, V>(part_w + (int64_t)blockIdx.y * k + col, sw, have);
  if (part_b) store<kFp32, V>(part_b + (int64_t)blockIdx.y * k + col, sb, have);
}

// out[c] = sum over the partial rows, in ascending order within each of 256 / L
// shares, then share by share; L lanes side by side.  blockIdx.y: 0 the weight, 1
// the bias.
template <int L>
__global__ __launch_bounds__(256) void norm_grad_final_kernel(const float* part_w, const float* part_b, int rows, int k,
                                                              float* dw, float* db) {
  constexpr int kShares = 256 / L;
  __shared__ float sum[kShares][L][V];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;
  const int lane = threadIdx.x % L, share = threadIdx.x / L;
  const int col = (blockIdx.x * L + lane) * V, have = k - col;
  float s[V] = {};
  const int per = (rows + kShares - 1) / kShares, r1 = min(rows, (share + 1) * per);
  if (have > 0) {
#pragma unroll 8
    for (int r = share * per; r < r1; ++r) {
      const Vec<kFp32, V> v = load<kFp32, V>(part + (int64_t)r * k + col, have);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) sum[share][lane][j] = s[j];
  __syncthreads();
  if (share != 0 || have <= 0) return;
#pragma unroll 16
  for (int r = 1; r < kShares; ++r)
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] += sum[r][lane][j];
  store<kFp32, V>(out + col, s, have);
}

__global__ __launch_bounds__(256) void zero_floats_kernel(float* p, int n) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) p[i] = 0.0f;
}

constexpr int64_t kStreamBytes = 16 << 20;       // outputs of less stay in the caches
constexpr int kWideFinal = 1024;

int vectors(int64_t k) { return (int)((k + V - 1) / V); }

// Slots per thread: with few rows, as few as 1024 threads can do with (all of a
// row's loads in flight from as many waves as possible); with more rows, 4 (more
// bytes in flight per wave, fewer waves to join in a reduction), as long as that
// leaves two waves.  Forward, where nothing but the row need be held, 8 for rows
// that 4 do not take (4096 x 28672 BF16 to fp32 and int8: 338 us by the kernel for
// longer rows, 168 so, which is the time of its bytes; 13824 values in 8 slots 111,
// in 4 94).  Backward 8 leave no room for the sums.
constexpr int kMaxSlots = 8, kMaxGradSlots = 4;
int slots_for(int nv, int64_t m_tok, int most) {
  int s = 1;
  if (m_tok >= 1024)
    while (s < 4 && nv >= 2 * s * 128) s *= 2;
  while (s < most && nv > 1024 * s) s *= 2;
  return s;
}
int threads_for(int nv, int slots) { return ((nv + slots - 1) / slots + 63) / 64 * 64; }

// workgroups that the chip holds at once
int resident(int threads, int waves_per_simd) {
  const int per_cu = 4 * waves_per_simd / (threads / 64);
  return 256 * (per_cu < 1 ? 1 : per_cu);
}

// the rows of an output of `bytes` in all
Rows rows_of(const void* out, int64_t k, int64_t bytes, int64_t held, int type) {
  if (bytes < kStreamBytes || k * type_bytes(type) % 128 != 0 || reinterpret_cast<uintptr_t>(out) % 128 != 0) return kAny;
  return k == held ? kWhole : kLines;
}

template <int TX, int TY, int SLOTS, bool HOLD> void forward_rows(const NormArgs& a, dim3 grid, dim3 block, hipStream_t s) {
  const Rows rows = rows_of(a.y, a.k, a.m_tok * a.k * type_bytes(TY), (int64_t)block.x * SLOTS * V, TY);
  if (rows == kWhole) hipLaunchKernelGGL((norm_kernel<TX, TY, SLOTS, HOLD, V, kWhole>), grid, block, 0, s, a);
  else if (rows == kLines) hipLaunchKernelGGL((norm_kernel<TX, TY, SLOTS, HOLD, V, kLines>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_kernel<TX, TY, SLOTS, HOLD, V, kAny>), grid, block, 0, s, a);
}

template <int TX, int TY> hipError_t forward(const NormArgs& a, hipStream_t s) {
  const int nv = vectors(a.k), slots = slots_for(nv, a.m_tok, kMaxSlots);
  if (nv > 1024 * kMaxSlots) {
    hipLaunchKernelGGL((norm_long_kernel<TX, TY>), dim3((unsigned)a.m_tok), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  const int threads = threads_for(nv, slots), waves = threads / 64;
  // 4 slots: the weights are held (4 waves per SIMD) unless without them one more workgroup fits
  // a CU (5): 4096 x 5120 BF16 to fp32 and int8 32 us held, 27 not; 16384 x 8192 BF16 108 and 134
  const bool hold = slots < 4 || (slots == 4 && 16 / waves == 20 / waves);
  const int64_t most = resident(threads, slots <= 2 ? 6 : slots == 4 && !hold ? 5 : 4);
  const dim3 grid((unsigned)(a.m_tok < most ? a.m_tok : most)), block((unsigned)threads);
  if (a.k < V) hipLaunchKernelGGL((norm_kernel<TX, TY, 1, true, 1, kAny>), grid, block, 0, s, a);
  else if (slots == 1) forward_rows<TX, TY, 1, true>(a, grid, block, s);
  else if (slots == 2) forward_rows<TX, TY, 2, true>(a, grid, block, s);
  else if (slots == 4 && hold) forward_rows<TX, TY, 4, true>(a, grid, block, s);
  else if (slots == 4) forward_rows<TX, TY, 4, false>(a, grid, block, s);
  else forward_rows<TX, TY, 8, false>(a, grid, block, s);
  return hipGetLastError();
}

struct GradPlan {
  int slots, threads;                            // slots 0: long rows
  int64_t parts;                                 // partial rows of the column sums
};
GradPlan grad_plan(int64_t m_tok, int64_t k) {
  const int nv = vectors(k);
  GradPlan p{0, 256, 0};
  if (nv <= 1024 * kMaxGradSlots) {
    p.slots = slots_for(nv, m_tok, kMaxGradSlots);
    p.threads = threads_for(nv, p.slots);
    p.parts = resident(p.threads, p.slots == 4 && p.threads <= 512 ? 3 : 4);
  } else {
    p.parts = 2048 / ((nv + 255) / 256);         // 8 workgroups a CU over the columns and the rows' shares
  }
  // narrow rows: a part takes 8 of them at least, so that joining the parts does not cost more than the rows;
  // the first few rows: one part, and no second launch
  const int64_t most = m_tok <= 4 ? 1 : m_tok < 4096 ? m_tok : std::max<int64_t>(512, m_tok / 8);
  if (p.parts > most) p.parts = most;
  return p;
}

template <int TX, int TD, int SLOTS, int MOST>
void backward_rows(const NormGradArgs& a, float* pw, float* pb, dim3 grid, dim3 block, hipStream_t s) {
  const Rows rows = rows_of(a.dx, a.k, a.m_tok * a.k * type_bytes(TX), (int64_t)block.x * SLOTS * V, TX);
  if (rows == kWhole) hipLaunchKernelGGL((norm_grad_kernel<TX, TD, SLOTS, V, MOST, kWhole>), grid, block, 0, s, a, pw, pb);
  else if (rows == kLines) hipLaunchKernelGGL((norm_grad_kernel<TX, TD, SLOTS, V, MOST, kLines>), grid, block, 0, s, a, pw, pb);
  else hipLaunchKernelGGL((norm_grad_kernel<TX, TD, SLOTS, V, MOST, kAny>), grid, block, 0, s, a, pw, pb);
}

template <int TX, int TD> hipError_t backward(const NormGradArgs& a, hipStream_t s) {
  const GradPlan p = grad_plan(a.m_tok, a.k);
  // one share of the rows: its sums are the outputs
  const bool join = p.parts > 1;
  float* pw = !a.dw ? nullptr : join ? a.ws : a.dw;
  float* pb = !a.db ? nullptr : join ? a.ws + p.parts * a.k : a.db;
  const dim3 grid((unsigned)p.parts), block((unsigned)p.threads);
  if (p.slots == 0) {
    float2* means = reinterpret_cast<float2*>(a.ws + 2 * p.parts * a.k);
    if (a.dx) hipLaunchKernelGGL((norm_grad_rows_kernel<TX, TD>), dim3((unsigned)a.m_tok), dim3(1024), 0, s, a, means);
    hipLaunchKernelGGL((norm_grad_columns_kernel<TX, TD>), dim3((unsigned)((vectors(a.k) + 255) / 256), (unsigned)p.parts),
                       dim3(256), 0, s, a, means, pw, pb);
  } else if (a.k < V) {
    hipLaunchKernelGGL((norm_grad_kernel<TX, TD, 1, 1, 1024, kAny>), grid, block, 0, s, a, pw, pb);
  } else if (p.slots == 1) {
    backward_rows<TX, TD, 1, 1024>(a, pw, pb, grid, block, s);
  } else if (p.slots == 2) {
    backward_rows<TX, TD, 2, 1024>(a, pw, pb, grid, block, s);
  } else if (p.threads <= 512) {
    backward_rows<TX, TD, 4, 512>(a, pw, pb, grid, block, s);
  } else {
    backward_rows<TX, TD, 4, 1024>(a, pw, pb, grid, block, s);
  }
  if (join && (a.dw || a.db)) {
    const int nv = vectors(a.k);
    if (nv < kWideFinal)                         // few columns: more shares of the parts
      hipLaunchKernelGGL(norm_grad_final_kernel<4>, dim3((unsigned)((nv + 3) / 4), 2), dim3(256), 0, s, pw, pb, (int)p.parts,
                         a.k, a.dw, a.db);
    else
      hipLaunchKernelGGL(norm_grad_final_kernel<16>, dim3((unsigned)((nv + 15) / 16), 2), dim3(256), 0, s, pw, pb,
                         (int)p.parts, a.k, a.dw, a.db);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, int tx, int ty, hipStream_t s) {
  return with_types(tx, ty, [&](auto x, auto y) { return forward<x.value, y.value>(a, s); });
}

// partial rows of both column sums; long rows: two means per row, 8-byte aligned
int64_t norm_grad_ws_bytes(int64_t m_tok, int64_t k) {
  if (m_tok == 0) return 0;
  const GradPlan p = grad_plan(m_tok, k);
  return (2 * p.parts * k * 4 + (p.slots == 0 ? m_tok * 8 : 0) + 255) / 256 * 256;
}

hipError_t launch_norm_backward(const NormGradArgs& a, int tx, int td, hipStream_t s) {
  if (a.m_tok == 0) {
    for (float* p : {a.dw, a.db})
      if (p) hipLaunchKernelGGL(zero_floats_kernel, dim3((unsigned)((a.k + 255) / 256)), dim3(256), 0, s, p, a.k);
    return hipGetLastError();
  }
  return with_types(tx, td, [&](auto x, auto d) { return backward<x.value, d.value>(a, s); });
}

}  // namespace step
}  // namespace sbl
