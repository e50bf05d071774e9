// The AdamW update of many tensors in one pass over their weights, gradients
// and states.
//
//   g' = g factor,  m' = b1 m + a1 g',  v' = b2 v + a2 (g' g')     (a = 1 - b)
//   w' = w (1 - lr wd) - (lr bias1) (m' / (sqrt(v') bias2 + eps))
// Every step is one IEEE fp32 operation, in this order, so results repeat
// bit for bit whatever the launch looks like.
//
// Weights.  BF16 masters may carry the 16 bits that BF16 drops: the pair is an
// fp32 number whose bits are (high << 16) + low, high the nearest BF16 value
// (ties away from zero), low in [-2^15, 2^15); a NaN is 0x7FC0 and 0.  An update
// far below half a BF16 step is then kept, at 4 bytes a weight instead of 6 for
// an fp32 copy.
//
// States in 8 bits: blocks of 256 consecutive values of a tensor share an fp32
// scale s = max(RN(amax RN(1 / 448)), 2^-126), and a value x is held as the e4m3
// number nearest to RN(x RN(1 / s)) (exponent 4 bits, mantissa 3, at most 448).
// m is rounded to nearest.  Of v the square root is held (half the exponent
// range), rounded at random in proportion: at b2 = 0.999 a step moves it by
// about 0.05% and half a step of e4m3 is 6%, so rounding to nearest would
// leave it where it is; at random it follows the average, with a deviation of
// about 15% (the walk's variance of |g^2/v - 1| (1 - b2) / 2 times a code's width
// a step, against a pull of 1 - b2 a step).  The 16 random bits are a hash of the
// value's place and the step's seed.  A root above zero is never held as zero:
// with m still there, the next step would divide by eps alone.
//
// Bound by memory: 28 bytes a weight with states in 32 bits (masters with
// their low bits, fp32 gradient), 16 with states in 8 bits: 124M weights 627 us
// (5.5 TB/s), 317M in 8 bits 919 (5.5).  With fewer bytes than that the 8-bit
// states are bound by their 85 operations a value: 54M FP16 weights and gradients
// 145 us, 1.3 times the bytes' time.  Everything goes past the caches (the next
// step is the next reader; 32-bit states 693 -> 627 us) but the 8-bit states'
// gradient and codes.
#include "sbl_step.h"

namespace sbl {
namespace step {

namespace {

constexpr int kThreads = 256;
constexpr int kMostChunk = 8192;                 // values per workgroup, where that leaves every CU four
constexpr int kLeastChunk = 2048;                // one round of 256 threads (8-bit states: 8 values each)
constexpr int kMaxItems = 40;                    // of one launch: their descriptors are its arguments (< 4 KB)

struct AdamBatch {
  AdamItem item[kMaxItems];
  uint32_t start[kMaxItems];                     // first workgroup of each item
  AdamStep step;
  int32_t count, chunk;
};
static_assert(sizeof(AdamBatch) <= 4096, "kernel arguments");

struct Factors {
  float b1, a1, b2, a2, eps;
  float c, decay, bias2, factor;
  uint32_t seed;
};

__device__ __forceinline__ float root_of(float v) { return __builtin_sqrtf(v); }

// one weight: m, v (32 bits) and w in place; the root of the new v
__device__ __forceinline__ float update(float& w, float g, float& m, float& v, const Factors& f) {
  g = g * f.factor;
  m = m * f.b1 + g * f.a1;
  v = v * f.b2 + (g * g) * f.a2;
  const float root = root_of(v);
  w = w * f.decay - (m / (root * f.bias2 + f.eps)) * f.c;
  return root;
}

__device__ __forceinline__ float join(uint16_t high, int16_t low) {
  return __builtin_bit_cast(float, ((uint32_t)high << 16) + (uint32_t)(int32_t)low);
}
__device__ __forceinline__ void split(float w, uint16_t& high, int16_t& low) {
  // one NaN for all: the carry would run through another's exponent and sign (0x7FFFE000 would be -0 and its low bits)
  const uint32_t bits = w == w ? __builtin_bit_cast(uint32_t, w) : 0x7FC00000u;
  high = (uint16_t)((bits + 0x8000u) >> 16);
  low = (int16_t)(uint16_t)(bits & 0xFFFFu);     // bits - (high << 16) modulo 2^16
}

// 16 bits each for values 2 pair and 2 pair + 1: the low and high half of a
// hash of the pair's number (two rounds of xor-shift and multiply; shifts and
// factors as published by C. Wellons, "Prospecting for Hash Functions", 2018)
constexpr uint32_t kNextPair = 0x9E3779B9u;      // what pair + 1 adds to pair * kNextPair + seed
__device__ __forceinline__ uint32_t dither(uint32_t h) {
  h ^= h >> 16;
  h *= 0x7FEB352Du;
  h ^= h >> 15;
  h *= 0x846CA68Bu;
  return h ^ (h >> 16);
}

// t >= 0 to a multiple of its e4m3 step, up with probability the rest over the
// step: `random` (16 bits) is added below the three mantissa bits, which are
// then cut off; below 2^-6 the step is 2^-9, as just above it
__device__ __forceinline__ float cut_e4m3(float t, uint32_t random) {
  const float least = t < 0x1p-6f ? 0x1p-6f : 0.0f;
  const uint32_t bits = (__builtin_bit_cast(uint32_t, t + least) + (random << 4)) & 0xFFF00000u;
  return __builtin_bit_cast(float, bits) - least;
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax * (float)(1.0 / 448.0), 0x1p-126f); }

// four numbers <-> four e4m3 bytes; |f| at most 448 but for rounding
__device__ __forceinline__ uint32_t to_e4m3(const float* f) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], r, true);
}
__device__ __forceinline__ void from_e4m3(uint32_t c, float* f) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  f[0] = lo.x;
  f[1] = lo.y;
  f[2] = hi.x;
  f[3] = hi.y;
}

// largest over the 32 lanes that share a block
__device__ __forceinline__ float max32(float x) {
  x = fmaxf(x, dpp<0xB1, 0xf>(x, x));
  x = fmaxf(x, dpp<0x4E, 0xf>(x, x));
  x = fmaxf(x, dpp<0x141, 0xf>(x, x));
  x = fmaxf(x, dpp<0x140, 0xf>(x, x));
  return fmaxf(x, __shfl_xor(x, 16, 64));
}

// weights of V values at i: loaded as fp32
template <int TW, bool LOW, int V>
__device__ __forceinline__ void load_w(const AdamItem& it, int64_t i, int have, float (&w)[V]) {
  typedef typename Mem<TW>::E E;
  const Vec<TW, V> v = have >= V ? load_once<TW, V>(static_cast<const E*>(it.w) + i) : load<TW, V>(static_cast<const E*>(it.w) + i, have);
  if constexpr (LOW) {
    const uint16_t* pl = reinterpret_cast<const uint16_t*>(it.low) + i;
    const Vec<kBf16, V> l = have >= V ? load_once<kBf16, V>(pl) : load<kBf16, V>(pl, have);
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = join(v.e[j], (int16_t)l.e[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = v[j];
  }
}
template <int TW, bool LOW, int V>
__device__ __forceinline__ void store_w(const AdamItem& it, int64_t i, int have, const float (&w)[V]) {
  typedef typename Mem<TW>::E E;
  if constexpr (LOW) {
    Loose<kBf16, V> h, l;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      int16_t low;
      split(w[j], h.v.e[j], low);
      l.v.e[j] = (uint16_t)low;
    }
    uint16_t *ph = static_cast<uint16_t*>(it.w) + i, *pl = reinterpret_cast<uint16_t*>(it.low) + i;
    if (have >= V) {
      put_bytes<true>(ph, h.v);
      put_bytes<true>(pl, l.v);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < have) {
          ph[j] = h.v.e[j];
          pl[j] = l.v.e[j];
        }
    }
  } else {
    store<TW, V, true>(static_cast<E*>(it.w) + i, w, have);
  }
}

// values [first, first + chunk) of a tensor whose states have 32 bits
template <int TW, bool LOW, int TG> __device__ void chunk32(const AdamItem& it, int64_t first, int chunk, const Factors& f) {
  constexpr int V = 4;
  const int64_t left = it.n - first;
  for (int at = threadIdx.x * V; at < chunk && at < left; at += kThreads * V) {
    const int64_t i = first + at;
    const int have = left - at < V ? (int)(left - at) : V;
    float w[V], mf[V], vf[V];
    load_w<TW, LOW, V>(it, i, have, w);
    Vec<TG, V> g;
    Vec<kFp32, V> m, v;
    if (have >= V) {
      g = load_once<TG, V>(static_cast<const typename Mem<TG>::E*>(it.g) + i);
      m = load_once<kFp32, V>(static_cast<const float*>(it.m) + i);
      v = load_once<kFp32, V>(static_cast<const float*>(it.v) + i);
    } else {
      g = load<TG, V>(static_cast<const typename Mem<TG>::E*>(it.g) + i, have);
      m = load<kFp32, V>(static_cast<const float*>(it.m) + i, have);
      v = load<kFp32, V>(static_cast<const float*>(it.v) + i, have);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      mf[j] = m[j];
      vf[j] = v[j];
      update(w[j], g[j], mf[j], vf[j], f);
    }
    store_w<TW, LOW, V>(it, i, have, w);
    store<kFp32, V, true>(static_cast<float*>(it.m) + i, mf, have);
    store<kFp32, V, true>(static_cast<float*>(it.v) + i, vf, have);
  }
}

// the same with states in 8 bits: 8 values a lane, 32 lanes a block
template <int TW, bool LOW, int TG> __device__ void chunk8(const AdamItem& it, int64_t first, int chunk, const Factors& f) {
  constexpr int V = 8;
  const int64_t left = it.n - first;
  uint8_t *cm = static_cast<uint8_t*>(it.m), *cv = static_cast<uint8_t*>(it.v);
  for (int at = threadIdx.x * V; at < chunk; at += kThreads * V) {
    const int64_t i = first + at, block = i >> 8;
    const int have = left - at <= 0 ? 0 : left - at < V ? (int)(left - at) : V;
    if ((at & ~255) >= left) continue;             // whole blocks past the end
    float w[V], mf[V], vf[V], root[V];
    uint32_t c[4] = {};
    load_w<TW, LOW, V>(it, i, have, w);
    const Vec<TG, V> g = load<TG, V>(static_cast<const typename Mem<TG>::E*>(it.g) + i, have);
    if (have == V) {
      const uint2 a = *reinterpret_cast<const uint2*>(cm + i), b = *reinterpret_cast<const uint2*>(cv + i);
      c[0] = a.x;
      c[1] = a.y;
      c[2] = b.x;
      c[3] = b.y;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < have) {
          c[j >> 2] |= (uint32_t)cm[i + j] << (8 * (j & 3));
          c[2 + (j >> 2)] |= (uint32_t)cv[i + j] << (8 * (j & 3));
        }
    }
    float sm = it.m_scale[block], sv = it.v_scale[block];
    from_e4m3(c[0], mf);
    from_e4m3(c[1], mf + 4);
    from_e4m3(c[2], vf);
    from_e4m3(c[3], vf + 4);
    float am = 0.0f, av = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      mf[j] = mf[j] * sm;
      vf[j] = vf[j] * sv;
      vf[j] = vf[j] * vf[j];
      root[j] = update(w[j], g[j], mf[j], vf[j], f);   // values past the end: all zeros
      am = fmaxf(am, fabsf(mf[j]));
      av = fmaxf(av, root[j]);
    }
    store_w<TW, LOW, V>(it, i, have, w);
    sm = scale_of(max32(am));
    sv = scale_of(max32(av));
    const float rm = 1.0f / sm, rv = 1.0f / sv;
    const uint32_t pair = (uint32_t)(i >> 1) * kNextPair + f.seed;
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const uint32_t d = dither(pair + (uint32_t)(j / 2) * kNextPair);
      mf[j] = mf[j] * rm;
      mf[j + 1] = mf[j + 1] * rm;
      const float lo = fminf(fmaxf(cut_e4m3(root[j] * rv, d & 0xFFFFu), 0x1p-9f), 448.0f);
      const float hi = fminf(fmaxf(cut_e4m3(root[j + 1] * rv, d >> 16), 0x1p-9f), 448.0f);
      root[j] = root[j] > 0.0f ? lo : 0.0f;
      root[j + 1] = root[j + 1] > 0.0f ? hi : 0.0f;
    }
    c[0] = to_e4m3(mf);
    c[1] = to_e4m3(mf + 4);
    c[2] = to_e4m3(root);
    c[3] = to_e4m3(root + 4);
    if (have == V) {
      *reinterpret_cast<uint2*>(cm + i) = uint2{c[0], c[1]};
      *reinterpret_cast<uint2*>(cv + i) = uint2{c[2], c[3]};
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < have) {
          cm[i + j] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
          cv[i + j] = (uint8_t)(c[2 + (j >> 2)] >> (8 * (j & 3)));
        }
    }
    if ((at & 255) == 0) {
      it.m_scale[block] = sm;
      it.v_scale[block] = sv;
    }
  }
}

template <int TW, bool LOW, int TG>
__device__ __forceinline__ void by_states(const AdamItem& it, int64_t first, int chunk, const Factors& f) {
  if (it.bits == 8) chunk8<TW, LOW, TG>(it, first, chunk, f);
  else chunk32<TW, LOW, TG>(it, first, chunk, f);
}
template <int TW, bool LOW>
__device__ __forceinline__ void by_gradient(const AdamItem& it, int64_t first, int chunk, const Factors& f) {
  const int tg = it.kind / 3;
  if (tg == kFp32) by_states<TW, LOW, kFp32>(it, first, chunk, f);
  else if (tg == kBf16) by_states<TW, LOW, kBf16>(it, first, chunk, f);
  else by_states<TW, LOW, kFp16>(it, first, chunk, f);
}

__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamBatch a) {
  int i = 0;                                     // the item that this workgroup belongs to
#pragma unroll
  for (int step = 32; step > 0; step >>= 1)
    if (i + step < a.count && a.start[i + step] <= blockIdx.x) i += step;
  const AdamItem it = a.item[i];
  const AdamSchedule t = a.step.schedule ? *a.step.schedule : a.step.now;
  const float lr = t.lr * it.lr_scale;
  const Factors f{a.step.b1, a.step.a1, a.step.b2, a.step.a2, a.step.eps, lr * t.bias1, 1.0f - lr * it.weight_decay,
                  t.bias2, t.factor, (uint32_t)t.seed};
  const int64_t first = (int64_t)(blockIdx.x - a.start[i]) * a.chunk;
  const int tw = it.kind % 3;
  if (tw == kFp32) by_gradient<kFp32, false>(it, first, a.chunk, f);
  else if (tw == kFp16) by_gradient<kFp16, false>(it, first, a.chunk, f);
  else if (it.low) by_gradient<kBf16, true>(it, first, a.chunk, f);
  else by_gradient<kBf16, false>(it, first, a.chunk, f);
}

}  // namespace

hipError_t launch_adamw(const AdamItem* items, int count, const AdamStep& step, hipStream_t s) {
  AdamBatch b{};
  b.step = step;
  int64_t all = 0;
  for (int i = 0; i < count; ++i) all += items[i].n;
  // small models: a workgroup's rounds follow each other, more workgroups do not
  b.chunk = all >= (int64_t)1024 * kMostChunk ? kMostChunk : kLeastChunk;
  uint32_t groups = 0;
  auto run = [&] {
    if (groups == 0) return hipSuccess;
    hipLaunchKernelGGL(adamw_kernel, dim3(groups), dim3(kThreads), 0, s, b);
    b.count = 0;
    groups = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < count; ++i) {
    const int64_t need = (items[i].n + b.chunk - 1) / b.chunk;
    if (need == 0) continue;
    // a grid holds fewer than 2^32 threads
    if (b.count == kMaxItems || (int64_t)groups + need > (int64_t(1) << 32) / kThreads - 1) {
      const hipError_t e = run();
      if (e != hipSuccess) return e;
    }
    b.item[b.count] = items[i];
    b.start[b.count++] = groups;
    groups += (uint32_t)need;
  }
  return run();
}

}  // namespace step
}  // namespace sbl
