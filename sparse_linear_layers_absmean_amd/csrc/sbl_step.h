// Internal declarations of what a training step needs around the layer and
// the head: the norm (k_norm.hip), the embedding (k_embed.hip) and the AdamW
// update (k_adamw.hip); their calls are in sbl_api_step.hip.
#pragma once

#include <type_traits>

#include "sbl_internal.h"

namespace sbl {
namespace step {

// numeric types, numbered as sbl_dtype
enum Type { kBf16 = 0, kFp16 = 1, kFp32 = 2 };
__host__ __device__ constexpr int64_t type_bytes(int t) { return t == kFp32 ? 4 : 2; }

// f(a, b) with two types as constants: the same, or fp32 and another
template <class F> hipError_t with_types(int a, int b, F f) {
  std::integral_constant<int, kBf16> bf16;
  std::integral_constant<int, kFp16> fp16;
  std::integral_constant<int, kFp32> fp32;
  if (a == kBf16) return b == kFp32 ? f(bf16, fp32) : f(bf16, bf16);
  if (a == kFp16) return b == kFp32 ? f(fp16, fp32) : f(fp16, fp16);
  return b == kBf16 ? f(fp32, bf16) : b == kFp16 ? f(fp32, fp16) : f(fp32, fp32);
}

// ---------------------------------------------------------------- norm

struct NormArgs {
  const void* x;                  // [m_tok][k]
  const float* w;                 // [k] or NULL (ones)
  const float* b;                 // [k] or NULL (zeros)
  int64_t m_tok;
  int32_t k;
  int32_t center;                 // subtract the mean (layer norm) or not (RMS norm)
  double eps;
  void* y;                        // [m_tok][k] or NULL
  int8_t* xq;                     // [m_tok][k] and
  float* gamma;                   // [m_tok], or both NULL
  float* mean;                    // [m_tok] or NULL
  float* rstd;                    // [m_tok] or NULL
};
hipError_t launch_norm_forward(const NormArgs& a, int x_type, int y_type, hipStream_t s);

struct NormGradArgs {
  const void* dy;                 // [m_tok][k]
  const void* x;                  // [m_tok][k]
  const float* mean;              // [m_tok] or NULL (zeros)
  const float* rstd;              // [m_tok]
  const float* w;                 // [k] or NULL
  int64_t m_tok;
  int32_t k;
  int32_t center;
  void* dx;                       // [m_tok][k] or NULL
  float* dw;                      // [k] or NULL
  float* db;                      // [k] or NULL
  float* ws;
};
int64_t norm_grad_ws_bytes(int64_t m_tok, int64_t k);
hipError_t launch_norm_backward(const NormGradArgs& a, int x_type, int dy_type, hipStream_t s);

// ---------------------------------------------------------------- embedding

struct EmbedArgs {
  const int64_t* ids;             // [m_tok]
  const void* table;              // [n_vocab][k]
  int64_t m_tok, n_vocab;
  int32_t k;
  float scale;
  void* out;                      // [m_tok][k]
};
hipError_t launch_embed_forward(const EmbedArgs& a, int table_type, int out_type, hipStream_t s);

struct EmbedGradArgs {
  const int64_t* ids;             // [m_tok]
  const void* dout;               // [m_tok][k]
  int64_t m_tok, n_vocab;
  int32_t k;
  float scale;
  void* dtable;                   // [n_vocab][k]
  bool add;                       // add to what dtable holds, or write all of it
  void* ws;
};
int64_t embed_grad_ws_bytes(int64_t m_tok, int64_t n_vocab, int64_t k, int out_type);
hipError_t launch_embed_backward(const EmbedGradArgs& a, int out_type, int table_type, hipStream_t s);

// ---------------------------------------------------------------- AdamW

struct AdamItem {
  void* w;
  int16_t* low;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float lr_scale, weight_decay;
  int32_t kind;                   // w_type + 3 * g_type
  int32_t bits;                   // of the states: 32 or 8
};

// the factors of one step, on the device or by value
struct AdamSchedule {
  float lr, bias1, bias2, factor, seed;
};

struct AdamStep {
  float b1, a1, b2, a2, eps;      // a = 1 - b
  AdamSchedule now;
  const AdamSchedule* schedule;   // or NULL: now
};
hipError_t launch_adamw(const AdamItem* items, int count, const AdamStep& step, hipStream_t s);

// ---------------------------------------------------------------- values in memory

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int T> struct Mem { typedef uint16_t E; };
template <> struct Mem<kFp32> { typedef float E; };

template <int T> __device__ __forceinline__ float to_f32(typename Mem<T>::E e) {
  if constexpr (T == kBf16) return __builtin_bit_cast(float, (uint32_t)e << 16);
  else if constexpr (T == kFp16) return (float)__builtin_bit_cast(_Float16, e);
  else return e;
}
// one rounding to nearest, ties to even (fp32: none)
template <int T> __device__ __forceinline__ typename Mem<T>::E from_f32(float f) {
  if constexpr (T == kBf16) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
  } else if constexpr (T == kFp16) {
    // f as an fp32 number first: else a product and its rounding to FP16 become one
    // instruction with one rounding (v_fma_mixlo_f16)
    asm("" : "+v"(f));
    return __builtin_bit_cast(uint16_t, (_Float16)f);
  } else {
    return f;
  }
}

// V consecutive values held as they lie in memory.  Rows of an odd number of
// 16-bit values start anywhere, so the type asks for no more alignment than an
// element has: gfx950 takes wide global accesses at any address.
template <int T, int V> struct Vec {
  typedef typename Mem<T>::E E;
  E e[V];
  __device__ __forceinline__ float operator[](int i) const { return to_f32<T>(e[i]); }
};
template <int T, int V> struct __attribute__((packed, aligned(sizeof(typename Mem<T>::E)))) Loose {
  Vec<T, V> v;
};

// n bytes at once, past the caches where STREAM (data that nothing reads soon)
template <int N> struct Words;
template <> struct Words<4> { typedef uint32_t T __attribute__((aligned(2), may_alias)); };
template <> struct Words<8> { typedef uint32_t T __attribute__((ext_vector_type(2), aligned(2), may_alias)); };
template <> struct Words<16> { typedef uint32_t T __attribute__((ext_vector_type(4), aligned(2), may_alias)); };
template <bool STREAM, class S> __device__ __forceinline__ void put_bytes(void* p, const S& v) {
  constexpr int N = sizeof(S);
  if constexpr (!STREAM || N < 4) {
    __builtin_memcpy(p, &v, N);
  } else if constexpr (N > 16) {
    struct Half {
      uint8_t b[16];
    } h[N / 16];
    __builtin_memcpy(h, &v, N);
#pragma unroll
    for (int i = 0; i < N / 16; ++i) put_bytes<true>(static_cast<uint8_t*>(p) + 16 * i, h[i]);
  } else {
    __builtin_nontemporal_store(__builtin_bit_cast(typename Words<N>::T, v), static_cast<typename Words<N>::T*>(p));
  }
}

// the V values at p, or its first `have` and zeros
template <int T, int V>
__device__ __forceinline__ Vec<T, V> load(const typename Mem<T>::E* p, int have) {
  if (have >= V) return reinterpret_cast<const Loose<T, V>*>(p)->v;
  Vec<T, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = i < have ? p[i] : (typename Mem<T>::E)0;
  return v;
}
template <int T, int V, bool STREAM = false>
__device__ __forceinline__ void store(typename Mem<T>::E* p, const float (&f)[V], int have) {
  if (have >= V) {
    Vec<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(f[i]);
    if constexpr (STREAM) put_bytes<true>(p, o);
    else reinterpret_cast<Loose<T, V>*>(p)->v = o;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < have) p[i] = from_f32<T>(f[i]);
  }
}

// Where a thread's V columns of a row of k >= V lie.  The vector that would
// pass the row's end (and those that begin past it) is moved back to end with
// the row, so that every load is a whole one, without a branch: its first
// `skip` columns are another thread's too (all of them where skip >= V).
struct Place {
  int col, skip;
};
template <int V> __device__ __forceinline__ Place place(int col, int k) {
  const int at = col < k - V ? col : k - V;
  return Place{at, col - at};
}
template <int T, int V> __device__ __forceinline__ Vec<T, V> load(const typename Mem<T>::E* p) {
  return reinterpret_cast<const Loose<T, V>*>(p)->v;
}
// the same, past the caches: values that are read once
template <int T, int V> __device__ __forceinline__ Vec<T, V> load_once(const typename Mem<T>::E* p) {
  constexpr int all = sizeof(Vec<T, V>), N = all > 16 ? 16 : all;
  if constexpr (N < 4) {
    return load<T, V>(p);
  } else {
    typename Words<N>::T w[all / N];
#pragma unroll
    for (int i = 0; i < all / N; ++i) w[i] = __builtin_nontemporal_load(reinterpret_cast<const typename Words<N>::T*>(p) + i);
    Vec<T, V> v;
    __builtin_memcpy(&v, w, all);
    return v;
  }
}
// The compiler knows nothing of v from here on: what it has made of v before
// (wider numbers, differences) is made again and not kept in registers meanwhile.
template <int T, int V> __device__ __forceinline__ void forget(Vec<T, V>& v) {
  if constexpr (sizeof(v) % 4 == 0) {
    uint32_t w[sizeof(v) / 4];
    __builtin_memcpy(w, &v, sizeof(v));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(v) / 4); ++i) asm("" : "+v"(w[i]));
    __builtin_memcpy(&v, w, sizeof(v));
  }
}

// element `col` of a row that begins at the same address in every lane: its byte
// offset in 32 bits, so that the address takes one vector register, not two
template <class E> __device__ __forceinline__ E* at_col(E* row, int col) {
  typedef typename std::conditional<std::is_const<E>::value, const uint8_t, uint8_t>::type B;
  return reinterpret_cast<E*>(reinterpret_cast<B*>(row) + (uint32_t)(col * (int)sizeof(E)));
}
// the columns that are this thread's own
template <int T, int V, bool STREAM = false>
__device__ __forceinline__ void store_own(typename Mem<T>::E* row, Place at, const float (&f)[V]) {
  typename Mem<T>::E* p = at_col(row, at.col);
  if (at.skip == 0) {
    store<T, V, STREAM>(p, f, V);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= at.skip) p[i] = from_f32<T>(f[i]);
  }
}

// ---------------------------------------------------------------- reductions over a wave

// x of another lane of the wave: DPP control words, and lane 63's value after the last
template <int CTRL, int ROWS> __device__ __forceinline__ float dpp(float x, float none) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x), CTRL,
                                                               ROWS, 0xf, false));
}
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp(double x, double none) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x), n = __builtin_bit_cast(uint64_t, none);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)n, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(n >> 32), (int)(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the wave's 64 lanes in a fixed order, in every lane: pairs, fours,
// eights and sixteens within each row of 16 lanes, then row after row.
template <class F> __device__ __forceinline__ F wave_sum(F x) {
  x += dpp<0xB1, 0xf>(x, (F)0);                 // quad_perm [1,0,3,2]
  x += dpp<0x4E, 0xf>(x, (F)0);                 // quad_perm [2,3,0,1]
  x += dpp<0x141, 0xf>(x, (F)0);                // row_half_mirror
  x += dpp<0x140, 0xf>(x, (F)0);                // row_mirror
  return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}
__device__ __forceinline__ float wave_max(float x) {
  x = larger(x, dpp<0xB1, 0xf>(x, x));
  x = larger(x, dpp<0x4E, 0xf>(x, x));
  x = larger(x, dpp<0x141, 0xf>(x, x));
  x = larger(x, dpp<0x140, 0xf>(x, x));
  return larger(larger(lane_value(x, 0), lane_value(x, 16)), larger(lane_value(x, 32), lane_value(x, 48)));
}

}  // namespace step
}  // namespace sbl
