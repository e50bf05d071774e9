// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: out[t] = scale * table[id[t]], one rounding to the output's type; a
// negative id gives zeros, an id past the table NaNs.  Bound by memory.
//
// Backward: dtable[v] = scale * sum of dout[t] over the tokens t with id[t] = v,
// in fp32, in ascending t, rounded once (added to what dtable holds first, if
// asked).  Without atomics on floats, so results repeat bit for bit.  Few tokens:
// few_kernel alone.  More:
//  1. sort_kernel: the tokens id by id, equal ids in order of t (`pos`, with
//     their ids `key`), and where each id's run lies (`run`).  Of 2^s workgroups
//     each owns the ids of one remainder by 2^s (neighbouring ids are often
//     alike in how many tokens they have: vocabularies are numbered by
//     frequency) and reads all token ids: to count its own, and those of
//     smaller remainders, after which its part of the order begins, so that no
//     workgroup waits for another.
//  2. sum_kernel: the sorted tokens in segments of S, a workgroup per segment
//     and chunk of columns, sums in registers while it walks its tokens.  A
//     run belongs to the segment that it begins in; a run longer than S (text
//     has a few ids that are a few per cent of all tokens) is split at the
//     segments' borders into fp32 partial rows.  Rows without a token are
//     zeroed by further workgroups of the launch (not when adding).
//  3. join_kernel: the partial rows of each long run, in order.
// Measured: 65536 tokens of 32000 ids x 3200 BF16 18 + 132 + 6 us (4.7 TB/s in
// sum_kernel); 16384 of 128256 x 5120, added, from fp32, 10 + 95 + 5 (5.1).
// sort_kernel's bound is every workgroup's pass over all ids (8 bytes each, from
// L2): 262144 tokens 51 us at least.
#include "sbl_host.h"
#include "sbl_step.h"

namespace sbl {
namespace step {

namespace {

// ---------------------------------------------------------------- forward

constexpr int kThreads = 256;

// n / d for n < 2^31: the factor is off by e < d <= 2^s, and n e < 2^(31 + s)
// leaves the quotient whole
struct Divider {
  uint32_t factor;
  int shift;
};
Divider divider(uint32_t d) {
  int s = 0;
  while ((uint64_t(1) << s) < d) ++s;            // 2^(s-1) < d <= 2^s: the factor lies in [2^31, 2^32)
  return Divider{(uint32_t)(((uint64_t(1) << (31 + s)) + d - 1) / d), 31 + s};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, Divider d) { return (uint32_t)(((uint64_t)n * d.factor) >> d.shift); }

// The output as one sequence of values, cut into vectors of V from its start
// whatever a row's length is, U of each thread: the ids, then the rows, of all U
// are in flight together, and stores are whole aligned vectors side by side.  A
// vector in which rows meet is taken value by value.  STREAM: many vectors,
// stored past the caches (16384 x 5120 BF16: 74 -> 50 us).
template <int TT, int TO, int V, int U, bool STREAM>
__global__ __launch_bounds__(kThreads) void embed_kernel(const EmbedArgs a, Divider by_k, uint32_t values) {
  typedef typename Mem<TT>::E ET;
  typedef typename Mem<TO>::E EO;
  const uint32_t k = (uint32_t)a.k, first = (blockIdx.x * (kThreads * U) + threadIdx.x) * V;
  const ET* table = static_cast<const ET*>(a.table);
  EO* out = static_cast<EO*>(a.out);
  auto inside = [&](int64_t id) { return id >= 0 && id < a.n_vocab; };
  auto value = [&](float x, int64_t id) { return id < 0 ? 0.0f : id >= a.n_vocab ? __builtin_nanf("") : x * a.scale; };
  uint32_t col[U];
  int64_t id[U];
  Vec<TT, V> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t n = first + u * (kThreads * V), row = divide(n < values ? n : 0, by_k);
    col[u] = (n < values ? n : 0) - row * k;
    id[u] = a.ids[row];
  }
#pragma unroll
  for (int u = 0; u < U; ++u)                    // whole vectors of the table alone (moved back where rows meet)
    v[u] = load<TT, V>(table + (inside(id[u]) ? id[u] * k : 0) + (col[u] < k - V ? col[u] : k - V));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t n = first + u * (kThreads * V);
    if (n >= values) break;
    float f[V];
    if (col[u] + V <= k) {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = value(v[u][j], id[u]);
      store<TO, V, STREAM>(out + n, f, V);
    } else {
      const uint32_t row = divide(n, by_k);
      for (uint32_t j = 0; j < V && n + j < values; ++j) {
        const bool next = col[u] + j >= k;
        const int64_t at = next ? a.ids[row + 1] : id[u];
        const uint32_t c = next ? col[u] + j - k : col[u] + j;
        out[n + j] = from_f32<TO>(value(inside(at) ? to_f32<TT>(table[at * k + c]) : 0.0f, at));
      }
    }
  }
}

template <int TT, int TO, int V, int U, bool STREAM> hipError_t forward_vectors(const EmbedArgs& a, hipStream_t s) {
  // rows of one launch: values are numbered in 31 bits, and every launch begins at a whole vector
  const int64_t most = ((int64_t(1) << 30) / a.k + 7) / 8 * 8;
  for (int64_t r = 0; r < a.m_tok; r += most) {
    EmbedArgs part = a;
    part.m_tok = a.m_tok - r < most ? a.m_tok - r : most;
    part.ids = a.ids + r;
    part.out = static_cast<typename Mem<TO>::E*>(a.out) + r * a.k;
    const uint32_t values = (uint32_t)(part.m_tok * a.k), each = kThreads * U * V;
    hipLaunchKernelGGL((embed_kernel<TT, TO, V, U, STREAM>), dim3((values + each - 1) / each), dim3(kThreads), 0, s, part,
                       divider((uint32_t)a.k), values);
  }
  return hipGetLastError();
}

template <int TT, int TO> hipError_t forward(const EmbedArgs& a, hipStream_t s) {
  // 16 bytes of the output (two such stores of a thread would each write half lines)
  constexpr int V = TO == kFp32 ? 4 : 8;
  if (a.k < V) return forward_vectors<TT, TO, 1, 1, false>(a, s);
  // few vectors: one of each thread, so that there are more waves
  if (a.m_tok * a.k < 4 * V * 1024 * kThreads) return forward_vectors<TT, TO, V, 1, false>(a, s);
  return forward_vectors<TT, TO, V, 4, true>(a, s);
}

// ---------------------------------------------------------------- backward: order

constexpr int kSortWaves = 16;
constexpr int kSortThreads = 64 * kSortWaves;
constexpr int kMaxRange = 1024;                  // ids per workgroup: a thread each, counters of 64 KB

// where the tokens of an id lie in the order
struct Run {
  int32_t begin, end;
};
// Workspace
struct Order {
  Run* run;                                      // [n_vocab + 1]; the last: all tokens
  int32_t* key;                                  // [m_tok] ids in order
  int32_t* pos;                                  // [m_tok] their tokens
};

struct SortArgs {
  const int64_t* ids;
  int32_t m_tok, n_vocab, bits, range;           // the workgroup's ids: d 2^bits + blockIdx.x, d < range
  Order o;
};

// Tokens that a wave remembers from its count.  More, and it reads the ids a second
// time: 262144 tokens of 131072 ids, the most frequent 3 per cent of them, 129 us
// with 192 and 58 with 768 (evenly drawn 51, all tokens of one id 298).
constexpr int kListed = 768;

__device__ __forceinline__ uint64_t lanes_below() { return (uint64_t(1) << (threadIdx.x & 63)) - 1; }

// f(t, id) for 64 tokens at a time of [t0, t1), the ids of 1024 in flight
// together; an id below 0 or past 32 bits comes as 2^32 - 1
template <class F> __device__ __forceinline__ void scan(const int64_t* ids, int t0, int t1, F f) {
  constexpr int U = 16;
  const int lane = threadIdx.x & 63;
  int t = t0;
  for (; t + 64 * U <= t1; t += 64 * U) {
    const uint2* p = reinterpret_cast<const uint2*>(ids) + t + lane;
    uint2 id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = p[64 * u];
#pragma unroll
    for (int u = 0; u < U; ++u) f(t + 64 * u + lane, id[u].y == 0 ? id[u].x : 0xFFFFFFFFu);
  }
  if (t >= t1) return;
  uint2 id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = t + 64 * u + lane;
    id[u] = reinterpret_cast<const uint2*>(ids)[at < t1 ? at : t1 - 1];
    if (at >= t1) id[u].y = 1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (t + 64 * u < t1) f(t + 64 * u + lane, id[u].y == 0 ? id[u].x : 0xFFFFFFFFu);
}

__global__ __launch_bounds__(kSortThreads) void sort_kernel(const SortArgs a) {
  extern __shared__ uint32_t count[];            // [wave][range]: counts, then the next place
  __shared__ uint32_t below[kSortWaves], sums[kSortWaves];
  __shared__ uint32_t list[kSortWaves][kListed]; // (token - t0) 2^10 + d, in order
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t mine0 = blockIdx.x, mask = (1u << a.bits) - 1;
  const uint32_t range = (uint32_t)a.range;
  for (uint32_t i = tid; i < kSortWaves * (uint32_t)a.range; i += kSortThreads) count[i] = 0;
  __syncthreads();
  // each wave takes a stretch of the tokens
  const int per = ((a.m_tok + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int t0 = wave * per, t1 = t0 + per < a.m_tok ? t0 + per : a.m_tok;
  uint32_t* mine = count + wave * a.range;
  uint32_t low = 0, listed = 0;                  // of the wave
  scan(a.ids, t0, t1, [&](int t, uint32_t id) {
    const uint32_t rest = id & mask;
    const uint64_t known = __ballot(id < (uint32_t)a.n_vocab);
    low += (uint32_t)__builtin_popcountll(known & __ballot(rest < mine0));
    const uint64_t inside = known & __ballot(rest == mine0);
    if (!inside) return;
    if (inside >> lane & 1) {
      const uint32_t d = id >> a.bits;
      atomicAdd(&mine[d], 1u);
      const uint32_t at = listed + (uint32_t)__builtin_popcountll(inside & lanes_below());
      if (at < kListed) list[wave][at] = (uint32_t)(t - t0) << 10 | d;
    }
    listed += (uint32_t)__builtin_popcountll(inside);
  });
  if (lane == 0) below[wave] = low;
  __syncthreads();
  // places of the workgroup's id `tid`: after the tokens of smaller remainders, the ids before it, the waves before each
  uint32_t total = 0;
  if (tid < (int)range)
    for (int w = 0; w < kSortWaves; ++w) total += count[w * a.range + tid];
  uint32_t upto = total;                         // inclusive scan over the workgroup
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t o = __shfl_up(upto, m, 64);
    if (lane >= m) upto += o;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  uint32_t base = upto - total;
  for (int w = 0; w < kSortWaves; ++w) base += below[w] + (w < wave ? sums[w] : 0);
  if (tid < (int)range) {
    const uint32_t v = ((uint32_t)tid << a.bits) + mine0;
    if (v < (uint32_t)a.n_vocab) a.o.run[v] = Run{(int32_t)base, (int32_t)(base + total)};
    // the last of all: past its last id no workgroup has a token
    if (tid == (int)range - 1 && blockIdx.x == gridDim.x - 1) a.o.run[a.n_vocab] = Run{0, (int32_t)(base + total)};
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t n = count[w * a.range + tid];
      count[w * a.range + tid] = base;
      base += n;
    }
  }
  __syncthreads();
  // 64 tokens of this wave in order, those inside the range (d < range) to their places
  auto put = [&](int t, uint32_t d) {
    uint64_t left = __ballot(d < range);
    while (left) {                               // the distinct ids among them
      const int first = __builtin_ctzll(left);
      const uint32_t which = (uint32_t)__builtin_amdgcn_readlane((int)d, first);
      const uint64_t group = __ballot(d == which);
      const uint32_t place = mine[which];        // this wave's counters: no other wave touches them
      if (d == which) {
        const uint32_t at = place + (uint32_t)__builtin_popcountll(group & lanes_below());
        a.o.key[at] = (int32_t)((d << a.bits) + mine0);
        a.o.pos[at] = t;
      }
      if (lane == first) mine[which] = place + (uint32_t)__builtin_popcountll(group);
      __builtin_amdgcn_wave_barrier();
      left &= ~group;
    }
  };
  if (listed <= kListed) {
    for (uint32_t i = 0; i < listed; i += 64) {
      const bool has = i + lane < listed;
      const uint32_t e = has ? list[wave][i + lane] : 0;
      put(t0 + (int)(e >> 10), has ? e & 1023u : range);
    }
  } else {                                       // too many to remember: read the ids again
    scan(a.ids, t0, t1, [&](int t, uint32_t id) {
      put(t, id < (uint32_t)a.n_vocab && (id & mask) == mine0 ? id >> a.bits : range);
    });
  }
}

// ---------------------------------------------------------------- backward: sums

// Up to here few_kernel.  777 tokens of 50257 ids x 1541 FP16 33 us, by the three
// kernels 39; 256 of 32000 x 3200, added, 11 and 18; but all of one id 23 and 14
// (1024 tokens x 3200: 108 and 26), for one workgroup then adds them up.
constexpr int kFewTokens = 1024;

struct SumArgs {
  const int64_t* ids;
  const void* dout;
  void* dtable;
  int32_t m_tok, n_vocab, k;
  float scale;
  int32_t segment;                               // S
  int32_t segments, chunks;                      // of columns: chunk_vecs vectors each
  int32_t chunk_vecs;
  int32_t zero_groups, zero_rows;                // workgroups that zero rows, after the others; rows of each wave
  Order o;
  float* part;                                   // [segments][2][k]: what a long run has in a segment that it comes
                                                 //   into [0], or begins in [1]
};

// One row's columns to memory.  LINES: rows are whole 128-byte lines, stored past
// the caches.
template <int TT, int V, bool ADD, bool LINES>
__device__ __forceinline__ void put(typename Mem<TT>::E* row, Place c, const float (&sum)[V], float scale,
                                    const Vec<TT, V>& old) {
  float f[V];
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = ADD ? old[j] + sum[j] * scale : sum[j] * scale;
  store_own<TT, V, LINES>(row, c, f);
}

// Zeros in the rows v0 + i of the bits i of `empty`.  Neighbouring ones are one
// stretch of memory, whose 128-byte lines are stored whole and past the caches
// (rows of an odd length begin anywhere; lines in parts past the caches are slower
// than within them).  One wave.
template <class E> __device__ __forceinline__ void zero_rows(E* table, uint64_t empty, int k, int v0) {
  const int lane = threadIdx.x & 63;
  while (empty) {
    const int from = __builtin_ctzll(empty);
    const uint64_t rest = ~(empty >> from);
    const int rows = rest ? __builtin_ctzll(rest) : 64 - from;
    empty = from + rows < 64 ? empty >> (from + rows) << (from + rows) : 0;
    E* p = table + (int64_t)(v0 + from) * k;
    const int64_t values = (int64_t)rows * k;
    const int per = 128 / (int)sizeof(E);        // at most 64: an edge is a value a lane
    int64_t head = (128 - (reinterpret_cast<uintptr_t>(p) & 127)) % 128 / sizeof(E);
    if (head > values) head = values;
    const int64_t lines = (values - head) / per, tail = head + lines * per;
    if (lane < head) p[lane] = (E)0;
    u32x4* piece = reinterpret_cast<u32x4*>(p + head);
    for (int64_t i = lane; i < lines * 8; i += 64) __builtin_nontemporal_store(u32x4{}, piece + i);
    if (tail + lane < values) p[tail + lane] = (E)0;
  }
}

template <int TD, int TT, int V, bool ADD, bool LINES> __global__ __launch_bounds__(kThreads) void sum_kernel(const SumArgs a) {
  typedef typename Mem<TD>::E ED;
  typedef typename Mem<TT>::E ET;
  ET* table = static_cast<ET*>(a.dtable);
  const int work = a.segments * a.chunks;
  const int lane = threadIdx.x & 63;
  if constexpr (!ADD) {
    if ((int)blockIdx.x >= work) {               // rows without a token
      const int wave = ((int)blockIdx.x - work) * (int)(blockDim.x >> 6) + (int)(threadIdx.x >> 6);
      const int v0 = wave * a.zero_rows, left = a.n_vocab - v0, n = left < a.zero_rows ? left : a.zero_rows;
      if (n <= 0) return;
      const Run mine = a.o.run[v0 + (lane < n ? lane : 0)];
      zero_rows(table, __ballot(lane < n && mine.begin == mine.end), a.k, v0);
      return;
    }
  }
  const int seg = (int)blockIdx.x / a.chunks, chunk = (int)blockIdx.x - seg * a.chunks;
  const int total = a.o.run[a.n_vocab].end, S = a.segment;
  const int i0 = seg * S;
  if (i0 >= total) return;
  const int i1 = i0 + S < total ? i0 + S : total;
  // (a thread past the chunk: no column of its own)
  const Place c = place<V>((int)threadIdx.x < a.chunk_vecs ? (chunk * a.chunk_vecs + (int)threadIdx.x) * V : a.k + V, a.k);
  // the tokens of this segment: from the first run that begins in it (or from
  // its start, inside a long run) to the end of the last one that begins in it
  // (or to its own end, inside a long run)
  const Run head = a.o.run[a.o.key[i0]], tail = a.o.run[a.o.key[i1 - 1]];
  const bool long_head = head.begin < i0 && head.end - head.begin > S;
  const bool long_tail = tail.end > i1 && tail.end - tail.begin > S;
  const int from = head.begin == i0 || long_head ? i0 : head.end;
  const int to = long_tail ? i1 : tail.end;
  const ED* dout = static_cast<const ED*>(a.dout);
  float sum[V] = {};
  constexpr int U = 8;                           // tokens whose loads are in flight
  for (int i = from; i < to; i += 64) {
    const int n = to - i < 64 ? to - i : 64;
    const int key = lane < n ? a.o.key[i + lane] : -1;
    const int pos = lane < n ? a.o.pos[i + lane] : 0;
    // the last token of its run among these (of a run that goes on: the very last, -1 here, if it ends there)
    const int after = i + lane + 1 < to ? (lane < n ? a.o.key[i + lane + 1] : -1) : -1;
    const uint64_t ends = __ballot(lane < n && after != key);
    for (int j = 0; j < n; j += U) {
      Vec<TD, V> d[U];
      Vec<TT, V> old[ADD ? U : 1];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + u >= n) break;
        const int t = __builtin_amdgcn_readlane(pos, j + u);
        d[u] = load_once<TD, V>(at_col(dout + (int64_t)t * a.k, c.col));
        if constexpr (ADD) {
          if (ends >> (j + u) & 1)
            old[u] = load<TT, V>(at_col(table + (int64_t)__builtin_amdgcn_readlane(key, j + u) * a.k, c.col));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + u >= n) break;
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += d[u][e];
        if (ends >> (j + u) & 1) {
          const int v = __builtin_amdgcn_readlane(key, j + u), at = i + j + u;
          const bool in_head = long_head && at < head.end, in_tail = long_tail && at == to - 1;
          if (in_head || in_tail) {
            const bool begins = in_tail && tail.begin >= i0;
            store_own<kFp32, V>(a.part + ((int64_t)seg * 2 + begins) * a.k, c, sum);
          } else {
            put<TT, V, ADD, LINES>(table + (int64_t)v * a.k, c, sum, a.scale, old[ADD ? u : 0]);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) sum[e] = 0.0f;
        }
      }
    }
  }
}

// The long run that begins in segment blockIdx.x / chunks, if one does (a run
// longer than a segment leaves no room for a second one).
template <int TT, int V, bool ADD, bool LINES> __global__ __launch_bounds__(kThreads) void join_kernel(const SumArgs a) {
  typedef typename Mem<TT>::E ET;
  const int seg = (int)blockIdx.x / a.chunks, chunk = (int)blockIdx.x - seg * a.chunks;
  const int total = a.o.run[a.n_vocab].end, S = a.segment;
  const int i0 = seg * S;
  if (i0 >= total) return;
  const int i1 = i0 + S < total ? i0 + S : total;
  const int v = a.o.key[i1 - 1];
  const Run r = a.o.run[v];
  if (r.begin < i0 || r.end <= i1 || r.end - r.begin <= S) return;
  if ((int)threadIdx.x >= a.chunk_vecs) return;
  const Place c = place<V>((chunk * a.chunk_vecs + (int)threadIdx.x) * V, a.k);
  ET* row = static_cast<ET*>(a.dtable) + (int64_t)v * a.k;
  Vec<TT, V> old{};
  if constexpr (ADD) old = load<TT, V>(at_col(row, c.col));
  float sum[V];
  const Vec<kFp32, V> first = load<kFp32, V>(at_col(a.part + ((int64_t)seg * 2 + 1) * a.k, c.col));
#pragma unroll
  for (int e = 0; e < V; ++e) sum[e] = first[e];
  const int last = (r.end - 1) / S;
#pragma unroll 8
  for (int s = seg + 1; s <= last; ++s) {
    const Vec<kFp32, V> p = load<kFp32, V>(at_col(a.part + (int64_t)s * 2 * a.k, c.col));
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] += p[e];
  }
  put<TT, V, ADD, LINES>(row, c, sum, a.scale, old);
}

// Few tokens: the whole gradient in one launch, without an order.  A workgroup per
// token and chunk of columns looks for the token's id among all ids; the first
// token of an id sums those of all.
template <int TD, int TT, int V, bool ADD, bool LINES> __global__ __launch_bounds__(kThreads) void few_kernel(const SumArgs a) {
  typedef typename Mem<TT>::E ET;
  __shared__ int32_t key[kFewTokens];
  __shared__ uint16_t same[kFewTokens];          // tokens of this workgroup's id, in order
  __shared__ int many;
  ET* table = static_cast<ET*>(a.dtable);
  const int lane = threadIdx.x & 63, work = a.m_tok * a.chunks;
  for (int t = threadIdx.x; t < a.m_tok; t += blockDim.x) {
    const int64_t id = a.ids[t];
    key[t] = id >= 0 && id < a.n_vocab ? (int32_t)id : -1;
  }
  __syncthreads();
  if constexpr (!ADD) {
    if ((int)blockIdx.x >= work) {               // rows without a token
      const int wave = ((int)blockIdx.x - work) * (int)(blockDim.x >> 6) + (int)(threadIdx.x >> 6);
      const int v0 = wave * a.zero_rows, left = a.n_vocab - v0, n = left < a.zero_rows ? left : a.zero_rows;
      if (n <= 0) return;
      uint64_t seen = 0;
      for (int t = lane; t < a.m_tok; t += 64) {
        const uint32_t d = (uint32_t)(key[t] - v0);
        if (key[t] >= v0 && d < 64) seen |= uint64_t(1) << d;
      }
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) seen |= (uint64_t)__shfl_xor((unsigned long long)seen, m, 64);
      zero_rows(table, ~seen & (n < 64 ? (uint64_t(1) << n) - 1 : ~uint64_t(0)), a.k, v0);
      return;
    }
  }
  const int token = (int)blockIdx.x / a.chunks, chunk = (int)blockIdx.x - token * a.chunks, v = key[token];
  if (v < 0) return;
  if (threadIdx.x < 64) {
    int n = 0;
    for (int t = 0; t < a.m_tok; t += 64) {
      const uint64_t hit = __ballot(t + lane < a.m_tok && key[t + lane < a.m_tok ? t + lane : 0] == v);
      if (hit >> lane & 1) same[n + __builtin_popcountll(hit & lanes_below())] = (uint16_t)(t + lane);
      n += __builtin_popcountll(hit);
    }
    if (lane == 0) many = n;
  }
  __syncthreads();
  if (same[0] != token) return;
  const Place c = place<V>((int)threadIdx.x < a.chunk_vecs ? (chunk * a.chunk_vecs + (int)threadIdx.x) * V : a.k + V, a.k);
  const typename Mem<TD>::E* dout = static_cast<const typename Mem<TD>::E*>(a.dout);
  ET* row = table + (int64_t)v * a.k;
  Vec<TT, V> old{};
  if constexpr (ADD) old = load<TT, V>(at_col(row, c.col));
  float sum[V] = {};
  constexpr int U = 8;                           // tokens whose loads are in flight
  for (int i = 0; i < many; i += 64) {
    const int n = many - i < 64 ? many - i : 64, pos = lane < n ? same[i + lane] : 0;
    for (int j = 0; j < n; j += U) {
      Vec<TD, V> d[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + u >= n) break;
        d[u] = load_once<TD, V>(at_col(dout + (int64_t)__builtin_amdgcn_readlane(pos, j + u) * a.k, c.col));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + u >= n) break;
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += d[u][e];
      }
    }
  }
  put<TT, V, ADD, LINES>(row, c, sum, a.scale, old);
}

// `words` 16-bit zeros, 16-byte aligned
__global__ __launch_bounds__(kThreads) void zero_kernel(uint16_t* p, int64_t words) {
  const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t i = t; i < words / 8; i += (int64_t)gridDim.x * kThreads) reinterpret_cast<u32x4*>(p)[i] = u32x4{};
  if (t < words % 8) p[words / 8 * 8 + t] = 0;
}

constexpr int64_t kAlign = 256;
int64_t rounded(int64_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

struct Plan {
  int bits, range, groups;                       // sorting workgroups: at most 2^bits, of `range` ids
  int vec;                                       // columns per thread
  int chunks, chunk_vecs, threads;
  int segment, segments;
  int64_t run, key, pos, part, bytes;          // the workspace
};

Plan plan_of(int64_t m_tok, int64_t n_vocab, int64_t k, int dout_type) {
  Plan p{};
  p.bits = 8;
  while ((n_vocab - 1) >> p.bits >= kMaxRange) ++p.bits;   // a wave remembers d in 10 bits
  p.range = (int)(((n_vocab - 1) >> p.bits) + 1);
  p.groups = (int)(n_vocab < int64_t(1) << p.bits ? n_vocab : int64_t(1) << p.bits);
  p.vec = dout_type == kFp32 ? 4 : 8;
  if (k < p.vec) p.vec = 1;
  const int64_t nv = (k + p.vec - 1) / p.vec;
  p.chunks = (int)((nv + kThreads - 1) / kThreads);
  // whole 128-byte lines to a chunk, whatever the table's type
  p.chunk_vecs = (int)(((nv + p.chunks - 1) / p.chunks + 15) / 16 * 16);
  p.threads = (p.chunk_vecs + 63) / 64 * 64;
  // long enough that partial rows are few, short enough that a batch makes 16 waves a CU
  p.segment = 64;
  while (p.segment > 8 && (m_tok / p.segment) * p.chunks * p.threads < 4096 * 64) p.segment /= 2;
  while (m_tok / p.segment > 4096) p.segment *= 2;
  p.segments = (int)((m_tok + p.segment - 1) / p.segment);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += rounded(bytes);
    return o;
  };
  p.run = take((n_vocab + 1) * 8);
  p.key = take(m_tok * 4);
  p.pos = take(m_tok * 4);
  p.part = take((int64_t)p.segments * 2 * k * 4);
  p.bytes = at;
  return p;
}

template <int TD, int TT, int V, bool ADD, bool LINES> hipError_t sums(const SumArgs& a, bool few, hipStream_t s) {
  const dim3 block((unsigned)((a.chunk_vecs + 63) / 64 * 64)), work((unsigned)(a.segments * a.chunks));
  const unsigned zero = ADD ? 0u : (unsigned)a.zero_groups;
  if (few) {
    hipLaunchKernelGGL((few_kernel<TD, TT, V, ADD, LINES>), dim3((unsigned)(a.m_tok * a.chunks) + zero), block, 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((sum_kernel<TD, TT, V, ADD, LINES>), dim3(work.x + zero), block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // (more tokens than few_kernel takes are always more than a segment: a run may be longer than one)
  hipLaunchKernelGGL((join_kernel<TT, V, ADD, LINES>), work, block, 0, s, a);
  return hipGetLastError();
}

template <int TD, int TT, int V, bool ADD> hipError_t by_row_length(const SumArgs& a, bool few, hipStream_t s) {
  if (a.k < V) return sums<TD, TT, 1, ADD, false>(a, few, s);
  if (a.k * type_bytes(TT) % 128 == 0 && reinterpret_cast<uintptr_t>(a.dtable) % 128 == 0)
    return sums<TD, TT, V, ADD, true>(a, few, s);
  return sums<TD, TT, V, ADD, false>(a, few, s);
}

template <int TD, int TT, int V> hipError_t backward(const SumArgs& a, bool add, bool few, hipStream_t s) {
  return add ? by_row_length<TD, TT, V, true>(a, few, s) : by_row_length<TD, TT, V, false>(a, few, s);
}

}  // namespace

hipError_t launch_embed_forward(const EmbedArgs& a, int tt, int to, hipStream_t s) {
  return with_types(tt, to, [&](auto t, auto o) { return forward<t.value, o.value>(a, s); });
}

int64_t embed_grad_ws_bytes(int64_t m_tok, int64_t n_vocab, int64_t k, int out_type) {
  return plan_of(m_tok, n_vocab, k, out_type).bytes;
}

hipError_t launch_embed_backward(const EmbedGradArgs& g, int td, int tt, hipStream_t s) {
  if (g.m_tok == 0) {                            // no token (and nothing to add): zeros
    const int64_t words = g.n_vocab * g.k * type_bytes(tt) / 2, want = (words + 8 * kThreads - 1) / (8 * kThreads);
    hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(want < 4096 ? want : 4096)), dim3(kThreads), 0, s,
                       static_cast<uint16_t*>(g.dtable), words);
    return hipGetLastError();
  }
  const Plan p = plan_of(g.m_tok, g.n_vocab, g.k, td);
  uint8_t* ws = static_cast<uint8_t*>(g.ws);
  const Order o{reinterpret_cast<Run*>(ws + p.run), reinterpret_cast<int32_t*>(ws + p.key),
                reinterpret_cast<int32_t*>(ws + p.pos)};
  const SortArgs sa{g.ids, (int32_t)g.m_tok, (int32_t)g.n_vocab, p.bits, p.range, o};
  const bool few = g.m_tok <= kFewTokens;
  if (!few) {
    static LdsLimit limit;
    hipError_t e = limit.raise((const void*)sort_kernel, kSortWaves * kMaxRange * 4);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sort_kernel, dim3((unsigned)p.groups), dim3(kSortThreads), (size_t)kSortWaves * p.range * 4, s, sa);
    e = hipGetLastError();                       // without an order the sums would read and write anywhere
    if (e != hipSuccess) return e;
  }
  // rows to zero: a few of each wave, so that there are many waves; at most 64 (the bits of a mask)
  int64_t zero_rows = 4;
  while (zero_rows < 64 && g.n_vocab / zero_rows > 8192) zero_rows *= 2;
  const int64_t rows = zero_rows * (p.threads / 64), zero = (g.n_vocab + rows - 1) / rows;
  const SumArgs a{g.ids, g.dout, g.dtable, (int32_t)g.m_tok, (int32_t)g.n_vocab, g.k, g.scale, p.segment, p.segments, p.chunks,
                  p.chunk_vecs, (int32_t)zero, (int32_t)zero_rows, o, reinterpret_cast<float*>(ws + p.part)};
  return with_types(td, tt, [&](auto d, auto t) { return backward<d.value, t.value, d.value == kFp32 ? 4 : 8>(a, g.add, few, s); });
}

}  // namespace step
}  // namespace sbl
