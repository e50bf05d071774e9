// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: out[t] = scale * table[id[t]], one rounding to the output's type; a
// negative id gives zeros, an id past the table NaNs.  Bound by memory.
//
// Backward: dtable[v] = scale * sum of dout[t] over the tokens t with id[t] = v,
// in fp32, in ascending t, rounded once (added to what dtable holds first, if
// asked).  Without atomics on floats, so results repeat bit for bit:
//  1. sort_kernel: the tokens in order of their ids, equal ids in order of t
//     (`pos`, with their ids `key`), and where each id's run begins (`start`).
//     Every workgroup owns a range of ids and reads all token ids twice: once
//     to count (its own ids, and how many tokens lie below its range: that is
//     where its part of the order begins, so that no workgroup waits for
//     another), once to place.
//  2. sum_kernel: the sorted tokens in segments of S, a workgroup per segment
//     and chunk of columns, sums in registers while it walks its tokens.  A
//     run belongs to the segment that it begins in; a run longer than S (text
//     has a few ids that are a few per cent of all tokens) is split at the
//     segments' borders into fp32 partial rows.  Rows without a token are
//     zeroed by further workgroups of the launch (not when adding).
//  3. join_kernel: the partial rows of each long run, in order.
#include "sbl_step.h"

namespace sbl {
namespace step {

namespace {

// ---------------------------------------------------------------- forward

constexpr int kThreads = 256;

// tx threads (a power of two) side by side in a row, V values each
template <int TT, int TO, int V>
__global__ __launch_bounds__(kThreads) void embed_kernel(const EmbedArgs a, int tx) {
  typedef typename Mem<TT>::E ET;
  typedef typename Mem<TO>::E EO;
  const int x = threadIdx.x & (tx - 1), y = threadIdx.x / tx, ty = kThreads / tx;
  const int64_t row = (int64_t)blockIdx.x * ty + y;
  if (row >= a.m_tok) return;
  const int64_t id = a.ids[row];
  EO* out = static_cast<EO*>(a.out) + row * a.k;
  const bool here = id >= 0 && id < a.n_vocab;
  const ET* in = static_cast<const ET*>(a.table) + (here ? id * a.k : 0);
  const float fill = id < 0 ? 0.0f : __builtin_nanf("");
  const int step = tx * V * gridDim.y;
  for (int c = (blockIdx.y * tx + x) * V; c < a.k; c += 4 * step) {
    Vec<TT, V> v[4] = {};
    if (here) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + u * step < a.k) v[u] = load<TT, V>(in + c + u * step, a.k - c - u * step);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (c + u * step >= a.k) break;
      float f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = here ? v[u][j] * a.scale : fill;
      store<TO, V>(out + c + u * step, f, a.k - c - u * step);
    }
  }
}

template <int TT, int TO> hipError_t forward(const EmbedArgs& a, hipStream_t s) {
  constexpr int V = 8;
  const int nv = (a.k + V - 1) / V;
  int tx = 1;
  while (tx < kThreads && tx < nv) tx *= 2;
  const int64_t gx = (a.m_tok + kThreads / tx - 1) / (kThreads / tx);
  // few rows: a row's columns over several workgroups
  int64_t gy = 1;
  while (gx * gy < 1024 && gy * tx < nv) gy *= 2;
  hipLaunchKernelGGL((embed_kernel<TT, TO, V>), dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), 0, s, a, tx);
  return hipGetLastError();
}

// ---------------------------------------------------------------- backward: order

constexpr int kSortWaves = 16;
constexpr int kSortThreads = 64 * kSortWaves;
constexpr int kMaxRange = 1008;                  // ids per workgroup (63 KB of counters)

// Workspace
struct Order {
  int32_t* start;                                // [n_vocab + 1] first sorted token of each id; the last: how many
  int32_t* key;                                  // [m_tok] ids in order
  int32_t* pos;                                  // [m_tok] their tokens
};

struct SortArgs {
  const int64_t* ids;
  int32_t m_tok, n_vocab, range;                 // ids per workgroup
  Order o;
};

__device__ __forceinline__ uint64_t lanes_below() { return (uint64_t(1) << (threadIdx.x & 63)) - 1; }

__global__ __launch_bounds__(kSortThreads) void sort_kernel(const SortArgs a) {
  extern __shared__ uint32_t count[];            // [wave][range]: counts, then the next place
  __shared__ uint32_t below[kSortWaves], sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t v0 = (int64_t)blockIdx.x * a.range;
  const uint32_t range = (uint32_t)(a.n_vocab - v0 < a.range ? a.n_vocab - v0 : a.range);
  for (uint32_t i = tid; i < kSortWaves * (uint32_t)a.range; i += kSortThreads) count[i] = 0;
  __syncthreads();
  // each wave takes a stretch of the tokens
  const int per = ((a.m_tok + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int t0 = wave * per, t1 = t0 + per < a.m_tok ? t0 + per : a.m_tok;
  uint32_t* mine = count + wave * a.range;
  uint32_t low = 0;
  for (int t = t0; t < t1; t += 256) {
    int64_t id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) id[u] = t + 64 * u + lane < t1 ? a.ids[t + 64 * u + lane] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      low += id[u] >= 0 && id[u] < v0;
      const uint64_t d = (uint64_t)(id[u] - v0);
      if (d < range) atomicAdd(&mine[d], 1u);
    }
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) low += __shfl_xor(low, m, 64);
  if (lane == 0) below[wave] = low;
  __syncthreads();
  // places of id v0 + tid: after the tokens below the range, the ids before it, the waves before each
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
    a.o.start[v0 + tid] = (int32_t)base;
    if (v0 + tid == a.n_vocab - 1) a.o.start[a.n_vocab] = (int32_t)(base + total);
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t n = count[w * a.range + tid];
      count[w * a.range + tid] = base;
      base += n;
    }
  }
  __syncthreads();
  for (int t = t0; t < t1; t += 256) {
    int64_t id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) id[u] = t + 64 * u + lane < t1 ? a.ids[t + 64 * u + lane] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint64_t d = (uint64_t)(id[u] - v0);
      uint64_t left = __ballot(d < range);
      while (left) {                             // the distinct ids among these 64 tokens
        const int first = __builtin_ctzll(left);
        const uint32_t which = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)d, first);
        const bool same = d < range && (uint32_t)d == which;
        const uint64_t group = __ballot(same);
        const uint32_t place = mine[which];      // this wave's counters: no other wave writes them
        if (same) {
          const uint32_t at = place + (uint32_t)__builtin_popcountll(group & lanes_below());
          a.o.key[at] = (int32_t)id[u];
          a.o.pos[at] = t + 64 * u + lane;
        }
        if (lane == first) mine[which] = place + (uint32_t)__builtin_popcountll(group);
        __builtin_amdgcn_wave_barrier();
        left &= ~group;
      }
    }
  }
}

// ---------------------------------------------------------------- backward: sums

struct SumArgs {
  const void* dout;
  void* dtable;
  int32_t m_tok, n_vocab, k;
  float scale;
  int32_t segment;                               // S
  int32_t segments, chunks;                      // of columns: chunk_vecs vectors each
  int32_t chunk_vecs;
  int32_t zero_groups;                           // workgroups that zero rows, after the others
  Order o;
  float* part;                                   // [segments][2][k]: what a long run has in a segment that it comes
                                                 //   into [0], or begins in [1]
};

// one row's columns to memory
template <int TT, int V, bool ADD>
__device__ __forceinline__ void put(typename Mem<TT>::E* row, int have, const float (&sum)[V], float scale,
                                    const Vec<TT, V>& old) {
  float f[V];
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = ADD ? old[j] + sum[j] * scale : sum[j] * scale;
  store<TT, V>(row, f, have);
}

// where the run of id `v` lies
struct Run {
  int begin, end;
};
__device__ __forceinline__ Run run_of(const Order& o, int v) { return Run{o.start[v], o.start[v + 1]}; }

template <int TD, int TT, int V, bool ADD> __global__ __launch_bounds__(kThreads) void sum_kernel(const SumArgs a) {
  typedef typename Mem<TD>::E ED;
  typedef typename Mem<TT>::E ET;
  ET* table = static_cast<ET*>(a.dtable);
  const int work = a.segments * a.chunks;
  const int lane = threadIdx.x & 63;
  if constexpr (!ADD) {
    if ((int)blockIdx.x >= work) {               // rows without a token: a wave each
      const int wave = ((int)blockIdx.x - work) * (kThreads / 64) + (threadIdx.x >> 6);
      const int waves = a.zero_groups * (kThreads / 64);
      for (int v = wave; v < a.n_vocab; v += waves) {
        const Run r = run_of(a.o, v);
        if (r.begin != r.end) continue;
        ET* row = table + (int64_t)v * a.k;
        const float none[V] = {};
        for (int c = lane * V; c < a.k; c += 64 * V) store<TT, V>(row + c, none, a.k - c);
      }
      return;
    }
  }
  const int seg = (int)blockIdx.x / a.chunks, chunk = (int)blockIdx.x - seg * a.chunks;
  const int total = a.o.start[a.n_vocab], S = a.segment;
  const int i0 = seg * S;
  if (i0 >= total) return;
  const int i1 = i0 + S < total ? i0 + S : total;
  const int col = threadIdx.x < a.chunk_vecs ? (chunk * a.chunk_vecs + (int)threadIdx.x) * V : a.k;
  const int have = a.k - col > 0 ? a.k - col : 0;
  // the tokens of this segment: from the first run that begins in it (or from
  // its start, inside a long run) to the end of the last one that begins in it
  // (or to its own end, inside a long run)
  const Run head = run_of(a.o, a.o.key[i0]), tail = run_of(a.o, a.o.key[i1 - 1]);
  const bool long_head = head.begin < i0 && head.end - head.begin > S;
  const bool long_tail = tail.end > i1 && tail.end - tail.begin > S;
  const int from = head.begin == i0 || long_head ? i0 : head.end;
  const int to = long_tail ? i1 : tail.end;
  const ED* dout = static_cast<const ED*>(a.dout) + col;
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
        d[u] = load<TD, V>(dout + (int64_t)t * a.k, have);
        if constexpr (ADD) {
          if (ends >> (j + u) & 1)
            old[u] = load<TT, V>(table + (int64_t)__builtin_amdgcn_readlane(key, j + u) * a.k + col, have);
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
            if (have > 0) store<kFp32, V>(a.part + ((int64_t)seg * 2 + begins) * a.k + col, sum, have);
          } else if (have > 0) {
            put<TT, V, ADD>(table + (int64_t)v * a.k + col, have, sum, a.scale, old[ADD ? u : 0]);
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
template <int TT, int V, bool ADD> __global__ __launch_bounds__(kThreads) void join_kernel(const SumArgs a) {
  typedef typename Mem<TT>::E ET;
  const int seg = (int)blockIdx.x / a.chunks, chunk = (int)blockIdx.x - seg * a.chunks;
  const int total = a.o.start[a.n_vocab], S = a.segment;
  const int i0 = seg * S;
  if (i0 >= total) return;
  const int i1 = i0 + S < total ? i0 + S : total;
  const int v = a.o.key[i1 - 1];
  const Run r = run_of(a.o, v);
  if (r.begin < i0 || r.end <= i1 || r.end - r.begin <= S) return;
  const int col = (chunk * a.chunk_vecs + (int)threadIdx.x) * V, have = a.k - col;
  if ((int)threadIdx.x >= a.chunk_vecs || have <= 0) return;
  ET* row = static_cast<ET*>(a.dtable) + (int64_t)v * a.k + col;
  Vec<TT, V> old{};
  if constexpr (ADD) old = load<TT, V>(row, have);
  float sum[V];
  const Vec<kFp32, V> first = load<kFp32, V>(a.part + ((int64_t)seg * 2 + 1) * a.k + col, have);
#pragma unroll
  for (int e = 0; e < V; ++e) sum[e] = first[e];
  const int last = (r.end - 1) / S;
#pragma unroll 4
  for (int s = seg + 1; s <= last; ++s) {
    const Vec<kFp32, V> p = load<kFp32, V>(a.part + (int64_t)s * 2 * a.k + col, have);
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] += p[e];
  }
  put<TT, V, ADD>(row, have, sum, a.scale, old);
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
  int range, groups;                             // ids per sorting workgroup
  int vec;                                       // columns per thread
  int chunks, chunk_vecs;
  int segment, segments;
  int64_t start, key, pos, part, bytes;          // the workspace
};

Plan plan_of(int64_t m_tok, int64_t n_vocab, int64_t k, int dout_type) {
  Plan p{};
  p.range = (int)((n_vocab + 255) / 256);
  if (p.range > kMaxRange) p.range = kMaxRange;
  p.groups = (int)((n_vocab + p.range - 1) / p.range);
  p.vec = dout_type == kFp32 ? 4 : 8;
  const int64_t nv = (k + p.vec - 1) / p.vec;
  p.chunks = (int)((nv + kThreads - 1) / kThreads);
  p.chunk_vecs = (int)((nv + p.chunks - 1) / p.chunks);
  // long enough that partial rows are few, short enough that a batch makes a workgroup or two per CU
  p.segment = 64;
  while (p.segment > 8 && (m_tok / p.segment) * p.chunks < 1024) p.segment /= 2;
  while (m_tok / p.segment > 4096) p.segment *= 2;
  p.segments = (int)((m_tok + p.segment - 1) / p.segment);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += rounded(bytes);
    return o;
  };
  p.start = take((n_vocab + 1) * 4);
  p.key = take(m_tok * 4);
  p.pos = take(m_tok * 4);
  p.part = take((int64_t)p.segments * 2 * k * 4);
  p.bytes = at;
  return p;
}

template <int TD, int TT, int V, bool ADD> hipError_t sums(const SumArgs& a, bool join, hipStream_t s) {
  hipLaunchKernelGGL((sum_kernel<TD, TT, V, ADD>), dim3((unsigned)(a.segments * a.chunks + (ADD ? 0 : a.zero_groups))),
                     dim3(kThreads), 0, s, a);
  if (join)
    hipLaunchKernelGGL((join_kernel<TT, V, ADD>), dim3((unsigned)(a.segments * a.chunks)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int TD, int TT, int V> hipError_t backward(const SumArgs& a, bool add, bool join, hipStream_t s) {
  return add ? sums<TD, TT, V, true>(a, join, s) : sums<TD, TT, V, false>(a, join, s);
}

}  // namespace

hipError_t launch_embed_forward(const EmbedArgs& a, int tt, int to, hipStream_t s) {
  if (tt == kBf16) return to == kFp32 ? forward<kBf16, kFp32>(a, s) : forward<kBf16, kBf16>(a, s);
  if (tt == kFp16) return to == kFp32 ? forward<kFp16, kFp32>(a, s) : forward<kFp16, kFp16>(a, s);
  return forward<kFp32, kFp32>(a, s);
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
  const Order o{reinterpret_cast<int32_t*>(ws + p.start), reinterpret_cast<int32_t*>(ws + p.key),
                reinterpret_cast<int32_t*>(ws + p.pos)};
  const SortArgs sa{g.ids, (int32_t)g.m_tok, (int32_t)g.n_vocab, p.range, o};
  hipLaunchKernelGGL(sort_kernel, dim3((unsigned)p.groups), dim3(kSortThreads), (size_t)kSortWaves * p.range * 4, s, sa);
  // rows to zero: at least four a wave, and no more than 8 workgroups a CU
  int64_t zero = (g.n_vocab + 15) / 16;
  if (zero > 2048) zero = 2048;
  const SumArgs a{g.dout, g.dtable, (int32_t)g.m_tok, (int32_t)g.n_vocab, g.k, g.scale, p.segment, p.segments, p.chunks,
                  p.chunk_vecs, (int32_t)zero, o, reinterpret_cast<float*>(ws + p.part)};
  const bool join = g.m_tok > p.segment;         // else no run is longer than a segment
  if (td == kFp32) {
    if (tt == kBf16) return backward<kFp32, kBf16, 4>(a, g.add, join, s);
    if (tt == kFp16) return backward<kFp32, kFp16, 4>(a, g.add, join, s);
    return backward<kFp32, kFp32, 4>(a, g.add, join, s);
  }
  if (td == kBf16) return backward<kBf16, kBf16, 8>(a, g.add, join, s);
  return backward<kFp16, kFp16, 8>(a, g.add, join, s);
}

}  // namespace step
}  // namespace sbl
