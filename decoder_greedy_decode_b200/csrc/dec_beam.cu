// dec_beam.cu -- beam search: the k best continuations of every group of
// beams, the contiguous cache that follows them, and the chosen sequences.
//
// Selection.  score(w, t) = s_w + x_wt - log sum_t exp(x_wt).  Within a row
// the order of the scores is the order of the logits, so one pass over the
// logits finds both what the row's sum needs and the only k candidates it can
// send: a CTA takes a chunk of a row in batches of 16 logits a thread (the
// next batch loads while one is used: the bound is HBM), keeps a running
// (max, sum exp) per thread and picks its k largest.  A second, dependent
// launch joins the chunks of each row, and the rows of each group, in fp64.
//
// The k largest of a chunk.  The k-th largest of the 64 maxima that groups of
// four threads find in the first two batches is a lower bound of the chunk's
// k-th largest logit.  A thread whose batch reaches it leaves a note (and the
// logits, while there is room), so a logit costs one maximum and one
// exponential; the logits noted that reach the bound (a few times k of random
// ones) find their place by counting the larger ones.  Keys (order of the logit, then the lower
// index) are unique 64-bit words.  Where too much reaches the bound (many
// equal logits, or -inf for most of a masked vocabulary, or rising ones), the
// chunk is read again with keys in place of logits: the bound of every batch
// is then exact enough that at most 64 k keys of a batch are gathered.
//
// Measured: 16 groups of 4 rows of 151936 fp32 logits 14.5 us (39 MB), 26.9 with
// a 64-bit key for every logit; one group 7.7 us; 4 groups of 32 rows, k = 32,
// 42 us.  One wave of CTAs: the loads alone take 7.6 us, the exponentials 1.1,
// and their phases coincide.  Both launches in one cooperative kernel took 5 us
// more than in two.
#include <cuda_runtime.h>

#include "dec.h"
#include "dec_paged.h"
#include "dec_ptx.cuh"
#include "dec_tc.cuh"

namespace dec {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 32;
constexpr int kMaxBeams = 32;
constexpr int kMaxLists = 128;   // chunks of a row
constexpr int kEach = 16;        // logits of a thread in a batch
constexpr int kBatch = kThreads * kEach;
constexpr int kRoom = 4 * kEach * kMaxK;   // gathered keys
// of which the first pass uses one half; the other holds its hits
constexpr int kKeys = kRoom / 2;
constexpr int kHits = 2048;                // a thread and batch that reach the bound: 2 bytes
constexpr int kKept = 64;                  // hits whose logits are kept
static_assert(kHits * 2 + kKept * kEach * 4 <= (kRoom - kKeys) * 8, "hits");
constexpr float kLog2e = 1.4426950408889634f;

struct BeamArgs {
  int G, W, V, k;
  const void* logits;
  long long row_stride;
  const float* scores;
  const uint8_t* done;
  int eos;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  uint8_t* out_done;
  int chunks, chunk;       // chunks of a row, logits of a chunk
  float2* stat;            // [G W][chunks] (max, sum of exp2((x - max) log2 e))
  unsigned long long* key; // [G W][chunks][k], descending, 0 = none
};

__device__ __forceinline__ unsigned long long key_of(float x, uint32_t i) {
  // (+ 0 makes -0 and 0 one value)
  return (static_cast<unsigned long long>(order_key(x + 0.f)) << 32) | static_cast<uint32_t>(~i);
}
__device__ __forceinline__ float logit_of(unsigned long long key) {
  const uint32_t u = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (a + b) c of two values at once (each operation rounded as by itself)
__device__ __forceinline__ float2 add_mul2(float a0, float a1, float b, float c) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
      "mov.b64 pa, {%2, %3};\n\t"
      "mov.b64 pb, {%4, %4};\n\t"
      "mov.b64 pc, {%5, %5};\n\t"
      "add.rn.f32x2 pa, pa, pb;\n\t"
      "mul.rn.f32x2 pa, pa, pc;\n\t"
      "mov.b64 {%0, %1}, pa;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
  return d;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void load(const float* p, float* x) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  }
};
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f(*p); }
  static __device__ __forceinline__ void load(const uint16_t* p, float* x) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(const BeamArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ __align__(16) unsigned long long s_key[kRoom + kMaxK];   // gathered keys, then the best so far
  __shared__ __align__(16) unsigned long long s_max[kThreads / 4];
  __shared__ unsigned long long s_bound;
  __shared__ float s_low;
  __shared__ float2 s_stat[kThreads / 32];
  __shared__ int s_n, s_hits;
  float (*s_val)[kEach] = reinterpret_cast<float (*)[kEach]>(s_key + kKeys);
  uint16_t* s_hit = reinterpret_cast<uint16_t*>(s_val + kKept);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x;
  const long long r = blockIdx.y + static_cast<long long>(blockIdx.z) * gridDim.y;
  pdl_trigger();
  if (r >= static_cast<long long>(a.G) * a.W) return;
  if (a.done && a.done[r]) return;   // its one candidate needs no logits
  const T* row = static_cast<const T*>(a.logits) + r * a.row_stride;
  // batches start on 16-byte boundaries: element i of the row is at i + mis
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int begin = c * a.chunk - mis, end = min(begin + a.chunk, a.V);
  const int batches = end > begin ? (end - begin + kBatch - 1) / kBatch : 0;
  // element e of vector j of this thread in batch b
  auto index = [&](int b, int j) { return begin + b * kBatch + (j * kThreads + tid) * N; };
  auto load = [&](int b, float (&x)[kEach]) {
    if (begin + b * kBatch >= 0 && begin + (b + 1) * kBatch <= end) {
#pragma unroll
      for (int j = 0; j < kEach / N; ++j) Vec<T>::load(row + index(b, j), &x[j * N]);
      return;
    }
#pragma unroll
    for (int j = 0; j < kEach / N; ++j) {
      const int i = index(b, j);
      if (i >= 0 && i + N <= end) {
        Vec<T>::load(row + i, &x[j * N]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          x[j * N + e] = i + e >= 0 && i + e < end ? Vec<T>::one(row + i + e) : -INFINITY;
      }
    }
  };
  auto largest = [&](const float (&x)[kEach]) {
    float m = x[0];
#pragma unroll
    for (int e = 1; e < kEach; ++e) m = fmaxf(m, x[e]);
    return m;   // (a NaN is skipped)
  };

  float x[kEach], y[kEach];
  load(0, x);
  load(1, y);   // (behind the chunk: -inf)
  if (tid == 0) {
    s_n = s_hits = 0;
    s_low = -INFINITY;
  }
  {
    float q = fmaxf(largest(x), largest(y));
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, o));
    float* quads = reinterpret_cast<float*>(s_max);
    if ((lane & 3) == 0) quads[tid >> 2] = q;
    __syncthreads();
    // a group's place among the 64: each of its threads compares with 16
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kThreads / 64; ++j) {
      const int i = 4 * (4 * j + (lane & 3));
      const float4 u = *reinterpret_cast<const float4*>(quads + i);
      const float v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) rank += v[e] > q || (v[e] == q && i + e < tid >> 2);
    }
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if (rank == a.k - 1) s_low = q;   // (one group's four threads)
    __syncthreads();
  }
  const float low = s_low;
  float m = -INFINITY, s = 0.f;
  auto use = [&](int b, const float (&v)[kEach]) {
    const float bm = largest(v);
    if (bm >= low && low > -INFINITY) {
      const int at = atomicAdd(&s_hits, 1);
      if (at < kHits) s_hit[at] = static_cast<uint16_t>(b * kThreads + tid);
      if (at < kKept) {
#pragma unroll
        for (int e = 0; e < kEach; e += 4)
          *reinterpret_cast<float4*>(s_val[at] + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
    // (all -inf so far: the sum is 0; a NaN or +inf makes it NaN)
    if (bm > m) {
      s *= ex2((m - bm) * kLog2e);
      m = bm;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < kEach; e += 2) {
      const float2 t = add_mul2(v[e], v[e + 1], -ref, kLog2e);
      s0 += ex2(t.x);
      s1 += ex2(t.y);
    }
    s += s0 + s1;
  };
#pragma unroll 1
  for (int b = 0; b < batches; b += 2) {
    use(b, x);
    if (b + 2 < batches) load(b + 2, x);
    if (b + 1 < batches) {
      use(b + 1, y);
      if (b + 3 < batches) load(b + 3, y);
    }
  }
  const float M = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m, Mr = M == -INFINITY ? 0.f : M;
  s = warp_sum(m == -INFINITY && s == 0.f ? 0.f : s * ex2((ref - Mr) * kLog2e));
  if (lane == 0) s_stat[warp] = make_float2(M, s);
  __syncthreads();

  // the logits of the hits that reach the bound
  const int hits = s_hits;
  if (low > -INFINITY && hits <= kHits) {
    for (int i = tid; i < hits * kEach; i += kThreads) {
      const int h = i / kEach, e = i % kEach, id = s_hit[h];
      const int at = begin + id / kThreads * kBatch + (e / N * kThreads + id % kThreads) * N + e % N;
      const float v = h < kKept ? s_val[h][e]
                      : at >= 0 && at < end ? Vec<T>::one(row + at) : -INFINITY;
      if (v >= low) {
        const int o = atomicAdd(&s_n, 1);
        if (o < kKeys) s_key[o] = key_of(v, at);
      }
    }
    __syncthreads();
  }
  int n = s_n;
  if (!(low > -INFINITY) || hits > kHits || n > kKeys) {
    // Once more, by keys: the best k so far stand behind the gathered ones.
    unsigned long long* best = s_key + kRoom;
    if (tid < a.k) best[tid] = 0;
    for (int b = 0; b < batches; ++b) {
      load(b, x);
      // the thread's largest logit, the first among equals
      float tm = -INFINITY;
      int ti = -1;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int i = index(b, e / N) + e % N;
        if (i >= 0 && i < end && (x[e] > tm || (ti < 0 && x[e] == tm))) {
          tm = x[e];
          ti = i;
        }
      }
      const unsigned long long mine = ti < 0 ? 0ull : key_of(tm, ti);
      unsigned long long quad = mine;
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, quad, o);
        quad = other > quad ? other : quad;
      }
      __syncthreads();   // s_n, s_max and s_key of the batch before have been read
      if ((lane & 3) == 0) s_max[tid >> 2] = quad;
      if (tid == 0) {
        s_n = 0;
        s_bound = 0;
      }
      __syncthreads();
      if (tid < kThreads / 4) {
        const unsigned long long q = s_max[tid];
        int rank = 0;
#pragma unroll 16
        for (int i = 0; i < kThreads / 4; ++i) rank += s_max[i] > q;
        if (q && rank == a.k - 1) s_bound = q;   // (fewer than k groups hold logits: all are gathered)
      }
      __syncthreads();
      const unsigned long long bound = max(s_bound, best[a.k - 1]);
      if (mine && mine >= bound) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int i = index(b, e / N) + e % N;
          if (x[e] == x[e] && i >= 0 && i < end) {
            const unsigned long long key = key_of(x[e], i);
            if (key >= bound) s_key[atomicAdd(&s_n, 1)] = key;
          }
        }
      }
      __syncthreads();
      n = s_n;
      // the k best of the gathered keys and the best so far
      const unsigned long long old = tid < a.k ? best[tid] : 0ull;
      int rank = 0;
      if (old) {
        rank = tid;
        for (int j = 0; j < n; ++j) rank += s_key[j] > old;
      }
      __syncthreads();
      unsigned long long put[kRoom / kThreads + 1];
      int to[kRoom / kThreads + 1];
#pragma unroll
      for (int u = 0; u <= kRoom / kThreads; ++u) {
        const int i = u < kRoom / kThreads ? tid + u * kThreads : kRoom;
        to[u] = kMaxK;
        put[u] = 0;
        if (u < kRoom / kThreads && i < n) {
          put[u] = s_key[i];
          to[u] = 0;
          for (int j = 0; j < n; ++j) to[u] += s_key[j] > put[u];
          for (int j = 0; j < a.k; ++j) to[u] += best[j] > put[u];
        }
      }
      __syncthreads();
      if (old && rank < a.k) best[rank] = old;
#pragma unroll
      for (int u = 0; u < kRoom / kThreads; ++u)
        if (put[u] && to[u] < a.k) best[to[u]] = put[u];
    }
    __syncthreads();
    if (tid < a.k) a.key[(r * a.chunks + c) * a.k + tid] = best[tid];
  } else {
    unsigned long long* out = a.key + (r * a.chunks + c) * a.k;
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long key = s_key[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += s_key[j] > key;
      if (rank < a.k) out[rank] = key;
    }
    if (tid >= n && tid < a.k) out[tid] = 0;
  }
  if (tid == 0) {
    float cm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) cm = fmaxf(cm, s_stat[w].x);
    const float cr = cm == -INFINITY ? 0.f : cm;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const float2 t = s_stat[w];
      sum += t.x == -INFINITY ? t.y : t.y * ex2((t.x - cr) * kLog2e);
    }
    a.stat[r * a.chunks + c] = make_float2(cm, sum);
  }
}

// The k best of a row from the sorted lists of its chunks, by one warp: a lane
// holds the first A keys of NL lists (a list that sends more of them is read
// on: a refill ahead of its use would have the whole warp wait for it).
template <int NL, int A>
__device__ __forceinline__ void merge_lists(const BeamArgs& a, const unsigned long long* lists,
                                            double own, double lse, uint32_t row0, double* sc,
                                            uint32_t* at,
                                            unsigned long long (&ahead)[NL][A]) {
  const int lane = threadIdx.x & 31;
  int pos[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) pos[i] = 0;
  for (int p = 0; p < a.k; ++p) {
    unsigned long long mine = ahead[0][0];
#pragma unroll
    for (int i = 1; i < NL; ++i) mine = max(mine, ahead[i][0]);
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(mine >> 32));
    const uint32_t lo = __reduce_max_sync(
        0xffffffffu, static_cast<uint32_t>(mine >> 32) == hi ? static_cast<uint32_t>(mine) : 0u);
    const unsigned long long best = (static_cast<unsigned long long>(hi) << 32) | lo;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (ahead[i][0] == best) {   // (keys are unique; a row holds at least k)
#pragma unroll
        for (int j = 1; j < A; ++j) ahead[i][j - 1] = ahead[i][j];
        ahead[i][A - 1] = 0;
        if (++pos[i] >= A && pos[i] < a.k)
          ahead[i][0] = __ldcg(lists + (i * 32 + lane) * a.k + pos[i]);
      }
    if (lane == 0) {
      const double v = own + static_cast<double>(logit_of(best)) - lse;
      sc[p] = v == v ? v : -INFINITY;
      at[p] = row0 + static_cast<uint32_t>(~lo);
    }
  }
}

// A row's sum and its k best candidates, best first, by one warp.
template <int NL, int A>
__device__ __forceinline__ void best_of_row(const BeamArgs& a, int w, double* sc, uint32_t* at,
                                            bool* s_done) {
  const int lane = threadIdx.x & 31;
  const long long r = static_cast<long long>(blockIdx.x) * a.W + w;
  // (loads first: the lists' heads do not wait for the row's sum)
  const unsigned long long* lists = a.key + r * a.chunks * a.k;
  const double own = a.scores[r];
  const bool done = a.done && a.done[r];
  if (lane == 0) s_done[w] = done;
  unsigned long long ahead[NL][A];
  float2 t[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int c = i * 32 + lane;
    const bool has = !done && c < a.chunks;
    t[i] = has ? __ldcg(&a.stat[r * a.chunks + c]) : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int j = 0; j < A; ++j) ahead[i][j] = has && j < a.k ? __ldcg(lists + c * a.k + j) : 0ull;
  }
  bool flat = !(own > -INFINITY);   // -inf or NaN: no candidate above -inf
  double lse = 0.0;
  if (!done && !flat) {
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i) M = fmaxf(M, t[i].x);
    M = warp_max(M);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      sum += static_cast<double>(t[i].x == -INFINITY ? t[i].y : t[i].y * ex2((t[i].x - M) * kLog2e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    lse = static_cast<double>(M) + log(sum);
    // a NaN or +inf in the row, or nothing but -inf
    flat = !(M > -INFINITY) || !(M < INFINITY) || !(sum < INFINITY);
  }
  const uint32_t row0 = static_cast<uint32_t>(w) * a.V;
  if (!flat && !done) {
    merge_lists<NL, A>(a, lists, own, lse, row0, sc, at, ahead);
    return;
  }
  for (int p = lane; p < a.k; p += 32) {
    if (flat) {
      sc[p] = -INFINITY;
      at[p] = row0 + p;
    } else if (p == 0) {
      sc[0] = own;
      at[0] = row0 + a.eos;
    } else {
      sc[p] = -INFINITY;
      at[p] = row0 + (p - 1 < a.eos ? p - 1 : p);
    }
  }
}

// One CTA per group: a warp per row, then one warp, a lane per row, takes the
// best of the rows' next candidates k times.
__global__ void __launch_bounds__(kMaxBeams * 32) groups_kernel(const BeamArgs a) {
  __shared__ double s_score[kMaxBeams * kMaxK];
  __shared__ uint32_t s_at[kMaxBeams * kMaxK];
  __shared__ bool s_done[kMaxBeams];   // (out_done may be done)
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  if (a.chunks <= 32)   // (one list to a lane; 16 keys ahead cost 16 groups of 4 15.7 for 14.4 us)
    best_of_row<1, 4>(a, w, s_score + w * a.k, s_at + w * a.k, s_done);
  else
    best_of_row<kMaxLists / 32, 2>(a, w, s_score + w * a.k, s_at + w * a.k, s_done);
  __syncthreads();
  if (w > 0) return;
  const bool row = lane < a.W;
  const double* sc = s_score + lane * a.k;
  const uint32_t* at = s_at + lane * a.k;
  int p = 0;
  // the order of doubles as that of integers (+ 0 makes -0 and 0 one value; 0
  // is below -inf: no candidate)
  auto order = [&](int p) {
    if (!row || p >= a.k) return 0ull;
    const unsigned long long u = __double_as_longlong(sc[p] + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
  };
  unsigned long long key = order(0);
  for (int i = 0; i < a.k; ++i) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
    const uint32_t lo = __reduce_max_sync(
        0xffffffffu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
    const unsigned best =
        __ballot_sync(0xffffffffu, key == ((static_cast<unsigned long long>(hi) << 32) | lo));
    if (lane == __ffs(best) - 1) {   // (among equals the lowest row)
      const long long o = static_cast<long long>(blockIdx.x) * a.k + i;
      const int token = static_cast<int>(at[p] - static_cast<uint32_t>(lane) * a.V);
      a.out_scores[o] = static_cast<float>(sc[p]);
      a.out_parents[o] = lane;
      a.out_tokens[o] = token;
      if (a.out_done) a.out_done[o] = s_done[lane] || token == a.eos;
      key = order(++p);
    }
  }
}

// ------------------------------------------------------- cache reordering
// A CTA takes the same few rows of one (layer, K or V, head) of every moved
// sequence: it copies the parents' rows to shared memory, waits, and writes
// them, so the cache changes in place although parents are themselves moved;
// the next plane loads while one is stored.  Bound by HBM (a parent of several
// is read once: its copies hit L2): 64 sequences of 200-420 rows of 28 layers,
// 48 of them moved, 524 us = 5.4 TB/s of DRAM traffic; one plane at a time
// 545, with 1 KB of a sequence 553; through bulk copies 728.
constexpr int kReThreads = 256;
constexpr int kRePiece = 512;    // bytes of a sequence in one CTA
constexpr int kRePlanes = 8;     // planes that a CTA takes in turn
constexpr int kReBatch = 64;

struct ReorderArgs {
  uint8_t* kv;
  float* scales;           // E4M3 caches
  int B, kv_batch, H, max_ctx, row_bytes, n_rows;  // n_rows of a piece
  long long planes;        // layers x 2 x heads
  const int32_t *parents, *rows;
  int* status;
};

__global__ void __launch_bounds__(kReThreads) reorder_kernel(const ReorderArgs a) {
  extern __shared__ __align__(16) uint8_t s_data[];   // [moved][kRePiece], then scales
  __shared__ int s_to[kReBatch], s_from[kReBatch], s_rows[kReBatch];
  __shared__ long long s_row[2][2][kReBatch];   // [buffer][from, to]
  __shared__ int s_n;
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * a.n_rows;
  int bad = 0;
  if (tid < 32) {
    int n = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + tid;
      const int p = b < a.B ? a.parents[b] : b, m = b < a.B ? a.rows[b] : 0;
      if (b < a.B && (p < 0 || p >= a.B)) bad |= DEC_DEV_BAD_PAGE;
      if (m < 0 || m > a.max_ctx) bad |= DEC_DEV_BAD_POSITION;
      const bool move = p != b && m > r0;
      const unsigned mask = __ballot_sync(0xffffffffu, move);
      if (move) {
        const int at = n + __popc(mask & ((1u << tid) - 1));
        s_to[at] = b;
        s_from[at] = p;
        s_rows[at] = min(a.n_rows, m - r0);
      }
      n += __popc(mask);
    }
    if (tid == 0) s_n = n;
  }
  if (__syncthreads_or(bad)) {
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && a.status) atomicOr(a.status, bad);
    return;
  }
  const int n = s_n;
  if (n == 0) return;
  constexpr int pieces = kRePiece / 16;
  const int room = n * kRePiece;   // bytes of one buffer
  float* s_scale = reinterpret_cast<float*>(s_data + 2 * room);
  auto load = [&](long long plane, int buf) {
    // where each moved sequence reads and writes, once for all its pieces
    if (tid < n) {
      const long long lk = plane / a.H, h = plane % a.H;   // (layer, K or V), head
      auto row_of = [&](int b) { return ((lk * a.kv_batch + b) * a.H + h) * a.max_ctx + r0; };
      s_row[buf][0][tid] = row_of(s_from[tid]);
      s_row[buf][1][tid] = row_of(s_to[tid]);
    }
    __syncthreads();
    for (int i = tid; i < n * pieces; i += kReThreads) {
      const int j = i / pieces, o = (i % pieces) * 16;
      if (o < s_rows[j] * a.row_bytes)
        cp_async16_cg(s_data + buf * room + i * 16, a.kv + s_row[buf][0][j] * a.row_bytes + o);
    }
    if (a.scales)
      for (int i = tid; i < n * a.n_rows; i += kReThreads) {
        const int j = i / a.n_rows, r = i % a.n_rows;
        if (r < s_rows[j])
          cp_async4(s_scale + buf * n * a.n_rows + i, a.scales + s_row[buf][0][j] + r);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int buf = 0;
  load(blockIdx.y, 0);
  for (long long plane = blockIdx.y; plane < a.planes; plane += gridDim.y, buf ^= 1) {
    if (plane + gridDim.y < a.planes) {   // the next plane loads while this one is stored
      load(plane + gridDim.y, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      cp_async_wait_all();
    }
    __syncthreads();
    for (int i = tid; i < n * pieces; i += kReThreads) {
      const int j = i / pieces, o = (i % pieces) * 16;
      if (o < s_rows[j] * a.row_bytes)
        *reinterpret_cast<uint4*>(a.kv + s_row[buf][1][j] * a.row_bytes + o) =
            *reinterpret_cast<const uint4*>(s_data + buf * room + i * 16);
    }
    if (a.scales)
      for (int i = tid; i < n * a.n_rows; i += kReThreads) {
        const int j = i / a.n_rows, r = i % a.n_rows;
        if (r < s_rows[j]) a.scales[s_row[buf][1][j] + r] = s_scale[buf * n * a.n_rows + i];
      }
    __syncthreads();
  }
}

__global__ void backtrace_kernel(int n, int G, int W, const int32_t* parents,
                                 const int32_t* tokens, int32_t* out) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= G * W) return;
  const int g = i / W;
  int w = i % W;
  int32_t* o = out + static_cast<long long>(i) * n;
  for (int t = n - 1; t >= 0; --t) {
    if (w < 0 || w >= W) {
      o[t] = -1;
      continue;
    }
    const long long e = (static_cast<long long>(t) * G + g) * W + w;
    o[t] = tokens[e];
    w = parents[e];
  }
}

struct Plan {
  int chunks, chunk;
  size_t stat, total;
};
// One wave of CTAs (four to an SM), as far as chunks of at least half a
// batch and at most kMaxLists of them to a row allow.
Plan plan_of(int rows, int V, int k, int sms) {
  Plan p{};
  const int len = V + 7;   // and the elements before the first 16-byte boundary
  int want = 4 * sms / rows;
  want = want < 1 ? 1 : want > kMaxLists ? kMaxLists : want;
  p.chunk = ((len + want - 1) / want + kBatch / 2 - 1) / (kBatch / 2) * (kBatch / 2);
  p.chunks = (len + p.chunk - 1) / p.chunk;
  p.stat = round256(sizeof(float2) * static_cast<size_t>(rows) * p.chunks);
  p.total = p.stat + round256(sizeof(unsigned long long) * static_cast<size_t>(rows) * p.chunks * k);
  return p;
}

bool bad_beams(int groups, int beams, int vocab, int k) {
  return groups < 1 || groups > 65535 || beams < 1 || beams > kMaxBeams || k < 1 || k > kMaxK ||
         vocab < k || vocab > 1000000;
}

template <typename T>
cudaError_t launch_beam_rows(const BeamArgs& a, cudaStream_t s) {
  const int rows = a.G * a.W;
  const int y = rows < 32768 ? rows : 32768;
  rows_kernel<T><<<dim3(a.chunks, y, (rows + y - 1) / y), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" size_t dec_beam_workspace_bytes(int groups, int beams, int vocab, int k) {
  if (bad_beams(groups, beams, vocab, k)) return 0;
  const int sms = device_sms();
  return plan_of(groups * beams, vocab, k, sms > 0 ? sms : 148).total;
}

extern "C" int dec_beam_select(int groups, int beams, int vocab, int k, int dtype,
                               const void* logits, long long row_stride, const float* scores,
                               const uint8_t* done, int eos, float* out_scores,
                               int32_t* out_parents, int32_t* out_tokens, uint8_t* out_done,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !workspace)
    return DEC_ERR_NULL;
  if (bad_beams(groups, beams, vocab, k)) return DEC_ERR_ARG;
  if (dtype != DEC_BF16 && dtype != DEC_F32) return DEC_ERR_DTYPE;
  if (eos < -1 || eos >= vocab || (done && eos < 0)) return DEC_ERR_ARG;
  if (groups * beams > 1 && row_stride < vocab) return DEC_ERR_SHAPE;
  if (!is_aligned(logits, dtype == DEC_BF16 ? 2 : 4) || !is_aligned(workspace, 256) ||
      !is_aligned(scores, 4) || !is_aligned(out_scores, 4) || !is_aligned(out_parents, 4) ||
      !is_aligned(out_tokens, 4))
    return DEC_ERR_ALIGN;
  if (k != beams && (out_scores == scores || (out_done && out_done == done))) return DEC_ERR_ARG;
  const int sms = device_sms();
  const Plan p = plan_of(groups * beams, vocab, k, sms > 0 ? sms : 148);
  if (workspace_bytes < p.total) return DEC_ERR_KV_SIZE;
  if (sms < 0) return sms;
  BeamArgs a{};
  a.G = groups;
  a.W = beams;
  a.V = vocab;
  a.k = k;
  a.logits = logits;
  a.row_stride = row_stride;
  a.scores = scores;
  a.done = done;
  a.eos = eos;
  a.out_scores = out_scores;
  a.out_parents = out_parents;
  a.out_tokens = out_tokens;
  a.out_done = out_done;
  a.chunks = p.chunks;
  a.chunk = p.chunk;
  a.stat = static_cast<float2*>(workspace);
  a.key = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) + p.stat);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  e = dtype == DEC_BF16 ? launch_beam_rows<uint16_t>(a, s) : launch_beam_rows<float>(a, s);
  if (e == cudaSuccess) e = launch_dependent(groups_kernel, dim3(groups), dim3(32 * beams), 0, s, a);
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}

extern "C" int dec_kv_reorder(int n_layers, int n_kv_heads, int head_dim, int dtype, int kv_batch,
                              int max_ctx, void* values, float* scales, int batch,
                              const int32_t* parents, const int32_t* rows, int* status,
                              void* stream) {
  if (!values || !parents || !rows) return DEC_ERR_NULL;
  if (n_layers < 1 || n_kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return DEC_ERR_SHAPE;
  if (dtype != DEC_KV_BF16 && dtype != DEC_KV_FP8_E4M3) return DEC_ERR_DTYPE;
  const bool fp8 = dtype == DEC_KV_FP8_E4M3;
  if (fp8 && !scales) return DEC_ERR_NULL;
  if (batch < 1 || batch > kReBatch || batch > kv_batch) return DEC_ERR_BATCH;
  if (max_ctx < 16 || max_ctx % 16) return DEC_ERR_ARG;
  if (!is_aligned(values, 16) || (fp8 && !is_aligned(scales, 4)) || !is_aligned(parents, 4) ||
      !is_aligned(rows, 4) || !is_aligned(status, 4))
    return DEC_ERR_ALIGN;
  ReorderArgs a{};
  a.kv = static_cast<uint8_t*>(values);
  a.scales = fp8 ? scales : nullptr;
  a.B = batch;
  a.kv_batch = kv_batch;
  a.H = n_kv_heads;
  a.max_ctx = max_ctx;
  a.row_bytes = head_dim * (fp8 ? 1 : 2);
  a.n_rows = kRePiece / a.row_bytes;
  a.planes = 2ll * n_layers * n_kv_heads;
  a.parents = parents;
  a.rows = rows;
  a.status = status;
  const int smem = 2 * batch * (kRePiece + (fp8 ? a.n_rows * 4 : 0));
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reorder_kernel, 2 * kReBatch * (kRePiece + 64), allowed);
  if (e != cudaSuccess) return cuda_failed(e);
  const unsigned x = static_cast<unsigned>((max_ctx + a.n_rows - 1) / a.n_rows);
  const long long per = (a.planes + kRePlanes - 1) / kRePlanes;
  const unsigned y = static_cast<unsigned>(per < 65535 ? per : 65535);
  reorder_kernel<<<dim3(x, y), kReThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}

extern "C" int dec_beam_backtrace(int n_steps, int groups, int beams, const int32_t* parents,
                                  const int32_t* tokens, int32_t* out, void* stream) {
  if (n_steps < 0 || groups < 1 || beams < 1 || static_cast<long long>(groups) * beams > (1 << 24))
    return DEC_ERR_ARG;
  if (n_steps == 0) return DEC_OK;
  if (!parents || !tokens || !out) return DEC_ERR_NULL;
  if (!is_aligned(parents, 4) || !is_aligned(tokens, 4) || !is_aligned(out, 4)) return DEC_ERR_ALIGN;
  const int n = groups * beams;
  backtrace_kernel<<<(n + 127) / 128, 128, 0, static_cast<cudaStream_t>(stream)>>>(
      n_steps, groups, beams, parents, tokens, out);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}
