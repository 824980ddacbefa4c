// dec_paged_append.cu -- rotary positions, and the append of new rows to a
// paged KV cache.
//
// Mathematics.  Pair i of a rotated head turns by p * f_i at position p.  The
// angle is kept in turns as a 64-bit binary fraction: p * phase_i modulo 2^64
// drops whole turns exactly, so the product is right to 2^-33 turns at any int32
// position (in fp32 it is off by p * f_i * 2^-24 radians, i.e. by 0.06 rad at
// p = 2^20).  Its top 32 bits (cut: 2^-32 turns) become fp32 half turns for the
// sine and cosine, rounded by at most 2^-26 turns, 1e-7 rad: what fp32 operands
// near a half turn hold.  The rotation itself is fp32, rounded once.
//
// Split.  A warp takes tokens, and the head rows of each four at a time:
// eight lanes hold a row, 16 (head_dim 128) or 8 (64) of its elements each, so
// loads and stores are 16 bytes a lane and one three-step butterfly reduces
// four rows (RMSNorm sums, E4M3 maxima).  Nothing passes through shared
// memory; the sines and cosines of a token are computed once by the warp,
// each lane a quarter of what its eight lanes need, and kept in registers
// for all rows.  The next rows are loaded before the present ones are used.
// The floor is HBM (every input read once, every output written once): 8192 x 32
// fp32 heads rotated alone take 45.1 us = 5.9 TB/s.  With norms and E4M3 pages
// issue is the bound: two thirds of the slots are used, the rest is lost to
// fixed latencies with the 20 warps an SM that the registers allow.  16384 tokens
// of 16 + 8 + 8 heads 50.2 us for 36 us of bytes; with a row per warp and IEEE
// divisions 180 us (193 instructions a row).
//
// E4M3 codes are RNE(x / scale) of the IEEE quotient.  The quotient comes from
// a correctly rounded reciprocal y of the scale by one residual step
// (Markstein 1990): q0 = x y, q = q0 + (x - q0 scale) y, which is the IEEE
// quotient while nothing underflows; rows with a maximum outside
// [2^-60, 2^100] are first brought near 1 by a power of two.
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "dec.h"
#include "dec_paged.h"
#include "dec_ptx.cuh"

namespace dec {
namespace {

constexpr int kWarps = 4;
constexpr int kCtas = 5;   // CTAs of an SM (96 registers a thread)

struct RowsArgs {
  int n_tokens, Hq, Hkv;              // Hkv = 0: rotation alone
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void* q_out;
  long long q_out_stride;
  const int32_t *positions, *seqs;
  const uint16_t *q_norm, *k_norm;
  float eps;
  int zero;                           // q_out rows of skipped tokens: 1 = zeroed
  const uint64_t* phases;             // null: no rotation
  int rot, inter;
  float mscale;
  const int32_t* table;
  int n_seqs, width;
  PoolView pool;
  int* status;
};

// Two fp32 operations in one instruction (each rounded as by itself).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
      "mov.b64 pa, {%2, %3};\n\t"
      "mov.b64 pb, {%4, %5};\n\t"
      "mul.rn.f32x2 pd, pa, pb;\n\t"
      "mov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\t"
      "mov.b64 pa, {%2, %3};\n\t"
      "mov.b64 pb, {%4, %5};\n\t"
      "mov.b64 pc, {%6, %7};\n\t"
      "fma.rn.f32x2 pd, pa, pb, pc;\n\t"
      "mov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float ld1(const uint16_t* p) { return bf16_to_f(*p); }
__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ void st1(uint16_t* p, float a) { *p = f_to_bf16(a); }
__device__ __forceinline__ void st1(float* p, float a) { *p = a; }

// N (8 or 4) consecutive elements as loaded.
template <typename T, int N>
struct Raw;
template <>
struct Raw<uint16_t, 8> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
  }
};
template <>
struct Raw<uint16_t, 4> {
  uint2 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
  }
};
template <int N>
struct Raw<float, N> {
  float4 w[N / 4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void get(float* x) const {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) x[4 * i] = w[i].x, x[4 * i + 1] = w[i].y, x[4 * i + 2] = w[i].z, x[4 * i + 3] = w[i].w;
  }
};
template <int N>
__device__ __forceinline__ void put(uint16_t* p, const float* x) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = f2_to_bf16x2(x[2 * i], x[2 * i + 1]);
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int N>
__device__ __forceinline__ void put(float* p, const float* x) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
template <int N>
__device__ __forceinline__ void put(uint8_t* p, const float* q) {   // quotients -> E4M3
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = f2_to_e4m3x2(q[4 * i], q[4 * i + 1]) |
           (static_cast<uint32_t>(f2_to_e4m3x2(q[4 * i + 2], q[4 * i + 3])) << 16);
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}
__device__ __forceinline__ void put1(uint16_t* p, float x) { st1(p, x); }
__device__ __forceinline__ void put1(float* p, float x) { st1(p, x); }
__device__ __forceinline__ void put1(uint8_t* p, float q) {
  *p = static_cast<uint8_t>(f2_to_e4m3x2(q, 0.f));
}

// Elements of a lane's vectors: 16 bytes of input, or what the lane holds of
// half a row.
template <typename T, int D>
constexpr int vector_of() {
  return 16 / sizeof(T) < D / 16 ? 16 / sizeof(T) : D / 16;
}

// Reductions over the eight lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Element of a row that pair p starts (a) and ends (b).  Half-split pairs
// (`half`): pair p < R/2 is elements (p, p + R/2), and the passed part is
// split the same way.  Otherwise (interleaved pairs, rows that are not
// rotated) pair p is elements 2p and 2p + 1.
template <int D>
__device__ __forceinline__ int first_of(int p, int R) {
  const int r = R >> 1;
  return p < r ? p : R + (p - r);
}
template <int D>
__device__ __forceinline__ int second_of(int p, int R) {
  const int r = R >> 1;
  return p < r ? p + r : R + (D - R) / 2 + (p - r);
}
// A lane's 2N = D/8 elements are runs of V consecutive ones, 8 V apart (the
// eight lanes of a row read 8 V elements side by side): x[k V + e] is element
// e of run k.  Half-split rows: run k < N/V holds the first elements of pairs
// 8 V k + V o + e, run k + N/V their second ones.
template <int D, int V>
__device__ __forceinline__ int run_at(bool half, int k, int o, int R) {
  constexpr int K = D / 16 / V;   // runs of first elements
  if (!half) return (8 * k + o) * V;
  return k < K ? first_of<D>((8 * k + o) * V, R) : second_of<D>((8 * (k - K) + o) * V, R);
}
// Pair that x[j], x[N + j] (half) or x[2j], x[2j + 1] are.
template <int D, int V>
__device__ __forceinline__ int pair_at(bool half, int j, int o) {
  return half ? (8 * (j / V) + o) * V + j % V : ((8 * (2 * j / V) + o) * V + 2 * j % V) / 2;
}

// How the pairs of a rotated row lie in a lane's registers.
enum Mode {
  kHalf,     // half-split pairs, R/2 a multiple of V: x[j] and x[N + j]
  kPairs,    // neighbours x[2j], x[2j + 1] (interleaved pairs, or no rotation)
  kScalar    // half-split pairs, any R: as kHalf, but every element for itself
};

// T: element of q, k and v; TO: of q_out.  CACHE 0: rotation alone; 1: bf16
// pages; 2: E4M3 pages.
template <int D, typename T, typename TO, int CACHE, Mode M>
__global__ void __launch_bounds__(kWarps * 32, kCtas) rows_kernel(const RowsArgs a, int per_token,
                                                                   unsigned inverse) {
  constexpr int N = D / 16;     // pairs of a lane
  constexpr int V = vector_of<T, D>(), K = 2 * N / V;
  const int lane = threadIdx.x & 31, oct = lane >> 3, o = lane & 7;
  // quads of q, k and v rows in this order: a quad is all of one kind, so what
  // it passes through is uniform (idle octets where heads are no multiple of 4)
  const int nq = (a.Hq + 3) / 4, nk = (a.Hkv + 3) / 4, quads = nq + 2 * nk;
  const int r = a.rot >> 1;
  // A job is a token's quads part, part + per_token, ...; a warp takes jobs
  // `hop` apart.
  const int jobs = a.n_tokens * per_token, hop = gridDim.x * kWarps;
  const int job0 = blockIdx.x * kWarps + (threadIdx.x >> 5);
  // token of a job, and its first quad
  auto token = [&](int job) { return inverse ? static_cast<int>(__umulhi(job, inverse)) : job; };
  auto part_of = [&](int job) { return job - token(job) * per_token; };
  if (job0 >= jobs) return;

  // where the lane's runs start in rows that are rotated, and in others
  // (neighbours in every mode)
  int split_at[K], plain_at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    plain_at[k] = run_at<D, V>(false, k, o, a.rot);
    split_at[k] = M == kPairs || !a.phases ? plain_at[k] : run_at<D, V>(true, k, o, a.rot);
  }
  // first element of token t, and the number of heads
  auto token_of = [&](int t, int kind) {
    const void* base = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    return static_cast<const T*>(base) + t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
  };
  auto heads_of = [&](int kind) { return kind == 0 ? a.Hq : a.Hkv; };
  // The next quad is loaded ahead, across the tokens of a warp.  Kind (0 q, 1 k,
  // 2 v) and token change in `enter`; from quad to quad only the head moves.
  Raw<T, V> raw[K];
  int fjob = job0, fquad = part_of(job0);
  int fend, flast, fhead, fat[K];   // quads of this kind end here; its last head; this octet's
  const T* fbase;
  auto enter = [&]() {
    const int kind = fquad < nq ? 0 : fquad < nq + nk ? 1 : 2;
    fend = kind == 0 ? nq : kind == 1 ? nq + nk : quads;
    flast = heads_of(kind) - 1;
    fhead = 4 * (fquad - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) + oct;
    fbase = token_of(token(fjob), kind);
#pragma unroll
    for (int k = 0; k < K; ++k) fat[k] = kind < 2 ? split_at[k] : plain_at[k];
  };
  auto fetch = [&]() {
    if (M == kScalar || fjob >= jobs) return;
    const int at = min(fhead, flast) * D;   // (an idle octet takes the last head)
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].load(fbase + (at + fat[k]));
    fquad += per_token;
    fhead += 4 * per_token;
    if (fquad >= fend) {
      if (fquad >= quads) {
        fjob += hop;
        if (fjob >= jobs) return;
        fquad = part_of(fjob);
      }
      enter();
    }
  };
  // position, sequence and page of the present job and of the next one: the
  // loads of a token's place are hidden behind the rows of the one before
  struct Spot {
    int pos, seq, page, bad;
  };
  auto look = [&](int job) {
    Spot w{-1, 0, -1, 0};
    if (job < jobs) {
      const int t = token(job);
      w.pos = a.positions[t];
      if (CACHE) w.seq = a.seqs ? a.seqs[t] : t;
    }
    return w;
  };
  auto find = [&](Spot& w) {
    if (!CACHE || w.pos < 0) return;
    const int slot = w.pos >> a.pool.shift;
    if (w.seq < 0 || w.seq >= a.n_seqs)
      w.bad = DEC_DEV_BAD_PAGE;
    else if (slot >= a.width)
      w.bad = DEC_DEV_BAD_POSITION;
    else
      w.page = a.table[static_cast<long long>(w.seq) * a.width + slot];
  };
  Spot now = look(job0), then = look(job0 + hop);
  uint64_t phase[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const int p = pair_at<D, V>(M != kPairs, oct * (N / 4) + j, o);
    phase[j] = a.phases && p < r ? a.phases[p] : 0;
  }
  if constexpr (M != kScalar) {
    enter();
    fetch();
  }

  find(now);
#pragma unroll 1
  for (int job = job0; job < jobs; job += hop) {
    const int t = token(job), part = part_of(job);
    const int pos = now.pos;
    bool keep = !CACHE || pos >= 0;   // (rotation alone: the row of padding is copied)
    long long row0 = 0;   // element of the token's row of head 0 in the pages
    if (CACHE && keep) {
      const int bad = now.bad | (!now.bad && (now.page < 0 || now.page >= a.pool.n_pages) ? DEC_DEV_BAD_PAGE : 0);
      if (bad) {
        if (a.status && lane == 0 && part == 0) atomicOr(a.status, bad);
        keep = false;
      }
      row0 = now.page * a.pool.page_stride + static_cast<long long>(pos & ((1 << a.pool.shift) - 1)) * D;
    }
    now = then;
    find(now);
    then = look(job + 2 * hop);
    const bool turned = a.phases && pos >= 0;

    // cosine and sine of the lane's pairs, packed as the rotation uses them:
    // of two neighbouring pairs (half-split), or twice the same pair
    constexpr int NC = M == kPairs ? N : N / 2;
    float2 c2[NC], s2[NC], n2[NC];   // cosine, sine, -sine (neighbours: s2 = (-sine, sine))
    if (turned) {
      float c[N / 4], s[N / 4];
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        // the angle in half turns, [-1, 1): the top 32 bits of the fraction
        const uint64_t ph = phase[j] * static_cast<uint64_t>(pos);
        sincospif(static_cast<float>(static_cast<int32_t>(ph >> 32)) * 0x1p-31f, &s[j], &c[j]);
        c[j] *= a.mscale;
        s[j] *= a.mscale;
      }
      float cs[N], sn[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        cs[j] = __shfl_sync(0xffffffffu, c[j % (N / 4)], j / (N / 4) * 8 + o);
        sn[j] = __shfl_sync(0xffffffffu, s[j % (N / 4)], j / (N / 4) * 8 + o);
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        if (M == kPairs) {
          c2[j] = make_float2(cs[j], cs[j]);
          s2[j] = make_float2(-sn[j], sn[j]);
        } else {
          c2[j] = make_float2(cs[2 * j], cs[2 * j + 1]);
          s2[j] = make_float2(sn[2 * j], sn[2 * j + 1]);
          n2[j] = make_float2(-sn[2 * j], -sn[2 * j + 1]);
        }
      }
    }
    // element of a rotated row that x[i] is, one by one
    auto element = [&](int i) {
      const int p = pair_at<D, V>(true, i % N, o);
      return i < N ? first_of<D>(p, a.rot) : second_of<D>(p, a.rot);
    };
    auto pair = [](const float* v, int i) { return make_float2(v[2 * i], v[2 * i + 1]); };
    auto set = [](float* v, int i, float2 y) {
      v[2 * i] = y.x;
      v[2 * i + 1] = y.y;
    };
    const bool whole = 2 * r == D;   // every pair turns

    // the token's row in q_out and in the pages, of head 0
    TO* const q_row = static_cast<TO*>(a.q_out) + t * a.q_out_stride;
    uint8_t* const k_row = a.pool.k + row0 * (CACHE == 1 ? 2 : 1);
    uint8_t* const v_row = a.pool.v + row0 * (CACHE == 1 ? 2 : 1);

    // four rows of one kind, this octet's of `head`
    auto rows = [&](auto tag, int head) {
      constexpr int kind = decltype(tag)::value;
      const bool live = keep && head < heads_of(kind);
      const bool loose = M == kScalar && kind < 2 && a.phases;   // element by element
      float x[2 * N];
      if constexpr (M != kScalar) {
#pragma unroll
        for (int k = 0; k < K; ++k) raw[k].get(x + k * V);
        fetch();
      } else {
        const T* p = token_of(t, kind) + min(head, heads_of(kind) - 1) * D;
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) x[i] = ld1(p + (loose ? element(i) : plain_at[i / V] + i % V));
      }
      const uint16_t* gain = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
      if (gain) {
        float g[2 * N];
        if (loose) {
#pragma unroll
          for (int i = 0; i < 2 * N; ++i) g[i] = ld1(gain + element(i));
        } else {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            Raw<uint16_t, V> w;
            w.load(gain + split_at[k]);
            w.get(g + k * V);
          }
        }
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fma2(pair(x, i), pair(x, i), ss);
        const float f = rsqrtf(row_sum(ss.x + ss.y) * (1.0f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < N; ++i) set(x, i, mul2(mul2(pair(x, i), make_float2(f, f)), pair(g, i)));
      }
      if (turned && kind < 2) {
        // a passed pair is not multiplied (cosine 1 and sine 0 would turn an
        // infinity in it into NaN)
        if constexpr (M == kPairs) {
          auto turn = [&](int j) {
            const float2 u = pair(x, j);
            return fma2(make_float2(u.y, u.x), s2[j], mul2(u, c2[j]));
          };
          if (whole) {
#pragma unroll
            for (int j = 0; j < N; ++j) set(x, j, turn(j));
          } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
              if (pair_at<D, V>(false, j, o) < r) set(x, j, turn(j));
          }
        } else {
          // pairs 2j, 2j + 1: both of one run, which turns or passes whole
          // (kScalar: each for itself)
          auto turn = [&](int j, bool first, bool second) {
            const float2 u = pair(x, j), v = pair(x, N / 2 + j);
            const float2 y = fma2(v, n2[j], mul2(u, c2[j]));
            const float2 z = fma2(u, s2[j], mul2(v, c2[j]));
            if (first) {
              x[2 * j] = y.x;
              x[N + 2 * j] = z.x;
            }
            if (second) {
              x[2 * j + 1] = y.y;
              x[N + 2 * j + 1] = z.y;
            }
          };
          if constexpr (M == kHalf) {
#pragma unroll
            for (int k = 0; k < K / 2; ++k)
              if ((8 * k + o) * V < r) {
#pragma unroll
                for (int j = k * V / 2; j < (k + 1) * V / 2; ++j) turn(j, true, true);
              }
          } else {
#pragma unroll
            for (int j = 0; j < NC; ++j)
              turn(j, pair_at<D, V>(true, 2 * j, o) < r, pair_at<D, V>(true, 2 * j + 1, o) < r);
          }
        }
      }
      auto write = [&](auto* p) {
        if (loose) {
#pragma unroll
          for (int i = 0; i < 2 * N; ++i) put1(p + element(i), x[i]);
        } else {
#pragma unroll
          for (int k = 0; k < K; ++k) put<V>(p + (kind < 2 ? split_at[k] : plain_at[k]), x + k * V);
        }
      };
      if (kind == 0) {
        if (live) {
          write(q_row + head * D);
        } else if (CACHE && !keep && a.zero && head < a.Hq) {
#pragma unroll
          for (int i = 0; i < 2 * N; ++i) x[i] = 0.f;
          write(q_row + head * D);
        }
        return;
      }
      if constexpr (CACHE > 0) {
        const int at = head << a.pool.shift;   // rows of the page before this one
        uint8_t* const row = kind == 1 ? k_row : v_row;
        if constexpr (CACHE == 1) {
          if (live) write(reinterpret_cast<uint16_t*>(row) + at * D);
        } else {
          float am = 0.f;
#pragma unroll
          for (int i = 0; i < 2 * N; ++i) am = fmaxf(am, fabsf(x[i]));
          am = fmaxf(row_max(am), 1.17549435e-38f);  // 2^-126
          float sc, den;   // the scale, and the scale times a power of two
          if (am >= 0x1p-60f && am <= 0x1p100f) {
            constexpr float y = 1.0f / 448.0f;
            const float s0 = am * y;
            den = sc = fmaf(fmaf(-s0, 448.0f, am), y, s0);
          } else {
            // far from 1: the row and its scale times a power of two, exact
            // where a code is not 0 (an infinite scale: 0, or NaN for infinities)
            sc = __fdiv_rn(am, 448.0f);
            const float u = am < 1.f ? 0x1p100f : isinf(sc) ? 0.f : 0x1p-60f;
            den = isinf(sc) ? 1.f : sc * u;
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) x[i] *= u;
          }
          const float inv = __frcp_rn(den);
          const float2 inv2 = make_float2(-inv, -inv), den2 = make_float2(den, den);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            // (the negative of the quotient, so that -0 stays -0)
            const float2 v = pair(x, i), q0 = mul2(v, inv2);
            const float2 q = fma2(fma2(q0, den2, v), inv2, q0);
            set(x, i, make_float2(-q.x, -q.y));
          }
          if (live) {
            write(row + at * D);
            if (o == 0) (kind == 1 ? a.pool.ks : a.pool.vs)[row0 / D + at] = sc;
          }
        }
      }
    };
    int quad = part;
#pragma unroll 1
    for (; quad < nq; quad += per_token) rows(std::integral_constant<int, 0>(), 4 * quad + oct);
    if constexpr (CACHE > 0) {
#pragma unroll 1
      for (; quad < nq + nk; quad += per_token) rows(std::integral_constant<int, 1>(), 4 * (quad - nq) + oct);
#pragma unroll 1
      for (; quad < quads; quad += per_token)
        rows(std::integral_constant<int, 2>(), 4 * (quad - nq - nk) + oct);
    }
  }
}

template <int D, typename T, typename TO, int CACHE>
cudaError_t launch_rows(const RowsArgs& a, int sms, cudaStream_t s) {
  // Warps of a token: one when the tokens alone give every SM its warps (the
  // angles are then computed once a token), up to one for four rows when
  // there are few tokens and latency counts.
  const int most = (a.Hq + 3) / 4 + 2 * ((a.Hkv + 3) / 4);
  const long long want = (32ll * sms + a.n_tokens - 1) / a.n_tokens;
  const int per_token = static_cast<int>(want < 1 ? 1 : want > most ? most : want);
  const long long jobs = static_cast<long long>(a.n_tokens) * per_token;
  if (jobs > (1ll << 30)) return cudaErrorInvalidValue;
  // job / per_token = the high word of job * inverse, as jobs * per_token < 2^32
  // (there are fewer tokens than 32 sms when per_token > 1); 0: per_token is 1
  const unsigned inverse = per_token > 1 ? static_cast<unsigned>(((1ull << 32) + per_token - 1) / per_token) : 0;
  const long long blocks = (jobs + kWarps - 1) / kWarps;
  const unsigned n = static_cast<unsigned>(blocks < kCtas * sms ? blocks : kCtas * sms);
  if (!a.phases || a.inter)
    rows_kernel<D, T, TO, CACHE, kPairs><<<n, kWarps * 32, 0, s>>>(a, per_token, inverse);
  else if (a.rot % (2 * vector_of<T, D>()) == 0)
    rows_kernel<D, T, TO, CACHE, kHalf><<<n, kWarps * 32, 0, s>>>(a, per_token, inverse);
  else
    rows_kernel<D, T, TO, CACHE, kScalar><<<n, kWarps * 32, 0, s>>>(a, per_token, inverse);
  return cudaGetLastError();
}

int check_rope(const dec_rope* r, int head_dim) {
  if (!r->phases) return DEC_ERR_NULL;
  if (r->rot_dim < 2 || r->rot_dim > head_dim || (r->rot_dim & 1)) return DEC_ERR_SHAPE;
  if (!is_aligned(r->phases, 8)) return DEC_ERR_ALIGN;
  return DEC_OK;
}

int check_stride(long long stride, int n, int heads, int D) {
  if (n <= 1) return DEC_OK;   // never used
  if (stride % 8) return DEC_ERR_ALIGN;
  if (stride < static_cast<long long>(heads) * D) return DEC_ERR_SHAPE;
  return DEC_OK;
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" int dec_rope_phases(int rot_dim, double theta, int scaling, double factor,
                               double orig_ctx, double alpha, double beta, uint64_t* phases) {
  if (!phases) return DEC_ERR_NULL;
  if (rot_dim < 2 || rot_dim > 128 || (rot_dim & 1)) return DEC_ERR_SHAPE;
  if (!(theta > 1.0) || !isfinite(theta)) return DEC_ERR_ARG;
  if (scaling < DEC_ROPE_NONE || scaling > DEC_ROPE_PARTS) return DEC_ERR_ARG;
  if (scaling != DEC_ROPE_NONE && (!(factor > 0.0) || !isfinite(factor))) return DEC_ERR_ARG;
  if (scaling == DEC_ROPE_NTK && rot_dim <= 2) return DEC_ERR_ARG;
  if (scaling == DEC_ROPE_PARTS &&
      (!(orig_ctx > 0.0) || !(beta > alpha) || !isfinite(orig_ctx) || !isfinite(alpha) ||
       !isfinite(beta)))
    return DEC_ERR_ARG;
  const long double two_pi = 6.283185307179586476925286766559L;
  long double base = theta;
  if (scaling == DEC_ROPE_NTK)
    base *= powl(static_cast<long double>(factor),
                 static_cast<long double>(rot_dim) / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    long double f = powl(base, -2.0L * i / rot_dim);
    if (scaling == DEC_ROPE_LINEAR) f /= factor;
    if (scaling == DEC_ROPE_PARTS) {
      long double g = (orig_ctx * f / two_pi - alpha) / (static_cast<long double>(beta) - alpha);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f = g * f + (1 - g) * f / factor;
    }
    long double turns = f / two_pi;
    turns -= floorl(turns);
    long double scaled = floorl(turns * 18446744073709551616.0L + 0.5L);
    phases[i] = scaled >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(scaled);
  }
  return DEC_OK;
}

extern "C" int dec_rope_apply(int n_tokens, int n_heads, int head_dim, int dtype, const void* x,
                              long long x_stride, void* out, long long out_stride,
                              const int32_t* positions, const dec_rope* rope, void* stream) {
  if (!rope) return DEC_ERR_NULL;
  if (n_tokens < 0) return DEC_ERR_BATCH;
  if (dtype != DEC_BF16 && dtype != DEC_F32) return DEC_ERR_DTYPE;
  if ((head_dim != 64 && head_dim != 128) || n_heads < 1 || n_heads > 65536) return DEC_ERR_SHAPE;
  int rc = check_rope(rope, head_dim);
  if (rc != DEC_OK) return rc;
  if (n_tokens == 0) return DEC_OK;
  if (!x || !out || !positions) return DEC_ERR_NULL;
  if (!is_aligned(x, 16) || !is_aligned(out, 16) || !is_aligned(positions, 4)) return DEC_ERR_ALIGN;
  if ((rc = check_stride(x_stride, n_tokens, n_heads, head_dim)) != DEC_OK) return rc;
  if ((rc = check_stride(out_stride, n_tokens, n_heads, head_dim)) != DEC_OK) return rc;
  if (x == out && n_tokens > 1 && x_stride != out_stride) return DEC_ERR_ARG;
  const int sms = device_sms();
  if (sms < 0) return sms;
  RowsArgs a{};
  a.n_tokens = n_tokens;
  a.Hq = n_heads;
  a.q = x;
  a.q_stride = x_stride;
  a.q_out = out;
  a.q_out_stride = out_stride;
  a.positions = positions;
  a.phases = rope->phases;
  a.rot = rope->rot_dim;
  a.inter = rope->interleaved != 0;
  a.mscale = rope->mscale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DEC_BF16)
    e = head_dim == 128 ? launch_rows<128, uint16_t, uint16_t, 0>(a, sms, s)
                        : launch_rows<64, uint16_t, uint16_t, 0>(a, sms, s);
  else
    e = head_dim == 128 ? launch_rows<128, float, float, 0>(a, sms, s)
                        : launch_rows<64, float, float, 0>(a, sms, s);
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}

extern "C" int dec_paged_append(const dec_pages* pool, const dec_page_map* map, int layer,
                                const dec_append* io, int* status, void* stream) {
  int rc = check_pool(pool);
  if (rc != DEC_OK) return rc;
  if ((rc = check_map(pool, map)) != DEC_OK) return rc;
  if (!io) return DEC_ERR_NULL;
  if (layer < 0 || layer >= pool->n_layers) return DEC_ERR_ARG;
  const int D = pool->head_dim, n = io->n_tokens;
  if (n < 0 || (!io->seqs && n > map->n_seqs)) return DEC_ERR_BATCH;
  if (io->dtype != DEC_BF16 && io->dtype != DEC_F32) return DEC_ERR_DTYPE;
  if (io->n_q_heads < 0 || io->n_q_heads > 65536) return DEC_ERR_SHAPE;
  if (io->rope && (rc = check_rope(io->rope, D)) != DEC_OK) return rc;
  if (n == 0) return DEC_OK;
  if (!io->k || !io->v || !io->positions) return DEC_ERR_NULL;
  if (io->n_q_heads ? (!io->q || !io->q_out) : (io->q || io->q_out)) return DEC_ERR_NULL;
  if (!(io->eps >= 0.f)) return DEC_ERR_ARG;
  if (!is_aligned(io->k, 16) || !is_aligned(io->v, 16) || !is_aligned(io->positions, 4) ||
      !is_aligned(io->seqs, 4) || !is_aligned(status, 4))
    return DEC_ERR_ALIGN;
  if (io->n_q_heads && (!is_aligned(io->q, 16) || !is_aligned(io->q_out, 16)))
    return DEC_ERR_ALIGN;
  if ((io->q_norm && !is_aligned(io->q_norm, 16)) || (io->k_norm && !is_aligned(io->k_norm, 16)))
    return DEC_ERR_ALIGN;
  if ((rc = check_stride(io->k_stride, n, pool->n_kv_heads, D)) != DEC_OK) return rc;
  if ((rc = check_stride(io->v_stride, n, pool->n_kv_heads, D)) != DEC_OK) return rc;
  if (io->n_q_heads && (rc = check_stride(io->q_stride, n, io->n_q_heads, D)) != DEC_OK) return rc;
  const int sms = device_sms();
  if (sms < 0) return sms;
  RowsArgs a{};
  a.n_tokens = n;
  a.Hq = io->n_q_heads;
  a.Hkv = pool->n_kv_heads;
  a.q = io->q;
  a.k = io->k;
  a.v = io->v;
  a.q_stride = io->q_stride;
  a.k_stride = io->k_stride;
  a.v_stride = io->v_stride;
  a.q_out = io->q_out;
  a.q_out_stride = static_cast<long long>(io->n_q_heads) * D;
  a.positions = io->positions;
  a.seqs = io->seqs;
  a.q_norm = static_cast<const uint16_t*>(io->q_norm);
  a.k_norm = static_cast<const uint16_t*>(io->k_norm);
  a.eps = io->eps;
  a.zero = io->zero_skipped != 0;
  if (io->rope) {
    a.phases = io->rope->phases;
    a.rot = io->rope->rot_dim;
    a.inter = io->rope->interleaved != 0;
    a.mscale = io->rope->mscale;
  }
  a.table = map->table;
  a.n_seqs = map->n_seqs;
  a.width = map->width;
  a.pool = layer_view(pool, layer);
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = pool->dtype == DEC_KV_FP8_E4M3, f32 = io->dtype == DEC_F32;
  cudaError_t e;
  if (D == 128) {
    if (f32)
      e = fp8 ? launch_rows<128, float, uint16_t, 2>(a, sms, s) : launch_rows<128, float, uint16_t, 1>(a, sms, s);
    else
      e = fp8 ? launch_rows<128, uint16_t, uint16_t, 2>(a, sms, s)
              : launch_rows<128, uint16_t, uint16_t, 1>(a, sms, s);
  } else {
    if (f32)
      e = fp8 ? launch_rows<64, float, uint16_t, 2>(a, sms, s) : launch_rows<64, float, uint16_t, 1>(a, sms, s);
    else
      e = fp8 ? launch_rows<64, uint16_t, uint16_t, 2>(a, sms, s)
              : launch_rows<64, uint16_t, uint16_t, 1>(a, sms, s);
  }
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}
