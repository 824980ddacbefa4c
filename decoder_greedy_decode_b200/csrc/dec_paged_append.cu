// dec_paged_append.cu -- rotary positions, and the append of new rows to a
// paged KV cache.
//
// Mathematics.  Pair i of a rotated head turns by p * f_i at position p.  The
// angle is kept in turns as a 64-bit binary fraction: p * phase_i modulo 2^64
// drops whole turns exactly, so the angle of any int32 position is right to
// 2^-33 turns (a product in fp32 is off by p * f_i * 2^-24 radians, i.e. by
// 0.06 rad at p = 2^20).  The rotation itself is fp32, rounded once.
//
// Split.  A warp takes one token and a few of its heads: the lanes hold the
// sine and cosine of their pairs in registers for all of them, a head row is
// 32 lanes x 2 pairs (head_dim 128) or 1 pair (64), so RMSNorm and the E4M3
// row maximum are warp reductions and nothing passes through shared memory.
// All head rows of a warp are loaded before the first is used (the loads are
// what bounds the kernel: every input is read once, every output written
// once).
#include <cuda_runtime.h>
#include <math.h>

#include "dec.h"
#include "dec_paged.h"
#include "dec_ptx.cuh"

namespace dec {
namespace {

constexpr int kWarps = 4;
constexpr int kHeadsPerWarp = 4;

struct RowsArgs {
  int n_tokens, Hq, Hkv;              // Hkv = 0: rotation alone
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void* q_out;
  long long q_out_stride;
  const int32_t *positions, *seqs;
  const uint16_t *q_norm, *k_norm;
  float eps;
  const uint64_t* phases;             // null: no rotation
  int rot, inter;
  float mscale;
  const int32_t* table;
  int n_seqs, width;
  PoolView pool;
  int* status;
};

template <typename T>
__device__ __forceinline__ float ld1(const T* p);
template <>
__device__ __forceinline__ float ld1<uint16_t>(const uint16_t* p) { return bf16_to_f(*p); }
template <>
__device__ __forceinline__ float ld1<float>(const float* p) { return *p; }
__device__ __forceinline__ void ld2(const uint16_t* p, float& a, float& b) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  a = bf16lo(w);
  b = bf16hi(w);
}
__device__ __forceinline__ void ld2(const float* p, float& a, float& b) {
  const float2 w = *reinterpret_cast<const float2*>(p);
  a = w.x;
  b = w.y;
}
__device__ __forceinline__ void st2(uint16_t* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = f2_to_bf16x2(a, b);
}
__device__ __forceinline__ void st2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void st1(uint16_t* p, float a) { *p = f_to_bf16(a); }
__device__ __forceinline__ void st1(float* p, float a) { *p = a; }

// Which elements a lane holds.  NP pairs a lane; x[2j], x[2j+1] are pair j.
// Rows whose pairs are neighbours (interleaved pairs, and rows without a
// rotation) are 2 NP consecutive elements.  Half-split pairs (i, i + R/2) of
// the rotated part, and the passed part split the same way, start at `lo` and
// `hi`; with NP = 2 both are two consecutive elements when R is a multiple of
// 4 (`vec`), else each element is addressed for itself.
template <int NP>
struct Slots {
  bool pairs;      // neighbouring pairs
  bool vec;
  int lo[NP], hi[NP];
};

template <int D>
__device__ __forceinline__ Slots<D / 64> half_slots(int lane, int R) {
  constexpr int NP = D / 64;
  Slots<NP> s;
  s.pairs = false;
  s.vec = NP == 2 && (R & 3) == 0;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int p = lane * NP + j;
    const int r = R >> 1;
    s.lo[j] = p < r ? p : R + (p - r);
    s.hi[j] = p < r ? p + r : R + (D - R) / 2 + (p - r);
  }
  return s;
}
template <int D>
__device__ __forceinline__ Slots<D / 64> pair_slots(int lane) {
  constexpr int NP = D / 64;
  Slots<NP> s;
  s.pairs = true;
  s.vec = true;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    s.lo[j] = 2 * (lane * NP + j);
    s.hi[j] = s.lo[j] + 1;
  }
  return s;
}

template <int NP, typename T>
__device__ __forceinline__ void load_row(const T* p, const Slots<NP>& s, float (&x)[2 * NP]) {
  if (s.pairs) {
#pragma unroll
    for (int j = 0; j < NP; ++j) ld2(p + s.lo[j], x[2 * j], x[2 * j + 1]);
  } else if (NP == 2 && s.vec) {
    ld2(p + s.lo[0], x[0], x[2]);
    ld2(p + s.hi[0], x[1], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      x[2 * j] = ld1(p + s.lo[j]);
      x[2 * j + 1] = ld1(p + s.hi[j]);
    }
  }
}
template <int NP, typename T>
__device__ __forceinline__ void store_row(T* p, const Slots<NP>& s, const float (&x)[2 * NP]) {
  if (s.pairs) {
#pragma unroll
    for (int j = 0; j < NP; ++j) st2(p + s.lo[j], x[2 * j], x[2 * j + 1]);
  } else if (NP == 2 && s.vec) {
    st2(p + s.lo[0], x[0], x[2]);
    st2(p + s.hi[0], x[1], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      st1(p + s.lo[j], x[2 * j]);
      st1(p + s.hi[j], x[2 * j + 1]);
    }
  }
}
// The E4M3 codes of a row (same slots), and its scale.
template <int NP>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scale, int lane,
                                            const Slots<NP>& s, const float (&x)[2 * NP]) {
  float am = 0.f;
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j) am = fmaxf(am, fabsf(x[j]));
  am = fmaxf(warp_max(am), 1.17549435e-38f);  // 2^-126
  const float sc = __fdiv_rn(am, 448.0f);
  if (lane == 0) *scale = sc;
  uint16_t c[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j)
    c[j] = f2_to_e4m3x2(__fdiv_rn(x[2 * j], sc), __fdiv_rn(x[2 * j + 1], sc));
  if (s.pairs) {
#pragma unroll
    for (int j = 0; j < NP; ++j) *reinterpret_cast<uint16_t*>(p + s.lo[j]) = c[j];
  } else if (NP == 2 && s.vec) {
    const uint32_t w = static_cast<uint32_t>(c[0]) | (static_cast<uint32_t>(c[NP - 1]) << 16);
    *reinterpret_cast<uint16_t*>(p + s.lo[0]) = static_cast<uint16_t>(__byte_perm(w, 0, 0x4420));
    *reinterpret_cast<uint16_t*>(p + s.hi[0]) = static_cast<uint16_t>(__byte_perm(w, 0, 0x4431));
  } else {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      p[s.lo[j]] = static_cast<uint8_t>(c[j]);
      p[s.hi[j]] = static_cast<uint8_t>(c[j] >> 8);
    }
  }
}

// T: element of q, k, v (and of q_out where TO = T).  CACHE 0: rotation alone;
// 1: bf16 pages; 2: E4M3 pages.
template <int D, typename T, typename TO, int CACHE>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const RowsArgs a, int q_units,
                                                            int k_units, int units) {
  constexpr int NP = D / 64;
  const int lane = threadIdx.x & 31;
  const long long job = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(job / units);
  const int u = static_cast<int>(job % units);
  if (t >= a.n_tokens) return;
  const int pos = a.positions[t];
  if (CACHE && pos < 0) return;   // (rotation alone: the row is copied)

  long long row0 = 0;   // element of the token's row of head 0 in the pages
  if (CACHE) {
    const int seq = a.seqs ? a.seqs[t] : t;
    const int slot = pos >> a.pool.shift;
    int page = -1;
    int bad = 0;
    if (seq < 0 || seq >= a.n_seqs) {
      bad = DEC_DEV_BAD_PAGE;
    } else if (slot >= a.width) {
      bad = DEC_DEV_BAD_POSITION;
    } else {
      page = a.table[static_cast<long long>(seq) * a.width + slot];
      if (page < 0 || page >= a.pool.n_pages) bad = DEC_DEV_BAD_PAGE;
    }
    if (bad) {
      if (a.status && lane == 0 && u == 0) atomicOr(a.status, bad);
      return;
    }
    row0 = page * a.pool.page_stride + static_cast<long long>(pos & ((1 << a.pool.shift) - 1)) * D;
  }

  // this warp's heads: of q, of k or of v
  const int part = u < q_units ? 0 : u < q_units + k_units ? 1 : 2;
  const int h0 = (part == 0 ? u : part == 1 ? u - q_units : u - q_units - k_units) * kHeadsPerWarp;
  const int nh = min(kHeadsPerWarp, (part == 0 ? a.Hq : a.Hkv) - h0);
  const bool turn = a.phases && part < 2 && pos >= 0;
  const Slots<NP> s = turn && !a.inter ? half_slots<D>(lane, a.rot) : pair_slots<D>(lane);
  const T* src = static_cast<const T*>(part == 0 ? a.q : part == 1 ? a.k : a.v) +
                 t * (part == 0 ? a.q_stride : part == 1 ? a.k_stride : a.v_stride) +
                 static_cast<long long>(h0) * D;

  float x[kHeadsPerWarp][2 * NP];
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i)
    if (i < nh) load_row<NP>(src + i * D, s, x[i]);

  float cs[NP], sn[NP];
  if (turn) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int p = lane * NP + j;
      cs[j] = 1.f;
      sn[j] = 0.f;
      if (p < (a.rot >> 1)) {
        // the angle in half turns, [-1, 1): the top 32 bits of the fraction
        const uint64_t ph = a.phases[p] * static_cast<uint64_t>(pos);
        sincospif(static_cast<float>(static_cast<int32_t>(ph >> 32)) * 0x1p-31f, &sn[j], &cs[j]);
        cs[j] *= a.mscale;
        sn[j] *= a.mscale;
      }
    }
  }
  const uint16_t* gain = part == 0 ? a.q_norm : part == 1 ? a.k_norm : nullptr;
  float g[2 * NP];
  if (gain) load_row<NP>(gain, s, g);

#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i) {
    if (i >= nh) break;
    if (gain) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * NP; ++e) ss = fmaf(x[i][e], x[i][e], ss);
      const float r = rsqrtf(warp_sum(ss) * (1.0f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 2 * NP; ++e) x[i][e] = x[i][e] * r * g[e];
    }
    if (turn) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float p = x[i][2 * j], q = x[i][2 * j + 1];
        // a passed pair is not multiplied (cos 1, sin 0 would turn an
        // infinity in it into NaN)
        if (lane * NP + j < (a.rot >> 1)) {
          x[i][2 * j] = p * cs[j] - q * sn[j];
          x[i][2 * j + 1] = q * cs[j] + p * sn[j];
        }
      }
    }
    if (part == 0) {
      store_row<NP>(static_cast<TO*>(a.q_out) + t * a.q_out_stride +
                        static_cast<long long>(h0 + i) * D,
                    s, x[i]);
    } else if (CACHE) {
      const long long e = row0 + (static_cast<long long>(h0 + i) << a.pool.shift) * D;
      uint8_t* base = part == 1 ? a.pool.k : a.pool.v;
      if (CACHE == 1)
        store_row<NP>(reinterpret_cast<uint16_t*>(base) + e, s, x[i]);
      else
        store_codes<NP>(base + e, (part == 1 ? a.pool.ks : a.pool.vs) + e / D, lane, s, x[i]);
    }
  }
}

template <int D, typename T, typename TO, int CACHE>
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s) {
  const int qu = (a.Hq + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const int ku = (a.Hkv + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const int units = qu + 2 * ku;
  const long long blocks = (static_cast<long long>(a.n_tokens) * units + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  rows_kernel<D, T, TO, CACHE><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(a, qu, ku,
                                                                                     units);
  return cudaGetLastError();
}

// Elements of T that a tensor of heads must be aligned to: 4 (two pairs).
bool bad_align(const void* p, int dtype) { return !is_aligned(p, dtype == DEC_BF16 ? 8 : 16); }

int check_rope(const dec_rope* r, int head_dim) {
  if (!r->phases) return DEC_ERR_NULL;
  if (r->rot_dim < 2 || r->rot_dim > head_dim || (r->rot_dim & 1)) return DEC_ERR_SHAPE;
  if (!is_aligned(r->phases, 8)) return DEC_ERR_ALIGN;
  return DEC_OK;
}

int check_stride(long long stride, int n, int heads, int D) {
  if (n <= 1) return DEC_OK;   // never used
  if (stride % 4) return DEC_ERR_ALIGN;
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
  if (bad_align(x, dtype) || bad_align(out, dtype)) return DEC_ERR_ALIGN;
  if ((rc = check_stride(x_stride, n_tokens, n_heads, head_dim)) != DEC_OK) return rc;
  if ((rc = check_stride(out_stride, n_tokens, n_heads, head_dim)) != DEC_OK) return rc;
  if (x == out && n_tokens > 1 && x_stride != out_stride) return DEC_ERR_ARG;
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
    e = head_dim == 128 ? launch_rows<128, uint16_t, uint16_t, 0>(a, s)
                        : launch_rows<64, uint16_t, uint16_t, 0>(a, s);
  else
    e = head_dim == 128 ? launch_rows<128, float, float, 0>(a, s)
                        : launch_rows<64, float, float, 0>(a, s);
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
  if (bad_align(io->k, io->dtype) || bad_align(io->v, io->dtype)) return DEC_ERR_ALIGN;
  if (io->n_q_heads && (bad_align(io->q, io->dtype) || bad_align(io->q_out, DEC_BF16)))
    return DEC_ERR_ALIGN;
  if ((io->q_norm && !is_aligned(io->q_norm, 4)) || (io->k_norm && !is_aligned(io->k_norm, 4)))
    return DEC_ERR_ALIGN;
  if ((rc = check_stride(io->k_stride, n, pool->n_kv_heads, D)) != DEC_OK) return rc;
  if ((rc = check_stride(io->v_stride, n, pool->n_kv_heads, D)) != DEC_OK) return rc;
  if (io->n_q_heads && (rc = check_stride(io->q_stride, n, io->n_q_heads, D)) != DEC_OK) return rc;
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
      e = fp8 ? launch_rows<128, float, uint16_t, 2>(a, s) : launch_rows<128, float, uint16_t, 1>(a, s);
    else
      e = fp8 ? launch_rows<128, uint16_t, uint16_t, 2>(a, s)
              : launch_rows<128, uint16_t, uint16_t, 1>(a, s);
  } else {
    if (f32)
      e = fp8 ? launch_rows<64, float, uint16_t, 2>(a, s) : launch_rows<64, float, uint16_t, 1>(a, s);
    else
      e = fp8 ? launch_rows<64, uint16_t, uint16_t, 2>(a, s)
              : launch_rows<64, uint16_t, uint16_t, 1>(a, s);
  }
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}
