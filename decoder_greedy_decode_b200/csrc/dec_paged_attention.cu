// dec_paged_attention.cu -- attention of one new token per sequence over a
// paged KV cache.
//
// Mathematics.  out = sum_j softmax_j(q . k_j / sqrt(D)) v_j with the running
// maximum m and sum l of an online softmax in fp32 (log2 units: a score is
// q . k * log2(e) / sqrt(D), exact bf16 products summed in fp32 by the tensor
// core).  A stretch of rows leaves (m, l, sum p v); stretches are joined by
// rescaling to the larger m.
//
// Bound and split.  Every K and V row is read once and used for the query
// heads of its KV head only: the bound is HBM.  The unit of work is a tile of
// 16 rows of one (sequence, KV head).  The tiles of all sequences, counted
// from the lengths on the device, are dealt in equal contiguous runs to the
// warps of a grid that just fills the GPU, so a ragged batch costs what its
// rows cost.  A warp works alone: it copies its tiles into a ring of its own
// (cp.async, several tiles ahead, across sequence boundaries), so no barrier
// holds the stream up.  A run that covers a whole (sequence, KV head) writes
// the output; otherwise it leaves its state in the workspace and a second,
// dependent launch joins the states in run order (the result does not depend
// on timing).
//
// Tile layout.  Every lane copies exactly the 16-byte pieces that it will use
// itself, into its own column of the ring ([piece][lane], free of bank
// conflicts), so a tile needs no barrier either.  For the scores the rows
// are the M of a 16x8x16 warp MMA and the heads its N; the order of the head
// elements along K is free as long as q uses the same, so a lane's 16-byte
// piece of a K row is its A fragment as it stands.  For the output, V^T is A
// (M = head elements, K = rows): the lane holds four rows of the same
// elements and one byte permute per register pairs two rows.  P goes from the
// score layout to the B fragment by a warp-wide 8x8 transpose.
//
// Rounding.  P enters the second MMA as two bf16 planes, hi = bf16(p) and
// lo = bf16(p - hi) (2^-17 relative; one plane would cost 2^-8).  lo may be 0
// or negative, so it meets V with infinities made finite: hi alone decides
// what an infinite element gives.  E4M3 codes
// are exact in f16 and stay codes: the K scale multiplies the score, the V
// scale multiplies p, whose planes are then f16 after a power-of-two factor F
// per head that keeps the largest p * scale near 2^14 (2^-22 relative, values
// below 2^-39 of the largest lost).  q is made f16 by a power of two per
// head, exact down to 2^-38 of the head's largest element.
#include <cuda_runtime.h>

#include "dec.h"
#include "dec_paged.h"
#include "dec_ptx.cuh"
#include "dec_tc.cuh"

namespace dec {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;     // rows of a tile
constexpr int kMaxHeads = 8;  // query heads per KV head (the N of the MMA)

struct PagedArgs {
  PoolView pool;
  const int32_t* table;
  int width;
  const int32_t* rows;
  int B, Hq, Hkv, rep;
  const uint16_t* q;
  long long q_stride;
  int window, max_rows;
  float* out;
  float* lse;
  float* part;     // [warps][2] states: rep x D sums, then rep x (m, l)
  int2* desc;      // [B][Hkv] (first warp, warps) of the states to join
  int* status;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8x8 matrix of 16-bit values spread over the warp (lane
// l holds row l/4, columns 2(l%4) and the next).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// BYTES (4, 8 or 16) global -> shared; zeros when !valid (src is not read).
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two bf16 values, infinities (and NaN) replaced by the largest finite value
// of their sign.
__device__ __forceinline__ uint32_t finite(uint32_t x) {
  uint32_t r;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7F7F7F7Fu));
  return r;
}
// Two E4M3 codes (low 16 bits) -> two f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(c)));
  return r;
}
__device__ __forceinline__ uint32_t f2_to_h2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// 2^e for a normal exponent.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// A warp's place in the list of tiles: sequence, KV head, tile of it.
struct Place {
  int b, g, tile, tiles;  // tiles: of one (sequence, KV head)
  int lo, len;            // rows [lo, len)
  __device__ __forceinline__ int row0() const { return (lo & ~(kTile - 1)) + tile * kTile; }
};

__device__ __forceinline__ int tiles_of(const PagedArgs& a, int n, int& lo) {
  lo = a.window > 0 && n > a.window ? n - a.window : 0;
  if (n < 1 || n > a.max_rows) return 0;
  return (n - (lo & ~(kTile - 1)) + kTile - 1) / kTile;
}
__device__ __forceinline__ void enter(const PagedArgs& a, Place& p) {
  p.g = 0;
  p.tile = 0;
  p.tiles = 0;
  while (p.b < a.B) {
    p.len = a.rows[p.b];
    p.tiles = tiles_of(a, p.len, p.lo);
    if (p.tiles) return;
    ++p.b;
  }
}
__device__ __forceinline__ void next(const PagedArgs& a, Place& p) {
  if (++p.tile < p.tiles) return;
  p.tile = 0;
  if (++p.g < a.Hkv) return;
  ++p.b;
  enter(a, p);
}

// Bytes of one tile in a warp's ring (K and V pieces, then E4M3 row scales).
template <int D, bool FP8>
constexpr int tile_bytes() {
  return FP8 ? 2 * kTile * D + kTile * 8 : 2 * kTile * D * 2;
}
template <int D, bool FP8>
constexpr int stages() {
  return FP8 ? (D == 128 ? 6 : 8) : (D == 128 ? 3 : 6);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 2) paged_kernel(const PagedArgs a) {
  constexpr int S = stages<D, FP8>();
  constexpr int TB = tile_bytes<D, FP8>();
  constexpr int ES = FP8 ? 1 : 2;               // bytes of an element
  constexpr int KP = D * ES / 64;               // 16-byte pieces of a K row per lane
  constexpr int MT = D / 16;                    // M tiles of V^T
  constexpr int VB = D * ES / 8 >= 16 ? 16 : 8; // bytes of a V piece
  constexpr int VP = D * ES / 8 / VB;           // pieces of a V row per lane
  constexpr int KBYTES = kTile * D * ES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sum[kWarps];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int nwarps = gridDim.x * kWarps;
  const int me = blockIdx.x * kWarps + warp;
  pdl_trigger();

  // The runs: total tiles, then this warp's first sequence.
  long long total = 0;
  {
    long long sum = 0;
    int lo;
    for (int b = threadIdx.x; b < a.B; b += kThreads) sum += tiles_of(a, a.rows[b], lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_sum[w];
    total *= a.Hkv;
  }
  const long long run = (total + nwarps - 1) / nwarps;
  const long long first = me * run;
  if (first >= total) return;
  const int count = static_cast<int>(min(run, total - first));
  // (each warp scans for itself: 32 sequences at a time)
  long long base = 0;
  Place ip;
  ip.b = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    int lo;
    const int b = b0 + lane;
    const long long n = b < a.B ? static_cast<long long>(tiles_of(a, a.rows[b], lo)) * a.Hkv : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + inc > first);
    if (hit) {
      const int l = __ffs(hit) - 1;
      ip.b = b0 + l;
      base += __shfl_sync(0xffffffffu, inc - n, l);
      break;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  enter(a, ip);
  ip.g = static_cast<int>((first - base) / ip.tiles);
  ip.tile = static_cast<int>((first - base) % ip.tiles);
  Place cp = ip;

  // ---- issue side: tile i of the run into ring slot i % S
  const uint32_t ring = smem_u32(smem) + warp * (S * TB);
  const int page_mask = (1 << a.pool.shift) - 1;
  int ids[2];       // page ids of the next tile's two row octets (-1: nothing needed)
  unsigned bad = 0; // bit s: the tile in slot s named a page out of range
  auto fetch_ids = [&]() {
    const int r0 = ip.row0();
    const int32_t* row = a.table + static_cast<long long>(ip.b) * a.width;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int r = r0 + 8 * o;
      ids[o] = (r + 7 >= ip.lo && r < ip.len) ? row[r >> a.pool.shift] : -2;
    }
  };
  int issued = 0;
  auto issue = [&]() {
    if (issued < count) {
      const int slot = issued % S;
      const uint32_t dst = ring + slot * TB;
      const int r0 = ip.row0();
      bool use[2];
      const uint8_t *kp[2], *vp[2];
      long long srow[2];
      unsigned wrong = 0;
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const bool ok = ids[o] >= 0 && ids[o] < a.pool.n_pages;
        if (!ok && ids[o] != -2) wrong = 1;
        use[o] = ok;
        const long long e =
            ok ? ids[o] * a.pool.page_stride +
                     ((static_cast<long long>(ip.g) << a.pool.shift) + ((r0 + 8 * o) & page_mask)) * D
               : 0;
        kp[o] = a.pool.k + e * ES;
        vp[o] = a.pool.v + e * ES;
        srow[o] = e / D;
      }
      bad = (bad & ~(1u << slot)) | (wrong << slot);
      auto in = [&](int r) { return r >= ip.lo && r < ip.len; };
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const bool ok = use[o] && in(r0 + 8 * o + g8);
#pragma unroll
        for (int c = 0; c < KP; ++c)
          copy_async<16>(dst + ((o * KP + c) * 32 + lane) * 16,
                         kp[o] + (ok ? g8 * (D * ES) + (4 * c + t4) * 16 : 0), ok);
      }
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * t4 + e;
          const bool ok = use[o] && in(r0 + 8 * o + r);
#pragma unroll
          for (int c = 0; c < VP; ++c)
            copy_async<VB>(dst + KBYTES + (((o * 2 + e) * VP + c) * 32 + lane) * VB,
                           vp[o] + (ok ? r * (D * ES) + (8 * c + g8) * VB : 0), ok);
        }
      if constexpr (FP8) {
        // row g8's four scales (K and V of rows g8 and g8 + 8), one a lane
        const int o = t4 & 1;
        const bool ok = use[o] && in(r0 + 8 * o + g8);
        copy_async<4>(dst + 2 * KBYTES + lane * 4,
                      (t4 < 2 ? a.pool.ks : a.pool.vs) + (ok ? srow[o] + g8 : 0), ok);
      }
      if (++issued < count) {
        next(a, ip);
        fetch_ids();
      }
    }
    copy_commit();
  };
  fetch_ids();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();

  // ---- compute side
  const float scale = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  uint32_t qb[KP * (FP8 ? 8 : 4)];  // B fragments of q^T (head g8), two registers a K step
  float sc0 = 0.f, sc1 = 0.f;       // score scale of heads 2 t4 and 2 t4 + 1
  float m0, m1, l0, l1;             // running maximum; this lane's share of the sum
  float w0 = 0.f, w1 = 0.f, F0 = 1.f, F1 = 1.f;  // E4M3: largest p * scale, factor
  float acc[MT][4];
  bool poison = false;
  int begin = cp.tile;              // first tile of the segment in this run

  auto start = [&]() {
    const uint16_t* qh = a.q + cp.b * a.q_stride + (static_cast<long long>(cp.g) * a.rep + g8) * D;
    float up = 1.f;
    if constexpr (FP8) {
      float am = 0.f;
      float x[KP][16];
#pragma unroll
      for (int c = 0; c < KP; ++c) {
        uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (g8 < a.rep) {
          w[0] = *reinterpret_cast<const uint4*>(qh + (4 * c + t4) * 16);
          w[1] = *reinterpret_cast<const uint4*>(qh + (4 * c + t4) * 16 + 8);
        }
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[c][2 * i] = bf16lo(u[i]);
          x[c][2 * i + 1] = bf16hi(u[i]);
          am = fmaxf(am, fmaxf(fabsf(x[c][2 * i]), fabsf(x[c][2 * i + 1])));
        }
      }
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      // 2^(14 - exponent): the head's largest element goes to [2^14, 2^15)
      const int ex = static_cast<int>(__float_as_uint(am) >> 23) - 127;
      int sh = 14 - ex;
      if (am == 0.f || ex > 127) sh = 0;   // zeros, or an infinity (which stays one)
      sh = min(sh, 126);
      up = pow2i(-sh);
      // in two steps: 2^sh may pass 2^127 / the smallest elements
      const float s1 = pow2i(sh / 2), s2 = pow2i(sh - sh / 2);
#pragma unroll
      for (int c = 0; c < KP; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          qb[c * 8 + i] = f2_to_h2(x[c][2 * i] * s1 * s2, x[c][2 * i + 1] * s1 * s2);
    } else {
#pragma unroll
      for (int c = 0; c < KP; ++c) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (g8 < a.rep) w = *reinterpret_cast<const uint4*>(qh + (4 * c + t4) * 8);
        qb[c * 4] = w.x;
        qb[c * 4 + 1] = w.y;
        qb[c * 4 + 2] = w.z;
        qb[c * 4 + 3] = w.w;
      }
    }
    sc0 = scale * __shfl_sync(0xffffffffu, up, (2 * t4) * 4);
    sc1 = scale * __shfl_sync(0xffffffffu, up, (2 * t4 + 1) * 4);
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    w0 = w1 = 0.f;
    F0 = F1 = 1.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    poison = false;
    begin = cp.tile;
  };
  auto over_rows = [&](float x) {   // maximum over the 8 lanes of a head pair
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
  };
  auto rescale = [&](float x0, float x1) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      acc[i][0] *= x0;
      acc[i][1] *= x1;
      acc[i][2] *= x0;
      acc[i][3] *= x1;
    }
  };

  auto tile_step = [&](uint32_t src) {
    // scores: rows g8 and g8 + 8, heads 2 t4 and 2 t4 + 1
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int c = 0; c < KP; ++c) {
      const uint4 x = lds128(src + (c * 32 + lane) * 16);
      const uint4 y = lds128(src + ((KP + c) * 32 + lane) * 16);
      const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
      if constexpr (FP8) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f16(s[j & 1], e4m3x2_to_h2(xa[j]), e4m3x2_to_h2(ya[j]), e4m3x2_to_h2(xa[j] >> 16),
                  e4m3x2_to_h2(ya[j] >> 16), qb[c * 8 + 2 * j], qb[c * 8 + 2 * j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          mma_bf16(s[j], xa[2 * j], ya[2 * j], xa[2 * j + 1], ya[2 * j + 1], qb[c * 4 + 2 * j],
                   qb[c * 4 + 2 * j + 1]);
      }
    }
    float ks0 = 1.f, ks1 = 1.f, vs0 = 1.f, vs1 = 1.f;
    if constexpr (FP8) {
      const uint4 f = lds128(src + 2 * KBYTES + g8 * 16);
      ks0 = __uint_as_float(f.x);
      ks1 = __uint_as_float(f.y);
      vs0 = __uint_as_float(f.z);
      vs1 = __uint_as_float(f.w);
    }
    float x0 = (s[0][0] + s[1][0]) * (sc0 * ks0), x1 = (s[0][1] + s[1][1]) * (sc1 * ks0);
    float x2 = (s[0][2] + s[1][2]) * (sc0 * ks1), x3 = (s[0][3] + s[1][3]) * (sc1 * ks1);
    const int r0 = cp.row0();
    if (r0 < cp.lo || r0 + kTile > cp.len) {
      const int ra = r0 + g8, rb = ra + 8;
      if (ra < cp.lo || ra >= cp.len) x0 = x1 = -INFINITY;
      if (rb < cp.lo || rb >= cp.len) x2 = x3 = -INFINITY;
    }
    const float t0 = fmaxf(x0, x2), t1 = fmaxf(x1, x3);
    const bool grow = t0 > m0 || t1 > m1;
    const bool up = __any_sync(0xffffffffu, grow);
    if (up) {
      const float n0 = fmaxf(m0, over_rows(t0)), n1 = fmaxf(m1, over_rows(t1));
      // (no score above -inf yet: nothing to rescale)
      const float e0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0);
      const float e1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= e0;
      l1 *= e1;
      w0 *= e0;
      w1 *= e1;
      rescale(e0, e1);
    }
    // (a maximum of -inf: every score so far is -inf, and p = 2^-inf = 0)
    const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
    x0 = ex2(x0 - b0);
    x1 = ex2(x1 - b1);
    x2 = ex2(x2 - b0);
    x3 = ex2(x3 - b1);
    l0 += x0 + x2;
    l1 += x1 + x3;
    uint32_t hi0, hi1, lo0, lo1;
    if constexpr (FP8) {
      x0 *= vs0;
      x1 *= vs0;
      x2 *= vs1;
      x3 *= vs1;
      const float u0 = fmaxf(x0, x2), u1 = fmaxf(x1, x3);
      // the factor keeps the largest p * scale in [2^13, 2^14): set anew
      // when the maximum moved, or when a value would pass 2^15
      if (__any_sync(0xffffffffu, up || u0 * F0 > 32768.f || u1 * F1 > 32768.f)) {
        w0 = fmaxf(w0, over_rows(u0));
        w1 = fmaxf(w1, over_rows(u1));
        auto factor = [](float w) {
          const int ex = static_cast<int>(__float_as_uint(w) >> 23) - 127;
          return pow2i(min(max(13 - ex, -126), 126));
        };
        const float f0 = factor(w0), f1 = factor(w1);
        // (the ratio may pass the range of one float: two halves)
        const int d0 = (__float_as_int(f0) - __float_as_int(F0)) / (1 << 23);
        const int d1 = (__float_as_int(f1) - __float_as_int(F1)) / (1 << 23);
        rescale(pow2i(d0 / 2), pow2i(d1 / 2));
        rescale(pow2i(d0 - d0 / 2), pow2i(d1 - d1 / 2));
        F0 = f0;
        F1 = f1;
      }
      x0 *= F0;
      x1 *= F1;
      x2 *= F0;
      x3 *= F1;
      hi0 = f2_to_h2(x0, x1);
      hi1 = f2_to_h2(x2, x3);
      const float2 a0 = h2_to_f2(hi0), a1 = h2_to_f2(hi1);
      lo0 = f2_to_h2(x0 - a0.x, x1 - a0.y);
      lo1 = f2_to_h2(x2 - a1.x, x3 - a1.y);
    } else {
      hi0 = f2_to_bf16x2(x0, x1);
      hi1 = f2_to_bf16x2(x2, x3);
      lo0 = f2_to_bf16x2(x0 - bf16lo(hi0), x1 - bf16hi(hi0));
      lo1 = f2_to_bf16x2(x2 - bf16lo(hi1), x3 - bf16hi(hi1));
    }
    hi0 = transpose8(hi0);
    hi1 = transpose8(hi1);
    lo0 = transpose8(lo0);
    lo1 = transpose8(lo1);
    // V^T: rows 2 t4, 2 t4 + 1 (octet 0) and the same of octet 1
    const uint32_t vsrc = src + KBYTES;
    if constexpr (!FP8) {
#pragma unroll
      for (int c = 0; c < VP; ++c) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = lds128(vsrc + ((e * VP + c) * 32 + lane) * 16);
        const uint32_t x[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w},
                                  {v[1].x, v[1].y, v[1].z, v[1].w},
                                  {v[2].x, v[2].y, v[2].z, v[2].w},
                                  {v[3].x, v[3].y, v[3].z, v[3].w}};
        // M tile: rows g8 = element 8 g8 + 2 i of this piece, rows g8 + 8 =
        // the next element
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = __byte_perm(x[0][i], x[1][i], 0x5410);
          const uint32_t a1 = __byte_perm(x[0][i], x[1][i], 0x7632);
          const uint32_t a2 = __byte_perm(x[2][i], x[3][i], 0x5410);
          const uint32_t a3 = __byte_perm(x[2][i], x[3][i], 0x7632);
          mma_bf16(acc[c * 4 + i], a0, a1, a2, a3, hi0, hi1);
          mma_bf16(acc[c * 4 + i], finite(a0), finite(a1), finite(a2), finite(a3), lo0, lo1);
        }
      }
    } else {
      uint32_t x[4][VB / 4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (VB == 16) {
          const uint4 v = lds128(vsrc + (e * 32 + lane) * 16);
          x[e][0] = v.x;
          x[e][1] = v.y;
          x[e][2] = v.z;
          x[e][3] = v.w;
        } else {
          const uint2 v = lds64(vsrc + (e * 32 + lane) * 8);
          x[e][0] = v.x;
          x[e][1] = v.y;
        }
      }
#pragma unroll
      for (int i = 0; i < VB / 4; ++i) {
        // codes of two rows side by side: (r0 d0, r1 d0, r0 d1, r1 d1), ...
        const uint32_t p0 = __byte_perm(x[0][i], x[1][i], 0x5140);
        const uint32_t p1 = __byte_perm(x[0][i], x[1][i], 0x7362);
        const uint32_t q0 = __byte_perm(x[2][i], x[3][i], 0x5140);
        const uint32_t q1 = __byte_perm(x[2][i], x[3][i], 0x7362);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t p = j ? p1 : p0, q = j ? q1 : q0;
          const uint32_t a0 = e4m3x2_to_h2(p), a1 = e4m3x2_to_h2(p >> 16);
          const uint32_t a2 = e4m3x2_to_h2(q), a3 = e4m3x2_to_h2(q >> 16);
          mma_f16(acc[2 * i + j], a0, a1, a2, a3, hi0, hi1);
          mma_f16(acc[2 * i + j], a0, a1, a2, a3, lo0, lo1);
        }
      }
    }
  };

  // The segment of (cp.b, cp.g) ends with the current tile.
  auto finish = [&]() {
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    const bool whole = begin == 0 && cp.tile + 1 == cp.tiles;
    const int h0 = 2 * t4, h1 = h0 + 1;
    if (begin == 0 && lane == 0) {
      // (the other warps of this (sequence, KV head) follow in order)
      const long long rest = cp.tiles - (cp.tile + 1);
      a.desc[static_cast<long long>(cp.b) * a.Hkv + cp.g] =
          make_int2(me, whole ? 0 : 1 + static_cast<int>((rest + run - 1) / run));
    }
    if (whole && poison) return;
    if (FP8) rescale(1.f / F0, 1.f / F1);
    // element of acc[i][0/1] and acc[i][2/3]
    auto elem = [&](int i) {
      return FP8 ? (D / 8) * g8 + 2 * i : 64 * (i / 4) + 8 * g8 + 2 * (i % 4);
    };
    float *o0, *o1;
    float z0 = 1.f, z1 = 1.f;
    if (whole) {
      o0 = a.out + (static_cast<long long>(cp.b) * a.Hq + static_cast<long long>(cp.g) * a.rep + h0) * D;
      o1 = o0 + D;
      z0 = 1.f / l0;
      z1 = 1.f / l1;
      if (g8 == 0 && a.lse) {
        float* ls = a.lse + static_cast<long long>(cp.b) * a.Hq + static_cast<long long>(cp.g) * a.rep;
        if (h0 < a.rep) ls[h0] = (m0 + log2f(l0)) * 0.6931471805599453f;
        if (h1 < a.rep) ls[h1] = (m1 + log2f(l1)) * 0.6931471805599453f;
      }
    } else {
      float* st = a.part + (static_cast<long long>(me) * 2 + (begin == 0)) * a.rep * (D + 2);
      o0 = st + h0 * D;
      o1 = o0 + D;
      if (g8 == 0) {
        float* ml = st + a.rep * D;
        const float nan = __int_as_float(0x7fffffff);   // marks a poisoned state
        if (h0 < a.rep) {
          ml[2 * h0] = poison ? nan : m0;
          ml[2 * h0 + 1] = l0;
        }
        if (h1 < a.rep) {
          ml[2 * h1] = poison ? nan : m1;
          ml[2 * h1 + 1] = l1;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int e = elem(i);
      if (h0 < a.rep) *reinterpret_cast<float2*>(o0 + e) = make_float2(acc[i][0] * z0, acc[i][2] * z0);
      if (h1 < a.rep) *reinterpret_cast<float2*>(o1 + e) = make_float2(acc[i][1] * z1, acc[i][3] * z1);
    }
  };

  start();
  for (int i = 0; i < count; ++i) {
    issue();
    copy_wait<S - 1>();
    if (FP8) __syncwarp();   // the scales are read by other lanes than copied them
    const int slot = i % S;
    if ((bad >> slot) & 1) {
      poison = true;
      if (a.status && lane == 0) atomicOr(a.status, DEC_DEV_BAD_PAGE);
    }
    tile_step(ring + slot * TB);
    if (FP8) __syncwarp();
    const bool last = cp.tile + 1 == cp.tiles;
    if (last || i + 1 == count) finish();
    if (i + 1 < count) {
      next(a, cp);
      if (last) start();
    }
  }
  copy_wait<0>();
}

// Joins the states of one (sequence, query head); also the outputs of empty
// sequences.  Four groups of 32 lanes take every fourth state.
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const PagedArgs a) {
  __shared__ float s_acc[4][D];
  __shared__ float s_ml[4][2];
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
  const int g = h / a.rep, hh = h % a.rep;
  const int grp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int n = a.rows[b];
  float* out = a.out + (static_cast<long long>(b) * a.Hq + h) * D;
  if (n < 0 || n > a.max_rows) {
    if (threadIdx.x == 0 && h == 0 && a.status) atomicOr(a.status, DEC_DEV_BAD_POSITION);
    return;
  }
  if (n == 0) {
    if (threadIdx.x < D) out[threadIdx.x] = 0.f;
    if (threadIdx.x == 0 && a.lse) a.lse[static_cast<long long>(b) * a.Hq + h] = -INFINITY;
    return;
  }
  const int2 d = a.desc[static_cast<long long>(b) * a.Hkv + g];
  if (d.y == 0) return;   // written by its one warp
  const long long stride = static_cast<long long>(a.rep) * (D + 2);
  constexpr int E = D / 32;
  float M = -INFINITY, L = 0.f, acc[E];
  bool poison = false;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i = grp; i < d.y; i += 4) {
    // the first state is its warp's last, the others their warps' first
    const float* st = a.part + (static_cast<long long>(d.x + i) * 2 + (i == 0)) * stride;
    const float m = __ldcg(st + a.rep * D + 2 * hh), l = __ldcg(st + a.rep * D + 2 * hh + 1);
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __ldcg(st + hh * D + e * 32 + lane);
    if (m != m) poison = true;
    const float nm = fmaxf(M, m);
    const float e0 = M == -INFINITY ? 0.f : ex2(M - nm), e1 = m == -INFINITY ? 0.f : ex2(m - nm);
    L = L * e0 + l * e1;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * e0 + v[e] * e1;
    M = nm;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[grp][e * 32 + lane] = acc[e];
  if (lane == 0) {
    s_ml[grp][0] = M;
    s_ml[grp][1] = L;
  }
  if (__syncthreads_or(poison)) return;
  if (threadIdx.x < D) {
    float m = -INFINITY, l = 0.f, x = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, s_ml[i][0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = s_ml[i][0] == -INFINITY ? 0.f : ex2(s_ml[i][0] - m);
      l += s_ml[i][1] * e;
      x += s_acc[i][threadIdx.x] * e;
    }
    out[threadIdx.x] = x / l;
    if (threadIdx.x == 0 && a.lse)
      a.lse[static_cast<long long>(b) * a.Hq + h] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, bool FP8>
cudaError_t launch_paged(const PagedArgs& a, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = kWarps * stages<D, FP8>() * tile_bytes<D, FP8>();
  cudaError_t e = allow_smem(paged_kernel<D, FP8>, smem, done);
  if (e != cudaSuccess) return e;
  paged_kernel<D, FP8><<<grid, kThreads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(join_kernel<D>, dim3(static_cast<unsigned>(a.B) * a.Hq), dim3(128), 0, s, a);
}

// CTAs of the grid: two to an SM.
int paged_grid(int sms) { return 2 * sms; }

size_t state_bytes(int grid, int rep, int D) {
  return round256(sizeof(float) * static_cast<size_t>(grid) * kWarps * 2 * rep * (D + 2));
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" size_t dec_paged_attention_workspace_bytes(const dec_pages* pool, int batch,
                                                      int n_q_heads) {
  if (check_pool(pool) != DEC_OK || batch < 1 || batch > 4096 || n_q_heads < 1 ||
      n_q_heads % pool->n_kv_heads || n_q_heads / pool->n_kv_heads > kMaxHeads)
    return 0;
  const int sms = device_sms();
  return state_bytes(paged_grid(sms > 0 ? sms : 148), n_q_heads / pool->n_kv_heads,
                     pool->head_dim) +
         round256(sizeof(int2) * static_cast<size_t>(batch) * pool->n_kv_heads);
}

extern "C" int dec_paged_attention(const dec_pages* pool, const dec_page_map* map, int layer,
                                   int batch, int n_q_heads, const void* q, long long q_stride,
                                   const int32_t* rows, int window, float* out, float* lse,
                                   void* workspace, size_t workspace_bytes, int* status,
                                   void* stream) {
  int rc = check_pool(pool);
  if (rc != DEC_OK) return rc;
  if ((rc = check_map(pool, map)) != DEC_OK) return rc;
  if (!q || !out || !workspace) return DEC_ERR_NULL;
  if (batch < 1 || batch > map->n_seqs) return DEC_ERR_BATCH;
  if (layer < 0 || layer >= pool->n_layers || window < 0) return DEC_ERR_ARG;
  const int D = pool->head_dim;
  if (n_q_heads < 1 || n_q_heads % pool->n_kv_heads ||
      n_q_heads / pool->n_kv_heads > kMaxHeads)
    return DEC_ERR_SHAPE;
  if (batch > 1 && q_stride < static_cast<long long>(n_q_heads) * D) return DEC_ERR_SHAPE;
  if (!is_aligned(q, 16) || (batch > 1 && q_stride % 8) || !is_aligned(workspace, 256) || !is_aligned(out, 8))
    return DEC_ERR_ALIGN;
  if (workspace_bytes < dec_paged_attention_workspace_bytes(pool, batch, n_q_heads))
    return DEC_ERR_KV_SIZE;
  const int sms = device_sms();
  if (sms < 0) return sms;
  PagedArgs a{};
  a.pool = layer_view(pool, layer);
  a.table = map->table;
  a.width = map->width;
  a.rows = rows ? rows : map->rows;
  a.B = batch;
  a.Hq = n_q_heads;
  a.Hkv = pool->n_kv_heads;
  a.rep = n_q_heads / pool->n_kv_heads;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.window = window;
  a.max_rows = map->width * pool->page_rows;
  a.out = out;
  a.lse = lse;
  const int grid = paged_grid(sms);
  a.part = static_cast<float*>(workspace);
  a.desc = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + state_bytes(grid, a.rep, D));
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (pool->dtype == DEC_KV_FP8_E4M3)
    e = D == 128 ? launch_paged<128, true>(a, grid, s) : launch_paged<64, true>(a, grid, s);
  else
    e = D == 128 ? launch_paged<128, false>(a, grid, s) : launch_paged<64, false>(a, grid, s);
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}
