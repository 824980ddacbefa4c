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
// 16 or 32 rows of one sequence.  The tiles of all sequences, counted from the
// lengths on the device, are dealt in equal contiguous runs to groups of
// warps of a grid that just fills the GPU, one warp of a group per KV head
// (neighbouring warps read neighbouring parts of the same pages), so a ragged
// batch costs what its rows cost.  A warp works alone: one lane copies its
// tiles into a ring of the warp's own, several ahead and across sequence
// boundaries, so no CTA barrier holds the stream up.  A run that covers a
// whole sequence writes its output; otherwise it leaves its state in the
// workspace and, after a barrier of the grid, the states are joined in run
// order (the result does not depend on timing).  TMA does the copies: loads alone
// (nothing computed) ran at 7.0 TB/s so, and at 5.2 TB/s with per-lane
// cp.async of the same rings (32 sequences of 16K to 32K rows).
//
// Measured (16 query heads on 8 KV heads of 128): 32 x 16K to 32K rows 470 us
// (6.8 TB/s); 64 x 2K to 4K rows E4M3 75.5 us (5.5 TB/s; loads alone 67, the
// barrier and the joins 4); 64 x 200 to 420 rows 20.6 us
// (4.0 TB/s; loads alone 15.7, the barrier 1.6, the joins 2); 795 rows 8.9 us
// (latencies: length, page ids, rows, barrier, join).
//
// Tile layout.  For the scores the rows are the M of a 16x8x16 warp MMA and
// the heads its N.  The order of the head elements along K is free as long as
// q uses the same, so a lane's 16-byte piece of a K row is its A fragment as
// it stands.  For the output, V^T is A (M = head elements, K = rows): the lane
// reads the same 16 bytes of four rows and one byte permute per register pairs
// two rows.  P goes from the score layout to the B fragment by a warp-wide 8x8
// transpose.  Rows of 128 bytes are swizzled by TMA (16-byte piece c of row r
// sits at c ^ (r mod 8)), and M index i of an octet of rows is row
// i ^ (i odd ? 4 : 0): with both, the K reads (two rows, four pieces) and the
// V reads (four rows, two pieces) of a quarter warp hit 32 different banks.
//
// Rounding.  P enters the second MMA as three bf16 planes, its 24 bits cut
// into 8 each: exact (one rounded plane would cost 2^-8, two 2^-17).  A
// tile's sums start from zero and are added to the running
// ones in fp32: the tensor core cuts, and a chain of thousands of tiles into
// one accumulator would drift (1.2e-5 of the output at 24K rows).  E4M3 codes
// are exact in f16 and stay codes: the K scale multiplies the score, the V
// scale multiplies p, whose planes are then f16 after a power-of-two factor F
// per head that keeps the largest p * scale near 2^14 (2^-23 relative, values
// below 2^-39 of the largest lost).  q is made f16 by a power of two per
// head: elements down to 2^-31 of the head's largest are exact (8 bits above
// f16's smallest step, 2^-24, with the largest in [2^14, 2^15)), smaller ones are
// off by at most 2^-39 of it.
//
// Waits.  Every wait for copies has a limit.  Whether it ran out is one decision
// of the warp, which then copies nothing more, lets what is in flight land (the
// limit once more) and marks its states, so that the joins leave those outputs.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_runtime.h>

#include "dec.h"
#include "dec_paged.h"
#include "dec_ptx.cuh"
#include "dec_tc.cuh"

namespace dec {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
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
  int2* desc;      // [B] (first worker, workers) whose states are joined
  int* status;
  unsigned long long timeout_ns;   // bound of a wait for copies
  int stall;       // warp of the grid that withholds its first copies (tests), or -1
};

// c += a b; with FIRST, c = a b.
template <bool F16, bool FIRST = false>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  const float z0 = FIRST ? 0.f : c[0], z1 = FIRST ? 0.f : c[1], z2 = FIRST ? 0.f : c[2],
              z3 = FIRST ? 0.f : c[3];
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
}
// The transpose of an 8x8 matrix of 16-bit values spread over the warp (lane
// l holds row l/4, columns 2(l%4) and the next).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Box at (element x, row y, page z) of a pool's tensor map.  x is 0 or 64
// elements of bf16 or 0 of E4M3: a multiple of 16 bytes.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                         uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
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
// Untiled bulk copy to a shared-memory address (bytes a multiple of 16, both
// addresses 16-byte aligned).
__device__ __forceinline__ void bulk_u32(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
// 2^e for a normal exponent.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Shape of the kernel for one head dimension and cache type.
template <int D, bool FP8>
struct Cfg {
  static constexpr int ES = FP8 ? 1 : 2;                   // bytes of an element
  // 16-row blocks of a tile (and of one softmax update), tiles of 8 KB: more
  // than one block spreads the update's fixed work and gives independent
  // chains, but 16 KB tiles would leave the ring too few slots
  static constexpr int NS = D * ES == 256 ? 1 : 2;
  static constexpr int TR = 16 * NS;                       // rows of a tile
  static constexpr int HB = TR * D * ES;                   // bytes of its K (or V) rows
  static constexpr int SB = FP8 ? 2 * TR * 4 : 0;          // bytes of its scales
  // CTAs of an SM.  E4M3 is bound by what its warps issue: 3 (64 sequences of
  // 2K to 4K rows: 95 us, 118 with 2).  bf16 heads of 128 want the registers of
  // 2 (32 sequences of 16K to 32K rows: 458 us, 496 with 3)
  static constexpr int CTAS = !FP8 && D == 128 ? 2 : 3;
  static constexpr int ROOM = (227 * 1024 / CTAS - 3 * 1024) / kWarps;   // a warp's share
  static constexpr int S = ROOM / (2 * HB + SB) < 8 ? ROOM / (2 * HB + SB) : 8;  // ring slots
  static constexpr int SMEM = 1024 + kWarps * S * (2 * HB + SB);
};

// A warp's place in the list of tiles: sequence, tile of it.
struct Place {
  int b, tile, tiles;     // tiles: of this sequence
  int lo, len;            // rows [lo, len)
};
template <int TR>
__device__ __forceinline__ int row0(const Place& p) {
  return (p.lo & ~(TR - 1)) + p.tile * TR;
}
template <int TR>
__device__ __forceinline__ int tiles_of(const PagedArgs& a, int n, int& lo) {
  lo = a.window > 0 && n > a.window ? n - a.window : 0;
  if (n < 1 || n > a.max_rows) return 0;
  return (n - (lo & ~(TR - 1)) + TR - 1) / TR;
}
template <int TR>
__device__ __forceinline__ void enter(const PagedArgs& a, Place& p) {
  p.tile = 0;
  p.tiles = 0;
  while (p.b < a.B) {
    p.len = a.rows[p.b];
    p.tiles = tiles_of<TR>(a, p.len, p.lo);
    if (p.tiles) return;
    ++p.b;
  }
}
template <int TR>
__device__ __forceinline__ void next(const PagedArgs& a, Place& p) {
  if (++p.tile < p.tiles) return;
  ++p.b;
  enter<TR>(a, p);
}

// Row of an octet that M index i stands for.
__device__ __forceinline__ int row_of(int i) { return i ^ ((i & 1) << 2); }

// This warp's run of tiles.  True if copies may still be on their way into the
// ring (a wait ran out, and so did the wait for the rest).
template <int D, bool FP8>
__device__ __forceinline__ bool run_tiles(const PagedArgs& a, const CUtensorMap& kmap,
                                          const CUtensorMap& vmap) {
  using C = Cfg<D, FP8>;
  constexpr int S = C::S, NS = C::NS, TR = C::TR, ES = C::ES, HB = C::HB, TB = 2 * HB;
  constexpr int RB = D * ES < 128 ? D * ES : 128;  // bytes of a row in a box
  constexpr int NB = D * ES / RB;               // boxes across a row
  constexpr int KP = D * ES / 64;               // 16-byte pieces of a K row per lane
  constexpr int MT = D / 16;                    // M tiles of V^T
  constexpr int VB = D * ES / 8 >= 16 ? 16 : 8; // bytes of a V piece
  constexpr int VP = D * ES / 8 / VB;           // pieces of a V row per lane
  constexpr int NO = TR / 8;                    // row octets of a tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_bar[kWarps][S];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int me = blockIdx.x * kWarps + warp;
  // neighbouring warps take the KV heads of the same rows
  const int workers = gridDim.x * kWarps / a.Hkv;
  const int worker = me / a.Hkv, g = me % a.Hkv;
  const uint32_t smem = (smem_u32(smem_raw) + 1023) & ~1023u;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&s_bar[warp][i], 1);
    fence_mbar_init();
  }

  // The runs: all tiles, then this warp's first one.  Every warp counts for
  // itself; the lengths of the first 128 sequences are loaded once.
  constexpr int R = 4;
  int known[R];
  long long total = 0;
  {
    int lo;
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int b = c * 32 + lane;
      known[c] = b < a.B ? tiles_of<TR>(a, a.rows[b], lo) : 0;
      total += known[c];
    }
    for (int b = R * 32 + lane; b < a.B; b += 32) total += tiles_of<TR>(a, a.rows[b], lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  const long long run = (total + workers - 1) / workers;
  const long long first = worker * run;
  if (worker >= workers || first >= total) return false;
  const int count = static_cast<int>(min(run, total - first));
  long long base = 0;   // tiles before the sequence that holds the first one
  Place ip;
  ip.b = -1;
  auto search = [&](int b0, int tiles) {   // among sequences b0 .. b0 + 31
    long long upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long before = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += before;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + upto > first);
    const int l = hit ? __ffs(hit) - 1 : 31;
    base += __shfl_sync(0xffffffffu, hit ? upto - tiles : upto, l);
    if (hit) ip.b = b0 + l;
  };
#pragma unroll
  for (int c = 0; c < R; ++c)
    if (ip.b < 0) search(c * 32, known[c]);
  for (int b0 = R * 32; ip.b < 0 && b0 < a.B; b0 += 32) {
    int lo;
    search(b0, b0 + lane < a.B ? tiles_of<TR>(a, a.rows[b0 + lane], lo) : 0);
  }
  enter<TR>(a, ip);
  ip.tile = static_cast<int>(first - base);
  Place cp = ip;

  // ---- issue side: tile i of the run into ring slot i % S
  const uint32_t ring = smem + warp * (S * TB);
  const uint32_t scales = smem + kWarps * (S * TB) + warp * (S * C::SB);
  const int P = 1 << a.pool.shift;
  const int BR = min(P, TR);   // rows of a box: a tile is 1 to 4 boxes, each in one page
  const uint64_t policy = policy_evict_first();
  int ids[NO];      // page ids of the next tile's boxes (-2: not needed)
  unsigned bad = 0; // bit s: the tile in slot s named a page out of range
  auto fetch_ids = [&]() {
    const int r0 = row0<TR>(ip);
    const int32_t* row = a.table + static_cast<long long>(ip.b) * a.width;
    if (BR == TR) {   // (the one box of a tile always holds rows)
      ids[0] = row[r0 >> a.pool.shift];
    } else {
#pragma unroll
      for (int o = 0; o < NO; ++o) {
        const int r = r0 + BR * o;
        ids[o] = (o * BR < TR && r + BR > ip.lo && r < ip.len) ? row[r >> a.pool.shift] : -2;
      }
    }
  };
  int issued = 0;
  auto issue = [&]() {
    if (issued >= count) return;
    const int slot = issued % S;
    auto outside = [&](int id) { return id < 0 || id >= a.pool.n_pages; };
    unsigned wrong = 0;
    int boxes = 1;
    if (BR == TR) {
      wrong = outside(ids[0]);
    } else {
      boxes = 0;
#pragma unroll
      for (int o = 0; o < NO; ++o)
        if (ids[o] != -2) {
          ++boxes;
          wrong |= outside(ids[o]);
        }
    }
    bad = (bad & ~(1u << slot)) | (wrong << slot);
    if (lane == 0 && (me != a.stall || issued > 0)) {
      uint64_t* bar = &s_bar[warp][slot];
      const uint32_t dst = ring + slot * TB, sdst = scales + slot * C::SB;
      constexpr int row_total = 2 * D * ES + (FP8 ? 8 : 0);   // bytes of a K and V row
      const int y = (g << a.pool.shift) + (row0<TR>(ip) & (P - 1));
      // boxes of one tile lie in different pages, at the same rows of them
      auto box = [&](int o, int page) {
        const uint32_t at = dst + o * BR * RB;
#pragma unroll
        for (int h = 0; h < NB; ++h) {
          load_box(at + h * (TR * RB), &kmap, h * 64, y, page, smem_u32(bar), policy);
          load_box(at + HB + h * (TR * RB), &vmap, h * 64, y, page, smem_u32(bar), policy);
        }
        if constexpr (FP8) {
          const long long e = page * (a.pool.page_stride / D) + y;
          bulk_u32(sdst + o * BR * 4, a.pool.ks + e, BR * 4, smem_u32(bar), policy);
          bulk_u32(sdst + (TR + o * BR) * 4, a.pool.vs + e, BR * 4, smem_u32(bar), policy);
        }
      };
      if (wrong) {
        mbar_arrive(bar);
      } else if (BR == TR) {
        mbar_arrive_expect_tx(bar, TR * row_total);
        box(0, ids[0]);
      } else {
        mbar_arrive_expect_tx(bar, boxes * BR * row_total);
#pragma unroll 1
        for (int o = 0; o * BR < TR; ++o) {
          int page = ids[0];
#pragma unroll
          for (int k = 1; k < NO; ++k) page = o == k ? ids[k] : page;
          if (page != -2) box(o, page);
        }
      }
    }
    if (++issued < count) {
      next<TR>(a, ip);
      fetch_ids();
    }
  };
  __syncwarp();
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
    const uint16_t* qh = a.q + cp.b * a.q_stride + (static_cast<long long>(g) * a.rep + g8) * D;
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

  // where a lane reads in a tile
  const int ra = row_of(g8), v0 = row_of(2 * t4), v1 = row_of(2 * t4 + 1);
  auto spot = [](int r, int piece) {   // byte of a 16-byte piece of row r
    return r * RB + ((RB == 128 ? piece ^ (r & 7) : piece ^ ((r >> 1) & 3)) << 4);
  };
  const int koff = spot(ra, t4);
  const int voff0 = VB == 16 ? spot(v0, g8) : spot(v0, g8 / 2) + (g8 & 1) * 8;
  const int voff1 = VB == 16 ? spot(v1, g8) : spot(v1, g8 / 2) + (g8 & 1) * 8;

  auto tile_step = [&](uint32_t src, uint32_t ssrc) {
    const int r0 = row0<TR>(cp);
    // a tile at an end of the sequence holds rows that are not part of it
    // (anything may stand there): their p is 0 and their V is made 0
    // (once for all blocks of a tile: branches among the blocks keep their
    // instructions apart, 79 against 75.5 us for 64 x 2K to 4K rows E4M3)
    const bool edge = r0 < cp.lo || r0 + TR > cp.len;
    auto in = [&](int r) { return r0 + r >= cp.lo && r0 + r < cp.len; };
    // scores of block n: rows 16 n + ra (x 0, 1) and 8 further (x 2, 3), heads
    // 2 t4 (x 0, 2) and 2 t4 + 1 (x 1, 3)
    float x[NS][4], vs[NS][2];
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      float s[2][4];
#pragma unroll
      for (int c = 0; c < KP; ++c) {
        // piece 4 c + t4 of the row
        const uint32_t at = src + n * 16 * RB +
                            (RB == 128 ? (c / 2) * (TR * RB) + (koff ^ ((c & 1) << 6)) : koff);
        const uint4 u = lds128(at), w = lds128(at + 8 * RB);
        const uint32_t xa[4] = {u.x, u.y, u.z, u.w}, ya[4] = {w.x, w.y, w.z, w.w};
        if constexpr (FP8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t k0 = e4m3x2_to_h2(xa[j]), k1 = e4m3x2_to_h2(ya[j]);
            const uint32_t k2 = e4m3x2_to_h2(xa[j] >> 16), k3 = e4m3x2_to_h2(ya[j] >> 16);
            if (c == 0 && j < 2)
              mma<true, true>(s[j], k0, k1, k2, k3, qb[2 * j], qb[2 * j + 1]);
            else
              mma<true>(s[j & 1], k0, k1, k2, k3, qb[c * 8 + 2 * j], qb[c * 8 + 2 * j + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (c == 0)
              mma<false, true>(s[j], xa[2 * j], ya[2 * j], xa[2 * j + 1], ya[2 * j + 1], qb[2 * j],
                               qb[2 * j + 1]);
            else
              mma<false>(s[j], xa[2 * j], ya[2 * j], xa[2 * j + 1], ya[2 * j + 1],
                         qb[c * 4 + 2 * j], qb[c * 4 + 2 * j + 1]);
          }
        }
      }
      float ks0 = 1.f, ks1 = 1.f;
      if constexpr (FP8) {
        const uint32_t at = ssrc + (16 * n + ra) * 4;
        ks0 = lds32(at);
        ks1 = lds32(at + 32);
        vs[n][0] = lds32(at + TR * 4);
        vs[n][1] = lds32(at + TR * 4 + 32);
      }
      x[n][0] = (s[0][0] + s[1][0]) * (sc0 * ks0);
      x[n][1] = (s[0][1] + s[1][1]) * (sc1 * ks0);
      x[n][2] = (s[0][2] + s[1][2]) * (sc0 * ks1);
      x[n][3] = (s[0][3] + s[1][3]) * (sc1 * ks1);
    }
    if (edge) {
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        if (!in(16 * n + ra)) {
          x[n][0] = x[n][1] = -INFINITY;
          vs[n][0] = 0.f;
        }
        if (!in(16 * n + ra + 8)) {
          x[n][2] = x[n][3] = -INFINITY;
          vs[n][1] = 0.f;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      t0 = fmaxf(t0, fmaxf(x[n][0], x[n][2]));
      t1 = fmaxf(t1, fmaxf(x[n][1], x[n][3]));
    }
    const bool up = __any_sync(0xffffffffu, t0 > m0 || t1 > m1);
    float e0 = 1.f, e1 = 1.f;   // what the sums so far are multiplied by
    if (up) {
      const float n0 = fmaxf(m0, over_rows(t0)), n1 = fmaxf(m1, over_rows(t1));
      // (no score above -inf yet: nothing to rescale)
      e0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0);
      e1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
      m0 = n0;
      m1 = n1;
      w0 *= e0;
      w1 *= e1;
    }
    // (a maximum of -inf: every score so far is -inf, and p = 2^-inf = 0)
    const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
    float p0 = 0.f, p1 = 0.f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      x[n][0] = ex2(x[n][0] - b0);
      x[n][1] = ex2(x[n][1] - b1);
      x[n][2] = ex2(x[n][2] - b0);
      x[n][3] = ex2(x[n][3] - b1);
      p0 += x[n][0] + x[n][2];
      p1 += x[n][1] + x[n][3];
    }
    l0 = fmaf(l0, e0, p0);
    l1 = fmaf(l1, e1, p1);
    // P^T as B fragments: planes of rows 0-7 and 8-15 of each block
    constexpr int NP = FP8 ? 2 : 3;
    uint32_t pb[NS][NP][2];
    if constexpr (FP8) {
      float u0 = 0.f, u1 = 0.f;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        x[n][0] *= vs[n][0];
        x[n][1] *= vs[n][0];
        x[n][2] *= vs[n][1];
        x[n][3] *= vs[n][1];
        u0 = fmaxf(u0, fmaxf(x[n][0], x[n][2]));
        u1 = fmaxf(u1, fmaxf(x[n][1], x[n][3]));
      }
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
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float y0 = x[n][2 * o] * F0, y1 = x[n][2 * o + 1] * F1;
          const uint32_t hi = f2_to_h2(y0, y1);
          const float2 h = h2_to_f2(hi);
          pb[n][0][o] = transpose8(hi);
          pb[n][1][o] = transpose8(f2_to_h2(y0 - h.x, y1 - h.y));
        }
    } else {
      // every plane is cut from what the ones before left, and positive where
      // p is (the floor is below any sum), so an infinite V element stays one
      auto rest = [](float v, float floor) {
        return fmaxf(v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), floor);
      };
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          float y0 = x[n][2 * o], y1 = x[n][2 * o + 1];
          const float f0 = fminf(y0, 0x1p-126f), f1 = fminf(y1, 0x1p-126f);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            pb[n][k][o] = transpose8(__byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x7632));
            y0 = rest(y0, f0);
            y1 = rest(y1, f1);
          }
        }
    }
    // V^T: the sums of a tile start from zero
    const uint32_t vsrc = src + HB;
    auto join = [&](float (&sum)[4], const float (&s)[4]) {
      sum[0] = fmaf(sum[0], e0, s[0]);
      sum[1] = fmaf(sum[1], e1, s[1]);
      sum[2] = fmaf(sum[2], e0, s[2]);
      sum[3] = fmaf(sum[3], e1, s[3]);
    };
#pragma unroll
    for (int c = 0; c < VP; ++c) {
      constexpr int W = VB / 4;
      uint32_t v[NS][4][W];   // rows v0, v1, v0 + 8, v1 + 8 of each block
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t at = vsrc + c * (TR * RB) + (16 * n + (e / 2) * 8) * RB + (e & 1 ? voff1 : voff0);
          if constexpr (VB == 16) {
            const uint4 u = lds128(at);
            v[n][e][0] = u.x;
            v[n][e][1] = u.y;
            v[n][e][W - 2] = u.z;
            v[n][e][W - 1] = u.w;
          } else {
            const uint2 u = lds64(at);
            v[n][e][0] = u.x;
            v[n][e][1] = u.y;
          }
        }
      if (edge) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!in(16 * n + (e / 2) * 8 + (e & 1 ? v1 : v0))) {
#pragma unroll
              for (int i = 0; i < W; ++i) v[n][e][i] = 0;
            }
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (!FP8) {
          // M tile: rows g8 = element 8 g8 + 2 i of this piece, rows g8 + 8 =
          // the next element
          float s[4];
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            const uint32_t a0 = __byte_perm(v[n][0][i], v[n][1][i], 0x5410);
            const uint32_t a1 = __byte_perm(v[n][0][i], v[n][1][i], 0x7632);
            const uint32_t a2 = __byte_perm(v[n][2][i], v[n][3][i], 0x5410);
            const uint32_t a3 = __byte_perm(v[n][2][i], v[n][3][i], 0x7632);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
              if (n == 0 && k == 0)
                mma<false, true>(s, a0, a1, a2, a3, pb[n][k][0], pb[n][k][1]);
              else
                mma<false>(s, a0, a1, a2, a3, pb[n][k][0], pb[n][k][1]);
            }
          }
          join(acc[c * 4 + i], s);
        } else {
          // codes of two rows side by side: (r0 d0, r1 d0, r0 d1, r1 d1), ...
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float s[4];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
              const uint32_t p = __byte_perm(v[n][0][i], v[n][1][i], j ? 0x7362 : 0x5140);
              const uint32_t q = __byte_perm(v[n][2][i], v[n][3][i], j ? 0x7362 : 0x5140);
              const uint32_t a0 = e4m3x2_to_h2(p), a1 = e4m3x2_to_h2(p >> 16);
              const uint32_t a2 = e4m3x2_to_h2(q), a3 = e4m3x2_to_h2(q >> 16);
#pragma unroll
              for (int k = 0; k < NP; ++k) {
                if (n == 0 && k == 0)
                  mma<true, true>(s, a0, a1, a2, a3, pb[n][k][0], pb[n][k][1]);
                else
                  mma<true>(s, a0, a1, a2, a3, pb[n][k][0], pb[n][k][1]);
              }
            }
            join(acc[2 * i + j], s);
          }
        }
      }
    }
  };

  // The run's part of sequence cp.b ends with the current tile.
  auto finish = [&]() {
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    const bool whole = begin == 0 && cp.tile + 1 == cp.tiles;
    const int h0 = 2 * t4, h1 = h0 + 1;
    if (begin == 0 && g == 0 && lane == 0) {
      // (the workers that share this sequence follow in order)
      const long long rest = cp.tiles - (cp.tile + 1);
      a.desc[cp.b] = make_int2(worker, whole ? 0 : 1 + static_cast<int>((rest + run - 1) / run));
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
      o0 = a.out + (static_cast<long long>(cp.b) * a.Hq + static_cast<long long>(g) * a.rep + h0) * D;
      o1 = o0 + D;
      z0 = 1.f / l0;
      z1 = 1.f / l1;
      if (g8 == 0 && a.lse) {
        float* ls = a.lse + static_cast<long long>(cp.b) * a.Hq + static_cast<long long>(g) * a.rep;
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

  // Whether the copies of tile i have landed within the limit.  One answer for
  // the warp: lanes that part ways here would miss each other's shuffles.
  auto landed = [&](int i, Spin1& sp) {
    bool ok = false;
    while (!(ok = mbar_wait(&s_bar[warp][i % S], (i / S) & 1, kWaitHintNs)) && !sp.expired()) {
    }
    return __all_sync(0xffffffffu, ok) != 0;
  };
  start();
  // A wait ran out: nothing of this run is written from here on, and nothing
  // more is copied.  Copies in flight get the limit once more to land.
  bool late = false, stuck = false;
  for (int i = 0; i < count; ++i) {
    const int slot = i % S;
    if (!late) {
      issue();
      Spin1 sp;
      sp.limit_ns = a.timeout_ns;
      late = !landed(i, sp);
      if (late) {
        Spin1 rest;
        rest.limit_ns = a.timeout_ns;
        for (int j = i; j < issued; ++j) stuck |= !landed(j, rest);
      }
    }
    if (late || ((bad >> slot) & 1)) {
      poison = true;
      if (a.status && lane == 0) atomicOr(a.status, late ? DEC_DEV_TIMEOUT : DEC_DEV_BAD_PAGE);
    }
    if (!poison) tile_step(ring + slot * TB, scales + slot * C::SB);
    __syncwarp();   // the slot may be refilled
    const bool last = cp.tile + 1 == cp.tiles;
    if (last || i + 1 == count) finish();
    if (i + 1 < count) {
      next<TR>(a, cp);
      if (last) start();
    }
  }
  return stuck;
}

// Joins the states of one (sequence, query head); also the outputs of empty
// sequences.  A warp takes up to 32 states (a lane each for the weights);
// sequences that more workers share are joined by their CTA.  The weights and
// the first sums load together (64 x 200 to 420 rows 21.3 -> 20.6 us).
struct Item {
  int2 d;          // first worker, workers (0: nothing to join)
  int g, hh;       // KV head, query head of its group
  float *out, *lse;
};
template <int D>
__device__ __forceinline__ Item item_at(const PagedArgs& a, int item, bool first_lane) {
  const int b = item / a.Hq, h = item % a.Hq;
  Item it{make_int2(0, 0), h / a.rep, h % a.rep, a.out + static_cast<long long>(item) * D,
          a.lse ? a.lse + item : nullptr};
  const int2 d = __ldcg(&a.desc[b]);   // (of no use for an empty sequence)
  const int n = a.rows[b];
  if (n < 0 || n > a.max_rows) {
    if (first_lane && h == 0 && a.status) atomicOr(a.status, DEC_DEV_BAD_POSITION);
  } else if (n == 0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) it.out[e * 32 + lane] = 0.f;
    if (first_lane && it.lse) *it.lse = -INFINITY;
  } else {
    it.d = d;
  }
  return it;
}
// State i: the first is its warp's last, the others their warps' first.
__device__ __forceinline__ const float* state_of(const PagedArgs& a, const Item& it, int D, int i) {
  const int words = a.rep * (D + 2);
  return a.part + (static_cast<long long>(it.d.x + i) * a.Hkv + it.g) * (2 * words) + (i == 0 ? words : 0);
}
// The sums of states first, first + step, ... of this lane's elements, loaded
// beside the weights instead of after them.
constexpr int kPre = 8;
template <int D>
__device__ __forceinline__ void preload(const PagedArgs& a, const Item& it, int first, int step,
                                        float (&v)[kPre][D / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < kPre; ++k) {
    const int i = first + k * step;
    if (i < it.d.y) {
      const float* p = state_of(a, it, D, i) + it.hh * D + lane;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) v[k][e] = __ldcg(p + 32 * e);
    }
  }
}
template <int D>
__device__ __forceinline__ void join_by_warp(const PagedArgs& a, const Item& it) {
  const int lane = threadIdx.x & 31, n = it.d.y;
  float v[kPre][D / 32];
  preload<D>(a, it, 0, 1, v);
  float m = -INFINITY, l = 0.f;
  if (lane < n) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(state_of(a, it, D, lane) + a.rep * D) + it.hh);
    m = ml.x;
    l = ml.y;
  }
  if (__any_sync(0xffffffffu, m != m)) return;   // poisoned
  const float M = warp_max(m);
  const float w = m == -INFINITY ? 0.f : ex2(m - M);
  l = warp_sum(l * w);
  float acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll
  for (int i = 0; i < kPre; ++i) {
    const float wi = __shfl_sync(0xffffffffu, w, i);   // (0 behind the last state)
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = i < n ? fmaf(v[i][e], wi, acc[e]) : acc[e];
  }
#pragma unroll 4
  for (int i = kPre; i < n; ++i) {
    const float* p = state_of(a, it, D, i) + it.hh * D + lane;
    const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(__ldcg(p + 32 * e), wi, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) it.out[e * 32 + lane] = acc[e] / l;
  if (lane == 0 && it.lse) *it.lse = (M + log2f(l)) * 0.6931471805599453f;
}
// s_w: two floats per worker; every thread of the CTA.
template <int D>
__device__ __forceinline__ void join_by_cta(const PagedArgs& a, const Item& it, float* s_w) {
  __shared__ float s_acc[kWarps][D];
  __shared__ float s_red[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = it.d.y;
  float v[kPre][D / 32];
  preload<D>(a, it, warp, kWarps, v);
  float m = -INFINITY;
  bool poison = false;
  float2* s_ml = reinterpret_cast<float2*>(s_w);
  for (int i = tid; i < n; i += kThreads) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(state_of(a, it, D, i) + a.rep * D) + it.hh);
    s_ml[i] = ml;
    poison |= ml.x != ml.x;
    m = fmaxf(m, ml.x);
  }
  m = warp_max(m);
  if (lane == 0) s_red[warp] = m;
  if (__syncthreads_or(poison)) return;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_red[w]);
  float l = 0.f;
  for (int i = tid; i < n; i += kThreads) {   // (the weight takes the place of m)
    const float2 ml = s_ml[i];
    const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
    l += ml.y * w;
    s_ml[i].x = w;
  }
  l = warp_sum(l);
  __syncthreads();   // s_red has been read, s_w is complete
  if (lane == 0) s_red[warp] = l;
  float acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll
  for (int k = 0; k < kPre; ++k) {
    const int i = warp + k * kWarps;
    if (i < n) {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(v[k][e], s_ml[i].x, acc[e]);
    }
  }
#pragma unroll 4
  for (int i = warp + kPre * kWarps; i < n; i += kWarps) {
    const float* p = state_of(a, it, D, i) + it.hh * D + lane;
    const float w = s_ml[i].x;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(__ldcg(p + 32 * e), w, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) s_acc[warp][e * 32 + lane] = acc[e];
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) l += s_red[w];
  for (int e = tid; e < D; e += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += s_acc[w][e];
    it.out[e] = x / l;
  }
  if (tid == 0 && it.lse) *it.lse = (m + log2f(l)) * 0.6931471805599453f;
  __syncthreads();   // before the shared arrays are used again
}

// One cooperative launch: all runs, a barrier of the grid, the joins.  (As two
// launches, the second one dependent, the host's part of a call was 9.1 us
// against 4.6, and the GPU's the same.)
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, Cfg<D, FP8>::CTAS) paged_kernel(
    const PagedArgs a, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Item s_many[kWarps];
  __shared__ int s_n;
  if (threadIdx.x == 0) s_n = 0;
  // (copies that may still land would overwrite the weights of join_by_cta)
  const bool stuck = __syncthreads_or(run_tiles<D, FP8>(a, kmap, vmap)) != 0;
  cooperative_groups::this_grid().sync();
  const int lane = threadIdx.x & 31;
  const long long items = static_cast<long long>(a.B) * a.Hq;
  const int hop = gridDim.x * kWarps;
  for (long long base = 0; base < items; base += hop) {
    // neighbouring items on different SMs
    const long long item = base + (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    if (item < items) {
      const Item it = item_at<D>(a, static_cast<int>(item), lane == 0);
      if (it.d.y > 32) {
        if (lane == 0) s_many[atomicAdd(&s_n, 1)] = it;
      } else if (it.d.y > 0) {
        join_by_warp<D>(a, it);
      }
    }
    __syncthreads();
    const int n = s_n;
    for (int i = 0; i < n && !stuck; ++i) join_by_cta<D>(a, s_many[i], reinterpret_cast<float*>(smem_raw));
    if (n) {   // (join_by_cta may end early for a poisoned sequence)
      __syncthreads();
      if (threadIdx.x == 0) s_n = 0;
    }
    __syncthreads();
  }
}

template <int D, bool FP8>
cudaError_t launch_paged(const PagedArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int grid,
                         cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = Cfg<D, FP8>::SMEM;
  cudaError_t e = allow_smem(paged_kernel<D, FP8>, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_kernel<D, FP8>, a, km, vm);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiledFn>(f);
}

std::atomic<unsigned long long> g_timeout_ns{2000000000ull};
std::atomic<int> g_stall{-1};

int tile_rows(const dec_pages* p) {
  if (p->dtype == DEC_KV_FP8_E4M3) return p->head_dim == 128 ? Cfg<128, true>::TR : Cfg<64, true>::TR;
  return p->head_dim == 128 ? Cfg<128, false>::TR : Cfg<64, false>::TR;
}

// Rows of the K (or V) pages of one layer: [page][head and row][element], a
// box = 128 bytes (64 of an E4M3 row of 64) of the rows of a tile in a page.
bool encode_pool(EncodeTiledFn enc, CUtensorMap* m, const void* base, const dec_pages* p) {
  const int tile = tile_rows(p);
  const bool fp8 = p->dtype == DEC_KV_FP8_E4M3;
  const cuuint64_t es = fp8 ? 1 : 2, D = p->head_dim;
  const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(p->n_kv_heads) * p->page_rows,
                              static_cast<cuuint64_t>(p->n_pages)};
  const cuuint64_t strides[2] = {D * es, static_cast<cuuint64_t>(p->page_stride) * es};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(D * es < 128 ? D : 128 / es),
                             static_cast<cuuint32_t>(p->page_rows < tile ? p->page_rows : tile), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D * es < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of the grid: one wave.
int paged_grid(const dec_pages* p, int sms) {
  if (p->dtype == DEC_KV_FP8_E4M3)
    return sms * (p->head_dim == 128 ? Cfg<128, true>::CTAS : Cfg<64, true>::CTAS);
  return sms * (p->head_dim == 128 ? Cfg<128, false>::CTAS : Cfg<64, false>::CTAS);
}

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
  return state_bytes(paged_grid(pool, sms > 0 ? sms : 148), n_q_heads / pool->n_kv_heads,
                     pool->head_dim) +
         round256(sizeof(int2) * static_cast<size_t>(batch));
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
  if (!is_aligned(q, 16) || (batch > 1 && q_stride % 8) || !is_aligned(workspace, 256) ||
      !is_aligned(out, 8) || !is_aligned(lse, 4) || !is_aligned(rows, 4) || !is_aligned(status, 4))
    return DEC_ERR_ALIGN;
  if (workspace_bytes < dec_paged_attention_workspace_bytes(pool, batch, n_q_heads))
    return DEC_ERR_KV_SIZE;
  const int sms = device_sms();
  if (sms < 0) return sms;
  if (paged_grid(pool, sms) * kWarps < pool->n_kv_heads) return DEC_ERR_DEVICE;   // (a warp per head)
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
  const int grid = paged_grid(pool, sms);
  a.part = static_cast<float*>(workspace);
  a.desc = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + state_bytes(grid, a.rep, D));
  a.status = status;
  a.timeout_ns = g_timeout_ns.load(std::memory_order_relaxed);
  a.stall = g_stall.load(std::memory_order_relaxed);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const EncodeTiledFn enc = encode_tiled();
  CUtensorMap km, vm;
  if (!enc || !encode_pool(enc, &km, a.pool.k, pool) || !encode_pool(enc, &vm, a.pool.v, pool))
    return cuda_failed(cudaErrorInvalidValue);
  if (pool->dtype == DEC_KV_FP8_E4M3)
    e = D == 128 ? launch_paged<128, true>(a, km, vm, grid, s)
                 : launch_paged<64, true>(a, km, vm, grid, s);
  else
    e = D == 128 ? launch_paged<128, false>(a, km, vm, grid, s)
                 : launch_paged<64, false>(a, km, vm, grid, s);
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}

extern "C" int dec_paged_attention_set_timeout_ns(unsigned long long ns) {
  if (ns < 1000000ull) return DEC_ERR_ARG;
  g_timeout_ns.store(ns, std::memory_order_relaxed);
  return DEC_OK;
}

extern "C" int dec_paged_attention_set_debug_stall(int warp_plus_one) {
  if (warp_plus_one < 0) return DEC_ERR_ARG;
  g_stall.store(warp_plus_one - 1, std::memory_order_relaxed);
  return DEC_OK;
}
