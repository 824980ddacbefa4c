// dec_pages.cu -- the pages of a paged KV cache: reserving, cropping and
// freeing them, copies on write, forks, compaction.
//
// A page is free when its count is 0: there is no list of free pages to keep,
// so forks and releases are count updates only, and which pages a call takes
// (the lowest free ones) depends on nothing but the counts.  The bookkeeping
// (tables and counts: a few hundred KB at most) runs in one CTA and is bound
// by latency; the data moves in a second, dependent launch over the whole GPU
// (a list of (from, to, rows) that the first one leaves in the workspace),
// bound by HBM: a copy on write moves the filled rows of its page, a compaction
// whole pages.  Measured: 256 of 1024 pages of 1.8 MB move in 158 us = 5.9 TB/s;
// a row more for each of 64 sequences 3.5 us, of 512 4.7 us (18 us with a warp
// for every sequence).
#include <cuda_runtime.h>

#include "dec.h"
#include "dec_paged.h"
#include "dec_ptx.cuh"
#include "dec_tc.cuh"

namespace dec {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSeqs = 4096;
constexpr int kScan = 8;       // pages a thread looks at per step of a scan

struct MapArgs {
  int32_t* table;
  int32_t* rows;
  int32_t* refs;
  int S, width, n_pages, shift;
  const int32_t* in;           // new_rows or parents
  int32_t* list;               // [n_pages] page ids
  int32_t* list2;              // [n_pages]
  int32_t* remap;              // [n_pages]
  int4* jobs;                  // (from, to, rows)
  int* n_jobs;
  int32_t* n_live;
  int* status;
};

// Exclusive prefix sum over the CTA (every thread); *total of all.
__device__ __forceinline__ int block_scan(int x, int* total, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();   // s_warp of the previous scan has been read
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += up;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp) - __shfl_sync(0xffffffffu, inc, 31);
  return before + inc - x;
}

// A thread looks after a sequence (kSeqs of them); pages to be released and
// long runs of new ones are walked by warps, from lists.
__global__ void __launch_bounds__(kThreads, 1) resize_kernel(const MapArgs a) {
  constexpr int kSeqs = kMaxSeqs / kThreads;
  constexpr int kFew = 4;            // new pages that a thread enters by itself
  __shared__ int s_warp[kWarps];
  __shared__ int s_last[kMaxSeqs];   // page that sequence s will write into, or -1
  __shared__ int s_pref[kMaxSeqs];   // its first entry in the list of new pages
  __shared__ uint16_t s_list[kMaxSeqs];   // shrinking sequences, and from its end those of long runs
  __shared__ int s_shrinks, s_longs, s_jobs, s_err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << a.shift;
  const int max_rows = a.width * P;
  pdl_trigger();
  int old[kSeqs], rows[kSeqs];   // rows now, and wanted (the same: nothing to do)
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const int s = tid + i * kThreads;
    old[i] = s < a.S ? a.rows[s] : 0;
    rows[i] = s < a.S ? a.in[s] : 0;
    if (rows[i] < 0) rows[i] = old[i];
  }
  if (tid == 0) {
    s_shrinks = s_longs = s_jobs = s_err = 0;
    *a.n_jobs = 0;
  }
  __syncthreads();
  auto pages = [&](int n) { return (n + P - 1) >> a.shift; };
  auto row_of = [&](int s) { return a.table + static_cast<long long>(s) * a.width; };
  // check everything before anything is changed
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const int s = tid + i * kThreads;
    if (s >= a.S) break;
    int last = -1;
    if (old[i] < 0 || old[i] > max_rows || rows[i] > max_rows) {
      atomicOr(&s_err, DEC_DEV_BAD_POSITION);
    } else {
      if (rows[i] > old[i] && (old[i] & (P - 1))) {
        last = row_of(s)[old[i] >> a.shift];
        if (last < 0 || last >= a.n_pages) atomicOr(&s_err, DEC_DEV_BAD_PAGE);
      }
      if (pages(rows[i]) < pages(old[i])) s_list[atomicAdd(&s_shrinks, 1)] = static_cast<uint16_t>(s);
    }
    s_last[s] = last;
  }
  __syncthreads();
  const int shrinks = s_shrinks;
  // pages behind the last row of every shrinking sequence
  auto each_freed = [&](auto visit) {
    for (int i = warp; i < shrinks; i += kWarps) {
      const int s = s_list[i], now = a.rows[s], n = a.in[s];
      const int32_t* row = row_of(s);
      for (int j = pages(n) + lane; j < pages(now); j += 32) visit(row[j]);
    }
  };
  if (shrinks) {
    each_freed([&](int page) {
      if (page < 0 || page >= a.n_pages) atomicOr(&s_err, DEC_DEV_BAD_PAGE);
    });
    __syncthreads();
  }
  if (s_err) {
    if (tid == 0 && a.status) atomicOr(a.status, s_err);
    return;
  }
  if (shrinks) {
    each_freed([&](int page) { atomicAdd(&a.refs[page], -1); });
    __syncthreads();
  }
  // copies on write, and how many new pages every sequence takes
  int need = 0;
  unsigned copies = 0;   // bit i: sequence tid + i kThreads copies its last page
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    if (i * kThreads >= a.S) break;
    const int s = tid + i * kThreads;
    int c = 0;
    if (s < a.S && rows[i] > old[i]) {
      const int x = s_last[s];
      if (x >= 0) {
        const int held = __ldcg(&a.refs[x]);
        int rank = 0;
        if (held > 1)
          for (int j = 0; j < s; ++j) rank += s_last[j] == x;
        if (rank < held - 1) copies |= 1u << i;   // (the last holder keeps the page)
      }
      c = ((copies >> i) & 1) + pages(rows[i]) - pages(old[i]);
    }
    int total;
    const int pre = block_scan(c, &total, s_warp);
    if (s < a.S) s_pref[s] = need + pre;
    need += total;
  }
  // the lowest free pages
  int found = 0;
  for (int p0 = 0; p0 < a.n_pages && found < need; p0 += kThreads * kScan) {
    unsigned free = 0;
    const int p = p0 + tid * kScan;
#pragma unroll
    for (int i = 0; i < kScan; ++i)
      if (p + i < a.n_pages && __ldcg(&a.refs[p + i]) == 0) free |= 1u << i;
    int total;
    int r = found + block_scan(__popc(free), &total, s_warp);
    for (int i = 0; i < kScan && r < need; ++i)
      if ((free >> i) & 1) a.list[r++] = p + i;
    found += total;
  }
  __syncthreads();
  if (found < need) {
    each_freed([&](int page) { atomicAdd(&a.refs[page], 1); });
    if (tid == 0 && a.status) atomicOr(a.status, DEC_DEV_NO_PAGES);
    return;
  }
  auto enter = [&](int32_t* row, int j, int at) {   // entry `at` of the list
    const int y = __ldcg(&a.list[at]);
    row[j] = y;
    a.refs[y] = 1;
    return y;
  };
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const int s = tid + i * kThreads;
    if (s >= a.S) break;
    if (rows[i] <= old[i]) continue;
    int32_t* row = row_of(s);
    int at = s_pref[s];
    if ((copies >> i) & 1) {
      const int x = s_last[s];
      const int y = enter(row, old[i] >> a.shift, at++);
      atomicSub(&a.refs[x], 1);
      a.jobs[atomicAdd(&s_jobs, 1)] = make_int4(x, y, old[i] & (P - 1), 0);
    }
    const int have = pages(old[i]), more = pages(rows[i]) - have;
    if (more > kFew) {
      s_pref[s] = at;
      s_list[kMaxSeqs - 1 - atomicAdd(&s_longs, 1)] = static_cast<uint16_t>(s);
    } else {
      for (int j = 0; j < more; ++j) enter(row, have + j, at + j);
    }
  }
  __syncthreads();
  for (int i = warp; i < s_longs; i += kWarps) {
    const int s = s_list[kMaxSeqs - 1 - i], now = a.rows[s], n = a.in[s];
    const int have = pages(now), more = pages(n) - have;
    for (int j = lane; j < more; j += 32) enter(row_of(s), have + j, s_pref[s] + j);
  }
  for (int i = warp; i < shrinks; i += kWarps) {
    const int s = s_list[i], now = a.rows[s], n = a.in[s];
    for (int j = pages(n) + lane; j < pages(now); j += 32) row_of(s)[j] = -1;
  }
  __syncthreads();   // (every warp has read the rows)
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const int s = tid + i * kThreads;
    if (s < a.S && rows[i] != old[i]) a.rows[s] = rows[i];
  }
  if (tid == 0) *a.n_jobs = s_jobs;
}

__global__ void __launch_bounds__(kThreads) compact_kernel(const MapArgs a) {
  __shared__ int s_warp[kWarps];
  const int tid = threadIdx.x;
  pdl_trigger();
  int mine = 0;
  for (int p = tid; p < a.n_pages; p += kThreads) mine += a.refs[p] > 0;
  int live;
  block_scan(mine, &live, s_warp);
  // the i-th live page from `live` on goes to the i-th free page below it
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < a.n_pages; p0 += kThreads * kScan) {
    unsigned hole = 0, move = 0;
    const int p = p0 + tid * kScan;
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      if (p + i >= a.n_pages) break;
      const bool held = a.refs[p + i] > 0;
      if (!held && p + i < live) hole |= 1u << i;
      if (held && p + i >= live) move |= 1u << i;
      a.remap[p + i] = p + i;
    }
    int th, tm;
    int h = holes + block_scan(__popc(hole), &th, s_warp);
    int m = movers + block_scan(__popc(move), &tm, s_warp);
    for (int i = 0; i < kScan; ++i) {
      if ((hole >> i) & 1) a.list[h++] = p + i;
      if ((move >> i) & 1) a.list2[m++] = p + i;
    }
    holes += th;
    movers += tm;
  }
  __syncthreads();
  for (int i = tid; i < movers; i += kThreads) {
    const int from = __ldcg(&a.list2[i]), to = __ldcg(&a.list[i]);
    a.remap[from] = to;
    a.refs[to] = a.refs[from];
    a.refs[from] = 0;
    a.jobs[i] = make_int4(from, to, 1 << a.shift, 0);
  }
  if (tid == 0) {
    *a.n_jobs = movers;
    *a.n_live = live;
  }
}

// A slice of table columns for all sequences (so that it can change in
// place); the last CTA takes the row counts.
constexpr int kForkThreads = 256;
constexpr int kForkCells = 7168;

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const MapArgs a, int cols) {
  __shared__ int s_cell[kForkCells];
  __shared__ int s_par[kMaxSeqs];
  const int tid = threadIdx.x;
  int bad = 0;
  for (int s = tid; s < a.S; s += kForkThreads) {
    const int p = a.in[s];
    s_par[s] = p;
    bad |= p >= a.S;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0 && blockIdx.x == 0 && a.status) atomicOr(a.status, DEC_DEV_BAD_PAGE);
    return;
  }
  if (blockIdx.x == gridDim.x - 1) {
    for (int s = tid; s < a.S; s += kForkThreads) s_cell[s] = a.rows[s];
    __syncthreads();
    for (int s = tid; s < a.S; s += kForkThreads) a.rows[s] = s_par[s] < 0 ? 0 : s_cell[s_par[s]];
    return;
  }
  const int c0 = blockIdx.x * cols, n = min(cols, a.width - c0);
  for (int i = tid; i < a.S * n; i += kForkThreads) {
    int e = a.table[static_cast<long long>(i / n) * a.width + c0 + i % n];
    if (e < -1 || e >= a.n_pages) {
      bad = 1;
      e = -1;
    }
    s_cell[i] = e;
  }
  if (__syncthreads_or(bad) && tid == 0 && a.status) atomicOr(a.status, DEC_DEV_BAD_PAGE);
  for (int i = tid; i < a.S * n; i += kForkThreads) {
    const int s = i / n, p = s_par[s];
    const int was = s_cell[i], now = p < 0 ? -1 : s_cell[p * n + i % n];
    a.table[static_cast<long long>(s) * a.width + c0 + i % n] = now;
    if (was == now) continue;
    if (now >= 0) atomicAdd(&a.refs[now], 1);
    if (was >= 0) atomicSub(&a.refs[was], 1);
  }
}

struct CopyArgs {
  uint8_t *k, *v;
  float *ks, *vs;
  long long layer_stride, page_stride;
  int L, H, D, es, shift;
  const int4* jobs;
  const int* n_jobs;
  int32_t* table;          // compaction: entries to renumber, or null
  const int32_t* remap;
  long long cells;
  int n_pages;
  int* status;
};

// A warp copies the rows of one head of one page: 8 loads of 512 bytes in
// flight (a page of 16 bf16 rows of 128 is 4 KB).  Many small CTAs that the
// GPU schedules as they finish: 256 pages of 1.8 MB at 5.9 TB/s with 16 to an
// SM, 5.7 with 4, 5.2 by bulk copies through a shared-memory ring.
__global__ void __launch_bounds__(256) copy_kernel(const CopyArgs a) {
  pdl_wait();
  const long long nthreads = static_cast<long long>(gridDim.x) * blockDim.x;
  if (a.table) {
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.cells;
         i += nthreads) {
      const int e = a.table[i];
      if (e >= 0 && e < a.n_pages)
        a.table[i] = a.remap[e];
      else if (e != -1 && a.status)
        atomicOr(a.status, DEC_DEV_BAD_PAGE);
    }
  }
  const int lane = threadIdx.x & 31;
  const int per = a.L * 2 * a.H;
  const long long items = static_cast<long long>(*a.n_jobs) * per;
  for (long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += static_cast<long long>(gridDim.x) * 8) {
    const int4 j = a.jobs[it / per];
    const int w = static_cast<int>(it % per);
    const int h = w % a.H, kv = (w / a.H) & 1, l = w / (2 * a.H);
    const long long in = (static_cast<long long>(h) << a.shift) * a.D + l * a.layer_stride;
    const long long from = j.x * a.page_stride + in, to = j.y * a.page_stride + in;
    uint8_t* base = kv ? a.v : a.k;
    const uint4* src = reinterpret_cast<const uint4*>(base + from * a.es);
    uint4* dst = reinterpret_cast<uint4*>(base + to * a.es);
    const int n = j.z * a.D * a.es / 16;
    for (int i0 = lane; i0 < n; i0 += 256) {
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + 32 * i < n) x[i] = src[i0 + 32 * i];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + 32 * i < n) dst[i0 + 32 * i] = x[i];
    }
    if (a.ks) {
      float* sc = kv ? a.vs : a.ks;
      for (int i = lane; i < j.z; i += 32) sc[to / a.D + i] = sc[from / a.D + i];
    }
  }
}

// A bit that another stream's kernel raises meanwhile is in *out or stays.
__global__ void take_status_kernel(int* status, int* out) { *out = atomicExch(status, 0); }

struct Layout {
  size_t list, list2, remap, jobs, total;
};
Layout layout_of(const dec_pages* p, const dec_page_map* m) {
  Layout l{};
  const size_t ids = round256(sizeof(int32_t) * static_cast<size_t>(p->n_pages));
  const size_t n = static_cast<size_t>(p->n_pages > m->n_seqs ? p->n_pages : m->n_seqs);
  l.list = 256;            // (the number of jobs comes first)
  l.list2 = l.list + ids;
  l.remap = l.list2 + ids;
  l.jobs = l.remap + ids;
  l.total = l.jobs + round256(sizeof(int4) * n);
  return l;
}

MapArgs map_args(const dec_pages* p, const dec_page_map* m, void* ws, int* status) {
  MapArgs a{};
  a.table = m->table;
  a.rows = m->rows;
  a.refs = m->refs;
  a.S = m->n_seqs;
  a.width = m->width;
  a.n_pages = p->n_pages;
  a.shift = log2_of(p->page_rows);
  a.status = status;
  if (ws) {
    const Layout l = layout_of(p, m);
    uint8_t* b = static_cast<uint8_t*>(ws);
    a.n_jobs = reinterpret_cast<int*>(b);
    a.list = reinterpret_cast<int32_t*>(b + l.list);
    a.list2 = reinterpret_cast<int32_t*>(b + l.list2);
    a.remap = reinterpret_cast<int32_t*>(b + l.remap);
    a.jobs = reinterpret_cast<int4*>(b + l.jobs);
  }
  return a;
}

// max_jobs: pages that may have to be copied.
cudaError_t launch_copy(const dec_pages* p, const dec_page_map* m, const MapArgs& ma, bool renumber,
                        long long max_jobs, int sms, cudaStream_t s) {
  CopyArgs c{};
  c.k = static_cast<uint8_t*>(p->k);
  c.v = static_cast<uint8_t*>(p->v);
  const bool fp8 = p->dtype == DEC_KV_FP8_E4M3;
  c.ks = fp8 ? p->k_scale : nullptr;
  c.vs = fp8 ? p->v_scale : nullptr;
  c.layer_stride = p->layer_stride;
  c.page_stride = p->page_stride;
  c.L = p->n_layers;
  c.H = p->n_kv_heads;
  c.D = p->head_dim;
  c.es = fp8 ? 1 : 2;
  c.shift = ma.shift;
  c.jobs = ma.jobs;
  c.n_jobs = ma.n_jobs;
  c.table = renumber ? m->table : nullptr;
  c.remap = ma.remap;
  c.cells = static_cast<long long>(m->n_seqs) * m->width;
  c.n_pages = p->n_pages;
  c.status = ma.status;
  const long long most = (max_jobs * c.L * 2 * c.H + 7) / 8;   // CTAs that could have work
  const unsigned n = static_cast<unsigned>(most < 16 * sms ? most : 16 * sms);
  return launch_dependent(copy_kernel, dim3(n), dim3(256), 0, s, c);
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" size_t dec_pages_workspace_bytes(const dec_pages* pool, const dec_page_map* map) {
  if (check_pool(pool) != DEC_OK || check_map(pool, map) != DEC_OK) return 0;
  return layout_of(pool, map).total;
}

static int check_pages_call(const dec_pages* pool, const dec_page_map* map, const void* in,
                            const void* ws, size_t ws_bytes, const int* status) {
  int rc = check_pool(pool);
  if (rc != DEC_OK) return rc;
  if ((rc = check_map(pool, map)) != DEC_OK) return rc;
  if (!in || !ws) return DEC_ERR_NULL;
  if (!is_aligned(in, 4) || !is_aligned(ws, 256) || !is_aligned(status, 4)) return DEC_ERR_ALIGN;
  return ws_bytes < layout_of(pool, map).total ? DEC_ERR_KV_SIZE : DEC_OK;
}

extern "C" int dec_pages_resize(const dec_pages* pool, const dec_page_map* map,
                                const int32_t* new_rows, void* workspace, size_t workspace_bytes,
                                int* status, void* stream) {
  const int rc = check_pages_call(pool, map, new_rows, workspace, workspace_bytes, status);
  if (rc != DEC_OK) return rc;
  const int sms = device_sms();
  if (sms < 0) return sms;
  MapArgs a = map_args(pool, map, workspace, status);
  a.in = new_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  resize_kernel<<<1, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_copy(pool, map, a, false, map->n_seqs, sms, s);
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}

extern "C" int dec_pages_compact(const dec_pages* pool, const dec_page_map* map, int32_t* n_live,
                                 void* workspace, size_t workspace_bytes, int* status,
                                 void* stream) {
  const int rc = check_pages_call(pool, map, n_live, workspace, workspace_bytes, status);
  if (rc != DEC_OK) return rc;
  const int sms = device_sms();
  if (sms < 0) return sms;
  MapArgs a = map_args(pool, map, workspace, status);
  a.n_live = n_live;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  compact_kernel<<<1, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_copy(pool, map, a, true, pool->n_pages, sms, s);
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}

extern "C" int dec_pages_fork(const dec_pages* pool, const dec_page_map* map,
                              const int32_t* parents, int* status, void* stream) {
  int rc = check_pool(pool);
  if (rc != DEC_OK) return rc;
  if ((rc = check_map(pool, map)) != DEC_OK) return rc;
  if (!parents) return DEC_ERR_NULL;
  if (!is_aligned(parents, 4) || !is_aligned(status, 4)) return DEC_ERR_ALIGN;
  MapArgs a = map_args(pool, map, nullptr, status);
  a.in = parents;
  // 8 cells to a thread, as far as columns allow
  int cols = 8 * kForkThreads / a.S;
  cols = cols > 16 ? 16 : cols < 1 ? 1 : cols;
  const int slices = (a.width + cols - 1) / cols;
  fork_kernel<<<slices + 1, kForkThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, cols);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}

extern "C" int dec_status_take(int* status, int* out, void* stream) {
  if (!status || !out) return DEC_ERR_NULL;
  if (!is_aligned(status, 4) || !is_aligned(out, 4)) return DEC_ERR_ALIGN;
  take_status_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(status, out);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DEC_OK : cuda_failed(e);
}
