// dec_paged.h -- host-side helpers and kernel views shared by the paged-cache
// and beam-search entry points.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "dec.h"

namespace dec {

// Records the runtime error for dec_last_cuda_error() and returns DEC_ERR_CUDA.
int cuda_failed(cudaError_t e);

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// One layer of a pool as the kernels address it: row r of head h of page p is
// element p * page_stride + (h << shift | r) * D.
struct PoolView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  long long page_stride;
  int n_pages;
  int shift;   // log2(page_rows)
};

inline int check_pool(const dec_pages* p) {
  if (!p || !p->k || !p->v) return DEC_ERR_NULL;
  if (p->dtype != DEC_KV_BF16 && p->dtype != DEC_KV_FP8_E4M3) return DEC_ERR_DTYPE;
  if (p->dtype == DEC_KV_FP8_E4M3 && (!p->k_scale || !p->v_scale)) return DEC_ERR_NULL;
  if (p->head_dim != 64 && p->head_dim != 128) return DEC_ERR_SHAPE;
  if (p->n_layers < 1 || p->n_kv_heads < 1 || p->n_kv_heads > 256 || p->n_pages < 1)
    return DEC_ERR_SHAPE;
  if (p->page_rows < 8 || p->page_rows > 1024 || (p->page_rows & (p->page_rows - 1)))
    return DEC_ERR_SHAPE;
  const long long page = static_cast<long long>(p->n_kv_heads) * p->page_rows * p->head_dim;
  if (p->layer_stride < page || p->page_stride < page || p->layer_stride % p->head_dim ||
      p->page_stride % p->head_dim)
    return DEC_ERR_SHAPE;
  if (!is_aligned(p->k, 16) || !is_aligned(p->v, 16)) return DEC_ERR_ALIGN;
  if (p->dtype == DEC_KV_FP8_E4M3 &&
      (!is_aligned(p->k_scale, 16) || !is_aligned(p->v_scale, 16) ||
       p->layer_stride % (4 * p->head_dim) || p->page_stride % (4 * p->head_dim)))
    return DEC_ERR_ALIGN;
  return DEC_OK;
}

inline int check_map(const dec_pages* p, const dec_page_map* m) {
  if (!m || !m->table || !m->rows || !m->refs) return DEC_ERR_NULL;
  if (m->n_seqs < 1 || m->n_seqs > 4096) return DEC_ERR_BATCH;
  if (m->width < 1 || static_cast<long long>(m->width) * p->page_rows > (1ll << 30) ||
      static_cast<long long>(m->n_seqs) * m->width > INT32_MAX)
    return DEC_ERR_SHAPE;
  if (!is_aligned(m->table, 4) || !is_aligned(m->rows, 4) || !is_aligned(m->refs, 4))
    return DEC_ERR_ALIGN;
  return DEC_OK;
}

inline int log2_of(int pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

inline PoolView layer_view(const dec_pages* p, int layer) {
  const bool fp8 = p->dtype == DEC_KV_FP8_E4M3;
  const long long off = layer * p->layer_stride;
  PoolView v{};
  v.k = static_cast<uint8_t*>(p->k) + off * (fp8 ? 1 : 2);
  v.v = static_cast<uint8_t*>(p->v) + off * (fp8 ? 1 : 2);
  v.ks = fp8 ? p->k_scale + off / p->head_dim : nullptr;
  v.vs = fp8 ? p->v_scale + off / p->head_dim : nullptr;
  v.page_stride = p->page_stride;
  v.n_pages = p->n_pages;
  v.shift = log2_of(p->page_rows);
  return v;
}

// SMs of the current device (DEC_ERR_* < 0 on failure).
inline int device_sms() {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? sms : cuda_failed(e);
}

// Raise a kernel's dynamic shared-memory limit once per device (the attribute
// belongs to the device's context).  `done` is a static of the call site.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch with programmatic stream serialisation: the kernel may start while
// its predecessor drains and must call pdl_wait() before it touches anything
// that the predecessor writes (or reads, if the kernel overwrites it).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dec
