// paged.cuh - what the paged-cache kernels (append, index, select, decode)
// share: the cache as kernel arguments, the search of a token's row, the
// host's argument checks.
#pragma once
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"

namespace msa {

constexpr int kMaxPageSize = 1024;
constexpr int kMaxRows = 65536;

// One pool (keys or values) of a paged cache, strides in elements.
struct PagedPool {
  void* base;
  int64_t page, token, head;
};
// The page table of a call.
struct PagedTable {
  const int32_t* pages;
  int64_t stride;
  int32_t rows, width;
  int32_t shift;       // log2 of the page size
  int32_t num_pages;
  int64_t* status;
};

__device__ __forceinline__ void raise_paged(int64_t* status, msa_status s) {
  atomicOr(reinterpret_cast<unsigned long long*>(status), 1ull << static_cast<int>(s));
}
// Page of position pos of row r, or -1 (with MSA_ERR_BAD_PAGE) if there is none.
__device__ __forceinline__ int32_t page_of(const PagedTable& t, int32_t r, int64_t pos) {
  const int64_t i = pos >> t.shift;
  int32_t p = -1;
  if (pos >= 0 && i < t.width) p = t.pages[int64_t(r) * t.stride + i];
  if (p < 0 || p >= t.num_pages) {
    raise_paged(t.status, MSA_ERR_BAD_PAGE);
    return -1;
  }
  return p;
}
// A row's length, or 0 (with MSA_ERR_BAD_PAGE) if its table is too short for it.
__device__ __forceinline__ int32_t row_length(const PagedTable& t, const int32_t* kv_len,
                                              int32_t r) {
  const int32_t n = kv_len[r];
  if (n < 0 || n > (int64_t(t.width) << t.shift)) {
    raise_paged(t.status, MSA_ERR_BAD_PAGE);
    return 0;
  }
  return n;
}

// Largest r in [0, rows) with offs[r] <= t (0 if there is none), by a whole
// warp: 32 probes a step, so that a batch of up to 1024 rows takes two
// dependent loads where halving takes ten.
__device__ __forceinline__ int32_t find_row_warp(const int32_t* offs, int32_t rows, int64_t t) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, n = rows;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) >> 5;
    const int32_t i = lo + lane * step;
    const bool le = lane * step < n && offs[i] <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, le));
    const int32_t k = hits > 0 ? hits - 1 : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// Checks row_offsets; one CTA's threads share the work.
__device__ __forceinline__ void check_offsets(const int32_t* offs, int32_t rows, int64_t T,
                                              int64_t* status) {
  bool bad = false;
  for (int32_t i = threadIdx.x; i < rows; i += blockDim.x) bad |= offs[i] > offs[i + 1];
  if (threadIdx.x == 0) bad |= offs[0] != 0 || offs[rows] > T;
  if (bad) raise_paged(status, MSA_ERR_BAD_OFFSETS);
}

template <typename T>
struct Pair;  // two 16-bit values <-> two fp32
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// ---------------------------------------------------------------- host side
// Lets a kernel use `bytes` of dynamic shared memory, once a device: `done` is
// the kernel's own, a bit for each device (the call is made every time on
// devices past 63).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}
int device_sm_count();
msa_status check_device();

// launch_k for a kernel in clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                           unsigned cluster, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = profiling_on() ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

inline bool paged_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool paged_aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int32_t log2_of(int32_t x) {
  int32_t s = 0;
  while ((int32_t(1) << s) < x) ++s;
  return s;
}
inline bool good_page_size(int32_t s) { return s >= 1 && s <= kMaxPageSize && (s & (s - 1)) == 0; }
inline bool good_strides(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 8 || s[i] % 8 || s[i] > (int64_t(1) << 48)) return false;
  return true;
}
inline msa_status check_cache(const msa_paged_cache* c) {
  if (!c || !c->k || !c->v || !c->status) return MSA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > INT32_MAX || !good_page_size(c->page_size) ||
      c->kv_heads < 1 || c->kv_heads > 64 || (c->head_dim != 64 && c->head_dim != 128) ||
      (c->dtype != MSA_BF16 && c->dtype != MSA_F16) || !good_strides(c->k_stride) ||
      !good_strides(c->v_stride))
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(c->k) || !paged_aligned(c->v) ||
      (reinterpret_cast<uintptr_t>(c->status) & 7u))
    return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}
inline msa_status check_index_cache(const msa_paged_index_cache* c) {
  if (!c || !c->keys || !c->means || !c->status) return MSA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > INT32_MAX || !good_page_size(c->page_size) ||
      c->heads < 1 || c->heads > 64 || c->dim < 8 || c->dim > 128 || c->dim % 8 ||
      !good_strides(c->key_stride))
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(c->keys) || !paged_aligned(c->means) ||
      (reinterpret_cast<uintptr_t>(c->status) & 7u))
    return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}
inline msa_status check_table(const msa_page_table* t, int32_t page_size) {
  if (!t || !t->pages || t->rows < 1 || t->rows > kMaxRows || t->width < 1 ||
      t->stride < t->width || int64_t(t->width) * page_size > (int64_t(1) << 30))
    return MSA_ERR_INVALID_ARG;
  return paged_aligned4(t->pages) ? MSA_OK : MSA_ERR_ALIGNMENT;
}
inline PagedTable table_args(const msa_page_table* t, int32_t page_size, int64_t num_pages,
                             int64_t* status) {
  return PagedTable{t->pages, t->stride, t->rows, t->width, log2_of(page_size),
                    int32_t(num_pages), status};
}

}  // namespace msa
