// paged_index.cu - the indexer over the paged cache: index keys and block
// means of new tokens, and the top-16 blocks of each row's newest token.
//
// Both follow select.cu, which forms the same means and scores over compact
// documents: a block's mean is its keys' fp32 sum in order of position divided
// by their number, a score the chain of fused multiply-adds channel by
// channel.  The order is kept exactly, so a token selects the same blocks
// here as there.
//
// k_paged_index   one CTA a block that got a token: it writes the block's new
//                 keys and sums old and new ones.  Blocks are found by their
//                 first new token (position a multiple of 128, or the row's
//                 first).
// k_paged_select  one cluster of CTAs a (row, index head): a lane scores a
//                 block, a warp keeps the best of its blocks in a list sorted
//                 across its lanes, and the lists are merged through shared
//                 memory, then through the cluster's.
#include <cooperative_groups.h>

#include <utility>

#include "paged.cuh"

namespace msa {
namespace {

constexpr int kIdxThreads = 256;
constexpr int kIdxPages = kBlock;  // pages of a block, one-token pages at most

struct IndexArgs {
  const __nv_bfloat16* ik;
  int64_t ik_stride;
  PagedPool keys;
  float* means;
  PagedTable table;
  const int32_t *offs, *start;
  int64_t T;
  int32_t heads, dim;
};

// Where the mean of the block that position last (its last key) lies in is kept.
__device__ __forceinline__ int64_t mean_slot(const PagedTable& t, int32_t page, int32_t last) {
  if (t.shift <= 7) return page;
  return (int64_t(page) << (t.shift - 7)) + ((last & ((1 << t.shift) - 1)) >> 7);
}

// Token t starts the new part of a block: its row, position and the number
// of the block's new tokens (0: t does not).
struct BlockStart {
  int32_t row, n_new;
  int64_t pos;
};
__device__ __forceinline__ BlockStart block_start(const IndexArgs& a, int64_t t, int32_t r) {
  BlockStart b{r, 0, 0};
  const int32_t o0 = a.offs[r], o1 = a.offs[r + 1];
  if (t < o0 || t >= o1) return b;
  b.pos = int64_t(a.start[r]) + (t - o0);
  if (t != o0 && (b.pos & 127) != 0) return b;
  const int64_t room = 128 - (b.pos & 127);
  b.n_new = int32_t(room < o1 - t ? room : o1 - t);
  return b;
}

__device__ void index_block(const IndexArgs& a, int64_t t, const BlockStart& b, int32_t* pages) {
  const int n_old = int(b.pos & 127);
  const int64_t first = b.pos - n_old;  // position of the block's first key
  const int n = n_old + b.n_new;
  const int64_t i0 = first >> a.table.shift;
  const int np = int(((first + n - 1) >> a.table.shift) - i0) + 1;
  __syncthreads();  // the list of the block before is no longer read
  bool bad = b.pos < 0;
  if (!bad)
    for (int i = threadIdx.x; i < np; i += kIdxThreads) {
      const int32_t p = page_of(a.table, b.row, (i0 + i) << a.table.shift);
      pages[i] = p;
      bad |= p < 0;
    }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    return;
  }
  __nv_bfloat16* keys = static_cast<__nv_bfloat16*>(a.keys.base);
  const int width = a.heads * a.dim;
  const int mask = (1 << a.table.shift) - 1;
  for (int ch = 2 * threadIdx.x; ch < width; ch += 2 * kIdxThreads) {
    const int h = ch / a.dim, c = ch % a.dim;
    __nv_bfloat16* col = keys + h * a.keys.head + c;
    const __nv_bfloat16* in = a.ik + t * a.ik_stride + ch;
    float s0 = 0.f, s1 = 0.f;
    // 32 keys' loads in flight, then their sum in order: the adds are one
    // chain either way, the loads need not be.
    for (int j0 = 0; j0 < n; j0 += 32) {
      uint32_t w[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const int j = j0 + u;
        w[u] = 0;
        if (j < n) {
          const int64_t p = first + j;
          const __nv_bfloat16* src =
              j < n_old ? col + pages[(p >> a.table.shift) - i0] * a.keys.page +
                              (p & mask) * a.keys.token
                        : in + int64_t(j - n_old) * a.ik_stride;
          w[u] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const int j = j0 + u;
        if (j < n) {
          const float2 f = Pair<__nv_bfloat16>::unpack(w[u]);
          s0 += f.x;
          s1 += f.y;
          if (j >= n_old) {
            const int64_t p = first + j;
            *reinterpret_cast<uint32_t*>(col + pages[(p >> a.table.shift) - i0] * a.keys.page +
                                         (p & mask) * a.keys.token) = w[u];
          }
        }
      }
    }
    const int64_t slot = mean_slot(a.table, pages[np - 1], int32_t(first + n - 1));
    *reinterpret_cast<float2*>(a.means + slot * width + ch) =
        make_float2(__fdiv_rn(s0, float(n)), __fdiv_rn(s1, float(n)));
  }
}

__global__ void __launch_bounds__(kIdxThreads) k_paged_index(const IndexArgs a) {
  __shared__ int32_t pages[kIdxPages];
  __shared__ int32_t hit[32];
  __shared__ int n_hits;
  grid_dep_wait();
  grid_dep_release();
  if (blockIdx.x == 0) check_offsets(a.offs, a.table.rows, a.T, a.table.status);
  if (a.T <= gridDim.x) {  // one token a CTA
    const int64_t t = blockIdx.x;
    const BlockStart b = block_start(a, t, find_row_warp(a.offs, a.table.rows, t));
    if (b.n_new > 0) index_block(a, t, b, pages);
    return;
  }
  for (int64_t t0 = blockIdx.x; t0 < a.T; t0 += 32ll * gridDim.x) {
    __syncthreads();
    if (threadIdx.x < 32) {
      const int64_t t = t0 + int64_t(threadIdx.x) * gridDim.x;
      bool starts = false;
      if (t < a.T) {
        int32_t lo = 0, hi = a.table.rows - 1;  // largest r with offs[r] <= t
        while (lo < hi) {
          const int32_t mid = (lo + hi + 1) >> 1;
          if (a.offs[mid] <= t) lo = mid; else hi = mid - 1;
        }
        starts = block_start(a, t, lo).n_new > 0;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, starts);
      if (starts) hit[__popc(m & ((1u << threadIdx.x) - 1))] = int32_t(t);
      if (threadIdx.x == 0) n_hits = __popc(m);
    }
    __syncthreads();
    const int n = n_hits;
    for (int i = 0; i < n; ++i) {
      const int64_t t = hit[i];
      const BlockStart b = block_start(a, t, find_row_warp(a.offs, a.table.rows, t));
      index_block(a, t, b, pages);
    }
  }
}

// ------------------------------------------------------------------ selection
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCluster = 8;

struct SelectArgs {
  const __nv_bfloat16* iq;
  const float* means;
  PagedTable table;
  const int32_t* kv_len;
  int32_t* q2k;
  int32_t heads, dim, force;
};

// A candidate as one 64-bit key, larger = ranked before: the score's bits made
// monotone, then the block's complement (equal scores: the lower block).
// 0 = no candidate.
__device__ __forceinline__ uint64_t rank_key(float score, int32_t v) {
  uint32_t u = __float_as_uint(score + 0.f);  // -0 ranks as +0
  u ^= (u >> 31) ? 0xffffffffu : 0x80000000u;
  return (uint64_t(u) << 32) | uint32_t(~v);
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int o) {
  return __shfl_xor_sync(0xffffffffu, x, o);
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t min64(uint64_t a, uint64_t b) { return a < b ? a : b; }
// Sorts a bitonic sequence of kN lanes (aligned groups), largest first.
template <int kN>
__device__ __forceinline__ uint64_t bitonic_merge(uint64_t x, int lane) {
#pragma unroll
  for (int o = kN / 2; o > 0; o >>= 1) {
    const uint64_t y = shfl_xor64(x, o);
    x = (lane & o) ? min64(x, y) : max64(x, y);
  }
  return x;
}
// Sorts the 32 lanes' values, largest first.
__device__ __forceinline__ uint64_t sort_desc(uint64_t x, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int o = k / 2; o > 0; o >>= 1) {
      const uint64_t y = shfl_xor64(x, o);
      const bool down = (lane & k) == 0;  // k == 32: every lane
      const bool low = (lane & o) == 0;
      x = (low == down) ? max64(x, y) : min64(x, y);
    }
  }
  return x;
}

__global__ void __launch_bounds__(kSelThreads) k_paged_select(const SelectArgs a) {
  namespace cg = cooperative_groups;
  __shared__ float sq[128];
  __shared__ uint64_t lists[kSelWarps][kTopK];
  __shared__ uint64_t from[kSelMaxCluster][kTopK];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int64_t unit = blockIdx.x / C;
  const int32_t r = int32_t(unit / a.heads), h = int32_t(unit % a.heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_release();
  const int32_t len = row_length(a.table, a.kv_len, r);
  const int32_t nb = int32_t((int64_t(len) + kBlock - 1) / kBlock), b = nb - 1;
  int32_t* out = a.q2k + (int64_t(h) * a.table.rows + r) * kTopK;
  if (nb <= kTopK) {  // the same for the whole cluster
    if (rank == 0 && threadIdx.x < kTopK)
      out[threadIdx.x] = int(threadIdx.x) < nb ? int(threadIdx.x) : -1;
    return;
  }
  auto started = cluster.barrier_arrive();
  for (int c = threadIdx.x; c < a.dim; c += kSelThreads)
    sq[c] = __bfloat162float(a.iq[(int64_t(r) * a.heads + h) * a.dim + c]);
  __syncthreads();
  const int32_t lo = a.force ? 1 : 0, hi = a.force ? b - 1 : b;
  uint64_t best = 0;  // the warp's best candidates, sorted over the lanes
  for (int32_t v0 = lo + (rank * kSelWarps + warp) * 32; v0 <= hi; v0 += C * kSelThreads) {
    const int32_t v = v0 + lane;
    uint64_t key = 0;
    if (v <= hi) {
      const int32_t last = min(v * kBlock + kBlock - 1, len - 1);
      const int32_t page = page_of(a.table, r, last);
      if (page >= 0) {
        const float4* m = reinterpret_cast<const float4*>(
            a.means + (mean_slot(a.table, page, last) * a.heads + h) * a.dim);
        float acc = 0.f;
#pragma unroll 8
        for (int c = 0; c < a.dim / 4; ++c) {
          const float4 s = m[c];
          acc = fmaf(sq[4 * c + 0], s.x, acc);
          acc = fmaf(sq[4 * c + 1], s.y, acc);
          acc = fmaf(sq[4 * c + 2], s.z, acc);
          acc = fmaf(sq[4 * c + 3], s.w, acc);
        }
        key = rank_key(acc, v);
      }
    }
    key = sort_desc(key, lane);
    // the larger of best[i] and key[31 - i] are the best 32 of both lists
    const uint64_t rev = __shfl_sync(0xffffffffu, key, 31 - lane);
    best = bitonic_merge<32>(max64(best, rev), lane);
  }
  if (lane < kTopK) lists[warp][lane] = best;
  __syncthreads();
  // merge the warps' lists pairwise: lanes 0..15 hold one, lanes 16..31 idle
  for (int n = kSelWarps / 2; n > 0; n >>= 1) {
    uint64_t x = 0;
    if (warp < n) {
      x = max64(lists[warp][lane & 15], lists[warp + n][15 - (lane & 15)]);
      x = bitonic_merge<16>(x, lane & 15);
    }
    __syncthreads();
    if (warp < n && lane < kTopK) lists[warp][lane] = x;
    __syncthreads();
  }
  cluster.barrier_wait(std::move(started));  // every CTA's shared memory is there
  if (C > 1) {
    if (threadIdx.x < kTopK)
      cluster.map_shared_rank(&from[rank][threadIdx.x], 0)[0] = lists[0][threadIdx.x];
    cluster.sync();
  }
  if (rank != 0 || warp != 0) return;
  uint64_t top = lists[0][lane & 15];
  for (int k = 1; k < C; ++k) {
    top = max64(top, from[k][15 - (lane & 15)]);
    top = bitonic_merge<16>(top, lane & 15);
  }
  // the chosen blocks in ascending order, unused slots last
  const int need = a.force ? kTopK - 2 : kTopK;
  int32_t mine = top == 0 ? INT32_MAX : int32_t(~uint32_t(top));
  if ((lane & 15) >= need) mine = (lane & 15) == need ? 0 : b;
  int place = 0;
#pragma unroll
  for (int k = 0; k < kTopK; ++k) {
    const int32_t x = __shfl_sync(0xffffffffu, mine, k);
    place += (x < mine || (x == mine && k < (lane & 15))) ? 1 : 0;
  }
  if (lane < kTopK) out[place] = mine == INT32_MAX ? -1 : mine;
}

cudaError_t launch_paged_select(const SelectArgs& a, cudaStream_t s) {
  // CTAs of a cluster: one for every 256 blocks that the table has room for.
  const int64_t room = ((int64_t(a.table.width) << a.table.shift) + kBlock - 1) / kBlock;
  int C = 1;
  while (C < kSelMaxCluster && room > int64_t(C) * kSelThreads) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(int64_t(a.table.rows) * a.heads * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = profiling_on() ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, k_paged_select, a);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_paged_index(const msa_paged_index_cache* cache,
                                      const msa_page_table* table, const int32_t* row_offsets,
                                      const int32_t* start_pos, int64_t T, const void* ik,
                                      int64_t ik_stride, msa_stream_t stream) {
  msa_status st = check_index_cache(cache);
  if (st != MSA_OK) return st;
  st = check_table(table, cache->page_size);
  if (st != MSA_OK) return st;
  if (!row_offsets || !start_pos || !ik || T < 1 || T > kMaxTokens || ik_stride % 8 ||
      ik_stride < int64_t(cache->heads) * cache->dim)
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(ik) || !paged_aligned4(row_offsets) || !paged_aligned4(start_pos))
    return MSA_ERR_ALIGNMENT;
  st = check_device();
  if (st != MSA_OK) return st;
  IndexArgs a{};
  a.ik = static_cast<const __nv_bfloat16*>(ik);
  a.ik_stride = ik_stride;
  a.keys = PagedPool{cache->keys, cache->key_stride[0], cache->key_stride[1], cache->key_stride[2]};
  a.means = cache->means;
  a.table = table_args(table, cache->page_size, cache->num_pages, cache->status);
  a.offs = row_offsets;
  a.start = start_pos;
  a.T = T;
  a.heads = cache->heads;
  a.dim = cache->dim;
  // An odd number of CTAs: blocks start 128 tokens apart, and an odd stride
  // spreads them over all CTAs.
  const int64_t most = int64_t(device_sm_count()) * 8 - 1;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin("paged_index", s);
  const cudaError_t e = launch_k(true, k_paged_index, dim3(unsigned(T < most ? T : most)),
                                 dim3(kIdxThreads), 0, s, a);
  launch_end("paged_index", s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

extern "C" msa_status msa_paged_select(const msa_paged_index_cache* cache,
                                       const msa_page_table* table, const int32_t* kv_len,
                                       const void* iq, int32_t force_local, int32_t* q2k,
                                       msa_stream_t stream) {
  msa_status st = check_index_cache(cache);
  if (st != MSA_OK) return st;
  st = check_table(table, cache->page_size);
  if (st != MSA_OK) return st;
  if (!kv_len || !iq || !q2k) return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(iq) || !paged_aligned(q2k) || !paged_aligned4(kv_len))
    return MSA_ERR_ALIGNMENT;
  st = check_device();
  if (st != MSA_OK) return st;
  SelectArgs a{};
  a.iq = static_cast<const __nv_bfloat16*>(iq);
  a.means = cache->means;
  a.table = table_args(table, cache->page_size, cache->num_pages, cache->status);
  a.kv_len = kv_len;
  a.q2k = q2k;
  a.heads = cache->heads;
  a.dim = cache->dim;
  a.force = force_local ? 1 : 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin("paged_select", s);
  const cudaError_t e = launch_paged_select(a, s);
  launch_end("paged_select", s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
