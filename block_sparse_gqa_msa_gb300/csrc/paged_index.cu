// paged_index.cu - the indexer over the paged cache: index keys and block
// means of new tokens, and the top-16 blocks of each row's newest token.
//
// Both follow select.cu, which forms the same means and scores over compact
// documents: a block's mean is its keys' fp32 sum in order of position divided
// by their number, a score the chain of fused multiply-adds channel by
// channel.  The order is kept exactly, so a token selects the same blocks
// here as there.
//
// k_paged_index   one CTA a block that got a token and 128 channels: it brings
//                 the block's keys, old and new, into shared memory with all
//                 loads in flight, writes the new ones to the cache and sums
//                 them in order.  Blocks are numbered over the rows and dealt
//                 out in turn.
//                 20494 prompt tokens of 4 x 128 channels (43 MB, 6.3 us at the
//                 copy rate): 11.5 us (44 with the block's keys summed as they
//                 came, 13.4 with them staged in registers, three CTAs an SM); 96 rows' next tokens: 5 us, four dependent loads.
// k_paged_select  one cluster of CTAs a (row, index head): a warp brings the
//                 means of 32 blocks to shared memory 32 channels at a time
//                 (rows coalesced), a lane scores a block, and the warp keeps
//                 the best 16 in order; the warps' lists meet in shared memory,
//                 the CTAs' in the cluster's.  Places in a list are counted.
//                 64 rows of up to 1024 blocks of 4 x 128 channels (68 MB, 10
//                 us): 21.5 us (62 with each lane reading its block's row from
//                 memory); 3 us before the first means come, the longest rows,
//                 two CTAs each, and the lists are the rest.  One row of 1024
//                 blocks: 4.8 to 5.0 us (5.3 with the lists sorted and merged, which made no
//                 difference to the batch).
#include <cooperative_groups.h>

#include <utility>

#include "paged.cuh"

namespace msa {
namespace {

constexpr int kIdxThreads = 256;
constexpr int kIdxSlice = 128;      // channels of one CTA
constexpr int kIdxChunks = kIdxSlice / 8;
constexpr int kIdxPages = kBlock;   // pages of a block, one-token pages at most

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

// The new part of a block: its row, the first of its new tokens, that token's
// position and their number.
struct NewBlock {
  int32_t row, t, n_new;
  int64_t pos;
};
// Blocks of row r that get a token (0: none, or the row's offsets or first
// position are bad; as for append, a row has no tokens past T).
__device__ __forceinline__ int32_t row_blocks(const IndexArgs& a, int32_t r) {
  const int64_t o0 = a.offs[r], o1 = min(int64_t(a.offs[r + 1]), a.T), p = a.start[r];
  if (o0 < 0 || o1 <= o0) return 0;
  if (p < 0) {
    raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    return 0;
  }
  return int32_t(((p + (o1 - o0) - 1) >> 7) - (p >> 7)) + 1;
}

struct IndexSmem {
  uint4 rows[kBlock][kIdxChunks];  // the block's keys, the CTA's channels
  int32_t pages[kIdxPages];
  int32_t sums[kIdxThreads / 32];
  NewBlock block;
};

__device__ __forceinline__ void index_block(const IndexArgs& a, IndexSmem& sm) {
  const NewBlock b = sm.block;
  const int n_old = int(b.pos & 127);
  const int64_t first = b.pos - n_old;  // position of the block's first key
  const int n = n_old + b.n_new;
  const int64_t i0 = first >> a.table.shift;
  const int np = int(((first + n - 1) >> a.table.shift) - i0) + 1;
  bool bad = false;
  for (int i = threadIdx.x; i < np; i += kIdxThreads) {
    const int32_t p = page_of(a.table, b.row, (i0 + i) << a.table.shift);
    sm.pages[i] = p;
    bad |= p < 0;
  }
  if (__syncthreads_or(bad)) return;
  const int width = a.heads * a.dim;
  const int mask = (1 << a.table.shift) - 1;
  // A thread's chunk is the same for all its keys.
  const int ch = blockIdx.y * kIdxSlice + int(threadIdx.x % kIdxChunks) * 8;
  if (ch < width) {
    __nv_bfloat16* col =
        static_cast<__nv_bfloat16*>(a.keys.base) + (ch / a.dim) * a.keys.head + ch % a.dim;
    const __nv_bfloat16* in = a.ik + b.t * a.ik_stride + ch;
    constexpr int kStep = kIdxThreads / kIdxChunks;
    constexpr int kEach = kBlock / kStep;
    const int j0 = int(threadIdx.x / kIdxChunks);
    auto place = [&](int j) {
      const int64_t p = first + j;
      return col + sm.pages[(p >> a.table.shift) - i0] * a.keys.page + (p & mask) * a.keys.token;
    };
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int j = j0 + u * kStep;
      if (j < n) {
        const __nv_bfloat16* src = j < n_old ? place(j) : in + int64_t(j - n_old) * a.ik_stride;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(
                         __cvta_generic_to_shared(&sm.rows[j][threadIdx.x % kIdxChunks]))),
                     "l"(src)
                     : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int j = j0 + u * kStep;
      if (j >= n_old && j < n)
        *reinterpret_cast<uint4*>(place(j)) = sm.rows[j][threadIdx.x % kIdxChunks];
    }
  }
  __syncthreads();
  const int c = blockIdx.y * kIdxSlice + 2 * int(threadIdx.x);
  if (2 * threadIdx.x < kIdxSlice && c < width) {
    const uint32_t* col = reinterpret_cast<const uint32_t*>(&sm.rows[0][0]) + threadIdx.x;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll 16
    for (int j = 0; j < n; ++j) {
      const float2 f = Pair<__nv_bfloat16>::unpack(col[j * (kIdxSlice / 2)]);
      s0 += f.x;
      s1 += f.y;
    }
    const int64_t slot = mean_slot(a.table, sm.pages[np - 1], int32_t(first + n - 1));
    *reinterpret_cast<float2*>(a.means + slot * width + c) =
        make_float2(__fdiv_rn(s0, float(n)), __fdiv_rn(s1, float(n)));
  }
}

__global__ void __launch_bounds__(kIdxThreads) k_paged_index(const IndexArgs a) {
  __shared__ IndexSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_release();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(a.offs, a.table.rows, a.T, a.table.status);
  // Blocks are numbered row by row and dealt out in turn: every thread counts
  // those of a stretch of rows, a scan gives their places.
  const int32_t rows = a.table.rows, each = (rows + kIdxThreads - 1) / kIdxThreads;
  const int32_t r0 = min(rows, tid * each), r1 = min(rows, r0 + each);
  int32_t mine = 0;
  for (int32_t r = r0; r < r1; ++r) mine += row_blocks(a, r);
  int32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.sums[warp] = incl;
  __syncthreads();
  int32_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kIdxThreads / 32; ++w) {
    if (w < warp) before += sm.sums[w];
    total += sm.sums[w];
  }
  before += incl - mine;
  for (int32_t x = blockIdx.x; x < total; x += gridDim.x) {
    if (x >= before && x < before + mine) {  // one thread: the block is in its stretch
      int32_t k = x - before;
      int32_t r = r0;
      for (int32_t n; k >= (n = row_blocks(a, r)); ++r) k -= n;
      const int32_t o0 = a.offs[r], o1 = int32_t(min(int64_t(a.offs[r + 1]), a.T));
      const int64_t p = a.start[r], first = k == 0 ? p : ((p >> 7) + k) << 7;
      NewBlock b;
      b.row = r;
      b.pos = first;
      b.t = o0 + int32_t(first - p);
      b.n_new = int32_t(min(128 - (first & 127), int64_t(o1 - b.t)));
      sm.block = b;
    }
    __syncthreads();
    index_block(a, sm);
    __syncthreads();  // the block is done
  }
}

// ------------------------------------------------------------------ selection
constexpr int kSelMaxCluster = 8;
// A warp's ring of slabs: 32 channels of the means of 32 blocks, a block's
// row 16 bytes longer than its 128 so that 8 rows' 16-byte reads hit
// different banks.
constexpr int kSlabRow = 144;
constexpr int kSlabBytes = 32 * kSlabRow;
constexpr int kSlabs = 3;

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
// How many of n keys (even, 16-byte aligned, shared memory) rank before x.
template <int kN>
__device__ __forceinline__ int ranked_before(const uint64_t* keys, uint64_t x) {
  int n = 0;
#pragma unroll
  for (int j = 0; j < kN; j += 2) {
    const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(keys + j);
    n += (k.x > x) + (k.y > x);
  }
  return n;
}

template <int kSelWarps>
__global__ void __launch_bounds__(kSelWarps * 32) k_paged_select(const SelectArgs a) {
  constexpr int kSelThreads = kSelWarps * 32;
  namespace cg = cooperative_groups;
  extern __shared__ __align__(128) uint8_t slabs[];
  __shared__ __align__(16) float sq[128];
  __shared__ __align__(16) uint64_t lists[kSelWarps][kTopK];
  __shared__ __align__(16) uint64_t from[kSelMaxCluster][kTopK];
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
  for (int i = threadIdx.x; i < C * kTopK; i += kSelThreads) from[0][i] = 0;
  auto started = cluster.barrier_arrive();
  const int32_t lo = a.force ? 1 : 0, hi = a.force ? b - 1 : b;
  const int32_t v_step = C * kSelThreads;
  int32_t fv = lo + (rank * kSelWarps + warp) * 32;  // first block of the group being fetched
  // The page of the lane's block in the group from v0 on, as the table has it;
  // loaded a group ahead.
  auto last_of = [&](int32_t v) { return min(v * kBlock + kBlock - 1, len - 1); };
  auto load_page = [&](int32_t v0) {
    return v0 + lane <= hi
               ? a.table.pages[int64_t(r) * a.table.stride + (last_of(v0 + lane) >> a.table.shift)]
               : 0;
  };
  int32_t next_page = load_page(fv);
  for (int c = threadIdx.x; c < a.dim; c += kSelThreads)
    sq[c] = __bfloat162float(a.iq[(int64_t(r) * a.heads + h) * a.dim + c]);
  // The warp's slabs in order: for every group of 32 blocks, its channels 32
  // at a time.  fetch runs kSlabs - 1 slabs ahead of the sums.
  const uint32_t ring = uint32_t(__cvta_generic_to_shared(slabs)) + warp * (kSlabs * kSlabBytes);
  const int per = (a.dim + 31) / 32;
  int fc = 0;        // the group's next slab
  int64_t row = -1;  // the lane's block in it: row of the means
  auto locate = [&]() {
    const int32_t page = next_page;
    row = -1;
    if (fv + lane <= hi) {
      if (page >= 0 && page < a.table.num_pages)
        row = mean_slot(a.table, page, last_of(fv + lane)) * a.heads + h;
      else
        raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    }
    next_page = load_page(fv + v_step);
  };
  if (fv <= hi) locate();
  auto fetch = [&](int stage) {
    if (fv > hi) return;
    const int c = fc * 32 + (lane & 7) * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // 4 rows of 128 bytes an instruction
      const int k = i * 4 + (lane >> 3);
      const int64_t m = __shfl_sync(0xffffffffu, row, k);
      const bool real = m >= 0 && c < a.dim;
      const float* src = real ? a.means + m * a.dim + c : a.means;
      asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(
                       ring + stage * kSlabBytes + k * kSlabRow + (lane & 7) * 16),
                   "l"(src), "r"(real ? 16 : 0)
                   : "memory");
    }
    if (++fc == per) {
      fc = 0;
      fv += v_step;
      if (fv <= hi) locate();
    }
  };
  uint64_t best = 0;  // the warp's best candidates, in order, in lanes 0 .. 15
  int32_t gv = fv;    // the group being summed
  int stage = 0;
  for (int i = 0; i < kSlabs - 1; ++i) {
    fetch(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __syncthreads();  // the query
  while (gv <= hi) {
    float acc = 0.f;
    for (int c = 0; c < per; ++c) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlabs - 2) : "memory");
      __syncwarp();
      fetch((stage + kSlabs - 1) % kSlabs);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const float4* m = reinterpret_cast<const float4*>(
          slabs + warp * (kSlabs * kSlabBytes) + stage * kSlabBytes + lane * kSlabRow);
      const int n4 = min(8, (a.dim - c * 32) / 4);
      const float4* q = reinterpret_cast<const float4*>(sq + c * 32);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k < n4) {
          const float4 s = m[k], t = q[k];
          acc = fmaf(t.x, s.x, acc);
          acc = fmaf(t.y, s.y, acc);
          acc = fmaf(t.z, s.z, acc);
          acc = fmaf(t.w, s.w, acc);
        }
      }
      stage = (stage + 1) % kSlabs;
    }
    uint64_t key = 0;
    if (gv + lane <= hi) {
      const int32_t v = gv + lane;
      const int32_t last = min(v * kBlock + kBlock - 1, len - 1);
      if (page_of(a.table, r, last) >= 0) key = rank_key(acc, v);
    }
    gv += v_step;
    // nothing here beats the last of the kept ones: most groups of a long row
    if (!__any_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, best, kTopK - 1))) continue;
    // Every candidate, new or kept, counts those that rank before it: its place
    // in the new list.  (In the slab just read, which the next fetch fills: 16
    // independent loads, where sorting and merging took 20 dependent exchanges.)
    uint64_t* sc = reinterpret_cast<uint64_t*>(slabs + warp * (kSlabs * kSlabBytes) +
                                               (stage + kSlabs - 1) % kSlabs * kSlabBytes);
    __syncwarp();  // the slab is read
    sc[lane] = key;
    if (lane < kTopK) {
      sc[32 + lane] = best;
      sc[32 + kTopK + lane] = 0;
    }
    __syncwarp();
    const int place = ranked_before<32 + kTopK>(sc, key);
    const int down = ranked_before<32>(sc, best);
    if (key != 0 && place < kTopK) sc[32 + kTopK + place] = key;
    if (best != 0 && lane + down < kTopK) sc[32 + kTopK + lane + down] = best;
    __syncwarp();
    best = lane < kTopK ? sc[32 + kTopK + lane] : 0;
  }
  // The warps' lists become the CTA's, in the first CTA of the cluster, the CTAs'
  // the unit's, by the same count.
  if (lane < kTopK) lists[warp][lane] = best;
  __syncthreads();
  cluster.barrier_wait(std::move(started));  // every CTA's shared memory is there
  if (threadIdx.x < kSelWarps * kTopK) {
    const uint64_t x = lists[0][threadIdx.x];
    const int place = ranked_before<kSelWarps * kTopK>(lists[0], x);
    if (x != 0 && place < kTopK) *cluster.map_shared_rank(&from[rank][place], 0) = x;
  }
  const uint64_t* last = from[0];
  if (C > 1) {
    cluster.sync();
    if (rank != 0) return;
    if (threadIdx.x < kTopK) lists[0][threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < C * kTopK; i += kSelThreads) {
      const uint64_t x = from[0][i];
      int place = 0;
      for (int k = 0; k < C; ++k) place += ranked_before<kTopK>(from[k], x);
      if (x != 0 && place < kTopK) lists[0][place] = x;
    }
    last = lists[0];
  }
  __syncthreads();
  if (warp != 0) return;
  const uint64_t top = last[lane & 15];
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

template <int kSelWarps>
cudaError_t launch_select_as(const SelectArgs& a, int cluster, cudaStream_t s) {
  constexpr int kSmem = kSelWarps * kSlabs * kSlabBytes;
  auto kernel = k_paged_select<kSelWarps>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, dim3(unsigned(int64_t(a.table.rows) * a.heads * cluster)),
                        dim3(kSelWarps * 32), kSmem, unsigned(cluster), s, a);
}

cudaError_t launch_paged_select(const SelectArgs& a, cudaStream_t s) {
  // A cluster's CTAs: one for every 128 blocks that the table has room for, while
  // the batch leaves SMs without any (64 rows of up to 1024 blocks: 27.3 us with 1,
  // 21.3 with 2, 22.7 with 4).  Four warps a CTA, four CTAs an SM; batches that would not be on
  // the chip at once so take two warps (256 rows of 64 blocks: 6.1 us, with
  // four 9.0; one row of 1024: 6.4, with four 4.8).
  const int64_t room = ((int64_t(a.table.width) << a.table.shift) + kBlock - 1) / kBlock;
  const int64_t units = int64_t(a.table.rows) * a.heads, sms = device_sm_count();
  int cluster = 1;
  while (cluster < kSelMaxCluster && room > int64_t(cluster) * 128 && units * cluster < 2 * sms)
    cluster *= 2;
  return units * cluster > 4 * sms ? launch_select_as<2>(a, cluster, s)
                                   : launch_select_as<4>(a, cluster, s);
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
  const int slices = (a.heads * a.dim + kIdxSlice - 1) / kIdxSlice;
  // Six CTAs an SM (their shared memory), no more than there can be blocks.
  int64_t most = int64_t(device_sm_count()) * 6 / slices;
  const int64_t blocks = T / kBlock + 2 * int64_t(table->rows);
  if (most > blocks) most = blocks;
  if (most > T) most = T;
  if (most < 1) most = 1;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin("paged_index", s);
  const cudaError_t e = launch_k(true, k_paged_index, dim3(unsigned(most), slices),
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
