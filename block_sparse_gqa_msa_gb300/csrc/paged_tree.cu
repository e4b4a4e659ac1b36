// paged_tree.cu - attention of each row's drafted tokens over the paged cache:
// over the cached keys (all, or each token's blocks) and over the drafted tokens
// on its own path.
//
// Mathematics.  The tokens of a row and the query heads that share a key head
// are the rows of matrix tiles: with n heads a key head and N tokens, N n rows
// against the same keys.  Over tiles of 128 keys, with a running reference m and
// sum l in base 2 (x = scale * log2(e) * <q, k>):
//   P = 2^(x - m), l += sum P, O += P V,
// O and l rescaled when m has to rise (see kMostSum);
// two such states join as M = max(m1, m2), l = l1 2^(m1 - M) + l2 2^(m2 - M), O
// likewise; at the end O / l, lse = ln2 (m + log2 l).  m, l, O are 32 bits; P is
// rounded to the cache's type for the product with V (the tensor cores take
// both in one type), which is off by 2^-8 (bf16) or 2^-11 (fp16) of a weight
// at most, as the output's own rounding is of the output.
//
// What bounds it.  A key and its value are read once for up to 256 rows, 4 * D
// bytes for 4 * D * rows flop: up to 256 rows HBM is the bound (at 6.8 TB/s and
// 1.9 PFLOP/s they meet at 280), beyond that the tensor cores.
//
// Tiles.  A CTA holds two query tiles of 128 rows (slots A and B) against one
// stream of key tiles, so that one slot's softmax runs while the tensor cores
// work for the other: S, softmax, P V and the next S, by turns.  A row
// with more than 256 matrix rows is several such items.  With 128 rows or fewer
// slot B takes the same queries and every other key tile, and the two states
// are joined in tensor memory's lanes at the end; the order of operations is the
// same.
//
// Split.  All items' key tiles, in order, are dealt out in runs of equal cost to the
// CTAs, one an SM; a run's place is found from the lengths on the device.  Items
// are ordered with the number of the 256-row group outermost: CTAs that read the
// same keys for other queries then do so at about the same time, and HBM is read
// once.  An item within one run is finished there; otherwise each run leaves its
// (m, l, O) in the workspace and k_paged_tree_join adds them up, in order.
//
// One warp fetches keys, three tiles ahead (heads of 64 channels: four), one values,
// two (four) tiles ahead, into the swizzled layout that the tensor cores read: from
// pages of 8 tokens or more by tensor copies of up to 64 tokens of a page, a lane
// each (by one lane of a warp that stays together they took as long); from smaller
// pages by copies of 16 bytes.  What lies behind a row's end may be anything: as a key it
// gives a score that a mask drops, as a value it would meet a weight of 0, so value
// rows that are not there are zeroed.  So are infinities and NaN in the values of
// drafted tokens, which not all of the row's tokens see: those that do get them added
// to their results.  (A look at every tile's values would take longer than its copy;
// what all cached tokens' values hold is taken as it is.)
//
// With q2k a first kernel (k_paged_tree_lists) makes, for each item, the list of
// the blocks that any of its tokens chose, and which tokens did.
//
// Measured.  8 rows of 64 tokens behind 12000 to 16384, 16 query heads a key head: 193
// us, 1.26 PFLOP/s; 32 rows of 10 to 32 tokens behind up to 12000: 157 us, 0.92
// PFLOP/s and 2.8 TB/s; 43 rows of 1 to 7 tokens behind up to 9000, heads of 64
// channels, 3 a key head: 95 us, 4.3 TB/s; one row of 8 tokens behind 2900: 22 us.
// A key tile of 128 keys for both slots takes 3500 cycles, 2200 of which the tensor
// cores need for it.  What holds a slot is its own chain: S (900 cycles), the softmax
// (1200), P V (700), and 100 for each barrier between them.
#include <algorithm>

#include "paged.cuh"
#include "sm100.cuh"

namespace msa {

#ifdef MSA_TEST_STARVE
// Test-only build: when set (4), one warp of CTA 0 of k_paged_tree does not tell of its
// part of the first queries, so that bounded waits run out and the call reports
// MSA_ERR_TIMEOUT.  Set by msa_test_starve.
__device__ int g_starve_tree;
cudaError_t test_set_starve_tree(int which) {
  return cudaMemcpyToSymbol(g_starve_tree, &which, sizeof which);
}
#endif

namespace {

constexpr int kNodes = 64;         // drafted tokens of a row
constexpr int kPairRows = 256;     // matrix rows of an item
constexpr int kTileRows = 128;
constexpr int kMaxRuns = 160;      // CTAs: no GB300 has more SMs
// Warps: one a slot that issues products, one that copies keys, one for values, four
// a slot for the softmax.  (With more than 12 a thread would have 128 registers, and
// the softmax's would not do.)
constexpr int kSoftWarps = 8, kCopyWarps = 2;
constexpr int kCopyWarp0 = 2, kSoftWarp0 = kCopyWarp0 + kCopyWarps;
constexpr int kTreeThreads = (kSoftWarp0 + kSoftWarps) * 32;
// Registers of a thread: 168 at launch; the softmax warps take over what the first
// four give up, 128 x 136 + 256 x 184 = 384 x 168: none of the roles spills then (with
// 72 and 216 the warps that issue products do, 32 rows of up to 12000 tokens 163 -> 190
// us).
constexpr int kSoftRegs = 184, kOtherRegs = 136;
// A row's reference m is set by its first tile, kLift below the maximum there.  In
// whole tiles no maximum is formed: m is raised where the weights sum up to more than
// kMostSum; in tiles with masks where the maximum is kRise above.  So the state is
// scaled a few times in a row at most.  bf16 has the range of 32 bits: weights up to
// 2^30 leave sums of 2^30 of them and values up to 2^60 inside it.  fp16 ends at 2^16:
// up to 2^15, and m 7 lower than the maximum so that a key far below it keeps its bits
// (as in paged_decode.cu).
constexpr float kRise = 8.f;
template <typename T>
constexpr float kLift = 0.f;
template <>
constexpr float kLift<__half> = 7.f;
template <typename T>
constexpr float kMostSum = 1073741824.f;
template <>
constexpr float kMostSum<__half> = 32768.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
  const void* q;
  PagedPool k, v;
  PagedTable table;
  const int32_t *offs, *kv_len, *parents, *q2k;
  void* o;
  float* lse;
  int64_t T;
  float scale_log2;     // scale * log2(e)
  int32_t kv_heads, group;
  int32_t layers;       // 256-row groups of the largest row there can be
  int32_t* counts;      // q2k: tiles of each item [layers][rows][kv_heads]
  int32_t* ids;         // q2k: its blocks, ascending (list_base)
  uint64_t* who;        // q2k: the tokens that chose them
  int4* joins;          // of each run that starts inside an item: the item's first
                        // run, its runs, layer row and key head (runs 0: it does not)
  float* part_ml;       // [2 runs][256][2]: m, l
  float* part_o;        // [2 runs][256][dim]
  int32_t box;          // tokens of a tensor copy (a power of two), 0: none are used
};

template <int kDim>
struct TreeShape {
  static constexpr uint32_t kTile = kTileRows * kDim * 2;
  static constexpr uint32_t kKStages = kDim == 128 ? 3 : 4, kVStages = kDim == 128 ? 2 : 4;
  static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = kK + kKStages * kTile;
  static constexpr uint32_t kRest = kV + kVStages * kTile;  // a TreeShared
  static constexpr uint32_t kTmO = 256;  // columns of O_A; O_B kDim further
};

// A row as the kernels see it; n == 0: nothing to attend for.
struct TreeRow {
  int32_t t0, n, len;
};
__device__ __forceinline__ bool row_fits(const TreeArgs& a, int32_t n, int32_t len) {
  return n <= kNodes && len >= 0 && int64_t(len) + n <= (int64_t(a.table.width) << a.table.shift);
}
__device__ __forceinline__ TreeRow tree_row(const TreeArgs& a, int32_t r) {
  const int32_t o0 = a.offs[r], o1 = a.offs[r + 1], len = a.kv_len[r];
  TreeRow v{o0, o1 - o0, len};
  if (o0 < 0 || o1 <= o0 || o1 > a.T || !row_fits(a, o1 - o0, len)) v.n = 0;
  return v;
}
__device__ __forceinline__ int32_t layer_count(const TreeArgs& a, int32_t n) {
  return (n * a.group + kPairRows - 1) / kPairRows;
}
__device__ __forceinline__ int32_t dense_tiles(const TreeRow& w) {
  return int32_t((int64_t(w.len) + w.n + kBlock - 1) / kBlock);
}
// First list entry of an item: 16 for each of its tokens; two items may share
// one token of a row, hence one more for each.
__device__ __forceinline__ int64_t list_base(const TreeArgs& a, int32_t row, int32_t layer,
                                             int32_t g, int32_t t0) {
  const int64_t all = a.T + 4 * int64_t(a.table.rows);
  return (g * all + t0 + layer * kPairRows / a.group + 4 * int64_t(row) + layer) * kTopK;
}

// ------------------------------------------------------------ lists of blocks
constexpr int kListThreads = 256;
constexpr int kHash = 2048;  // places for up to 64 x 16 blocks
__global__ void __launch_bounds__(kListThreads) k_paged_tree_lists(const TreeArgs a) {
  __shared__ int32_t key[kHash];
  __shared__ unsigned long long who[kHash];
  __shared__ int32_t uniq[kNodes * kTopK], place[kNodes * kTopK];
  __shared__ int32_t n_uniq;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < kHash; i += kListThreads) {
    key[i] = -1;
    who[i] = 0;
  }
  if (tid == 0) n_uniq = 0;
  grid_dep_wait();
  grid_dep_release();
  const int32_t item = blockIdx.x;  // (layer * rows + row) * kv_heads + g
  const int32_t g = item % a.kv_heads, row = item / a.kv_heads % a.table.rows;
  const int32_t layer = item / a.kv_heads / a.table.rows;
  const TreeRow w = tree_row(a, row);
  if (layer >= layer_count(a, w.n)) {
    if (tid == 0) a.counts[item] = 0;
    return;
  }
  __syncthreads();
  const int32_t j0 = layer * kPairRows / a.group;
  const int32_t j1 = min(w.n, ((layer + 1) * kPairRows + a.group - 1) / a.group);
  const int32_t blocks = int32_t((int64_t(w.len) + kBlock - 1) / kBlock);
  const int32_t* slots = a.q2k + (int64_t(g) * a.T + w.t0) * kTopK;
  for (int i = j0 * kTopK + tid; i < j1 * kTopK; i += kListThreads) {
    const int32_t v = slots[i];
    if (v == -1) continue;
    if (v < 0 || v >= blocks) {
      raise_paged(a.table.status, MSA_ERR_BAD_Q2K);
      continue;
    }
    // at most half the places fill up, so a free one is found
    uint32_t h = (uint32_t(v) * 2654435761u) >> 21;
    for (;;) {
      const int32_t old = atomicCAS(&key[h], -1, v);
      if (old == -1 || old == v) break;
      h = (h + 1) % kHash;
    }
    atomicOr(&who[h], 1ull << (i / kTopK));
  }
  __syncthreads();
  for (int i = tid; i < kHash; i += kListThreads) {
    const bool used = key[i] >= 0;
    const uint32_t m = __ballot_sync(0xffffffffu, used);
    int32_t at = 0;
    if (lane == 0 && m) at = atomicAdd(&n_uniq, __popc(m));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1));
    if (used) {
      uniq[at] = key[i];
      place[at] = i;
    }
  }
  __syncthreads();
  const int32_t n = n_uniq;
  const int64_t base = list_base(a, row, layer, g, w.t0);
  for (int i = tid; i < n; i += kListThreads) {
    const int32_t v = uniq[i];
    int32_t rank = 0;
    for (int k = 0; k < n; ++k) rank += uniq[k] < v;
    a.ids[base + rank] = v;
    a.who[base + rank] = who[place[i]];
  }
  if (tid == 0) a.counts[item] = n + 1;  // and the drafted tokens' tile
}

// ------------------------------------------------------------ dealing out
// Runs are equal in cost: a key tile costs 8 where both slots work on it, 5 where one
// does (3500 and 2200 cycles), and where there are many tiles to a run an item costs
// kItemCost beside its tiles (its queries, its first and last tile on their own, its
// results; 18 for 34: 43 rows of small trees 102 -> 106 us, 32 rows of up to 12000 tokens
// 160 -> 166).  Where that leaves enough runs, a run has tiles of one item alone: items
// are then rounded up to whole runs of 2^kShort, twice or four times as much.
constexpr int kPairCost = 8, kSplitCost = 5, kItemCost = 34;
constexpr int kManyTiles = 8;
constexpr int kShort = 3, kShorts = 3;
static_assert((1 << kShort) >= kPairCost, "no run is empty");
constexpr int kStretches = kTreeThreads;
struct TreePrefix {
  int32_t at[kStretches];     // the cost of tiles before each of a CTA's stretches of
  int32_t items[kStretches];  // layer rows (layer * rows + row), and the items there
  int4 sums[kTreeThreads / 32];
  int32_t total;
  int32_t item;  // an item's own cost
  int32_t pad;   // log2 of a run's, where items are rounded up to whole runs, or 0
  int32_t runs;
  int32_t each;  // layer rows of a stretch
};
__device__ __forceinline__ int32_t item_rows(const TreeArgs& a, const TreeRow& w, int32_t layer) {
  return min(kPairRows, w.n * a.group - layer * kPairRows);
}
__device__ __forceinline__ int32_t tile_cost(const TreeArgs& a, const TreeRow& w, int32_t layer) {
  return item_rows(a, w, layer) > kTileRows ? kPairCost : kSplitCost;
}
__device__ __forceinline__ int32_t item_tiles(const TreeArgs& a, const TreeRow& w, int32_t lr,
                                              int32_t g) {
  if (a.q2k) return a.counts[int64_t(lr) * a.kv_heads + g];
  return lr / a.table.rows < layer_count(a, w.n) ? dense_tiles(w) : 0;
}
// What an item of so many tiles takes of the runs, its own cost apart.  (kFew: the page
// table says that there are few tiles; else nothing is rounded up.)
template <bool kFew>
__device__ __forceinline__ int32_t item_span(int32_t tiles, int32_t cost, int32_t pad) {
  return !kFew || pad == 0 || tiles == 0 ? tiles * cost : (((tiles - 1) * cost >> pad) + 1) << pad;
}
// The spans and the number of a layer row's items.
template <bool kFew>
__device__ __forceinline__ int2 layer_row_cost(const TreeArgs& a, int32_t lr, int32_t pad) {
  const int32_t layer = lr / a.table.rows;
  const TreeRow w = tree_row(a, lr - layer * a.table.rows);
  if (layer >= layer_count(a, w.n)) return make_int2(0, 0);
  const int32_t cost = tile_cost(a, w, layer);
  if (!a.q2k) return make_int2(item_span<kFew>(dense_tiles(w), cost, pad) * a.kv_heads, a.kv_heads);
  int32_t n = 0;
  for (int32_t g = 0; g < a.kv_heads; ++g) n += item_span<kFew>(item_tiles(a, w, lr, g), cost, pad);
  return make_int2(n, a.kv_heads);
}
template <bool kFew>
__device__ __forceinline__ void make_tree_prefix(const TreeArgs& a, TreePrefix& s, int32_t grid) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int32_t all = a.table.rows * a.layers, threads = blockDim.x;
  const int32_t each = (all + threads - 1) / threads;
  const int32_t r0 = min(all, tid * each), r1 = min(all, r0 + each);
  int32_t pad = 0;
  int2 total;
  auto sum_up = [&]() {
    int2 mine = make_int2(0, 0);
    for (int32_t r = r0; r < r1; ++r) {
      const int2 c = layer_row_cost<kFew>(a, r, pad);
      mine.x += c.x;
      mine.y += c.y;
    }
    int2 incl = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t x = __shfl_up_sync(0xffffffffu, incl.x, o);
      const int32_t y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) {
        incl.x += x;
        incl.y += y;
      }
    }
    if (lane == 31) s.sums[warp] = make_int4(incl.x, incl.y, 0, 0);
    __syncthreads();
    int2 before = make_int2(0, 0);
    total = before;
    for (int w = 0; w < warps; ++w) {
      const int4 v = s.sums[w];
      if (w < warp) {
        before.x += v.x;
        before.y += v.y;
      }
      total.x += v.x;
      total.y += v.y;
    }
    s.at[tid] = before.x + incl.x - mine.x;
    s.items[tid] = before.y + incl.y - mine.y;
  };
  sum_up();
  if (kFew && total.x <= grid << (kShort + kShorts - 1)) {
    // how many runs there would be of each short length
    int32_t n[kShorts] = {};
    for (int32_t r = r0; r < r1; ++r)
#pragma unroll
      for (int k = 0; k < kShorts; ++k) n[k] += layer_row_cost<true>(a, r, kShort + k).x >> (kShort + k);
    __syncthreads();  // the sums are read
#pragma unroll
    for (int k = 0; k < kShorts; ++k) n[k] = __reduce_add_sync(0xffffffffu, n[k]);
    if (lane == 0) s.sums[warp] = make_int4(n[0], n[1], n[2], 0);
    __syncthreads();
    int4 sum = make_int4(0, 0, 0, 0);
    for (int w = 0; w < warps; ++w) {
      sum.x += s.sums[w].x;
      sum.y += s.sums[w].y;
      sum.z += s.sums[w].z;
    }
    pad = sum.x <= grid ? kShort : sum.y <= grid ? kShort + 1 : sum.z <= grid ? kShort + 2 : 0;
    __syncthreads();
    if (pad > 0) sum_up();
  }
  if (tid == 0) {
    const int32_t item = pad == 0 && total.x >= kManyTiles * kPairCost * grid ? kItemCost : 0;
    s.item = item;
    s.pad = pad;
    s.total = total.x + item * total.y;
    // no run shorter than a tile behind an item's own cost, so that none is empty
    s.runs = pad > 0 ? s.total >> pad
                     : min(s.total > 0 ? max(s.total / (kPairCost + item), 1) : 0, grid);
    s.each = each;
  }
  __syncthreads();
}
// Run c: cost run_start(c) to run_start(c + 1), the tiles that begin there.
__device__ __forceinline__ int32_t run_start(const TreePrefix& s, int32_t c) {
  return int32_t(int64_t(s.total) * c / s.runs);
}
__device__ __forceinline__ int32_t run_of(const TreePrefix& s, int32_t at) {
  int32_t c = int32_t(int64_t(at) * s.runs / s.total);
  while (run_start(s, c + 1) <= at) ++c;
  return c;
}

// A walk over the items of a run.  All lanes alike.
template <bool kFew>
struct TreeWalk {
  const TreeArgs& a;
  int32_t lr, g;      // layer row and key head of the item
  int32_t row, layer;
  TreeRow w;
  int32_t tiles;      // of the item
  int32_t cost;       // of a tile
  int32_t own, pad;   // as in the prefix
  int32_t at;         // where the item's first tile begins
  int32_t hi;         // the run's end
  int32_t i0, i1;     // the segment
  __device__ __forceinline__ explicit TreeWalk(const TreeArgs& args) : a(args) {}
  __device__ __forceinline__ void enter_row() {
    layer = lr / a.table.rows;
    row = lr - layer * a.table.rows;
    w = tree_row(a, row);
    cost = tile_cost(a, w, layer);
  }
  __device__ __forceinline__ void end_at() {
    i1 = min(tiles, (hi - at + cost - 1) / cost);
  }
  // The first tile that begins at lo or later; there is one before `end`.
  __device__ __forceinline__ void begin(const TreePrefix& s, int32_t lo, int32_t end) {
    own = s.item;
    pad = s.pad;
    hi = end;
    int a0 = 0, a1 = blockDim.x;  // the last stretch that starts at or before lo
    while (a1 - a0 > 1) {
      const int mid = (a0 + a1) >> 1;
      if (s.at[mid] + own * s.items[mid] <= lo) a0 = mid; else a1 = mid;
    }
    int32_t pos = s.at[a0] + own * s.items[a0];
    const int32_t last = a.table.rows * a.layers - 1;
    for (lr = a0 * s.each; lr < last; ++lr) {
      const int2 c = layer_row_cost<kFew>(a, lr, pad);
      if (pos + c.x + own * c.y > lo) break;
      pos += c.x + own * c.y;
    }
    enter_row();
    for (g = 0;; ++g) {
      tiles = item_tiles(a, w, lr, g);
      at = pos + own;
      pos = at + item_span<kFew>(tiles, cost, pad);
      if (pos > lo || g + 1 == a.kv_heads) break;
    }
    i0 = lo > at ? (lo - at + cost - 1) / cost : 0;
    end_at();
    if (i0 >= i1) next();
  }
  __device__ __forceinline__ bool next() {
    for (;;) {
      at += item_span<kFew>(tiles, cost, pad) + own;  // of the next item
      if (at >= hi) return false;
      if (++g == a.kv_heads) {
        g = 0;
        do {
          if (++lr >= a.table.rows * a.layers) return false;
          enter_row();
        } while (layer >= layer_count(a, w.n));
      }
      tiles = item_tiles(a, w, lr, g);
      i0 = 0;
      end_at();
      if (i1 > 0) return true;
    }
  }
  __device__ __forceinline__ int32_t rows_here() const { return item_rows(a, w, layer); }
};

// ------------------------------------------------------------ the main kernel
constexpr int kMaxStages = 4;
struct TreeBars {
  uint64_t q_full[2], q_empty, k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages],
      v_empty[kMaxStages], s_full[2], p_full[2], o_full[2], o_free[2], ml, part, turn[2][4], fin[2];
};
struct TreeShared {
  TreeBars bars;
  // Keys of a tile whose pages are there.  A ring of 8 tiles: keys are six tiles ahead
  // of a slot's softmax at most (those of the tile after its next wait for its next S).
  uint4 there[8];
  // Drafted tokens of a segment with values that are not finite.  Values are four
  // segments ahead of one whose results are read at most.
  uint64_t odd[8];
  float2 states[2][kTileRows];    // (m, l) of the slots, where they are joined
  uint32_t tmem_base;
  uint32_t filled[2];             // tiles of keys and of values that were copied
  int abort;
};
// The prefix is done with before the first values arrive where it lies.
template <int kDim>
constexpr uint32_t kTreeSmem = TreeShape<kDim>::kRest + sizeof(TreeShared);
static_assert(kTreeSmem<128> <= 227 * 1024, "shared memory of a CTA");
static_assert(sizeof(TreePrefix) <= TreeShape<64>::kTile, "the prefix fits a stage");

__device__ __forceinline__ void cp_async16_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
// First key of an item's tile and the end of its keys.
struct TileKeys {
  int32_t first, end;
  bool drafted;   // it may hold drafted tokens
  uint64_t who;   // q2k: which tokens chose it
};
template <typename Walk>
__device__ __forceinline__ TileKeys tile_keys(const TreeArgs& a, const Walk& s, int64_t base,
                                              int32_t i) {
  if (!a.q2k) {
    const int32_t f = i * kBlock;
    return TileKeys{f, min(f + kBlock, s.w.len + s.w.n), true, ~0ull};
  }
  if (i + 1 == s.tiles)  // (aligned for the copies: cached keys in it are masked)
    return TileKeys{s.w.len & -max(a.box, 1), s.w.len + s.w.n, true, 0ull};
  const int32_t f = a.ids[base + i] * kBlock;
  return TileKeys{f, min(f + kBlock, s.w.len), false, a.who[base + i]};
}

// Offset of 16 bytes of a row in a tile that the tensor cores read.
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (chunk >> 3) * 16384u + row * 128u + (((chunk & 7) ^ (row & 7)) << 4);
}

// The keys of a tile that a row sees: those of the cached tokens, if it chose them,
// and of the drafted ones those on its path.
__device__ __forceinline__ void tile_words(const TileKeys& t, int32_t len, bool chose,
                                           uint64_t path, uint32_t (&w)[4]) {
  const int32_t cached = chose ? min(max(len - t.first, 0), kBlock) : 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int32_t n = cached - 32 * c;
    w[c] = n >= 32 ? ~0u : n > 0 ? (1u << n) - 1 : 0u;
  }
  if (t.drafted && t.end > len) {
    const int32_t off = len - t.first;  // place of drafted token 0
    uint64_t lo = 0, hi = 0;
    if (off <= 0) {
      lo = -off < 64 ? path >> -off : 0;
    } else if (off < 64) {
      lo = path << off;
      hi = path >> (64 - off);
    } else {
      hi = path << (off - 64);
    }
    w[0] |= uint32_t(lo);
    w[1] |= uint32_t(lo >> 32);
    w[2] |= uint32_t(hi);
    w[3] |= uint32_t(hi >> 32);
  }
}

// The copying warps' side, of keys or of values.
template <typename T, int kDim, typename Walk>
struct Copier {
  using S = TreeShape<kDim>;
  static constexpr int kHalves = kDim / 64;  // tensor copies of a box
  const TreeArgs& a;
  const PagedPool& pool;
  const CUtensorMap* map;
  bool values;
  int lane;

  // With boxes: the page of the lane's box of a tile, else of key 32 grp + lane, as the
  // table has it (of some key of the row, if that one is not in it: nothing here waits
  // for the load).
  __device__ __forceinline__ int32_t page(const int32_t* pages, const TileKeys& t, int grp) const {
    const int32_t at = a.box > 0 ? lane / kHalves * a.box : 32 * grp + lane;
    return pages[min(t.first + min(at, kBlock - 1), t.end - 1) >> a.table.shift];
  }
  // Such a page; -1: not one of the pool; kNoKey: the key is not in the row.
  static constexpr int32_t kNoKey = INT32_MIN;
  __device__ __forceinline__ int32_t checked(const TileKeys& t, int32_t p, int grp) const {
    const int32_t at = a.box > 0 ? lane / kHalves * a.box : 32 * grp + lane;
    if (at >= kBlock || t.first + at >= t.end) return kNoKey;
    if (p >= 0 && p < a.table.num_pages) return p;
    if (!values) raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    return -1;
  }
  // Zeros into rows r0 .. r1 - 1 of a tile.
  __device__ __forceinline__ void zero(uint32_t tile, int r0, int r1) const {
    constexpr int kChunks = kDim / 8;
    for (int i = max(r0, 0) * kChunks + lane; i < r1 * kChunks; i += 32)
      st_shared_v4(tile + tile_at(i / kChunks, i % kChunks), 0, 0, 0, 0);
  }
  // Zeros over what is not finite in the drafted tokens' values of a tile.  Returns
  // which tokens had any.
  __device__ __forceinline__ uint64_t clear(const Walk& s, const TileKeys& t, uint32_t tile) const {
    constexpr int kChunks = kDim / 8;
    // all ones in the exponent; one more makes a carry of that
    constexpr uint32_t kExp = kLift<T> == 0.f ? 0x7f807f80u : 0x7c007c00u;
    constexpr uint32_t kOne = kLift<T> == 0.f ? 0x00800080u : 0x04000400u;
    const int off = s.w.len - t.first;  // row of drafted token 0
    const int r0 = max(off, 0), r1 = min(t.end - t.first, kBlock);
    uint32_t had[2] = {0u, 0u};
#pragma unroll 2
    for (int i = r0 * kChunks + lane; i < r1 * kChunks; i += 32) {
      const uint32_t at = tile + tile_at(i / kChunks, i % kChunks);
      uint4 v = ld_shared_v4(at);
      auto carry = [&](uint32_t w) { return ((w & kExp) + kOne) & 0x80008000u; };
      if (carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w)) {
        auto kept = [&](uint32_t w) { return w & ~((carry(w) >> 15) * 0xffffu); };
        st_shared_v4(at, kept(v.x), kept(v.y), kept(v.z), kept(v.w));
        const int j = i / kChunks - off;
        had[j >> 5] |= 1u << (j & 31);
      }
    }
    return uint64_t(__reduce_or_sync(0xffffffffu, had[0])) |
           uint64_t(__reduce_or_sync(0xffffffffu, had[1])) << 32;
  }
  // Fills a tile and has its barrier told when all of it has landed; false: a wait gave
  // up.  p: the lane's page; there: of keys, the mask of those that are; odd: of values,
  // the segment's drafted tokens with some that are not finite.
  __device__ __forceinline__ bool fill(const Walk& s, const int32_t* pages, const TileKeys& t, int32_t p,
                                       uint32_t tile, uint32_t bar, uint4* there, uint64_t& part,
                                       uint32_t& parts, uint64_t* odd,
                                       volatile int* abort_flag) const {
    const int32_t mask = (1 << a.table.shift) - 1;
    const bool drafted = t.drafted && t.end > s.w.len;
    if (a.box > 0) {
      p = checked(t, p, 0);
      const bool bad = __any_sync(0xffffffffu, p == -1);
      const bool mine = p >= 0;
      const int boxes = __popc(__ballot_sync(0xffffffffu, mine)) / kHalves;
      // values of a tile that is not whole, or of drafted tokens: zeros where they belong
      // before it is told of
      const bool rest = values && (t.end - t.first < kBlock || bad || drafted);
      const uint32_t to = rest ? smem_u32(&part) : bar;
      if (!values && lane == 0) *there = make_uint4(~0u, ~0u, ~0u, ~0u);
      if (!values && bad) {
        __syncwarp();
        if (p == -1 && lane % kHalves == 0)
          for (int k = lane / kHalves * a.box, e = k + a.box; k < e; ++k)
            atomicAnd(reinterpret_cast<uint32_t*>(there) + k / 32, ~(1u << (k % 32)));
        __syncwarp();
      }
      if (lane == 0) {
        if (boxes > 0)
          mbar_arrive_expect_tx(to, uint32_t(boxes * a.box) * kDim * 2);
        else
          mbar_arrive(to);
      }
      __syncwarp();
      const int b = lane / kHalves * a.box, half = lane % kHalves;
      if (mine)
        tma_load_4d(tile + half * 16384u + b * 128u, map, to, half * 64, s.g, (t.first + b) & mask,
                    p);
      if (rest) {
        // what no box covers now, the rest of the last one when it is there
        const int end = t.end - t.first, covered = (end + a.box - 1) & -a.box;
        zero(tile, covered, kBlock);
        if (bad) {
          for (int l = 0; l < 32; l += kHalves)
            if (__shfl_sync(0xffffffffu, p, l) == -1)
              zero(tile, l / kHalves * a.box, (l / kHalves + 1) * a.box);
        }
        if (!mbar_wait_warp(to, parts++ & 1, abort_flag)) {
          mbar_wait_drain(to, (parts - 1) & 1);
          return false;
        }
        zero(tile, end, covered);
        if (drafted) {
          if (a.q2k) zero(tile, 0, s.w.len - t.first);
          __syncwarp();
          const uint64_t had = clear(s, t, tile);
          if (lane == 0) *odd |= had;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      }
      return true;
    }
    constexpr int kChunks = kDim / 8, kAtOnce = 32 / kChunks;
    const int sub = lane / kChunks, c = lane % kChunks;
    const T* base = static_cast<const T*>(pool.base) + s.g * pool.head + c * 8;
    for (int grp = 0; grp < kBlock / 32; ++grp) {
      if (grp > 0) p = page(pages, t, grp);
      p = checked(t, p, grp);
      const uint32_t lost = __ballot_sync(0xffffffffu, p == -1);
      if (!values && lane == 0) reinterpret_cast<uint32_t*>(there)[grp] = ~lost;
#pragma unroll 4
      for (int x = 0; x < 32 / kAtOnce; ++x) {
        const int key = x * kAtOnce + sub;
        const int32_t pg = __shfl_sync(0xffffffffu, p, key);
        const int32_t slot = (t.first + 32 * grp + key) & mask;
        cp_async16_zero(tile + tile_at(32 * grp + key, c),
                        pg >= 0 ? base + pg * pool.page + slot * pool.token
                                : static_cast<const T*>(pool.base),
                        pg >= 0);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (values && drafted) {
      __syncwarp();
      const uint64_t had = clear(s, t, tile);
      if (lane == 0) *odd |= had;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    return true;
  }
};

// Tensor memory in the layout of matrix fragments: 16 lanes x 32 columns; thread t
// gets, of each 8 columns, columns 2 (t % 4) and the next of lane t / 4 in r[4 k],
// r[4 k + 1], of lane t / 4 + 8 in the next two.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// P = 2^(s c2 - mref) of one tile row (tensor memory columns [cs, cs + 128) of
// the thread's lane) as pairs of T into pk.  Returns the sum of the 32-bit values.
template <typename T>
__device__ __forceinline__ float tree_row_exp(uint32_t cs, float c2, float mref,
                                              uint32_t (&pk)[64]) {
  const uint64_t cc = f2_pack(__float_as_uint(c2), __float_as_uint(c2));
  const uint64_t nm = f2_pack(__float_as_uint(-mref), __float_as_uint(-mref));
  uint64_t ls[2] = {0ull, 0ull};
  auto expo = [&](const uint32_t (&r)[16], int c) {
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const uint64_t x2 = f2_fma(f2_pack(r[j], r[j + 1]), cc, nm);
      const float p0 = fast_exp2(f2_lo(x2)), p1 = fast_exp2(f2_hi(x2));
      ls[(j >> 1) & 1] =
          f2_add(ls[(j >> 1) & 1], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
      pk[8 * c + (j >> 1)] = Pair<T>::pack(p0, p1);
    }
  };
  // chunk c+1 loads while chunk c is exponentiated
  uint32_t r0[16], r1[16];
  tmem_ld16(cs, r0);
  tmem_ld_wait();
  reg_fence16(r0);
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    tmem_ld16(cs + 16 * c + 16, r1);
    expo(r0, c);
    tmem_ld_wait();
    reg_fence16(r1);
    if (c < 6) tmem_ld16(cs + 16 * c + 32, r0);
    expo(r1, c + 1);
    if (c < 6) {
      tmem_ld_wait();
      reg_fence16(r0);
    }
  }
  const uint64_t s2 = f2_add(ls[0], ls[1]);
  return f2_lo(s2) + f2_hi(s2);
}

// A row's state: reference and sum of weights.
struct RowState {
  float m, l;
};
// The row's largest score.
__device__ __forceinline__ float tree_row_max(uint32_t cs) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld32(cs + 32 * c, r);
    tmem_ld_wait();
    reg_fence32(r);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      m0 = fmax3(m0, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
      m1 = fmax3(m1, __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
    }
  }
  return fmaxf(m0, m1);
}
// The same for tiles with masks (the keys whose bit is not set in words give 0) and
// where the reference has to rise: the maximum first, O (complete up to the slot's step
// before; there is none where `begins`) and the sum scaled, then the weights, stored
// over the scores that have been read.
template <typename T, int kDim>
__device__ __forceinline__ RowState tree_masked_tile(uint32_t cs, uint32_t co,
                                                     const uint32_t (&words)[4], float c2,
                                                     RowState st, bool begins) {
  // (rolled loops: this code runs a few times in a run, and is fetched each time)
  uint32_t w[4] = {words[0], words[1], words[2], words[3]};
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld32(cs + 32 * c, r);
    tmem_ld_wait();
    reg_fence32(r);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = (w[0] >> (j + e)) & 1u ? __uint_as_float(r[j + e]) : -INFINITY;
      m0 = fmax3(m0, x[0], x[1]);
      m1 = fmax3(m1, x[2], x[3]);
    }
    const uint32_t next = w[0];
    w[0] = w[1];
    w[1] = w[2];
    w[2] = w[3];
    w[3] = next;
  }
  const float to = fmaxf(m0, m1) * c2 - kLift<T>;  // (-infinity without keys)
  const bool raise = to > st.m + kRise;
  if (__any_sync(0xffffffffu, raise)) {
    const float f = raise ? fast_exp2(st.m - to) : 1.f;
    st.l *= f;
    if (raise) st.m = to;
    if (!begins) {
#pragma unroll 1
      for (int c = 0; c < kDim / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(co + 32 * c, o);
        tmem_ld_wait();
        reg_fence32(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st32_nc(co + 32 * c, o);
      }
    }
  }
  const float m = st.m == -INFINITY ? 0.f : -st.m;
  const uint64_t cc = f2_pack(__float_as_uint(c2), __float_as_uint(c2));
  const uint64_t nm = f2_pack(__float_as_uint(m), __float_as_uint(m));
  uint64_t ls[2] = {0ull, 0ull};
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32], p[16];
    tmem_ld32(cs + 32 * c, r);
    tmem_ld_wait();
    reg_fence32(r);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint64_t x2 = f2_fma(f2_pack(r[j], r[j + 1]), cc, nm);
      const float p0 = (w[0] >> j) & 1u ? fast_exp2(f2_lo(x2)) : 0.f;
      const float p1 = (w[0] >> j) & 2u ? fast_exp2(f2_hi(x2)) : 0.f;
      ls[(j >> 1) & 1] =
          f2_add(ls[(j >> 1) & 1], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
      p[j >> 1] = Pair<T>::pack(p0, p1);
    }
    tmem_st16(cs + 16 * c, p);
    w[0] = w[1];
    w[1] = w[2];
    w[2] = w[3];
  }
  const uint64_t s2 = f2_add(ls[0], ls[1]);
  st.l += f2_lo(s2) + f2_hi(s2);
  return st;
}

// The tokens on the path of token `node` of a row (bit i: token i), by a warp:
// paths of twice the length six times over.
__device__ __forceinline__ uint64_t path_of(const TreeArgs& a, const TreeRow& w, int node) {
  if (!a.parents) return node >= 63 ? ~0ull : (2ull << node) - 1;
  const int lane = threadIdx.x & 31;
  int up[2];
  uint64_t path[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 32 * h;
    up[h] = j < w.n ? a.parents[w.t0 + j] : -1;
    if (up[h] < -1 || up[h] >= j) {
      raise_paged(a.table.status, MSA_ERR_BAD_TREE);
      up[h] = -1;
    }
    path[h] = 1ull << j;
  }
#pragma unroll 1
  for (int step = 0; step < 6; ++step) {
    uint64_t add[2];
    int further[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t p0 = __shfl_sync(0xffffffffu, path[0], up[h] & 31);
      const uint64_t p1 = __shfl_sync(0xffffffffu, path[1], up[h] & 31);
      const int u0 = __shfl_sync(0xffffffffu, up[0], up[h] & 31);
      const int u1 = __shfl_sync(0xffffffffu, up[1], up[h] & 31);
      add[h] = up[h] < 0 ? 0ull : up[h] < 32 ? p0 : p1;
      further[h] = up[h] < 0 ? -1 : up[h] < 32 ? u0 : u1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      path[h] |= add[h];
      up[h] = further[h];
    }
  }
  const uint64_t p0 = __shfl_sync(0xffffffffu, path[0], node & 31);
  const uint64_t p1 = __shfl_sync(0xffffffffu, path[1], node & 31);
  return node < 32 ? p0 : p1;
}

// Products and their commits by one lane of a warp that stays together: operands
// then live in the registers that all lanes share, from which the tensor cores take
// them.  (With lane 0 alone in a branch an instruction took 80 cycles to issue.)
__device__ __forceinline__ void mma_ss_one(uint32_t one, uint32_t d, uint64_t a, uint64_t b,
                                           uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts_one(uint32_t one, uint32_t d, uint32_t a, uint64_t b,
                                           uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar),
      "r"(one)
      : "memory");
}

// The tensor cores' side of slot x, one warp: S of its first key tile, then P V of a
// tile and S of its next one.  Issuing waits for the tensor cores, and a wait for a
// barrier that is there already takes 100 cycles: with one warp for both slots the
// tensor cores had nothing to do for half of the time, with one each they work for
// one slot while the other's warp waits.
template <typename T, int kDim, typename Walk>
__device__ __forceinline__ void tree_mma_role(const TreeArgs& a, TreeBars& bars, Walk& walk, int x,
                                              uint32_t tmem, uint32_t sbase,
                                              volatile int* abort_flag) {
  using S = TreeShape<kDim>;
  constexpr bool kBf = kLift<T> == 0.f;
  constexpr uint32_t idS = kBf ? idesc_bf16_f32(128, 128, 0, 0) : idesc_f16_f32(128, 128, 0, 0);
  constexpr uint32_t idPV = kBf ? idesc_bf16_f32(128, kDim, 0, 1) : idesc_f16_f32(128, kDim, 0, 1);
  const uint32_t one = (threadIdx.x & 31) == 0;
  auto wait = [&](uint64_t& bar, uint32_t ph) {
    return mbar_wait_warp(smem_u32(&bar), ph & 1, abort_flag);
  };
  const uint64_t dq = sdesc_sw128(sbase + S::kQ, 16u, 1024u);
  const uint64_t dk = sdesc_sw128(sbase + S::kK, 16u, 1024u);
  const uint64_t dv = sdesc_sw128(sbase + S::kV, 16384u, 1024u);
  constexpr uint64_t kStage = S::kTile >> 4;
  const uint32_t to_s = tmem + 128 * x, to_o = tmem + S::kTmO + kDim * x;
  uint32_t nt = 0, np = 0, segs = 0;  // tiles, this slot's P V, segments
  bool ok = true;
  do {
    const bool split = walk.rows_here() <= kTileRows;
    const int tiles = walk.i1 - walk.i0;
    const int step = split ? 2 : 1, first = split ? x : 0;  // the slot's tiles
    const uint64_t bq = dq + (split ? 0 : x) * kStage;
    // a tile's barrier counts both slots; in a tile of one slot that one counts twice
    auto release = [&](uint64_t& bar) {
      commit_one(one, smem_u32(&bar));
      if (split) commit_one(one, smem_u32(&bar));
    };
    auto key_there = [&](int i) -> bool {
      const uint32_t t = nt + i;
      return wait(bars.k_full[t % S::kKStages], t / S::kKStages);
    };
    auto issue_s = [&](int i) {
      const uint32_t t = nt + i, stg = t % S::kKStages;
      const uint64_t bk = dk + stg * kStage;
#pragma unroll
      for (int kk = 0; kk < kDim / 16; ++kk) {
        const uint64_t off = uint64_t((kk >> 2) * 1024 + (kk & 3) * 2);
        mma_ss_one(one, to_s, bq + off, bk + off, idS, kk > 0);
      }
      commit_one(one, smem_u32(&bars.s_full[x]));
      release(bars.k_empty[stg]);
      if (x == 0 && i + step >= tiles) commit_one(one, smem_u32(&bars.q_empty));
    };
    ok = wait(bars.q_full[x], segs) && (!split || wait(bars.q_full[x ^ 1], segs));
    if (ok && first < tiles) {
      ok = key_there(first);
      tc_fence_after();
      if (ok) issue_s(first);
    }
    for (int i = first; ok && i < tiles; i += step) {
      const uint32_t t = nt + i, stg = t % S::kVStages;
      if (i == first && segs > 0 && !wait(bars.o_free[x], segs - 1)) { ok = false; break; }
      // (the next keys have long been there: asked for behind P they cost their wait)
      if (!wait(bars.v_full[stg], t / S::kVStages) ||
          (i + step < tiles && !key_there(i + step)) || !wait(bars.p_full[x], np)) {
        ok = false;
        break;
      }
      ++np;
      tc_fence_after();
      const uint64_t bv = dv + stg * kStage;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts_one(one, to_o, to_s + kk * 8, bv + uint64_t(kk) * 128u, idPV,
                   (kk > 0 || i > first) ? 1u : 0u);
      release(bars.v_empty[stg]);
      // (products of one thread run in order: S may overwrite P)
      if (i + step < tiles)
        issue_s(i + step);
      else
        commit_one(one, smem_u32(&bars.o_full[x]));
    }
    nt += tiles;
    ++segs;
  } while (ok && walk.next());
  commit_one(one, smem_u32(&bars.fin[x]));
  mbar_wait_drain(smem_u32(&bars.fin[x]), 0);
}

template <typename T, int kDim, bool kFew>
__global__ void __launch_bounds__(kTreeThreads, 1)
    k_paged_tree(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v) {
  using S = TreeShape<kDim>;
  extern __shared__ __align__(1024) uint8_t smem[];
  TreeShared& sh = *reinterpret_cast<TreeShared*>(smem + S::kRest);
  TreePrefix& prefix = *reinterpret_cast<TreePrefix*>(smem + S::kV);
  TreeBars& bars = sh.bars;
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sh.abort;
  if (sbase & 1023u) {  // (no static shared memory, so it is aligned: the swizzle needs that)
    if (tid == 0) raise_paged(a.table.status, MSA_ERR_TIMEOUT);
    return;
  }
  if (tid == 0) {
    sh.abort = 0;
    auto init = [](uint64_t& b, uint32_t n) { mbar_init(smem_u32(&b), n); };
    for (int i = 0; i < kMaxStages; ++i) {
      init(bars.k_full[i], 1);
      init(bars.k_empty[i], 2);
      init(bars.v_full[i], 1);
      init(bars.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      init(bars.s_full[i], 1);
      init(bars.p_full[i], 4);
      init(bars.o_full[i], 1);
      init(bars.o_free[i], kSoftWarps);
      init(bars.q_full[i], 4);
      init(bars.fin[i], 1);
    }
    init(bars.ml, kSoftWarps);
    init(bars.part, 1);
    init(bars.q_empty, 1);
    for (int i = 0; i < 8; ++i) init(bars.turn[i >> 2][i & 3], 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sh.tmem_base), 512);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_release();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  if (blockIdx.x == 0) check_offsets(a.offs, a.table.rows, a.T, a.table.status);
  // rows that do not fit: their tokens see nothing
  for (int32_t r = blockIdx.x; r < a.table.rows; r += gridDim.x) {
    const int32_t o0 = a.offs[r], o1 = a.offs[r + 1], len = a.kv_len[r], n = o1 - o0;
    if (o0 < 0 || o1 <= o0 || o1 > a.T || row_fits(a, n, len)) continue;
    if (tid == 0)
      raise_paged(a.table.status, n > kNodes ? MSA_ERR_BAD_TREE : MSA_ERR_BAD_PAGE);
    const int64_t heads = int64_t(a.kv_heads) * a.group;
    uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.o) + o0 * heads * kDim);
    for (int64_t i = tid; i < n * heads * (kDim / 8); i += kTreeThreads)
      o[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = tid; i < n * heads; i += kTreeThreads) a.lse[o0 * heads + i] = -INFINITY;
  }
  make_tree_prefix<kFew>(a, prefix, gridDim.x);
  const int32_t runs = prefix.runs;
  const int32_t run = blockIdx.x;
  TreeWalk<kFew> walk(a);
  if (run < runs) walk.begin(prefix, run_start(prefix, run), run_start(prefix, run + 1));
  // If the run starts inside an item: the item's first run, its runs, layer row and head.
  if (tid == kTreeThreads - 1) {
    int4 join = make_int4(0, 0, 0, 0);
    if (run < runs && walk.i0 > 0) {
      join.x = run_of(prefix, walk.at);
      join.y = run_of(prefix, walk.at + (walk.tiles - 1) * walk.cost) + 1 - join.x;
      join.z = walk.lr;
      join.w = walk.g;
    }
    a.joins[run] = join;
  }
  __syncthreads();  // the prefix is read
  if (run < runs) {
    if (warp < kSoftWarp0) {
      // (one instruction for the group of warps, in front of its roles: PTX asks for that)
      fewer_registers<kOtherRegs>();
      if (warp >= kCopyWarp0) {
        // ---------------- copies: one warp keys, one values
        const bool values = warp != kCopyWarp0;
        const Copier<T, kDim, TreeWalk<kFew>> copy{a, values ? a.v : a.k,
                                                   values ? &map_v : &map_k, values, lane};
        const uint32_t stages = values ? S::kVStages : S::kKStages;
        uint64_t* const full = values ? bars.v_full : bars.k_full;
        uint64_t* const empty = values ? bars.v_empty : bars.k_empty;
        const uint32_t tiles_at = sbase + (values ? S::kV : S::kK);
        uint32_t nt = 0, stage = 0, round = 0, parts = 0, segs = 0;
        bool ok = true;
        do {
          uint64_t* const odd = &sh.odd[segs++ & 7];
          if (values && lane == 0) *odd = 0;
          const int64_t base =
              a.q2k ? list_base(a, walk.row, walk.layer, walk.g, walk.w.t0) : 0;
          TileKeys t = tile_keys(a, walk, base, walk.i0);
          const int32_t* const pages = a.table.pages + walk.row * a.table.stride;
          int32_t page = copy.page(pages, t, 0);
          for (int32_t i = walk.i0; i < walk.i1; ++i, ++nt) {
            // the pages of the next tile, while this one is waited for
            TileKeys t1 = t;
            int32_t page1 = 0;
            if (i + 1 < walk.i1) {
              t1 = tile_keys(a, walk, base, i + 1);
              page1 = copy.page(pages, t1, 0);
            }
            ok = (round == 0 ||
                  mbar_wait_warp(smem_u32(&empty[stage]), (round - 1) & 1, abort_flag)) &&
                 copy.fill(walk, pages, t, page, tiles_at + stage * S::kTile,
                           smem_u32(&full[stage]), &sh.there[nt & 7], bars.part, parts, odd,
                           abort_flag);
            if (!ok) break;
            if (++stage == stages) {
              stage = 0;
              ++round;
            }
            t = t1;
            page = page1;
          }
        } while (ok && walk.next());
        if (lane == 0) sh.filled[values] = nt;
      } else {
        // ---------------- tensor cores
        tree_mma_role<T, kDim>(a, bars, walk, warp, tmem, sbase, abort_flag);
      }
    } else {
      // ---------------- softmax and results of slot x (warps 4-7: A, 8-11: B)
      more_registers<kSoftRegs>();
      const int x = (warp - kSoftWarp0) >> 2, quad = warp & 3;
      const int trow = quad * 32 + lane;  // tile row = lane of tensor memory
      const uint32_t lane_base = uint32_t(quad * 32) << 16;
      const uint32_t cs = tmem + lane_base + 128 * x;
      const uint32_t co = tmem + lane_base + S::kTmO;
      uint32_t nt = 0, nx = 0, segs = 0, joins = 0, no[2] = {0, 0};
      // Where the slots have rows of their own, their warps on one scheduler take turns:
      // side by side both slots would be at their softmax, and then both at the tensor
      // cores.
      int32_t turns = -(1 - x);  // (slot A's first needs no leave)
      auto my_turn = [&]() {
        const int32_t n = turns++;
        return n < 0 || mbar_wait_warp(smem_u32(&bars.turn[x][quad]), n & 1, abort_flag);
      };
      auto pass_turn = [&]() {
        if (lane == 0) mbar_arrive(smem_u32(&bars.turn[x ^ 1][quad]));
      };
      // What the warp knows of its segment.
      bool split, real, used;
      int32_t node, qrow, tiles;
      int64_t base;
      uint64_t path;
      // Enters the walk's segment and fetches its queries, once the products with the
      // ones before them are done: each warp its own rows of its slot's tile, or half of
      // them where both slots have one.
      auto enter = [&](bool was_split) -> bool {
        const int32_t rows = walk.rows_here();
        split = rows <= kTileRows;
        const int32_t m = (split ? 0 : x * kTileRows) + trow;  // matrix row of the item
        real = m < rows;
        used = m - lane < rows;  // a row of the warp is one
        const int32_t mr = walk.layer * kPairRows + (real ? m : 0);
        node = mr / a.group;
        base = a.q2k ? list_base(a, walk.row, walk.layer, walk.g, walk.w.t0) : 0;
        tiles = walk.i1 - walk.i0;
        qrow = (walk.w.t0 + node) * (a.kv_heads * a.group) + walk.g * a.group + mr -
               node * a.group;
        // Slot x's products with its tile are done: its softmax has read them.  Where slot
        // B helps to fill A's tile it waits for A's; after a segment that both had on one
        // tile they have met.
        if (segs > 0 && x == 1 && split && !was_split &&
            !mbar_wait_warp(smem_u32(&bars.q_empty), (segs - 1) & 1, abort_flag))
          return false;
        ++segs;
        constexpr int kChunks = kDim / 8, kAtOnce = 32 / kChunks;
        const int sub = lane / kChunks, c = lane % kChunks;
        const uint32_t tile = sbase + S::kQ + (split ? 0 : x) * S::kTile;
        const T* q = static_cast<const T*>(a.q) + c * 8;
#pragma unroll 4
        for (int i = split ? x * 16 : 0; i < (split ? x * 16 + 16 : 32); i += kAtOnce) {
          const int32_t from = __shfl_sync(0xffffffffu, real ? qrow : -1, i + sub);
          cp_async16_zero(tile + tile_at(quad * 32 + i + sub, c),
                          q + int64_t(max(from, 0)) * kDim, from >= 0);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
#ifdef MSA_TEST_STARVE
        if (!(g_starve_tree == 4 && blockIdx.x == 0 && segs == 1 && warp == kSoftWarp0))
#endif
        if (lane == 0) mbar_arrive(smem_u32(&bars.q_full[x]));
        path = 0;
        // (does the segment reach the drafted tokens?)
        if (a.q2k ? walk.i1 == walk.tiles : int64_t(walk.i1) * kBlock > walk.w.len)
          path = path_of(a, walk.w, node);
        return true;
      };
      bool ok = enter(false), more = true;
      while (ok && more) {
        const int steps = split ? (tiles + 1 - x) / 2 : tiles;
        RowState st{-INFINITY, 0.f};
        for (int k = 0; k < steps; ++k) {
          const int i = split ? 2 * k + x : k;
          const uint32_t t = nt + i;
          const TileKeys tk = tile_keys(a, walk, base, walk.i0 + i);
          const bool chose = real && ((tk.who >> node) & 1);
          // (the turn first: it has come before S, so that its wait costs nothing)
          if ((!split && !my_turn()) ||
              !mbar_wait_warp(smem_u32(&bars.s_full[x]), nx & 1, abort_flag)) {
            ok = false;
            break;
          }
          ++nx;
          if (!used) {  // no row of the warp is one: what P holds there does not matter
            if (!split) pass_turn();
            if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[x]));
            continue;
          }
          tc_fence_after();
          // Tiles of cached keys alone: a row sees all of them or none.  Whether all are there
          // is looked at behind the weights, by when it has been read.
          const uint4 there = sh.there[t & 7];
          auto complete = [&]() { return (there.x & there.y & there.z & there.w) == ~0u; };
          bool plain = tk.first + kBlock <= walk.w.len;
          if (plain && k == 0) {  // the first tile sets the reference
            plain = complete();
            if (plain) {
              const float mx = tree_row_max(cs);
              if (chose) st.m = mx * a.scale_log2 - kLift<T>;
            }
          }
          if (plain) {
            uint32_t pk[64];
            const float ls = tree_row_exp<T>(cs, a.scale_log2, st.m, pk);
            // The sum tells when the reference has to rise (it is infinite where the row
            // has seen no key so far).
            const bool low = ls <= kMostSum<T>;
            if (!__all_sync(0xffffffffu, chose && low && complete())) {
              plain = complete() && !__any_sync(0xffffffffu, chose && !low);
#pragma unroll
              for (int e = 0; e < 64; ++e) pk[e] = chose ? pk[e] : 0u;
            }
            if (plain) {
              if (chose) st.l += ls;
              // P over the first 64 columns of S (all of S has been read)
              tmem_st32_nc(cs, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
              tmem_st32_nc(cs + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
            }
          }
          if (!plain) {
            const uint32_t all = chose ? ~0u : 0u;
            uint32_t words[4] = {all, all, all, all};
            tile_words(tk, walk.w.len, chose, real ? path : 0ull, words);
            words[0] &= there.x;
            words[1] &= there.y;
            words[2] &= there.z;
            words[3] &= there.w;
            st = tree_masked_tile<T, kDim>(cs, co + kDim * x, words, a.scale_log2, st, k == 0);
          }
          if (!split) pass_turn();
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[x]));
        }
        if (!ok) break;
        nt += tiles;
        // ---- results.  Two states of the same rows are joined here, half of the
        // columns by each slot's warps.  The next segment begins before, so that its
        // first products and softmax need not wait for this one's results.
        const bool was_split = split, two = split && tiles > 1;
        const bool whole = walk.i0 == 0 && walk.i1 == walk.tiles;
        // the row's place among the results or the parts, -1: none
        const int32_t place =
            !real ? -1
            : whole ? qrow
                    : (2 * run + (walk.i0 > 0 ? 0 : 1)) * kPairRows + (split ? 0 : x * kTileRows) + trow;
        float M = st.m, l = st.l, f0 = x == 0 ? 1.f : 0.f, f1 = x == 1 ? 1.f : 0.f;
        if (was_split) {
          // the states before these are read (a round of the barrier for writing, one
          // for reading)
          if (joins > 0 && !mbar_wait_warp(smem_u32(&bars.ml), 1, abort_flag)) break;
          sh.states[x][trow] = make_float2(st.m, st.l);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.ml));
          if (!mbar_wait_warp(smem_u32(&bars.ml), 0, abort_flag)) break;
          const float2 s0 = sh.states[0][trow], s1 = sh.states[1][trow];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.ml));
          ++joins;
          M = fmaxf(s0.x, s1.x);
          f0 = s0.x == -INFINITY ? 0.f : fast_exp2(s0.x - M);
          f1 = s1.x == -INFINITY ? 0.f : fast_exp2(s1.x - M);
          l = s0.y * f0 + s1.y * f1;
        }
        const uint64_t was_path = place >= 0 ? path : 0;
        const uint64_t* const odd = &sh.odd[(segs - 1) & 7];
        const int32_t was_row = walk.row, was_g = walk.g, was_len = walk.w.len;
        more = walk.next();
        if (more && !(ok = enter(was_split))) break;
        const bool use0 = was_split || x == 0, use1 = two || (!was_split && x == 1);
        if (use0 && !mbar_wait_warp(smem_u32(&bars.o_full[0]), no[0] & 1, abort_flag)) break;
        if (use1 && !mbar_wait_warp(smem_u32(&bars.o_full[1]), no[1] & 1, abort_flag)) break;
        ++no[0];
        if (two || !was_split) ++no[1];
        tc_fence_after();
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;  // l == 0: no key was seen
          f0 *= inv;
          f1 *= inv;
        }
        const int c0 = was_split ? x * (kDim / 2) : 0, c1 = was_split ? c0 + kDim / 2 : kDim;
#pragma unroll 1
        for (int h = 0; h < 32; h += 16) {  // 16 rows at a time
          float fa[2], fb[2];               // of lane's rows h + lane / 4 and 8 further
          int32_t to[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int src = h + lane / 4 + 8 * e;
            fa[e] = __shfl_sync(0xffffffffu, f0, src);
            fb[e] = __shfl_sync(0xffffffffu, f1, src);
            to[e] = __shfl_sync(0xffffffffu, place, src);
          }
          if (!__any_sync(0xffffffffu, to[0] >= 0 || to[1] >= 0)) continue;
#pragma unroll 1
          for (int c = c0; c < c1; c += 32) {
            uint32_t u[16], v[16];
            if (use0) tmem_ld_frag(co + (uint32_t(h) << 16) + c, u);
            if (use1) tmem_ld_frag(co + (uint32_t(h) << 16) + kDim + c, v);
            tmem_ld_wait();
            reg_fence16(u);
            reg_fence16(v);
            // (4 lanes' stores are a sector of 32 bytes, or half of one)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int64_t at = int64_t(to[e]) * kDim + c + 2 * (lane & 3);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float o[2];
#pragma unroll
                for (int z = 0; z < 2; ++z)
                  o[z] = (use0 ? __uint_as_float(u[4 * k + 2 * e + z]) * fa[e] : 0.f) +
                         (use1 ? __uint_as_float(v[4 * k + 2 * e + z]) * fb[e] : 0.f);
                if (to[e] < 0) continue;
                if (whole)
                  *reinterpret_cast<uint32_t*>(static_cast<T*>(a.o) + at + 8 * k) =
                      Pair<T>::pack(o[0], o[1]);
                else
                  *reinterpret_cast<float2*>(a.part_o + at + 8 * k) = make_float2(o[0], o[1]);
              }
            }
          }
        }
        // Values of drafted tokens on the row's path that are not finite.
        const uint64_t seen = was_path & *odd;
        if (__any_sync(0xffffffffu, seen != 0)) {
          __syncwarp();
          for (uint64_t left = seen; left != 0; left &= left - 1) {
            const int64_t key = int64_t(was_len) + __ffsll(static_cast<long long>(left)) - 1;
            const int32_t page =
                a.table.pages[was_row * a.table.stride + (key >> a.table.shift)];
            if (page < 0 || page >= a.table.num_pages) continue;
            const T* v = static_cast<const T*>(a.v.base) + page * a.v.page + was_g * a.v.head +
                         (key & ((int64_t(1) << a.table.shift) - 1)) * a.v.token;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
              const float add = float(v[c]);
              if (fabsf(add) <= 3.4e38f) continue;
              const int64_t at = int64_t(place) * kDim + c;
              if (whole) {
                T& o = static_cast<T*>(a.o)[at];
                o = T(float(o) + add);
              } else {
                a.part_o[at] += add;
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {  // O_x counts 8: all warps have read both, or slot x's its own
          mbar_arrive(smem_u32(&bars.o_free[x]));
          mbar_arrive(smem_u32(&bars.o_free[was_split ? x ^ 1 : x]));
        }
        if (place >= 0 && (!was_split || x == 0)) {
          if (whole)
            a.lse[place] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
          else
            *reinterpret_cast<float2*>(a.part_ml + int64_t(place) * 2) = make_float2(M, l);
        }
      }
    }
  }
  // ---------------- teardown
  tc_fence_before();
  __syncthreads();
  // (behind the barrier: any of the roles may be the last to give up)
  if (*abort_flag) {
    if (tid == 0) raise_paged(a.table.status, MSA_ERR_TIMEOUT);
    // Tensor copies that nobody has waited for land before the CTA ends: a thread a stage,
    // its last copy.  (With whole warps in turn heads of 64 channels spill registers.)
    const bool values = tid >= kMaxStages;
    const uint32_t stages = values ? S::kVStages : S::kKStages, n = sh.filled[values];
    const uint32_t stage = tid % kMaxStages;
    if (tid < 2 * kMaxStages && stage < stages && stage < n)
      mbar_wait_drain(smem_u32(&(values ? bars.v_full : bars.k_full)[stage]),
                      (n - 1 - stage) / stages & 1);
    __syncwarp();
  }
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ joining runs
// CTAs (x, ..) stand for run x + 1, if that run starts inside an item; the CTAs of an
// item share its rows.  A warp takes kJoinRows rows at a time, its lanes the channels.
// (Where each worked out for itself from the lengths what it joins, that was half of
// its time.)
constexpr int kJoinThreads = 256;
template <typename T, int kDim, int kJoinRows, int kLoads>
__global__ void __launch_bounds__(kJoinThreads) k_paged_tree_join(const TreeArgs a) {
  constexpr int kPer = kDim / 32;
  struct __align__(4 * kPer) Chunk {
    float x[kPer];
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t run = int32_t(blockIdx.x) + 1;
  grid_dep_wait();  // every CTA waits: this grid must not end before the runs
  grid_dep_release();
  const int4 join = a.joins[run];
  const int32_t first = join.x;
  const int n = join.y;
  if (n == 0) return;
  const int32_t layer = join.z / a.table.rows, g = join.w;
  const TreeRow w_row = tree_row(a, join.z - layer * a.table.rows);
  const int32_t rows = item_rows(a, w_row, layer);
  constexpr int kWarps = kJoinThreads / 32;
  const int share = ((run - first - 1) * gridDim.y + blockIdx.y) * kWarps + warp;
  const int shares = (n - 1) * gridDim.y * kWarps;
  for (int32_t m0 = share * kJoinRows; m0 < rows; m0 += shares * kJoinRows) {
    float M[kJoinRows], l[kJoinRows], acc[kJoinRows][kPer] = {};
#pragma unroll
    for (int w = 0; w < kJoinRows; ++w) {
      M[w] = -INFINITY;
      l[w] = 0.f;
    }
    for (int i0 = 0; i0 < n; i0 += kLoads) {
      Chunk o[kJoinRows][kLoads];
      float2 ml[kJoinRows][kLoads];
#pragma unroll
      for (int w = 0; w < kJoinRows; ++w)
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int i = i0 + u;
          ml[w][u] = make_float2(-INFINITY, 0.f);
          o[w][u] = Chunk{};
          if (i < n && m0 + w < rows) {
            const int64_t part =
                (2 * int64_t(first + i) + (i == 0 ? 1 : 0)) * kPairRows + m0 + w;
            ml[w][u] = *reinterpret_cast<const float2*>(a.part_ml + part * 2);
            o[w][u] = reinterpret_cast<const Chunk*>(a.part_o + part * kDim)[lane];
          }
        }
#pragma unroll
      for (int w = 0; w < kJoinRows; ++w)
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const float top = fmaxf(M[w], ml[w][u].x);
          const float f = M[w] == -INFINITY ? 0.f : fast_exp2(M[w] - top);
          const float g = ml[w][u].x == -INFINITY ? 0.f : fast_exp2(ml[w][u].x - top);
          M[w] = top;
          l[w] = l[w] * f + ml[w][u].y * g;
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[w][e] = acc[w][e] * f + o[w][u].x[e] * g;
        }
    }
#pragma unroll
    for (int w = 0; w < kJoinRows; ++w) {
      if (m0 + w >= rows) break;
      const int32_t mr = layer * kPairRows + m0 + w, node = mr / a.group;
      const int64_t orow = (int64_t(w_row.t0) + node) * (a.kv_heads * a.group) + g * a.group + mr -
                           node * a.group;
      const float inv = l[w] == 0.f ? 0.f : 1.f / l[w];
      uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<T*>(a.o) + orow * kDim + lane * kPer);
#pragma unroll
      for (int e = 0; e < kPer; e += 2)
        o[e / 2] = Pair<T>::pack(acc[w][e] * inv, acc[w][e + 1] * inv);
      if (lane == 0) a.lse[orow] = l[w] == 0.f ? -INFINITY : kLn2 * (M[w] + log2f(l[w]));
    }
  }
}

int32_t tree_layers(int64_t T, int32_t group) {
  return int32_t((std::min<int64_t>(T, kNodes) * group + kPairRows - 1) / kPairRows);
}
// Where things lie in the workspace.
struct TreeLayout {
  size_t joins, ml, o, counts, ids, who, total;
  TreeLayout(int32_t rows, int64_t T, int32_t kv_heads, int32_t group, int32_t dim) {
    const size_t lists = size_t(kv_heads) * (size_t(T) + 4 * size_t(rows)) * kTopK;
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t was = at;
      at = align_up(at + n, 256);
      return was;
    };
    joins = take(sizeof(int4) * kMaxRuns);
    ml = take(sizeof(float) * 2 * 2 * kMaxRuns * kPairRows);
    o = take(sizeof(float) * 2 * kMaxRuns * kPairRows * size_t(dim));
    counts = take(sizeof(int32_t) * size_t(tree_layers(T, group)) * rows * kv_heads);
    ids = take(sizeof(int32_t) * lists);
    who = take(sizeof(uint64_t) * lists);
    total = at;
  }
};

}  // namespace
CUresult make_map_pages(CUtensorMap* m, const void* base, bool bf16, int32_t dim, int32_t heads,
                        int32_t page_size, int64_t pages, int64_t head_stride,
                        int64_t token_stride, int64_t page_stride, int32_t rows);  // msa_api.cu
namespace {

template <typename T, int kDim, bool kFew>
cudaError_t launch_tree_as(TreeArgs a, cudaStream_t s) {
  auto kernel = k_paged_tree<T, kDim, kFew>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, kTreeSmem<kDim>, done);
  if (e != cudaSuccess) return e;
  if (a.q2k) {
    launch_begin("paged_tree_lists", s);
    e = launch_k(true, k_paged_tree_lists,
                 dim3(unsigned(int64_t(a.layers) * a.table.rows * a.kv_heads)),
                 dim3(kListThreads), 0, s, a);
    launch_end("paged_tree_lists", s);
    if (e != cudaSuccess) return e;
  }
  // tensor copies where a page holds 8 tokens (whole rows of the swizzle) and a map
  // can be made of the pools
  CUtensorMap map[2] = {};
  const int32_t page_size = 1 << a.table.shift;
  a.box = page_size >= 8 ? std::min(page_size, 64) : 0;
  for (int i = 0; i < 2 && a.box > 0; ++i) {
    const PagedPool& p = i ? a.v : a.k;
    if (make_map_pages(&map[i], p.base, kLift<T> == 0.f, kDim, a.kv_heads, page_size,
                       a.table.num_pages, p.head, p.token, p.page, a.box) != CUDA_SUCCESS)
      a.box = 0;
  }
  const int grid = std::min(device_sm_count(), kMaxRuns);
  launch_begin("paged_tree", s);
  e = launch_k(true, kernel, dim3(unsigned(grid)), dim3(kTreeThreads), kTreeSmem<kDim>, s, a,
               map[0], map[1]);
  launch_end("paged_tree", s);
  if (e != cudaSuccess || grid == 1) return e;
  launch_begin("paged_tree_join", s);
  // A run for each CTA, and with many items (as many as rows and key heads, of so many
  // matrix rows) several CTAs for a run's share of an item's rows, 16 a pass (one row
  // 29.0 us with four CTAs a run, 26.7 with one; 32 rows of up to 12000 tokens 247 us
  // with four and 310 with one).
  const int64_t tokens = (a.T + a.table.rows - 1) / a.table.rows;
  const int64_t rows = int64_t(a.table.rows) * a.kv_heads * std::min<int64_t>(tokens * a.group, kPairRows);
  const int64_t shares = std::min<int64_t>(rows / (grid * 16) + 1, 4);
  // (few items have many parts: eight at a time; many have two or three: more rows at a
  // time, 32 rows of up to 12000 tokens 160 -> 157 us)
  e = launch_k(true, shares == 1 ? k_paged_tree_join<T, kDim, 2, 8> : k_paged_tree_join<T, kDim, 4, 2>,
               dim3(unsigned(grid - 1), unsigned(shares)), dim3(kJoinThreads), 0, s, a);
  launch_end("paged_tree_join", s);
  return e;
}

template <typename T, int kDim>
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  // Few tiles by the table's width: runs of one item alone may do (one row of 2900
  // tokens 29.7 -> 26.5 us; in larger calls the question alone costs 2.5 us).
  const int64_t tiles = (int64_t(a.table.width) << a.table.shift) / kBlock + 2;
  const int64_t most = int64_t(a.layers) * a.table.rows * a.kv_heads * tiles;
  return most <= int64_t(std::min(device_sm_count(), kMaxRuns)) * 8
             ? launch_tree_as<T, kDim, true>(a, s)
             : launch_tree_as<T, kDim, false>(a, s);
}

bool good_tree(const msa_paged_cache* cache, int32_t rows, int64_t T, int32_t q_heads) {
  return rows >= 1 && rows <= kMaxRows && T >= 1 && T <= kMaxTokens && q_heads >= 1 &&
         q_heads % cache->kv_heads == 0 && q_heads / cache->kv_heads <= 16;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_paged_tree_workspace_bytes(const msa_paged_cache* cache, int32_t rows,
                                                     int64_t T, int32_t q_heads, size_t* bytes) {
  const msa_status st = check_cache(cache);
  if (st != MSA_OK) return st;
  if (!bytes || !good_tree(cache, rows, T, q_heads)) return MSA_ERR_INVALID_ARG;
  *bytes = TreeLayout(rows, T, cache->kv_heads, q_heads / cache->kv_heads, cache->head_dim).total;
  return MSA_OK;
}

extern "C" msa_status msa_paged_tree(const msa_paged_cache* cache, const msa_page_table* table,
                                     const int32_t* row_offsets, const int32_t* kv_len,
                                     const int32_t* parents, int64_t T, const void* q,
                                     int32_t q_heads, float softmax_scale, const int32_t* q2k,
                                     void* o, float* lse, void* workspace, size_t workspace_bytes,
                                     msa_stream_t stream) {
  msa_status st = check_cache(cache);
  if (st != MSA_OK) return st;
  st = check_table(table, cache->page_size);
  if (st != MSA_OK) return st;
  if (!row_offsets || !kv_len || !q || !o || !lse || !workspace ||
      !good_tree(cache, table->rows, T, q_heads))
    return MSA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale > 1e30f) return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(q) || !paged_aligned(o) || !paged_aligned(workspace) ||
      !paged_aligned4(row_offsets) || !paged_aligned4(kv_len) || !paged_aligned4(parents) ||
      !paged_aligned4(q2k) || !paged_aligned4(lse))
    return MSA_ERR_ALIGNMENT;
  const int32_t group = q_heads / cache->kv_heads, layers = tree_layers(T, group);
  // tiles and their cost are counted in 32 bits
  if (int64_t(table->rows) * cache->kv_heads * layers * table->width * cache->page_size >
      (int64_t(1) << 34))
    return MSA_ERR_INVALID_ARG;
  const TreeLayout at(table->rows, T, cache->kv_heads, group, cache->head_dim);
  if (workspace_bytes < at.total) return MSA_ERR_WORKSPACE;
  st = check_device();
  if (st != MSA_OK) return st;
  TreeArgs a{};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.q = q;
  a.k = PagedPool{cache->k, cache->k_stride[0], cache->k_stride[1], cache->k_stride[2]};
  a.v = PagedPool{cache->v, cache->v_stride[0], cache->v_stride[1], cache->v_stride[2]};
  a.table = table_args(table, cache->page_size, cache->num_pages, cache->status);
  a.offs = row_offsets;
  a.kv_len = kv_len;
  a.parents = parents;
  a.q2k = q2k;
  a.o = o;
  a.lse = lse;
  a.T = T;
  a.scale_log2 = softmax_scale * kLog2e;
  a.kv_heads = cache->kv_heads;
  a.group = group;
  a.layers = layers;
  a.joins = reinterpret_cast<int4*>(ws + at.joins);
  a.part_ml = reinterpret_cast<float*>(ws + at.ml);
  a.part_o = reinterpret_cast<float*>(ws + at.o);
  a.counts = reinterpret_cast<int32_t*>(ws + at.counts);
  a.ids = reinterpret_cast<int32_t*>(ws + at.ids);
  a.who = reinterpret_cast<uint64_t*>(ws + at.who);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == MSA_BF16)
    e = cache->head_dim == 128 ? launch_tree<__nv_bfloat16, 128>(a, s)
                               : launch_tree<__nv_bfloat16, 64>(a, s);
  else
    e = cache->head_dim == 128 ? launch_tree<__half, 128>(a, s) : launch_tree<__half, 64>(a, s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
