// paged_decode.cu - attention of one new token of each row over the paged
// cache, over all its keys or over the blocks that q2k names.
//
// Mathematics.  For row r and key head g the (up to 16) query heads that
// share g form the 16 rows of one matrix tile.  Over the keys in any order,
// with running maximum m and sum l in base 2 (x = scale * log2(e) * <q, k>):
//   m' = max(m, max x),  l' = l 2^(m-m') + sum 2^(x-m'),
//   O' = O 2^(m-m') + 2^(x-m') V
// (any m' serves that keeps the powers in range, see kLift), and two such states join as M = max(m1, m2), l = l1 2^(m1-M) + l2 2^(m2-M),
// O likewise; at the end O / l and lse = ln2 (m + log2 l).  m, l, O are 32
// bits throughout.  The weights 2^(x-m') enter the product with V as the sum of
// two numbers of the cache's type, the second what rounding to the first leaves
// over (as far as the type's smallest step lets it): with one number O was 0.0021 off (relative, bf16, of
// which the output's own rounding is 0.0017), with two 0.0017, and the second
// product costs 1 % of the time.
//
// What bounds it.  Each key and value is used for 16 query heads at most:
// 4 * 16 * D flop on 4 * D bytes, 16 flop a byte, so HBM is the bound (at 6.8
// TB/s 109 TFLOP/s, which keep the tensor pipe 28 % busy) and the 16-row
// register-level matrix instruction has the right shape: the tile's rows are
// the 16 heads, where a 128-row tensor-memory tile would be seven eighths
// empty.
//
// Split.  A unit is a (row, key head); its keys are cut into tiles of 8 KB a
// warp.  All units' tiles, in order, are dealt out in runs to the CTAs, so a
// batch of any lengths is balanced and a single long row occupies the whole
// chip; a run's place is found from the lengths on the device, so nothing
// comes back to the host.  SMs do not get equal shares of the memory's
// bandwidth (with equal runs they ended 7 % apart), so part of the tiles is
// kept back in short runs, each a CTA of the same grid: a CTA that ends its
// run takes the next short one over from the hardware's queue of CTAs not
// started yet (cluster launch control), in the midst of its copies.  A run is
// cut into segments at unit borders.  A unit that lies within one run is
// finished there; otherwise each run leaves its (m, l, O) in the workspace
// and k_paged_join adds them up, in order: which CTA works on a run changes
// from call to call, the runs and the sums do not.
//
// A warp works alone on its share of each tile (16 keys of 128 channels, 32 of
// 64: 8 KB of keys and values): it fetches them with asynchronous copies into
// its own ring of three stages, across unit and run borders, and waits for
// other warps only where a segment ends.  Two stages are in flight while it
// waits, 128 KB an SM; with the third one filled before the wait as well
// (192 KB) the same calls took 3 % longer, the requests being in each other's
// way.
//
// Measured (bf16, 64 heads on 4, 128 channels): 9 rows of 65536 to 131072
// tokens, all keys, 1.85 GB: 269 to 278 us, 6.6 to 6.9 TB/s, as fast as a
// plain copy (285 without the short runs; 277 or less with head-major pages).
// 128 rows of 500 to 16384 tokens, selected blocks, 508 MB: 89 us, 5.7 TB/s:
// the first bytes come after 4 us, the runs end up to 8 % apart, the join
// takes 3.5 us.  77 rows of up to 12000 tokens, 24 heads on 8 of 64 channels,
// 950 MB: 149 to 165 us, 5.8 to 6.4 TB/s: a head's 128 bytes a token are read
// alone (head-major pages: 147).  One row: 7.0 us for 1000 tokens, 8.8 for 16
// blocks; dependent loads (length and slots, page, keys) and one join in the
// cluster are the time.
#include <cooperative_groups.h>

#include "asked_once.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace msa {
namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kGroup = 16;   // query heads of a matrix tile
// The m of a running state is renewed only when a score is 8 (in base 2) above
// the maximum that it was set by, so the state is scaled a few times in a unit
// and not in most of its first tiles.  m is set kLift below that maximum, so
// weights are up to 2^(8 + kLift), sums of 2^30 of them far inside 32 bits.
// bf16 has the range of 32 bits: 0.  fp16 ends at 2^16 and its half step is
// 2^-25 at least: with m 7 lower a weight of 2^15 still fits, and what a key far
// below the maximum gives is off by 2^-32 of the maximum's weight at most (with
// no lift every key 17.3 nats below was lost from O and not from l, and 131072
// such keys beside one dominant key are 0.4 % of the sum).
constexpr float kRise = 8.f;
template <typename T>
constexpr float kLift = 0.f;
template <>
constexpr float kLift<__half> = 7.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int kDim>
struct DecodeShape {
  static constexpr int kWarpKeys = 2048 / kDim;              // keys of a warp in a tile
  static constexpr int kTileKeys = kDecWarps * kWarpKeys;    // 64 or 128
  static constexpr int kTilesPerBlock = kBlock / kTileKeys;  // 2 or 1
  static constexpr int kRow = kDim * 2;                      // bytes of a key
  static constexpr int kStageBytes = 2 * kWarpKeys * kRow;   // 8 KB
  static constexpr int kStages = 3;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kStateBytes = kGroup * kDim * 4;      // of O in 32 bits
  static_assert(kStateBytes <= kStageBytes, "a warp's state fits a stage");
  static constexpr int kSmem = kDecWarps * kRing;            // 96 KB a CTA
  static constexpr int kSmemCluster = kSmem + kStateBytes;   // 104 KB
};

// Runs of a call: one for each CTA that is on the chip at once (two an SM),
// and as many short ones (a multiple of 4).  The workspace is sized without a
// device: no GB300 has more than 160 SMs.
constexpr int kTailShare = 12;  // one in so many tiles is kept back for the short runs
// In calls of so many tiles a CTA and more (160 rows of 16 blocks, 67 tiles: 115
// us with short runs, 112 without; 77 rows of 64-channel heads, 95: 167 and 173).
constexpr int kTailFrom = 80;
constexpr int kMaxSlots = 160 * 2;
constexpr int kMaxGrid = kMaxSlots * 2;

// Few units that are not long: a cluster of CTAs takes each, and no second
// kernel is needed.
constexpr int kMaxCluster = 8;
constexpr int kClusterTiles = 8;  // of a CTA at most, by the room in the table
constexpr int kSmallUnit = 4;     // tiles of a unit that is not worth dividing

struct DecodeArgs {
  const void* q;
  PagedPool k, v;
  PagedTable table;
  const int32_t* kv_len;
  const int32_t* q2k;  // or null
  void* o;
  float* lse;
  float scale_log2;    // scale * log2(e)
  int32_t kv_heads, group;
  int32_t slots;       // first runs
  int32_t cluster;     // CTAs of a unit, where units are not dealt out in runs
  float* part_ml;      // [2 grid][2][16]: m, l
  float* part_o;       // [2 grid][16][dim]
};

__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4],
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Tiles of one unit of a row of len keys, an upper bound where blocks are
// selected (at least one, so that rows without keys are written too).
template <int kDim>
__device__ __forceinline__ int32_t unit_tiles(int32_t len, bool sparse) {
  using S = DecodeShape<kDim>;
  if (sparse && len > kTopK * kBlock) return kTopK * S::kTilesPerBlock;
  return max(int32_t((int64_t(len) + S::kTileKeys - 1) / S::kTileKeys), 1);
}

// How n tiles are dealt out to runs: by the numbers alone.  The first runs are
// equal.  The short ones shrink in four steps, 7 : 5 : 3 : 1: the CTAs that end
// first take the longest.  No run is empty.
struct Deal {
  int32_t first;    // tiles of the first runs
  int32_t q0, r0;   // a first run's tiles, and how many runs have one more
  int32_t step, e, r1;  // a short run's: 7, 5, 3 or 1 times step, + e, one more for r1 of them
  int32_t c0, runs; // first runs, all runs
  __device__ __forceinline__ Deal(int32_t n, int32_t slots, int32_t grid) {
    const bool tail = grid > slots && n >= slots * kTailFrom;
    first = tail ? n - n / kTailShare : n;
    c0 = min(n, slots);
    runs = tail ? grid : c0;
    q0 = first / c0;
    r0 = first - q0 * c0;
    step = e = r1 = 0;
    if (tail) {
      const int32_t R = runs - c0, rest = n - first;
      step = rest / (4 * R);
      e = (rest - 4 * R * step) / R;
      r1 = rest - 4 * R * step - e * R;
    }
  }
  // First tile of run c (c == runs: the end of the last).
  __device__ __forceinline__ int32_t start(int32_t c) const {
    if (c <= c0) return q0 * c + min(c, r0);
    const int32_t k = c - c0, R4 = (runs - c0) / 4, s = min(k / R4, 3);
    // runs before the step, weighted: 0, 7, 12, 15 times R4
    return first + step * (s * (8 - s) * R4 + (7 - 2 * s) * (k - s * R4)) + e * k + min(k, r1);
  }
};
// The run of c0 .. c1 - 1 that tile t lies in (run c0 starts at or before it).
// A whole warp.
__device__ __forceinline__ int32_t run_of(const Deal& deal, int32_t c0, int32_t c1, int32_t t) {
  const int lane = threadIdx.x & 31;
  while (c1 - c0 > 1) {
    const int32_t step = (c1 - c0 + 31) >> 5, c = c0 + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, c < c1 && deal.start(c) <= t);
    c0 += (__popc(le) - 1) * step;
    c1 = min(c1, c0 + step);
  }
  return c0;
}
static_assert(kTailFrom >= kTailShare, "a tile for every short run");

// What a CTA keeps in shared memory to find the place of a tile: the tiles
// before each of kDecThreads stretches of rows.
struct Prefix {
  int32_t at[kDecThreads];
  int32_t sums[kDecWarps];
  int32_t total;
  int32_t each;  // rows of a stretch
};
__device__ __forceinline__ int32_t checked_len(const DecodeArgs& a, int32_t n) {
  return n < 0 || n > (int64_t(a.table.width) << a.table.shift) ? 0 : n;
}
// A length, in the kernel that starts before its wait from the second level of
// the cache, where those that wrote it have left it.
template <bool kEarly>
__device__ __forceinline__ int32_t length_of(const DecodeArgs& a, int32_t r) {
  return kEarly ? __ldcg(a.kv_len + r) : a.kv_len[r];
}
// Every one of the first kDecThreads threads sums the tiles of a stretch of
// rows; a scan over them.
template <int kDim, bool kEarly>
__device__ __forceinline__ void make_prefix(const DecodeArgs& a, Prefix& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t rows = a.table.rows;
  const int32_t each = (rows + kDecThreads - 1) / kDecThreads;
  const int32_t r0 = min(rows, tid * each), r1 = tid < kDecThreads ? min(rows, r0 + each) : r0;
  int32_t mine = 0;
  for (int32_t r = r0; r < r1; ++r) {
    const int32_t n = length_of<kEarly>(a, r);
    if (checked_len(a, n) != n && blockIdx.x == 0) raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    mine += unit_tiles<kDim>(checked_len(a, n), a.q2k != nullptr) * a.kv_heads;
  }
  int32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31 && warp < kDecWarps) s.sums[warp] = incl;
  __syncthreads();
  int32_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += s.sums[w];
    total += s.sums[w];
  }
  if (tid < kDecThreads) s.at[tid] = before + incl - mine;
  if (tid == 0) {
    s.total = total;
    s.each = each;
  }
  __syncthreads();
}

// A tile's row, its length and the first tile of the row.  A whole warp.
struct RowPlace {
  int32_t row, len, tiles, start;
};
template <int kDim, bool kEarly>
__device__ __forceinline__ RowPlace locate(const DecodeArgs& a, const Prefix& s, int32_t t) {
  const int lane = threadIdx.x & 31;
  const bool sparse = a.q2k != nullptr;
  int k = -1;  // the last stretch that starts at or before t
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w)
    k += __popc(__ballot_sync(0xffffffffu, s.at[w * 32 + lane] <= t));
  RowPlace p;
  p.start = s.at[k];
  if (s.each == 1) {
    p.row = k;
    p.len = checked_len(a, length_of<kEarly>(a, k));
    p.tiles = unit_tiles<kDim>(p.len, sparse);
    return p;
  }
  const int32_t end = min(a.table.rows, (k + 1) * s.each);
#pragma unroll 1
  for (int32_t r0 = k * s.each;; r0 += 32) {
    const int32_t r = r0 + lane;
    const int32_t len = r < end ? checked_len(a, length_of<kEarly>(a, r)) : 0;
    const int32_t tiles = unit_tiles<kDim>(len, sparse);
    const int32_t mine = r < end ? tiles * a.kv_heads : 0;
    int32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, p.start + incl > t);
    if (past || r0 + 32 >= end) {
      const int src = past ? __ffs(past) - 1 : 31;
      p.row = min(r0 + src, end - 1);
      p.len = __shfl_sync(0xffffffffu, len, src);
      p.tiles = __shfl_sync(0xffffffffu, tiles, src);
      p.start += __shfl_sync(0xffffffffu, incl - mine, src);
      return p;
    }
    p.start += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The hardware's queue of CTAs that have not started: a request takes the next
// one off it, whose index arrives in shared memory.
constexpr int kAnswers = 8;
struct Queue {
  uint4 answer[kAnswers];
  uint64_t bar[kAnswers];
};
__device__ __forceinline__ void take_cta(uint32_t answer, uint32_t bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(answer),
      "r"(bar)
      : "memory");
}
// The CTA taken, or -1: there was none left.
__device__ __forceinline__ int32_t taken_cta(uint32_t answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(answer)
      : "memory");
  return ok ? int32_t(x) : -1;
}

// A part of a unit that one CTA works on: its tiles i0 .. i1 - 1.
struct Segment {
  int32_t run, row, head, i0, i1, tiles;
};
struct NextRun {
  int32_t run, row, head, len, tiles, i, n;
};

// The place of run c.
template <int kDim>
__device__ __forceinline__ void find_run(const DecodeArgs& a, const Prefix& prefix,
                                         const Deal& deal, int32_t c, NextRun* next) {
  const int32_t lo = deal.start(c), n = deal.start(c + 1) - lo;
  const RowPlace p = locate<kDim, false>(a, prefix, lo);
  const int32_t h = (lo - p.start) / p.tiles;
  if ((threadIdx.x & 31) == 0)
    *next = NextRun{c, p.row, h, p.len, p.tiles, lo - p.start - h * p.tiles, n};
  __syncwarp();
}
// The answer to the CTA's request number n (1, 2, ..): the run taken, or -1.
__device__ __forceinline__ int32_t await_run(const DecodeArgs& a, Queue* ctas, uint32_t n) {
  const int b = n % kAnswers;
  int32_t c = -1;
  if (mbar_wait_drain(smem_u32(&ctas->bar[b]), ((n - 1) / kAnswers) & 1))
    c = taken_cta(smem_u32(&ctas->answer[b]));
  else
    raise_paged(a.table.status, MSA_ERR_TIMEOUT);
  fence_proxy_async_smem();  // the place is written again by a later request
  return __shfl_sync(0xffffffffu, c, 0);
}
constexpr int kSegQueue = 8;  // the fetch is three tiles, so at most as many segments, ahead
// Tiles before a run's end at which the next one is asked for, and at which its
// place is looked up: each wait on the way is hidden by the tiles in flight.
constexpr int kAskAt = 6;
constexpr int kFindAt = 3;

// The fetching side of a warp: walks the runs' tiles ahead of the sums and
// leaves each segment that it enters in a queue.  All its state is the same
// in all lanes except page and slots.  The warps of a CTA walk the same runs:
// warp 0 asks for the next one, all read the answer.  Answer n sits in place n
// mod 8.  A fetch is three tiles ahead of its warp's sums, and warps meet where
// a segment ends: where warp 0's fetch is in its run n + 8, eight tiles or
// more past run n, its sums are past run n and have met the others' there,
// whose fetches, ahead of their sums, have all read answer n.
template <typename T, int kDim, bool kCluster>
struct Fetch {
  using S = DecodeShape<kDim>;
  static constexpr int kChunks = kDim / 8;          // 16-byte chunks of a key
  static constexpr int kRowsAtOnce = 32 / kChunks;  // keys one copy instruction covers
  static constexpr int kCopies = S::kWarpKeys / kRowsAtOnce;
  static constexpr int kWhole = S::kWarpKeys == 32 ? 5 : 4;  // log2 of a warp's keys
  const DecodeArgs& a;
  int32_t* blocks;   // the unit's blocks (sparse), shared memory
  Segment* queue;
  const Prefix& prefix;
  Queue* ctas;
  NextRun* next;     // shared memory of the warp
  int lane, warp;
  int32_t run;       // the run at hand
  uint32_t n_run;    // runs found
  bool more;         // there may be further runs
  bool asked;        // for the next one
  bool found;        // the next one
  int32_t left;      // tiles of the run after the current segment
  int32_t row, head, len, tiles, i, i1, n_blocks, n_seg;
  int32_t next_len, slots;  // of the next unit, loaded ahead
  int32_t j;         // first key of the warp's part of the tile at hand, -1: none
  int32_t page;      // its page as the table has it, unchecked

  __device__ __forceinline__ void load_slots(int32_t r, int32_t h) {
    if (a.q2k && lane < kTopK && r < a.table.rows)
      slots = a.q2k[(int64_t(h) * a.table.rows + r) * kTopK + lane];
  }
  __device__ __forceinline__ void prefetch_queries(int32_t r, int32_t h) {
    if (lane * 64 < a.group * kDim)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          static_cast<const T*>(a.q) + (int64_t(r) * a.kv_heads + h) * a.group * kDim +
          lane * 64));
  }
  // Enters the unit (row, head) at tile i: its blocks (the distinct valid
  // slots, in slot order, but the row's last block, which may be short, at the
  // end), its place in the queue, and a look ahead.
  __device__ __forceinline__ void enter(bool opens) {
    if (a.q2k) {
      const int32_t nb = int32_t((int64_t(len) + kBlock - 1) / kBlock);
      const int32_t v = slots;
      const bool ok = lane < kTopK && v >= 0 && v < nb;
      if (lane < kTopK && len > 0 && v != -1 && !ok) raise_paged(a.table.status, MSA_ERR_BAD_Q2K);
      const uint32_t same = __match_any_sync(0xffffffffu, ok ? v : -1 - lane);
      const bool keep = ok && (__ffs(same) - 1) == lane;
      const uint32_t m = __ballot_sync(0xffffffffu, keep);
      const uint32_t end = __ballot_sync(0xffffffffu, keep && v == nb - 1);
      n_blocks = __popc(m);
      __syncwarp();  // the list before is read
      if (keep)
        blocks[(end >> lane) & 1 ? n_blocks - 1 : __popc(m & ~end & ((1u << lane) - 1))] = v;
    }
    if (lane == 0) queue[n_seg % kSegQueue] = Segment{run, row, head, i, i1, tiles};
    ++n_seg;
    __syncwarp();
    if (opens) prefetch_queries(row, head);
    if (left > 0) {  // the next unit: its length, slots and queries
      const int32_t r = head + 1 == a.kv_heads ? row + 1 : row;
      const int32_t h = head + 1 == a.kv_heads ? 0 : head + 1;
      next_len = a.kv_len[r];
      load_slots(r, h);
      prefetch_queries(r, h);
    }
  }
  // Before the first tile: the run to begin lies in *next.
  __device__ __forceinline__ void init(bool tail) {
    n_run = 1;
    n_seg = 0;
    more = tail;
    found = true;
    left = 0;
    i = 0;
    i1 = 1;
    j = -1;
  }
  // On to the next tile: of the segment, of the run's next unit, of the next run.
  __device__ __forceinline__ void advance() {
    if (i1 == 0) return;  // nothing is left
    if (++i == i1) {
      const bool opens = left == 0;
      if (opens) {
        if (!found) {
          i1 = 0;
          j = -1;
          return;
        }
        run = next->run;
        row = next->row;
        head = next->head;
        len = next->len;
        tiles = next->tiles;
        i = next->i;
        left = next->n;
        if (!kCluster) load_slots(row, head);  // a cluster's unit is known before its length
        n_blocks = 0;
        asked = found = false;
      } else {
        if (++head == a.kv_heads) {
          head = 0;
          ++row;
          len = checked_len(a, next_len);
          tiles = unit_tiles<kDim>(len, a.q2k != nullptr);
        }
        i = 0;
      }
      i1 = min(tiles, i + left);
      left -= i1 - i;
      enter(opens);
    }
    look();
    if (!more) return;
    const int32_t rest = left + (i1 - i);
    if (!asked && rest <= kAskAt) {
      asked = true;
      const int b = n_run % kAnswers;
      if (warp == 0 && lane == 0) take_cta(smem_u32(&ctas->answer[b]), smem_u32(&ctas->bar[b]));
    }
    if (!found && rest <= kFindAt) {
      const int32_t c = await_run(a, ctas, n_run);
      more = found = c >= 0;
      if (found) {
        ++n_run;
        find_run<kDim>(a, prefix, Deal(prefix.total, a.slots, gridDim.x), c, next);
      }
    }
  }
  // The warp's first key in tile i and its page (loaded, not looked at yet).
  // Where a page holds all the warp's keys every lane loads that page, else
  // lane l the page of key j + l.
  __device__ __forceinline__ void look() {
    j = -1;
    if (a.q2k) {
      const int32_t s = i / S::kTilesPerBlock;
      if (s < n_blocks)
        j = blocks[s] * kBlock + (i % S::kTilesPerBlock) * S::kTileKeys + warp * S::kWarpKeys;
    } else {
      j = i * S::kTileKeys + warp * S::kWarpKeys;
    }
    if (j >= len) j = -1;
    page = -1;
    if (j < 0) return;
    const int32_t* t = a.table.pages + int64_t(row) * a.table.stride;
    if (a.table.shift >= kWhole)
      page = t[j >> a.table.shift];
    else if (lane < S::kWarpKeys && j + lane < len)
      page = t[(j + lane) >> a.table.shift];
  }
  // Starts the copies of the tile at hand into a stage: the keys, then the
  // values; a key's 16-byte chunk c sits at c ^ (key & 7), so that the 8 rows
  // of a matrix load hit different banks.  Keys that are not there become
  // zeros (a masked key's weight is 0, and 0 times what lies there must be 0).
  // Returns the mask of the keys that are there.
  __device__ __forceinline__ uint32_t copy(uint32_t stage) const {
    if (j < 0) return 0;
    const int sub = lane / kChunks, c = lane % kChunks;
    const int mask = (1 << a.table.shift) - 1;
    const T* kb = static_cast<const T*>(a.k.base) + head * a.k.head + c * 8;
    const T* vb = static_cast<const T*>(a.v.base) + head * a.v.head + c * 8;
    constexpr int kValues = S::kWarpKeys * S::kRow;
    if (a.table.shift >= kWhole) {
      if (page < 0 || page >= a.table.num_pages) {
        raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
        return 0;
      }
      const int n = len - j;
      const int64_t slot = (j & mask) + (sub < n ? sub : 0);
      kb += page * a.k.page + slot * a.k.token;
      vb += page * a.v.page + slot * a.v.token;
      const int64_t k_step = a.k.token * kRowsAtOnce, v_step = a.v.token * kRowsAtOnce;
      const uint32_t lane_at = stage + sub * S::kRow + ((c ^ sub) << 4);
#pragma unroll
      for (int x = 0; x < kCopies; ++x) {
        const uint32_t dst =
            (lane_at ^ (((x * kRowsAtOnce) & 7) << 4)) + x * kRowsAtOnce * S::kRow;
        const bool real = x * kRowsAtOnce + sub < n;
        cp_async16_if(dst, kb, real);
        cp_async16_if(dst + kValues, vb, real);
        if ((x + 1) * kRowsAtOnce + sub < n) {  // else nothing is read: a real key's address
          kb += k_step;
          vb += v_step;
        }
      }
      return n >= S::kWarpKeys ? 0xffffffffu >> (32 - S::kWarpKeys) : (1u << n) - 1;
    }
    const bool due = lane < S::kWarpKeys && j + lane < len;
    const bool good = due && page >= 0 && page < a.table.num_pages;
    if (due && !good) raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    const uint32_t there = __ballot_sync(0xffffffffu, good);
#pragma unroll 1
    for (int x = 0; x < kCopies; ++x) {
      const int key = x * kRowsAtOnce + sub;
      const int32_t p = __shfl_sync(0xffffffffu, good ? page : -1, key);
      const uint32_t dst = stage + key * S::kRow + ((c ^ (key & 7)) << 4);
      const int64_t slot = (j + key) & mask;
      cp_async16_if(dst, p >= 0 ? kb + p * a.k.page + slot * a.k.token : a.k.base, p >= 0);
      cp_async16_if(dst + kValues, p >= 0 ? vb + p * a.v.page + slot * a.v.token : a.v.base,
                    p >= 0);
    }
    return there;
  }
};

// kCluster: a cluster of CTAs takes one unit, in equal parts, and joins them in
// its shared memory.
template <typename T, int kDim, bool kCluster>
__global__ void __launch_bounds__(kDecThreads, 2) k_paged_decode(const DecodeArgs a) {
  using S = DecodeShape<kDim>;
  constexpr int kSteps = kDim / 16;            // k-steps of the first product
  constexpr int kCols = kDim / 8;              // column tiles of the second
  constexpr int kKeyTiles = S::kWarpKeys / 8;  // column tiles of the first
  constexpr uint32_t kAllSeen = 0xffffffffu >> (32 - S::kWarpKeys);
  extern __shared__ __align__(256) uint8_t smem[];  // rows of keys begin on their own size
  __shared__ Prefix prefix;
  __shared__ Queue ctas;
  __shared__ NextRun next[kDecWarps];
  __shared__ int32_t blocks[kDecWarps][kTopK];
  __shared__ Segment queue[kDecWarps][kSegQueue];
  __shared__ float ml[2][kDecWarps][kGroup];
  __shared__ float state_ml[2][kGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r_lo = lane >> 2;  // the lane's matrix rows: r_lo and r_lo + 8
  const int col = (lane & 3) * 2;
  const uint32_t ring = smem_u32(smem) + warp * S::kRing;
  [[maybe_unused]] float* state = reinterpret_cast<float*>(smem + S::kSmem);  // the CTA's part (cluster)
  Fetch<T, kDim, kCluster> fetch{a, blocks[warp], queue[warp], prefix, &ctas, &next[warp], lane, warp};
  if (!kCluster && tid == 0) {
    for (int i = 0; i < kAnswers; ++i) mbar_init(smem_u32(&ctas.bar[i]), 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  grid_dep_release();
  bool tail = false;
  if constexpr (kCluster) {
    const int rank = blockIdx.x % a.cluster;
    const int32_t unit = blockIdx.x / a.cluster;
    const int32_t row = unit / a.kv_heads, n = a.kv_len[row];
    fetch.load_slots(row, unit % a.kv_heads);
    const int32_t len = checked_len(a, n);
    if (n != len && tid == 0) raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    const int32_t tiles = unit_tiles<kDim>(len, a.q2k != nullptr);
    const int32_t i0 = int32_t(int64_t(tiles) * rank / a.cluster);
    const int32_t i1 = int32_t(int64_t(tiles) * (rank + 1) / a.cluster);
    if (lane == 0) next[warp] = NextRun{0, row, unit % a.kv_heads, len, tiles, i0, i1 - i0};
    __syncwarp();
  } else {
    make_prefix<kDim, false>(a, prefix);
    const Deal deal(prefix.total, a.slots, gridDim.x);
    if (blockIdx.x >= deal.runs) return;
    tail = deal.runs > deal.c0;
    find_run<kDim>(a, prefix, deal, blockIdx.x, &next[warp]);
  }

  fetch.init(tail);
  [[maybe_unused]] const bool idle = next[warp].n == 0;  // (only in a cluster)

  uint32_t qa[kSteps][4];           // the query heads as the left operand
  float acc[kCols][4];              // O
  float m0, m1, l0, l1;
  uint32_t there[S::kStages - 1] = {};  // of the tiles in flight: the keys that are there
  Segment g;
  int seg = 0;
  int32_t left = 0;                 // tiles of the segment
  int stage = 0;
  // A step starts the copies of the tile kStages - 1 further, into the stage that
  // the last step has freed, then works on its own tile.  The first steps only
  // fill the ring (the very first has no tile yet: the run is begun in it).
  int fill = S::kStages;
#pragma unroll 1
  while (!kCluster || !idle) {
    const uint32_t kb = ring + stage * S::kStageBytes, vb = kb + S::kWarpKeys * S::kRow;
    const uint32_t seen = there[0];
    if (fill == 0 && left == 0) {  // the next segment; heads past the group are zeros
      g = queue[warp][seg % kSegQueue];
      left = g.i1 - g.i0;
      const T* q = static_cast<const T*>(a.q) +
                   (int64_t(g.row) * a.kv_heads + g.head) * a.group * kDim + col;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint32_t* lo = reinterpret_cast<const uint32_t*>(q + r_lo * kDim + s * 16);
        const uint32_t* hi = reinterpret_cast<const uint32_t*>(q + (r_lo + 8) * kDim + s * 16);
        qa[s][0] = r_lo < a.group ? lo[0] : 0;
        qa[s][1] = r_lo + 8 < a.group ? hi[0] : 0;
        qa[s][2] = r_lo < a.group ? lo[4] : 0;
        qa[s][3] = r_lo + 8 < a.group ? hi[4] : 0;
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    if (fill == 0) cp_async_wait<S::kStages - 2>();
    __syncwarp();
    {
      const int free = stage == 0 ? S::kStages - 1 : stage - 1;
#pragma unroll
      for (int s = 0; s + 1 < S::kStages - 1; ++s) there[s] = there[s + 1];
      there[S::kStages - 2] = fetch.copy(ring + free * S::kStageBytes);
      cp_async_commit();
      fetch.advance();
    }
    if (fill == 0 && seen != 0) {
      float x[kKeyTiles][4];
#pragma unroll
      for (int n = 0; n < kKeyTiles; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
      for (int n = 0; n < kKeyTiles; n += 2) {
        // matrices: keys 0-7 / 8-15 by channels 0-7 / 8-15 of the step
        const int key = n * 8 + (lane & 7) + ((lane >> 4) << 3);
        const uint32_t at = kb + key * S::kRow + ((((lane >> 3) & 1) ^ (key & 7)) << 4);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b[4];
          ldsm4(b, at ^ (k << 5));
          mma16816<T>(x[n], qa[k], b[0], b[1]);
          mma16816<T>(x[n + 1], qa[k], b[2], b[3]);
        }
      }
      // Scores and maxima; base 2 comes with the scale.
      if (seen != kAllSeen) {
#pragma unroll
        for (int n = 0; n < kKeyTiles; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((seen >> (n * 8 + col + (e & 1))) & 1)) x[n][e] = -INFINITY;
      }
      float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
      for (int n = 0; n < kKeyTiles; ++n) {
        top0 = fmaxf(top0, fmaxf(x[n][0], x[n][1]));
        top1 = fmaxf(top1, fmaxf(x[n][2], x[n][3]));
      }
      top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
      top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
      top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 2)) * a.scale_log2;
      top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 2)) * a.scale_log2;
      constexpr float kAbove = kLift<T> + kRise;
      if (__any_sync(0xffffffffu, top0 > m0 + kAbove || top1 > m1 + kAbove)) {
        const float n0 = fmaxf(m0, top0 - kLift<T>), n1 = fmaxf(m1, top1 - kLift<T>);
        const float f0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
        const float f1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          acc[n][0] *= f0;
          acc[n][1] *= f0;
          acc[n][2] *= f1;
          acc[n][3] *= f1;
        }
      }
      const float z0 = m0 == -INFINITY ? 0.f : -m0, z1 = m1 == -INFINITY ? 0.f : -m1;
#pragma unroll
      for (int n = 0; n < kKeyTiles; ++n) {
        x[n][0] = fast_exp2(fmaf(x[n][0], a.scale_log2, z0));
        x[n][1] = fast_exp2(fmaf(x[n][1], a.scale_log2, z0));
        x[n][2] = fast_exp2(fmaf(x[n][2], a.scale_log2, z1));
        x[n][3] = fast_exp2(fmaf(x[n][3], a.scale_log2, z1));
        l0 += x[n][0] + x[n][1];
        l1 += x[n][2] + x[n][3];
      }
#pragma unroll
      for (int k = 0; k < kKeyTiles; k += 2) {
        // weights as two numbers of the cache's type, the second what the first leaves
        uint32_t pa[4], pb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = x[k + (e >> 1)][(e & 1) * 2], v = x[k + (e >> 1)][(e & 1) * 2 + 1];
          pa[e] = Pair<T>::pack(u, v);
          const float2 r = Pair<T>::unpack(pa[e]);
          pb[e] = Pair<T>::pack(u - r.x, v - r.y);
        }
        // matrices: keys 0-7 / 8-15 by channels 0-7 / 8-15 of the pair of column tiles
        const int key = k * 8 + (lane & 15);
        const uint32_t at = vb + key * S::kRow + (((lane >> 4) ^ (key & 7)) << 4);
#pragma unroll
        for (int n = 0; n < kCols; n += 2) {
          uint32_t b[4];
          ldsm4_t(b, at ^ (n << 4));
          mma16816<T>(acc[n], pa, b[0], b[1]);
          mma16816<T>(acc[n + 1], pa, b[2], b[3]);
          mma16816<T>(acc[n], pb, b[0], b[1]);
          mma16816<T>(acc[n + 1], pb, b[2], b[3]);
        }
      }
    }
    const int worked = stage;
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
    if (fill > 0) {
      --fill;
      continue;
    }
    if (--left > 0) continue;

    // ---- the segment's end: join the warps.  Each leaves its state in the stage
    // that it has just worked on, which the next step fills: a row's 16-byte
    // piece p sits at p ^ (2 (row & 3)), so that 4 rows' writes hit all banks.
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if ((lane & 3) == 0) {
      ml[0][warp][r_lo] = m0;
      ml[0][warp][r_lo + 8] = m1;
      ml[1][warp][r_lo] = l0;
      ml[1][warp][r_lo + 8] = l1;
    }
    uint8_t* const states = smem + worked * S::kStageBytes;  // the warps', kRing apart
    {
      float* mine = reinterpret_cast<float*>(states + warp * S::kRing) + (col & 2);
      const int swz = (r_lo & 3) << 1;
      __syncwarp();  // the stage is read
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        const int at = ((2 * n + (col >> 2)) ^ swz) * 4;
        *reinterpret_cast<float2*>(mine + r_lo * kDim + at) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2*>(mine + (r_lo + 8) * kDim + at) =
            make_float2(acc[n][2], acc[n][3]);
      }
    }
    __syncthreads();
    const bool whole = !kCluster && g.i0 == 0 && g.i1 == g.tiles;
    const int64_t slot = 2 * int64_t(g.run) + (g.i0 > 0 ? 0 : 1);
    const int64_t unit = int64_t(g.row) * a.kv_heads + g.head;
    const int h = tid / 8;  // the thread's row of the result, 4 channels of each 32
    float M = -INFINITY, l = 0.f, f[kDecWarps];
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ml[0][w][h]);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float m = ml[0][w][h];
      f[w] = m == -INFINITY ? 0.f : fast_exp2(m - M);
      l += ml[1][w][h] * f[w];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // l == 0: no key was seen
#pragma unroll
    for (int c = 0; c < kDim / 32; ++c) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(
            states + w * S::kRing + h * (kDim * 4) + ((c * 8 + tid % 8) ^ ((h & 3) << 1)) * 16);
        v.x += u.x * f[w];
        v.y += u.y * f[w];
        v.z += u.z * f[w];
        v.w += u.w * f[w];
      }
      const int ch = c * 32 + (tid % 8) * 4;
      if (kCluster)
        *reinterpret_cast<float4*>(state + h * kDim + ch) = v;
      else if (!whole)
        *reinterpret_cast<float4*>(a.part_o + (slot * kGroup + h) * kDim + ch) = v;
      else if (h < a.group)
        *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + (unit * a.group + h) * kDim + ch) =
            make_uint2(Pair<T>::pack(v.x * inv, v.y * inv), Pair<T>::pack(v.z * inv, v.w * inv));
    }
    if (tid % 8 == 0) {
      if (kCluster) {
        state_ml[0][h] = M;
        state_ml[1][h] = l;
      } else if (!whole) {
        a.part_ml[slot * (2 * kGroup) + h] = M;
        a.part_ml[slot * (2 * kGroup) + kGroup + h] = l;
      } else if (h < a.group) {
        a.lse[unit * a.group + h] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
      }
    }
    __syncthreads();  // the states are read
    if (++seg == fetch.n_seg) break;  // the fetch is ahead: it would have entered the next one
  }
  cp_async_wait<0>();
  if constexpr (kCluster) {
    // Every CTA joins the parts of its share of the results, a thread 4 channels.
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    if (idle) {
      for (int e = tid; e < kGroup * kDim; e += kDecThreads) state[e] = 0.f;
      if (tid < kGroup) {
        state_ml[0][tid] = -INFINITY;
        state_ml[1][tid] = 0.f;
      }
    }
    cluster.sync();
    for (int it = int(cluster.block_rank()) * kDecThreads + tid; it < kGroup * (kDim / 4);
         it += a.cluster * kDecThreads) {
      const int h = it / (kDim / 4), ch = it % (kDim / 4) * 4;
      float pm[kMaxCluster], pl[kMaxCluster], M = -INFINITY;
      float4 po[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (c < a.cluster) {
          pm[c] = *cluster.map_shared_rank(&state_ml[0][h], c);
          pl[c] = *cluster.map_shared_rank(&state_ml[1][h], c);
          po[c] = *reinterpret_cast<const float4*>(
              cluster.map_shared_rank(state + h * kDim + ch, c));
          M = fmaxf(M, pm[c]);
        }
      }
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (c < a.cluster) {
          const float f = pm[c] == -INFINITY ? 0.f : fast_exp2(pm[c] - M);
          l += pl[c] * f;
          o.x += po[c].x * f;
          o.y += po[c].y * f;
          o.z += po[c].z * f;
          o.w += po[c].w * f;
        }
      }
      if (h < a.group) {
        const int64_t out = int64_t(blockIdx.x / a.cluster) * a.group + h;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + out * kDim + ch) =
            make_uint2(Pair<T>::pack(o.x * inv, o.y * inv), Pair<T>::pack(o.z * inv, o.w * inv));
        if (ch == 0) a.lse[out] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
      }
    }
    cluster.sync();  // nobody reads this CTA's state any more
  }
}

// Joins the parts of the units that several runs share.  CTA x stands for run
// x + 1, if that run starts inside a unit; the CTAs of one unit share its
// heads.  A warp works on a head, alone or with others that take the head's
// parts in turn, its lanes over the channels: the parts' states are merged as
// the keys' were, then the warps'.  With few rows this kernel is a good part of
// the call's time, so all that follows from the lengths is worked out before
// the wait for the runs' end.  (The lengths are there: k_paged_decode lets this
// kernel start after its own wait for what came before.)
template <typename T, int kDim, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32, 48 / kJoinWarps) k_paged_join(const DecodeArgs a) {
  constexpr int kPer = kDim / 32;
  constexpr int kLoads = 4;
  struct __align__(4 * kPer) Chunk {
    float x[kPer];
  };
  __shared__ Chunk so[kJoinWarps][32];
  __shared__ float sm[kJoinWarps], sl[kJoinWarps];
  __shared__ Prefix prefix;
  __shared__ int32_t s_first, s_parts, s_unit;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t run = int32_t(blockIdx.x) + 1;
  make_prefix<kDim, true>(a, prefix);
  if (warp == 0) {
    const Deal deal(prefix.total, a.slots, int32_t(gridDim.x) + 1);
    int32_t first = 0, parts = 0, unit = 0;
    if (run < deal.runs) {
      const int32_t lo = deal.start(run);
      const RowPlace p = locate<kDim, true>(a, prefix, lo);
      const int32_t head = (lo - p.start) / p.tiles, u0 = p.start + head * p.tiles;
      if (u0 < lo) {  // the run starts inside the unit
        unit = p.row * a.kv_heads + head;
        first = run_of(deal, 0, run, u0);
        parts = run_of(deal, run, deal.runs, u0 + p.tiles - 1) + 1 - first;
      }
    }
    if (lane == 0) {
      s_first = first;
      s_parts = parts;
      s_unit = unit;
    }
  }
  __syncthreads();
  const int32_t first = s_first;  // the run that the unit starts in
  const int n = s_parts;          // parts; n - 1 CTAs
  grid_dep_wait();  // every CTA waits: this grid must not end before the runs
  grid_dep_release();
  if (n == 0) return;
  int shares = 1;                  // of the 16 heads
  while (shares < kGroup && 2 * shares <= n - 1) shares *= 2;
  const int share = run - first - 1;
  if (share >= shares) return;
  const int heads = kGroup / shares;    // of this CTA
  const int ways = max(kJoinWarps / heads, 1);  // warps of a head
  const int way = warp % ways;
  // (one pass, but where few warps have all heads)
  for (int h = share * heads + warp / ways; h < (share + 1) * heads; h += kJoinWarps) {
    // part 0: the run that the unit starts in; then the runs that start inside it
    float M = -INFINITY, l = 0.f, acc[kPer] = {};
    for (int i0 = way; i0 < n; i0 += kLoads * ways) {
      Chunk o[kLoads];
      float m[kLoads], pl[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int i = i0 + u * ways;
        m[u] = -INFINITY;
        pl[u] = 0.f;
        o[u] = Chunk{};
        if (i < n) {
          const int32_t s = 2 * (first + i) + (i == 0 ? 1 : 0);
          m[u] = a.part_ml[s * (2 * kGroup) + h];
          pl[u] = a.part_ml[s * (2 * kGroup) + kGroup + h];
          o[u] = reinterpret_cast<const Chunk*>(a.part_o + (s * kGroup + h) * kDim)[lane];
        }
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const float top = fmaxf(M, m[u]);
        const float f = M == -INFINITY ? 0.f : fast_exp2(M - top);
        const float g = m[u] == -INFINITY ? 0.f : fast_exp2(m[u] - top);
        M = top;
        l = l * f + pl[u] * g;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * f + o[u].x[e] * g;
      }
    }
    if (ways > 1) {
      Chunk mine;
#pragma unroll
      for (int e = 0; e < kPer; ++e) mine.x[e] = acc[e];
      so[warp][lane] = mine;
      if (lane == 0) {
        sm[warp] = M;
        sl[warp] = l;
      }
      __syncthreads();
      if (way != 0) return;
      // a lane a way's state, then the ways' sums with their weights
      const float mw = lane < ways ? sm[warp + lane] : -INFINITY;
      M = mw;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
      l = lane < ways ? sl[warp + lane] * f : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll
      for (int w0 = 0; w0 < kJoinWarps; w0 += 4) {
        if (w0 >= ways) break;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float g = __shfl_sync(0xffffffffu, f, w0 + u);  // 0 past the ways
          const Chunk o = so[min(warp + w0 + u, kJoinWarps - 1)][lane];
          if (w0 + u < ways) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] += o.x[e] * g;
          }
        }
      }
    }
    if (h >= a.group) return;
    const int64_t out = int64_t(s_unit) * a.group + h;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<T*>(a.o) + out * kDim + lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) o[e / 2] = Pair<T>::pack(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0) a.lse[out] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
  }
}

size_t decode_workspace(int32_t dim) {
  return sizeof(float) * 2 * kMaxGrid * (2 * kGroup + kGroup * size_t(dim));
}

// Clusters of this kernel that fit on the chip at once (GPCs of unlike size
// leave SMs over), asked for once a device and size.
template <typename T, int kDim>
int cluster_room(void (*kernel)(DecodeArgs), int cluster) {
  static AskedOnce<64, kMaxCluster> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return known.get(dev, cluster - 1, [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(cluster));
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = DecodeShape<kDim>::kSmemCluster;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(cluster);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
    cudaGetLastError();  // no room known: no clusters
    return -1;
  });
}

template <typename T, int kDim>
cudaError_t launch_decode(DecodeArgs a, cudaStream_t s) {
  using S = DecodeShape<kDim>;
  a.slots = device_sm_count() * 2;
  if (a.slots > kMaxSlots) a.slots = kMaxSlots;
  // What the room in the table allows: the lengths are on the device.  A table much
  // wider than its rows need sends few short rows without blocks through runs and a
  // join (one row of 1000 tokens 7.1 us, 8.2 with a table for 131072; 9 rows of up
  // to 300 tokens 7.2 and 8.8; 8 rows of up to 2048 10.0 and 11.9); selected
  // blocks are 16 a row at most, and larger batches take runs in any case.
  int64_t unit = (int64_t(a.table.width) << a.table.shift) / S::kTileKeys + 1;
  if (a.q2k && unit > kTopK * S::kTilesPerBlock) unit = kTopK * S::kTilesPerBlock;
  const int64_t units = int64_t(a.table.rows) * a.kv_heads;
  // Clusters: as many CTAs a unit as the chip has room for at once, 8 at most.
  // Blocks make units of like length; units of all keys may differ, so those
  // must be short.  Whole units for CTAs pay only if they nearly fill the chip,
  // and a second wave of clusters never does (64 heads on 4, 128 channels,
  // selected blocks, with clusters / with runs and a join: 9 rows, clusters of 7,
  // 13.9 / 19 us; 24 rows, of 3, 23.7 / 28.4; 32 rows, of 2, 29.8 / 34.0; 76 rows,
  // of 1, 56 / 60; but 48 rows, of 1, 49 / 44, and 128 rows, of 1, 100 / 93).
  // Clusters of 8 near the room there is get in one another's way.
  auto clustered = k_paged_decode<T, kDim, true>;
  static std::atomic<uint64_t> done_c{0};
  cudaError_t e = allow_smem(clustered, S::kSmemCluster, done_c);
  if (e != cudaSuccess) return e;
  int cluster = kMaxCluster;
  while (cluster > 1 &&
         (unit < 2 * cluster ||
          units * cluster * 8 > a.slots * (cluster == kMaxCluster ? 7 : 8) ||
          units > cluster_room<T, kDim>(clustered, cluster)))
    --cluster;
  const bool fits = cluster > 1 || (units <= a.slots && (unit <= kSmallUnit ||
                                                         units * 4 >= a.slots * 3));
  if (fits && unit <= cluster * (a.q2k ? kTopK * S::kTilesPerBlock : kClusterTiles)) {
    a.cluster = cluster;
    launch_begin("paged_decode", s);
    e = launch_cluster(clustered, dim3(unsigned(units * cluster)), dim3(kDecThreads),
                       S::kSmemCluster, unsigned(cluster), s, a);
    launch_end("paged_decode", s);
    return e;
  }
  auto kernel = k_paged_decode<T, kDim, false>;
  static std::atomic<uint64_t> done{0};
  e = allow_smem(kernel, S::kSmem, done);
  if (e != cudaSuccess) return e;
  // Short runs only where there can be enough tiles for them.
  const int grid =
      a.slots + (unit * units >= int64_t(a.slots) * kTailFrom ? a.slots / 4 * 4 : 0);
  launch_begin("paged_decode", s);
  e = launch_k(true, kernel, dim3(unsigned(grid)), dim3(kDecThreads), S::kSmem, s, a);
  launch_end("paged_decode", s);
  if (e != cudaSuccess) return e;
  launch_begin("paged_join", s);
  // All of its CTAs should be on the chip while the runs end: three an SM with
  // 16 warps, six with 8, whose warps take two heads where a CTA has all 16
  // (256 rows of 16 blocks: 173 us with 16 warps, 171 with 8; 128 rows, without
  // short runs: 91 and 93).
  e = grid > a.slots ? launch_k(true, k_paged_join<T, kDim, 8>, dim3(unsigned(grid - 1)),
                                dim3(8 * 32), 0, s, a)
                     : launch_k(true, k_paged_join<T, kDim, 16>, dim3(unsigned(grid - 1)),
                                dim3(16 * 32), 0, s, a);
  launch_end("paged_join", s);
  return e;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_paged_decode_workspace_bytes(const msa_paged_cache* cache, int32_t rows,
                                                       int32_t q_heads, size_t* bytes) {
  const msa_status st = check_cache(cache);
  if (st != MSA_OK) return st;
  if (!bytes || rows < 1 || rows > kMaxRows || q_heads < 1 || q_heads % cache->kv_heads ||
      q_heads / cache->kv_heads > kGroup)
    return MSA_ERR_INVALID_ARG;
  *bytes = decode_workspace(cache->head_dim);
  return MSA_OK;
}

extern "C" msa_status msa_paged_decode(const msa_paged_cache* cache, const msa_page_table* table,
                                       const int32_t* kv_len, const void* q, int32_t q_heads,
                                       float softmax_scale, const int32_t* q2k, void* o,
                                       float* lse, void* workspace, size_t workspace_bytes,
                                       msa_stream_t stream) {
  msa_status st = check_cache(cache);
  if (st != MSA_OK) return st;
  st = check_table(table, cache->page_size);
  if (st != MSA_OK) return st;
  if (!kv_len || !q || !o || !lse || !workspace || q_heads < 1 || q_heads % cache->kv_heads ||
      q_heads / cache->kv_heads > kGroup)
    return MSA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale > 1e30f) return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(q) || !paged_aligned(o) || !paged_aligned(workspace) ||
      !paged_aligned4(kv_len) || !paged_aligned4(q2k) || !paged_aligned4(lse))
    return MSA_ERR_ALIGNMENT;
  // tiles are counted in 32 bits
  if (int64_t(table->rows) * cache->kv_heads * table->width * cache->page_size > (int64_t(1) << 36))
    return MSA_ERR_INVALID_ARG;
  if (workspace_bytes < decode_workspace(cache->head_dim)) return MSA_ERR_WORKSPACE;
  st = check_device();
  if (st != MSA_OK) return st;
  DecodeArgs a{};
  a.q = q;
  a.k = PagedPool{cache->k, cache->k_stride[0], cache->k_stride[1], cache->k_stride[2]};
  a.v = PagedPool{cache->v, cache->v_stride[0], cache->v_stride[1], cache->v_stride[2]};
  a.table = table_args(table, cache->page_size, cache->num_pages, cache->status);
  a.kv_len = kv_len;
  a.q2k = q2k;
  a.o = o;
  a.lse = lse;
  a.scale_log2 = softmax_scale * kLog2e;
  a.kv_heads = cache->kv_heads;
  a.group = q_heads / cache->kv_heads;
  a.part_ml = static_cast<float*>(workspace);
  a.part_o = a.part_ml + 2 * kMaxGrid * 2 * kGroup;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == MSA_BF16)
    e = cache->head_dim == 128 ? launch_decode<__nv_bfloat16, 128>(a, s)
                               : launch_decode<__nv_bfloat16, 64>(a, s);
  else
    e = cache->head_dim == 128 ? launch_decode<__half, 128>(a, s)
                               : launch_decode<__half, 64>(a, s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
