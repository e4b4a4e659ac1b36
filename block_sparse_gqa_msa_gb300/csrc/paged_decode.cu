// paged_decode.cu - attention of one new token of each row over the paged
// cache, over all its keys or over the blocks that q2k names.
//
// Mathematics.  For row r and key head g the (up to 16) query heads that
// share g form the 16 rows of one matrix tile.  Over the keys in any order,
// with running maximum m and sum l in base 2 (x = scale * log2(e) * <q, k>):
//   m' = max(m, max x),  l' = l 2^(m-m') + sum 2^(x-m'),
//   O' = O 2^(m-m') + 2^(x-m') V,
// and two such states join as M = max(m1, m2), l = l1 2^(m1-M) + l2 2^(m2-M),
// O likewise; at the end O / l and lse = ln2 (m + log2 l).  m, l, O are 32
// bits throughout.  The weights 2^(x-m') <= 1 are rounded to the cache's type
// for the matrix product with V: one rounding of half a step relative to each
// weight, independent from key to key, so it stays below the one rounding of
// the output that follows.
//
// What bounds it.  Each key and value is used for 16 query heads at most:
// 4 * 16 * D flop on 4 * D bytes, 16 flop a byte, so HBM is the bound (at 6.8
// TB/s 109 TFLOP/s, a few per cent of the tensor pipe) and the 16-row
// register-level matrix instruction has the right shape: the tile's rows are
// the 16 heads, where a 128-row tensor-memory tile would be seven eighths
// empty.
//
// Split.  A unit is a (row, key head); its keys are cut into tiles of 64.  All
// units' tiles, in order, are dealt out in equal runs to the CTAs (two an
// SM), so a batch of any lengths is balanced and a single long row occupies
// the whole chip; the run's place is found from the lengths on the device, so
// nothing comes back to the host.  A run is cut into segments at unit
// borders.  A unit that lies within one run is finished there; otherwise
// each of its CTAs leaves its (m, l, O) in the workspace and k_paged_join adds
// them up, in order, so results do not depend on timing.
//
// A warp works alone on its share of each tile (16 keys of 128 channels, 32 of
// 64: 8 KB of keys and values): it fetches them with asynchronous copies into
// its own ring of stages, two stages ahead and across segment borders, and
// waits for other warps only where a segment ends.
#include "paged.cuh"

namespace msa {
namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kGroup = 16;   // query heads of a matrix tile
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
  // the warps' states meet 32 channels at a time, rows 40 floats apart
  // (8 rows' 8-byte writes then hit all banks once)
  static constexpr int kMergeRow = 40;
  static constexpr int kMergeBytes = kDecWarps * kGroup * kMergeRow * 4;
  static constexpr int kSmem = kDecWarps * kRing + kMergeBytes;  // 106 KB a CTA
};

// What a CTA leaves for the join about the unit that its run starts inside.
struct JoinRec {
  int32_t unit;   // row * kv_heads + key head
  int32_t parts;  // CTAs after the unit's first one that hold a part of it; 0: no join here
};

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
  JoinRec* rec;        // [grid]
  float* part_ml;      // [2 grid][2][16]: m, l
  float* part_o;       // [2 grid][16][dim]
};

__device__ __forceinline__ float exp2_fast(float x) {  // to 2^-22, results below 2^-126 are 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
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

// Tiles of one unit of a row of len keys (at least one, so that rows without
// keys are written too).
template <int kDim>
__device__ __forceinline__ int32_t unit_tiles(int32_t len, bool sparse) {
  using S = DecodeShape<kDim>;
  int32_t n;
  if (sparse) {
    const int32_t nb = int32_t((int64_t(len) + kBlock - 1) / kBlock);
    n = min(nb, kTopK) * S::kTilesPerBlock;
  } else {
    n = int32_t((int64_t(len) + S::kTileKeys - 1) / S::kTileKeys);
  }
  return max(n, 1);
}

// Start of CTA c's run of the n tiles, dealt to `ctas` <= n CTAs (so no run is
// empty); the last CTA whose run starts before tile e is (e * ctas - 1) / n.
__device__ __forceinline__ int64_t run_start(int64_t n, int64_t c, int64_t ctas) {
  return n * c / ctas;
}

// A place in the list of all tiles.
struct Place {
  int64_t total;       // tiles of the call
  int64_t ctas;        // CTAs they are dealt to
  int64_t lo, hi;      // the CTA's run
  int64_t unit_start;  // first tile of the unit that lo lies in
  int32_t row, head, tiles, len;
};

// Finds the CTA's run.  Every thread sums the tiles of a stretch of rows; a
// scan over the threads' sums gives the total and, for the one stretch that
// holds lo, its place.
template <int kDim>
__device__ __forceinline__ Place find_place(const DecodeArgs& a, int64_t* sums, Place* found) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool sparse = a.q2k != nullptr;
  const int32_t rows = a.table.rows;
  const int32_t each = (rows + kDecThreads - 1) / kDecThreads;
  const int32_t r0 = min(rows, tid * each), r1 = min(rows, r0 + each);
  const int64_t most = int64_t(a.table.width) << a.table.shift;
  int64_t mine = 0;
  int32_t first_len = 0;
  for (int32_t r = r0; r < r1; ++r) {
    int32_t n = a.kv_len[r];
    if (n < 0 || n > most) {
      if (blockIdx.x == 0) raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
      n = 0;
    }
    if (r == r0) first_len = n;
    mine += int64_t(unit_tiles<kDim>(n, sparse)) * a.kv_heads;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  int64_t at = before + incl - mine;  // tiles before the thread's rows
  const int64_t ctas = total < gridDim.x ? total : gridDim.x;
  const int64_t lo = run_start(total, blockIdx.x, ctas);  // total and more past the last CTA
  if (tid == 0) found->ctas = ctas;
  if (lo >= at && lo < at + mine) {
    int32_t len = first_len;
    for (int32_t r = r0; r < r1; ++r) {
      if (r > r0) {
        len = a.kv_len[r];
        if (len < 0 || len > most) len = 0;
      }
      const int32_t tiles = unit_tiles<kDim>(len, sparse);
      const int64_t here = int64_t(tiles) * a.kv_heads;
      if (lo < at + here) {
        Place p;
        p.total = total;
        p.ctas = ctas;
        p.lo = lo;
        p.hi = run_start(total, blockIdx.x + 1, ctas);
        p.head = int32_t((lo - at) / tiles);
        p.unit_start = at + int64_t(p.head) * tiles;
        p.row = r;
        p.tiles = tiles;
        p.len = len;
        *found = p;
        break;
      }
      at += here;
    }
  }
  __syncthreads();
  return *found;
}

// A part of a unit that one CTA works on: its tiles i0 .. i1 - 1.
struct Segment {
  int32_t row, head, i0, i1, tiles;
};
constexpr int kSegQueue = 8;  // the fetch is at most kStages tiles, so segments, ahead

// The fetching side of a warp: walks the run's tiles ahead of the sums and
// leaves each segment that it enters in a queue.  All its state is the same
// in all lanes except page and slots.
template <typename T, int kDim>
struct Fetch {
  using S = DecodeShape<kDim>;
  static constexpr int kChunks = kDim / 8;          // 16-byte chunks of a key
  static constexpr int kRowsAtOnce = 32 / kChunks;  // keys one copy instruction covers
  static constexpr int kCopies = S::kWarpKeys / kRowsAtOnce;
  static constexpr int kWhole = S::kWarpKeys == 32 ? 5 : 4;  // log2 of a warp's keys
  const DecodeArgs& a;
  int32_t* blocks;   // the unit's blocks (sparse), shared memory
  Segment* queue;
  int lane, warp;
  int64_t left;      // tiles of the run after the current segment
  int32_t row, head, len, tiles, i, i1, n_blocks, n_seg;
  int32_t next_len, slots;  // of the next unit, loaded ahead
  int32_t j;         // first key of the warp's part of the tile at hand, -1: none
  int32_t page;      // its page as the table has it, unchecked

  __device__ __forceinline__ int32_t checked(int32_t n) const {
    return n < 0 || n > (int64_t(a.table.width) << a.table.shift) ? 0 : n;
  }
  __device__ __forceinline__ void load_slots(int32_t r, int32_t h) {
    if (a.q2k && lane < kTopK && r < a.table.rows)
      slots = a.q2k[(int64_t(h) * a.table.rows + r) * kTopK + lane];
  }
  // Enters the unit (row, head) at tile i: its blocks (the distinct valid
  // slots, in slot order), its place in the queue, and a look ahead.
  __device__ __forceinline__ void enter() {
    if (a.q2k) {
      const int32_t nb = int32_t((int64_t(len) + kBlock - 1) / kBlock);
      const int32_t v = slots;
      const bool ok = lane < kTopK && v >= 0 && v < nb;
      if (lane < kTopK && len > 0 && v != -1 && !ok) raise_paged(a.table.status, MSA_ERR_BAD_Q2K);
      const uint32_t same = __match_any_sync(0xffffffffu, ok ? v : -1 - lane);
      const bool keep = ok && (__ffs(same) - 1) == lane;
      const uint32_t m = __ballot_sync(0xffffffffu, keep);
      n_blocks = __popc(m);
      __syncwarp();  // the list before is read
      if (keep) blocks[__popc(m & ((1u << lane) - 1))] = v;
    }
    if (lane == 0) queue[n_seg % kSegQueue] = Segment{row, head, i, i1, tiles};
    ++n_seg;
    __syncwarp();
    if (left > 0) {  // the next unit: its length, slots and queries
      const int32_t r = head + 1 == a.kv_heads ? row + 1 : row;
      const int32_t h = head + 1 == a.kv_heads ? 0 : head + 1;
      next_len = a.kv_len[r];
      load_slots(r, h);
      if (lane * 64 < a.group * kDim)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            static_cast<const T*>(a.q) + (int64_t(r) * a.kv_heads + h) * a.group * kDim +
            lane * 64));
    }
  }
  __device__ __forceinline__ void begin(const Place& p) {
    row = p.row;
    head = p.head;
    len = p.len;
    tiles = p.tiles;
    i = int32_t(p.lo - p.unit_start);
    const int64_t n = p.hi - p.lo;
    i1 = int32_t(min(int64_t(tiles), i + n));
    left = n - (i1 - i);
    n_blocks = 0;
    n_seg = 0;
    slots = -1;
    load_slots(row, head);
    enter();
    look();
  }
  __device__ __forceinline__ void advance() {
    if (i1 == 0) return;  // the run is done
    if (++i == i1) {
      if (left == 0) {
        i1 = 0;
        j = -1;
        return;
      }
      if (++head == a.kv_heads) {
        head = 0;
        ++row;
        len = checked(next_len);
        tiles = unit_tiles<kDim>(len, a.q2k != nullptr);
      }
      i = 0;
      i1 = int32_t(min(int64_t(tiles), left));
      left -= i1;
      enter();
    }
    look();
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
      const int64_t slot = j & mask;
      kb += page * a.k.page + slot * a.k.token;
      vb += page * a.v.page + slot * a.v.token;
      const int n = len - j;
      if (n >= S::kWarpKeys) {
#pragma unroll
        for (int x = 0; x < kCopies; ++x) {
          const int key = x * kRowsAtOnce + sub;
          const uint32_t dst = stage + key * S::kRow + ((c ^ (key & 7)) << 4);
          cp_async16(dst, kb + key * a.k.token);
          cp_async16(dst + kValues, vb + key * a.v.token);
        }
        return 0xffffffffu >> (32 - S::kWarpKeys);
      }
#pragma unroll 4
      for (int x = 0; x < kCopies; ++x) {
        const int key = x * kRowsAtOnce + sub;
        const uint32_t dst = stage + key * S::kRow + ((c ^ (key & 7)) << 4);
        const bool real = key < n;  // else nothing is read; the address is the first key's
        cp_async16_if(dst, kb + (real ? key : 0) * a.k.token, real);
        cp_async16_if(dst + kValues, vb + (real ? key : 0) * a.v.token, real);
      }
      return (1u << n) - 1;
    }
    const bool due = lane < S::kWarpKeys && j + lane < len;
    const bool good = due && page >= 0 && page < a.table.num_pages;
    if (due && !good) raise_paged(a.table.status, MSA_ERR_BAD_PAGE);
    const uint32_t there = __ballot_sync(0xffffffffu, good);
#pragma unroll 4
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

template <typename T, int kDim>
__global__ void __launch_bounds__(kDecThreads, 2) k_paged_decode(const DecodeArgs a) {
  using S = DecodeShape<kDim>;
  constexpr int kSteps = kDim / 16;            // k-steps of the first product
  constexpr int kCols = kDim / 8;              // column tiles of the second
  constexpr int kKeyTiles = S::kWarpKeys / 8;  // column tiles of the first
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sums[kDecWarps];
  __shared__ Place found;
  __shared__ int32_t blocks[kDecWarps][kTopK];
  __shared__ Segment queue[kDecWarps][kSegQueue];
  __shared__ float ml[2][kDecWarps][kGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r_lo = lane >> 2;  // the lane's matrix rows: r_lo and r_lo + 8
  const int col = (lane & 3) * 2;
  grid_dep_wait();
  grid_dep_release();
  const Place p = find_place<kDim>(a, sums, &found);
  if (blockIdx.x >= p.ctas) {
    if (tid == 0) a.rec[blockIdx.x] = JoinRec{0, 0};
    return;
  }
  if (tid == 0) {
    // The unit that the run starts inside, for the join: the first CTA that
    // starts inside it records how many parts follow.
    JoinRec rec{0, 0};
    const int64_t c = blockIdx.x;
    if (p.unit_start < p.lo && run_start(p.total, c - 1, p.ctas) <= p.unit_start) {
      const int64_t last = ((p.unit_start + p.tiles) * p.ctas - 1) / p.total;
      rec.unit = p.row * a.kv_heads + p.head;
      rec.parts = int32_t(last - c + 1);
    }
    a.rec[c] = rec;
  }

  const uint32_t ring = uint32_t(__cvta_generic_to_shared(smem)) + warp * S::kRing;
  float* merge = reinterpret_cast<float*>(smem + kDecWarps * S::kRing);
  Fetch<T, kDim> fetch{a, blocks[warp], queue[warp], lane, warp};
  fetch.begin(p);
  uint32_t there[S::kStages - 1];  // of the tiles in flight: the keys that are there
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    there[s] = fetch.copy(ring + s * S::kStageBytes);
    cp_async_commit();
    fetch.advance();
  }

  int64_t left = p.hi - p.lo;
  int stage = 0;
  for (int seg = 0; left > 0; ++seg) {
    const Segment g = queue[warp][seg % kSegQueue];
    left -= g.i1 - g.i0;

    // ---- the query heads as the left operand; heads past the group are zeros
    uint32_t qa[kSteps][4];
    {
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
    }
    float acc[kCols][4];
#pragma unroll
    for (int n = 0; n < kCols; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    // ---- the keys
#pragma unroll 1
    for (int32_t i = g.i0; i < g.i1; ++i) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      const uint32_t seen = there[0];
      const uint32_t kb = ring + stage * S::kStageBytes, vb = kb + S::kWarpKeys * S::kRow;
      // the stage freed by the last tile takes the tile kStages - 1 ahead
      {
        const int free = stage == 0 ? S::kStages - 1 : stage - 1;
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
#pragma unroll
        for (int s = 0; s + 1 < S::kStages - 1; ++s) there[s] = there[s + 1];
        there[S::kStages - 2] = fetch.copy(ring + free * S::kStageBytes);
        cp_async_commit();
        fetch.advance();
      }
      if (seen == 0) continue;

      float x[kKeyTiles][4];
#pragma unroll
      for (int n = 0; n < kKeyTiles; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
      for (int n = 0; n < kKeyTiles; n += 2) {
        // matrices: keys 0-7 / 8-15 by channels 0-7 / 8-15 of the step
        const int key = n * 8 + (lane & 7) + ((lane >> 4) << 3);
        const uint32_t rowp = kb + key * S::kRow;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b[4];
          ldsm4(b, rowp + (((2 * k + ((lane >> 3) & 1)) ^ (key & 7)) << 4));
          mma16816<T>(x[n], qa[k], b[0], b[1]);
          mma16816<T>(x[n + 1], qa[k], b[2], b[3]);
        }
      }
      // scores in base 2, masked
      float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
      for (int n = 0; n < kKeyTiles; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool on = (seen >> (n * 8 + col + (e & 1))) & 1;
          x[n][e] = on ? x[n][e] * a.scale_log2 : -INFINITY;
        }
        top0 = fmaxf(top0, fmaxf(x[n][0], x[n][1]));
        top1 = fmaxf(top1, fmaxf(x[n][2], x[n][3]));
      }
      top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
      top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
      top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 2));
      top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 2));
      if (__any_sync(0xffffffffu, top0 > m0 || top1 > m1)) {
        const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
        const float f0 = n0 == -INFINITY ? 1.f : exp2_fast(m0 - n0);
        const float f1 = n1 == -INFINITY ? 1.f : exp2_fast(m1 - n1);
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
      const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int n = 0; n < kKeyTiles; ++n) {
        x[n][0] = exp2_fast(x[n][0] - z0);
        x[n][1] = exp2_fast(x[n][1] - z0);
        x[n][2] = exp2_fast(x[n][2] - z1);
        x[n][3] = exp2_fast(x[n][3] - z1);
        l0 += x[n][0] + x[n][1];
        l1 += x[n][2] + x[n][3];
      }
#pragma unroll
      for (int k = 0; k < kKeyTiles; k += 2) {
        const uint32_t pa[4] = {
            Pair<T>::pack(x[k][0], x[k][1]), Pair<T>::pack(x[k][2], x[k][3]),
            Pair<T>::pack(x[k + 1][0], x[k + 1][1]), Pair<T>::pack(x[k + 1][2], x[k + 1][3])};
        // matrices: keys 0-7 / 8-15 by channels 0-7 / 8-15 of the pair of column tiles
        const int key = k * 8 + (lane & 15);
        const uint32_t rowp = vb + key * S::kRow;
#pragma unroll
        for (int n = 0; n < kCols; n += 2) {
          uint32_t b[4];
          ldsm4_t(b, rowp + (((n + (lane >> 4)) ^ (key & 7)) << 4));
          mma16816<T>(acc[n], pa, b[0], b[1]);
          mma16816<T>(acc[n + 1], pa, b[2], b[3]);
        }
      }
    }

    // ---- join the warps: every state is brought to the common maximum
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if ((lane & 3) == 0) {
      ml[0][warp][r_lo] = m0;
      ml[0][warp][r_lo + 8] = m1;
    }
    __syncthreads();
    float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      M0 = fmaxf(M0, ml[0][w][r_lo]);
      M1 = fmaxf(M1, ml[0][w][r_lo + 8]);
    }
    const float f0 = m0 == -INFINITY ? 0.f : exp2_fast(m0 - M0);
    const float f1 = m1 == -INFINITY ? 0.f : exp2_fast(m1 - M1);
    if ((lane & 3) == 0) {
      ml[1][warp][r_lo] = l0 * f0;
      ml[1][warp][r_lo + 8] = l1 * f1;
    }
    const bool whole = g.i0 == 0 && g.i1 == g.tiles;
    const int64_t slot = 2 * int64_t(blockIdx.x) + (g.i0 > 0 ? 0 : 1);
    const int64_t unit = int64_t(g.row) * a.kv_heads + g.head;
    const int h = tid / 8;  // the thread's row of the result, 4 channels of each 32
    float M = -INFINITY, l = 0.f, inv = 0.f;
#pragma unroll
    for (int c = 0; c < kDim / 32; ++c) {
      float* mine = merge + warp * (kGroup * S::kMergeRow);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float* x = acc[c * 4 + n];
        *reinterpret_cast<float2*>(mine + r_lo * S::kMergeRow + n * 8 + col) =
            make_float2(x[0] * f0, x[1] * f0);
        *reinterpret_cast<float2*>(mine + (r_lo + 8) * S::kMergeRow + n * 8 + col) =
            make_float2(x[2] * f1, x[3] * f1);
      }
      __syncthreads();
      if (c == 0) {
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          M = fmaxf(M, ml[0][w][h]);
          l += ml[1][w][h];
        }
        inv = l == 0.f ? 0.f : 1.f / l;  // l == 0: no key was seen
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(
            merge + (w * kGroup + h) * S::kMergeRow + (tid % 8) * 4);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      const int ch = c * 32 + (tid % 8) * 4;
      if (!whole)
        *reinterpret_cast<float4*>(a.part_o + (slot * kGroup + h) * kDim + ch) = v;
      else if (h < a.group)
        *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + (unit * a.group + h) * kDim + ch) =
            make_uint2(Pair<T>::pack(v.x * inv, v.y * inv), Pair<T>::pack(v.z * inv, v.w * inv));
      __syncthreads();  // the buffers are read
    }
    if (tid % 8 == 0) {
      if (!whole) {
        a.part_ml[slot * (2 * kGroup) + h] = M;
        a.part_ml[slot * (2 * kGroup) + kGroup + h] = l;
      } else if (h < a.group) {
        a.lse[unit * a.group + h] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
      }
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of the units that several CTAs share.  CTA (c, y): the unit
// that run c starts inside, if c is the first such run; a warp a (head, part of
// the parts), lanes over the channels.
constexpr int kJoinThreads = 512;
constexpr int kJoinWays = 4;    // warps that share a head
constexpr int kJoinHeads = kJoinThreads / 32 / kJoinWays;
template <typename T, int kDim>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const DecodeArgs a) {
  constexpr int kPer = kDim / 32;
  __shared__ float so[kJoinThreads / 32][kDim];
  __shared__ float sl[kJoinThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int way = warp / kJoinHeads;
  const int h = blockIdx.y * kJoinHeads + warp % kJoinHeads;
  grid_dep_wait();
  grid_dep_release();
  const int64_t c = int64_t(blockIdx.x) + 1;
  const JoinRec rec = a.rec[c];
  if (rec.parts == 0 || blockIdx.y * kJoinHeads >= a.group) return;
  const int n = rec.parts + 1;
  // part 0: the unit's first CTA, whose run goes on past it; then the CTAs
  // that start inside the unit
  auto slot = [&](int i) { return i == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + i); };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, a.part_ml[slot(i) * (2 * kGroup) + h]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[kPer] = {};
  float l = 0.f;
#pragma unroll 4
  for (int i = way; i < n; i += kJoinWays) {
    const int64_t s = slot(i);
    const float m = a.part_ml[s * (2 * kGroup) + h];
    const float f = m == -INFINITY ? 0.f : exp2_fast(m - M);
    l += f * a.part_ml[s * (2 * kGroup) + kGroup + h];
    const float* o = a.part_o + (s * kGroup + h) * kDim + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] += f * o[e];
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = acc[e];
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  if (way != 0 || h >= a.group) return;
#pragma unroll
  for (int w = 1; w < kJoinWays; ++w) {
    l += sl[warp + w * kJoinHeads];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] += so[warp + w * kJoinHeads][lane * kPer + e];
  }
  const int64_t out = int64_t(rec.unit) * a.group + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<T*>(a.o) + out * kDim + lane * kPer);
#pragma unroll
  for (int e = 0; e < kPer; e += 2) o[e / 2] = Pair<T>::pack(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) a.lse[out] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
}

int decode_grid() { return device_sm_count() * 2; }
// The workspace is sized without a device: no GB300 has more SMs than this.
constexpr int kMaxGrid = 160 * 2;

size_t decode_workspace(int32_t dim) {
  return align_up(sizeof(JoinRec) * kMaxGrid, 256) +
         sizeof(float) * 2 * kMaxGrid * (2 * kGroup + kGroup * size_t(dim));
}

template <typename T, int kDim>
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s) {
  using S = DecodeShape<kDim>;
  auto kernel = k_paged_decode<T, kDim>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::kSmem);
  if (e != cudaSuccess) return e;
  int grid = decode_grid();
  if (grid > kMaxGrid) grid = kMaxGrid;
  launch_begin("paged_decode", s);
  e = launch_k(true, kernel, dim3(unsigned(grid)), dim3(kDecThreads), S::kSmem, s, a);
  launch_end("paged_decode", s);
  if (e != cudaSuccess) return e;
  launch_begin("paged_join", s);
  e = launch_k(true, k_paged_join<T, kDim>,
               dim3(unsigned(grid - 1), unsigned((a.group + kJoinHeads - 1) / kJoinHeads)),
               dim3(kJoinThreads), 0, s, a);
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
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.rec = reinterpret_cast<JoinRec*>(w);
  w += align_up(sizeof(JoinRec) * kMaxGrid, 256);
  a.part_ml = reinterpret_cast<float*>(w);
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
