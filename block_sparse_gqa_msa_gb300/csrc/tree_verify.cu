// tree_verify.cu - which drafted tokens of a row stay, by given random
// numbers, and the token behind them.
//
// Mathematics: at a token with target distribution p and drafting distribution
// q, drafts are tried one after the other against what is left of p: r = p,
// S = 1; draft x is kept if u q(x) < r(x) / S, else r = max(r / S - q, 0),
// S = sum r.  Keeping with probability min(1, r(x) / (S q(x))) and going on from
// the rest leaves p as the distribution of what is kept.  Without q a draft is
// no random choice: kept if u S < r(x), else r(x) = 0.  The token behind the last
// kept one is drawn from r by its running sum.
//
// r(x) of one token follows from p(x), q(x) and the S so far, so the walk needs
// a pass over the vocabulary only for each S behind a rejection, and one for the
// last draw.  All drafts' p(x) and q(x) are loaded side by side before the walk.
//
// A cluster of CTAs takes a row, each a run of the vocabulary, each warp a run
// of that; all walk alike.  Sums: the running sum's steps are as narrow as 1 /
// vocab, where 32 bits would draw a neighbour, and 64-bit additions are 1/64 as
// fast here as 32-bit ones (they would take ten times as long as the reading).
// So a lane adds in pairs of 32-bit numbers (the sum and what its rounding lost,
// exact two-sums).  What was lost is itself rounded at every addition, so its error
// grows with the square of their number: in one pair for all, 151000 values of a thread
// block were up to 2^-37 of the sum off, 2^20 values 2^-31.  Hence a pair takes 16
// additions and then goes into a sum of three numbers.  With u = 2^-24 and s what a
// lane's two pairs add up, the 16 are off by (1 + .. + 16) u^2 s, putting the two
// together by 50 u^2 s, at most 1024 sums of three by 2^29 u^3 of the lane's sum, a pair
// of that by u^2, five exchanges between lanes by 40 u^2 of the warp's: less than 2^-40
// of the sum.  (Adding the pairs up in 64 bits: 128 rows of 151000 60.5 us, not 56.5.)
// The drawn token's run is then added again, finer, until a warp looks at 32 values at
// a time.
//
// Measured: one row, 32000 tokens in the vocabulary, 9.5 us; 40 rows, 100003, no q,
// 16.6; 128 rows, 151000, with q, 56.5 (125 MB, two passes in the longest rows).
// A pass of a row by itself takes about 20 us there: a value costs 14 to 20
// instructions, and eight loads of a lane are on their way at a time.  16 bytes a load
// are as fast; a ring of asynchronous copies (80 to 100 us) and loads kept in
// registers for the next step (84, they spill) are slower.
#include <cooperative_groups.h>

#include <algorithm>

#include "paged.cuh"

namespace msa {
namespace {

constexpr int kTree = 64;
constexpr int kVerWarps = 16;
constexpr int kVerThreads = kVerWarps * 32;
constexpr int kVerCluster = 8;
constexpr int kVerLoads = 8;  // values of each distribution that a lane has in flight
constexpr int kVerRun = 24576;  // values of a CTA in calls of more rows than fit the chip

struct VerifyArgs {
  const float *target, *draft;  // draft may be null
  int64_t target_stride, draft_stride;
  const int32_t *tokens, *parents, *offs;
  const float *u, *u_last;
  int32_t *path, *count, *last;
  int64_t T;
  int32_t vocab, max_path, cluster;
};

// a + b in a; returns what its rounding lost, exactly.
__device__ __forceinline__ float two_sum(float& a, float b) {
  const float s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  const float lost = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  a = s;
  return lost;
}
// A sum in two 32-bit numbers.
struct Pair32 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {  // exact but for lo's own rounding
    lo = __fadd_rn(lo, two_sum(hi, x));
  }
  __device__ __forceinline__ void add(const Pair32& o) {
    add(o.hi);
    lo = __fadd_rn(lo, o.lo);
  }
  __device__ __forceinline__ double value() const { return double(hi) + double(lo); }
};
__device__ __forceinline__ Pair32 warp_sum(Pair32 s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Pair32 t{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)};
    // both lanes of a pair must get the same bits: the lower lane's sum first
    if (threadIdx.x & o) {
      const Pair32 x = s;
      s = t;
      t = x;
    }
    s.add(t);
  }
  return s;
}
// A sum of such sums in three numbers.
struct Sum32 {
  float hi, mid, lo;
  __device__ __forceinline__ void add(const Pair32& o) {
    const float a = two_sum(hi, o.hi);
    const float b = two_sum(mid, a);
    lo = __fadd_rn(lo, __fadd_rn(b, two_sum(mid, o.lo)));
  }
  // As a pair, lo no more than hi's rounding.
  __device__ __forceinline__ Pair32 pair() const {
    Pair32 s{hi, 0.f};
    s.lo = __fadd_rn(two_sum(s.hi, mid), lo);
    return s;
  }
};
// Sum of v over the lanes up to this one, of the first kLanes lanes.
template <int kLanes>
__device__ __forceinline__ double scan(double v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += y;
  }
  return v;
}

// What is left of a token's distribution: p's row, q's, the factors so far, the
// tokens that were rejected (without q).
struct Rest {
  const float *p, *q;
  const float* f;      // shared
  const int32_t* out;  // shared
  int n;               // rejections
  bool drawn;
  // r from p for the values x0, x0 + 32, ..; factors and tokens outermost.
  template <int kN>
  __device__ __forceinline__ void left(float (&r)[kN], const float (&q_x)[kN], int32_t x0) const {
    if (drawn) {
      for (int i = 0; i < n; ++i) {
        const float g = f[i];
#pragma unroll
        for (int e = 0; e < kN; ++e) r[e] = fmaxf(__fsub_rn(__fmul_rn(r[e], g), q_x[e]), 0.f);
      }
    } else {
      for (int i = 0; i < n; ++i) {
        const int32_t d = out[i] - x0;
#pragma unroll
        for (int e = 0; e < kN; ++e) r[e] = d == 32 * e ? 0.f : r[e];
      }
    }
  }
  template <int kN>
  __device__ __forceinline__ void load(float (&r)[kN], int32_t x0, int32_t hi) const {
    float q_x[kN] = {};
    const bool two = drawn && n > 0;
    if (x0 + 32 * (kN - 1) < hi) {
#pragma unroll
      for (int e = 0; e < kN; ++e) r[e] = p[x0 + 32 * e];
      if (two) {
#pragma unroll
        for (int e = 0; e < kN; ++e) q_x[e] = q[x0 + 32 * e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) r[e] = x0 + 32 * e < hi ? p[x0 + 32 * e] : 0.f;
      if (two) {
#pragma unroll
        for (int e = 0; e < kN; ++e) q_x[e] = x0 + 32 * e < hi ? q[x0 + 32 * e] : 0.f;
      }
    }
    left(r, q_x, x0);
  }
};

// Sum of r over [lo, hi), by a warp.
constexpr int kVerFold = 4;  // steps of 2 x 4 additions to a pair
static_assert(kVerFold * kVerLoads / 2 == 16, "the sums' bound");
__device__ __forceinline__ Pair32 run_sum(const Rest& rest, int32_t lo, int32_t hi) {
  const int lane = threadIdx.x & 31;
  Sum32 sum{0.f, 0.f, 0.f};
  for (int32_t x0 = lo + lane; x0 < hi;) {
    Pair32 s[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
    for (int i = 0; i < kVerFold && x0 < hi; ++i, x0 += 32 * kVerLoads) {
      float r[kVerLoads];
      rest.load(r, x0, hi);
#pragma unroll
      for (int e = 0; e < kVerLoads; ++e) s[e & 1].add(r[e]);
    }
    s[0].add(s[1]);
    sum.add(s[0]);
  }
  return warp_sum(sum.pair());
}

__global__ void __launch_bounds__(kVerThreads, 2) k_tree_verify(const VerifyArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int32_t par[kTree], tok[kTree], out[kTree];
  __shared__ float us[kTree], pv[kTree], qv[kTree], factor[kTree];
  __shared__ double warp_total[kVerWarps];
  __shared__ double total[2];  // the CTA's, of this pass and the one before
  __shared__ int32_t path[kTree];
  __shared__ int32_t sh_cur, sh_last, sh_n, sh_lo, sh_hi;  // what warp 0 has the others sum
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(cluster.block_rank());
  const int32_t r = blockIdx.x / a.cluster;
  grid_dep_wait();
  grid_dep_release();
  const int64_t t0 = a.offs[r], t1 = a.offs[r + 1];
  const int n = t0 >= 0 && t0 < t1 && t1 <= a.T && t1 - t0 <= kTree ? int(t1 - t0) : 0;
  int32_t* const row_path = a.path + int64_t(r) * a.max_path;
  if (n == 0) {
    if (rank == 0) {
      for (int i = tid; i < a.max_path; i += kVerThreads) row_path[i] = -1;
      if (tid == 0) {
        a.count[r] = 0;
        a.last[r] = -1;
      }
    }
    return;  // all CTAs of the cluster
  }
  if (tid < n) {
    const int64_t t = t0 + tid;
    const int32_t x = a.tokens[t];
    const float u = a.u[t];
    int32_t up = a.parents ? a.parents[t] : tid - 1;
    if (tid == 0 || up < 0 || up >= tid || x < 0 || x >= a.vocab) up = -1;
    par[tid] = up;
    tok[tid] = x;
    us[tid] = u;
    if (up >= 0) {
      const float p = a.target[(t0 + up) * a.target_stride + x];
      qv[tid] = a.draft ? a.draft[(t0 + up) * a.draft_stride + x] : 0.f;
      pv[tid] = p;
    }
  }
  __syncthreads();

  // The CTA's run of the vocabulary; the w-th 16th of a run.
  const int32_t V = a.vocab;
  const int32_t c0 = int32_t(int64_t(V) * rank / a.cluster);
  const int32_t c1 = int32_t(int64_t(V) * (rank + 1) / a.cluster);
  auto part = [](int32_t lo, int32_t hi, int w) {
    return lo + int32_t(int64_t(hi - lo) * w / kVerWarps);
  };
  auto rest_of = [&](int cur, int rejected) {
    return Rest{a.target + (t0 + cur) * a.target_stride,
                a.draft ? a.draft + (t0 + cur) * a.draft_stride : nullptr, factor, out, rejected,
                a.draft != nullptr};
  };
  // Warp 0 walks, and has all warps sum where it needs a sum (64-bit operations of 16
  // warps would get in one another's way): the walks of the cluster's CTAs are alike.
  int passes = 0;
  int cur = 0, kept = 1, rejected = 0, j = 1;
  double S = 1.0, R = 0.0, before = 0.0;
  double each = 0.0;     // a lane: the sum of the cluster's CTA number lane
  double run = 0.0;      // a lane: the CTA's sums up to warp number lane
  bool summed = false;   // R is the sum of the rest
  bool walking = true;
  const int32_t up0 = lane < n ? par[lane] : -1, up1 = lane + 32 < n ? par[lane + 32] : -1;
  if (tid == 0) path[0] = 0;
  for (;;) {
    if (warp == 0) {
      while (walking) {
        // the next child of cur from j on
        const uint64_t kids =
            uint64_t(__ballot_sync(0xffffffffu, lane >= j && up0 == cur)) |
            uint64_t(__ballot_sync(0xffffffffu, lane + 32 >= j && up1 == cur)) << 32;
        if (kids == 0 || kept == a.max_path) {
          walking = false;
          break;
        }
        const int kid = __ffsll(static_cast<long long>(kids)) - 1;
        float mine[1] = {pv[kid]};
        const float q[1] = {qv[kid]};
        bool keep;
        if (a.draft) {
          if (rejected > 0 && !summed) break;  // (to the sum, and back here)
          if (rejected > 0) S = R;
          float f = rejected == 0 ? 1.f : S > 0.0 ? float(1.0 / S) : 0.f;
          if (isinf(f)) f = 0.f;  // infinity times r would leave no distribution
          rest_of(cur, rejected).left(mine, q, tok[kid]);
          keep = double(us[kid]) * double(q[0]) < double(mine[0]) * double(f);
          if (!keep) {
            __syncwarp();
            if (lane == 0) factor[rejected] = f;
          }
        } else {
          rest_of(cur, rejected).left(mine, q, tok[kid]);
          keep = mine[0] > 0.f && double(us[kid]) * S < double(mine[0]);
          if (!keep) {
            S -= double(mine[0]);
            __syncwarp();
            if (lane == 0) out[rejected] = tok[kid];
          }
        }
        __syncwarp();
        j = kid + 1;
        summed = false;
        if (keep) {
          cur = kid;
          if (lane == 0) path[kept] = kid;
          ++kept;
          S = 1.0;
          rejected = 0;
        } else {
          ++rejected;
        }
      }
      if (!walking && summed && !(R > 0.0) && rejected > 0) {  // nothing is left: p itself
        rejected = 0;
        summed = false;
      }
      if (lane == 0) {
        sh_cur = summed ? -1 : cur;
        sh_last = cur;
        sh_n = rejected;
      }
    }
    __syncthreads();
    const int at = sh_cur;
    if (at < 0) break;
    const int32_t w0 = part(c0, c1, warp), w1 = part(c0, c1, warp + 1);
    const Pair32 s = run_sum(rest_of(at, sh_n), w0, w1);
    if (lane == 0) warp_total[warp] = s.value();
    __syncthreads();
    const int b = passes++ & 1;
    if (warp == 0) {
      run = scan<kVerWarps>(lane < kVerWarps ? warp_total[lane] : 0.0);
      if (lane == kVerWarps - 1) total[b] = run;
    }
    cluster.sync();  // (total[] alternates: one barrier a pass is enough)
    if (warp == 0) {
      each = lane < a.cluster ? *cluster.map_shared_rank(&total[b], lane) : 0.0;
      const double sum = scan<kVerCluster>(each);
      R = __shfl_sync(0xffffffffu, sum, a.cluster - 1);
      before = __shfl_sync(0xffffffffu, sum, rank > 0 ? rank - 1 : 0);
      if (rank == 0) before = 0.0;
      summed = true;
    }
  }

  // ---- the last token
  cluster.barrier_arrive();  // this CTA has read the others' shared memory
  // The first of the cluster's CTAs, of its warps, of their parts, whose sum passes
  // the goal; where rounding or a goal past the sum leaves none, the last with
  // anything in it.  up_to: the sum up to the lane's part, v: of it.
  double goal = 0.0, base = before;
  auto choose = [&](double up_to, double v, int parts) {
    const uint32_t past = __ballot_sync(0xffffffffu, lane < parts && v > 0.0 && up_to > goal);
    const uint32_t some = __ballot_sync(0xffffffffu, lane < parts && v > 0.0);
    return past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
  };
  auto narrow = [&](double sums) {  // sums: up to warp number lane
    double prev = __shfl_up_sync(0xffffffffu, sums, 1);
    if (lane == 0) prev = 0.0;
    const int w = choose(base + sums, sums - prev, kVerWarps);
    base += __shfl_sync(0xffffffffu, prev, w);
    return w;
  };
  if (warp == 0) {
    const bool any = R > 0.0 && !isinf(R);
    goal = double(a.u_last[r]) * R;
    int32_t lo = 0, hi = 0;
    if (any && choose(scan<kVerCluster>(each), each, a.cluster) == rank) {
      const int w = narrow(run);
      lo = part(c0, c1, w);
      hi = part(c0, c1, w + 1);
    }
    if (lane == 0) {
      sh_lo = lo;
      sh_hi = hi;
      if (rank == 0) {
        a.count[r] = kept;
        if (!any) a.last[r] = -1;
      }
    }
    if (rank == 0)
      for (int i = lane; i < a.max_path; i += 32) row_path[i] = i < kept ? path[i] : -1;
  }
  __syncthreads();
  const int32_t r0 = sh_lo, r1 = sh_hi;
  if (r0 < r1) {  // this CTA has it: the run's 16th part, then 32 values at a time
    const Rest rest = rest_of(sh_last, sh_n);
    const Pair32 s = run_sum(rest, part(r0, r1, warp), part(r0, r1, warp + 1));
    if (lane == 0) warp_total[warp] = s.value();
    __syncthreads();
    if (warp == 0) {
      const int w = narrow(scan<kVerWarps>(lane < kVerWarps ? warp_total[lane] : 0.0));
      const int32_t s0 = part(r0, r1, w), s1 = part(r0, r1, w + 1);
      int32_t found = -1, some = -1;
      for (int32_t x0 = s0; x0 < s1 && found < 0; x0 += 32) {
        float v[1];
        rest.load(v, x0 + lane, s1);
        const double incl = scan<32>(double(v[0]));
        const uint32_t past = __ballot_sync(0xffffffffu, v[0] > 0.f && base + incl > goal);
        const uint32_t any = __ballot_sync(0xffffffffu, v[0] > 0.f);
        if (past)
          found = x0 + __ffs(past) - 1;
        else if (any)
          some = x0 + 31 - __clz(any);
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) a.last[r] = found >= 0 ? found : some;
    }
  }
  cluster.barrier_wait();
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_tree_verify(const float* target, int64_t target_stride,
                                      const float* draft, int64_t draft_stride,
                                      const int32_t* tokens, const int32_t* parents,
                                      const int32_t* row_offsets, int32_t rows, int64_t T,
                                      int32_t vocab, const float* u, const float* u_last,
                                      int32_t max_path, int32_t* path, int32_t* count,
                                      int32_t* last, msa_stream_t stream) {
  if (!target || !tokens || !row_offsets || !u || !u_last || !path || !count || !last)
    return MSA_ERR_INVALID_ARG;
  if (rows < 1 || rows > kMaxRows || T < 1 || T > kMaxTokens || vocab < 1 ||
      vocab > (1 << 24) || max_path < 1 || max_path > kTree || target_stride < vocab ||
      (draft && draft_stride < vocab))
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned4(target) || !paged_aligned4(draft) || !paged_aligned4(tokens) ||
      !paged_aligned4(parents) || !paged_aligned4(row_offsets) || !paged_aligned4(u) ||
      !paged_aligned4(u_last) || !paged_aligned4(path) || !paged_aligned4(count) ||
      !paged_aligned4(last))
    return MSA_ERR_ALIGNMENT;
  const msa_status st = check_device();
  if (st != MSA_OK) return st;
  VerifyArgs a{};
  a.target = target;
  a.draft = draft;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.tokens = tokens;
  a.parents = parents;
  a.offs = row_offsets;
  a.u = u;
  a.u_last = u_last;
  a.path = path;
  a.count = count;
  a.last = last;
  a.T = T;
  a.vocab = vocab;
  a.max_path = max_path;
  // As many CTAs a row as are on the chip at once (2 an SM), none with less than a pass
  // of its loads to do.  With q, where rows of several passes keep the others waiting,
  // twice as many where each still has kVerRun values: half of the rows begin as others
  // end (100 rows, 151000 tokens: 63.5 -> 50.5 us, 200 rows, 65536: 58 -> 43; below it
  // 128 rows, 40000: 26 -> 30; without q 128 rows, 151000: 34 -> 38).
  auto chip = [&](int n) { return int64_t(rows) * n <= int64_t(device_sm_count()) * 2; };
  int cluster = 1;
  while (cluster < kVerCluster && vocab >= cluster * 2 * kVerThreads * 4 &&
         (chip(cluster * 2) ||
          (draft && chip(cluster) && vocab >= int64_t(cluster) * 2 * kVerRun)))
    cluster *= 2;
  a.cluster = cluster;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin("tree_verify", s);
  const cudaError_t e = launch_cluster(k_tree_verify, dim3(unsigned(rows) * cluster),
                                       dim3(kVerThreads), 0, unsigned(cluster), s, a);
  launch_end("tree_verify", s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
