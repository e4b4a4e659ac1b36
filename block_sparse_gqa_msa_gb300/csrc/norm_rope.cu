// norm_rope.cu - norm of every query and key head with the rotation by
// position in the same pass, and its gradient.
//
// Mathematics: over a head's channels n = 1 / sqrt(mean(x^2) + eps), y = x n w,
// then pairs turn by position * inv_freq (angles in 64 bits, turn_of).  The
// turn is orthogonal, so the gradient turns dy back, g, and then
//   dx = n (g w - u mean(g w u)), dw = sum g u, u = x n.
// Nothing but x is kept for it: n is formed again from the x that is read
// anyway.
//
// Both are bound by HBM: x in and y out (forward), x and dy in and dx out.  A
// lane holds 16 channels of a head (8 pairs and both of their halves), so a
// head is 8 or 4 lanes, its sums two or three exchanges, and the rotation needs
// none.  A warp takes an equal run of all tokens' heads and forms a token's
// angles once.  It works alone: each lane
// copies its own channels into its own places of a ring in shared memory, 8 KB a
// warp ahead of the sums, across tokens; 128 KB an SM are on their way at any
// time, and no registers are held for them.
//
// Measured (16384 tokens of 64 + 4 heads of 128 channels): 93 us forward, 6.1 TB/s,
// and 141 the gradient, 6.1 TB/s, of a plain copy's 6.8; 9 tokens of 24 + 8 heads
// of 64 channels 3.2 us.  With the loads in registers, a head's at a time, the two
// took 300 us together instead of 265.  Few heads do not hide a token's angles: 16384
// tokens of 16 + 2 heads of 128 channels 29 us without rotation, 42 with all turned.
#include <algorithm>

#include "paged.cuh"

namespace msa {
namespace {

constexpr int kNormThreads = 512;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kRing = 8192;  // bytes of a warp's ring
constexpr int kNormSmem = kNormWarps * kRing;

struct NormArgs {
  const void* x[2];       // queries, keys
  const void* dy[2];      // backward
  void* y[2];             // results, or dx
  int64_t stride[2];
  const void* w[2];
  const int32_t* positions;
  const float* inv_freq;
  float* part;            // backward: [CTAs][2][dim]
  float* dw[2];
  int64_t T;
  int32_t heads[2];
  int32_t rot, w_type, parts;
  float eps;
};

__device__ __forceinline__ float weight_at(const void* w, int type, int i) {
  if (type == MSA_F32) return static_cast<const float*>(w)[i];
  if (type == MSA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
  return __half2float(static_cast<const __half*>(w)[i]);
}

// The lane's place in a head: two runs of 8 channels.  Of a head whose halves
// pair, run 0 holds the first and run 1 the second channels of 8 pairs, or
// both are runs of the channels that are not turned.
template <int kDim, bool kInter>
struct Place {
  int c0, c1;
  bool turn0, turn1;
  __device__ __forceinline__ Place(int sub, int rot) {
    if (kInter) {
      c0 = sub * 8;
      c1 = c0 + kDim / 2;
    } else if (sub * 16 < rot) {
      c0 = sub * 8;
      c1 = c0 + rot / 2;
    } else {
      c0 = rot + (sub - rot / 16) * 8;
      c1 = c0 + (kDim - rot) / 2;
    }
    turn0 = c0 < rot;
    turn1 = c1 < rot;
  }
};

// Angles of a token, left in the warp's shared memory, then the lane's 8.
template <int kDim, bool kInter>
__device__ __forceinline__ void angles(const NormArgs& a, int32_t pos, float2* mine,
                                       const Place<kDim, kInter>& at, float (&c)[8],
                                       float (&s)[8]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (a.rot > 0) {
    for (int i = lane; i < a.rot / 2; i += 32) mine[i] = turn_of(pos, a.inv_freq[i]);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // pair of the lane's channels: (c0 + i, c1 + i), or 4 pairs in each run
    const bool turned = kInter && i >= 4 ? at.turn1 : at.turn0;
    const int pair = kInter ? (i < 4 ? at.c0 / 2 + i : at.c1 / 2 + i - 4) : at.c0 + i;
    const float2 v = turned ? mine[pair] : make_float2(1.f, 0.f);
    c[i] = v.x;
    s[i] = v.y;
  }
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = Pair<T>::unpack(w[i]);
    x[2 * i] = p.x;
    x[2 * i + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(Pair<T>::pack(x[0], x[1]), Pair<T>::pack(x[2], x[3]),
                    Pair<T>::pack(x[4], x[5]), Pair<T>::pack(x[6], x[7]));
}
// Turns the lane's 16 channels (run 0 in x[0..7], run 1 in x[8..15]); back: by
// the negative angle.
template <bool kInter, bool kBack>
__device__ __forceinline__ void rotate16(float* x, const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = kInter ? 2 * i : i, q = kInter ? 2 * i + 1 : i + 8;
    const float u = x[p], v = x[q], sn = kBack ? -s[i] : s[i];
    x[p] = u * c[i] - v * sn;
    x[q] = v * c[i] + u * sn;
  }
}
template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kN>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

// A warp's place in its run of groups.  A group is 32 / kLanes heads of the queries
// or of the keys of a token, a head to kLanes lanes; the tokens' groups are dealt out
// in equal runs.
struct Cursor {
  int64_t t;
  int32_t g;
  int32_t left;
  int32_t groups_q, groups;
  __device__ __forceinline__ void next() {
    --left;
    if (++g == groups) {
      g = 0;
      ++t;
    }
  }
};

// Forward, or the gradient: then each CTA's sums of dw go to the workspace,
// k_norm_rope_join adds them up in order.
template <typename T, int kDim, bool kInter, bool kBack>
__global__ void __launch_bounds__(kNormThreads, 1) k_norm_rope(const NormArgs a) {
  constexpr int kLanes = kDim / 16, kPer = 32 / kLanes;
  constexpr int kParts = kBack ? 4 : 2;             // copies of a lane in a group
  constexpr int kDepth = kRing / (kParts * 512);    // groups on their way
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float sw[2][kDim];
  __shared__ float2 turns[kNormWarps][kDim / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place<kDim, kInter> at(lane % kLanes, a.rot);
  const int slot = lane / kLanes;
  grid_dep_wait();
  grid_dep_release();
  Cursor work;
  work.groups_q = (a.heads[0] + kPer - 1) / kPer;
  work.groups = work.groups_q + (a.heads[1] + kPer - 1) / kPer;
  {
    const int64_t all = a.T * work.groups, runs = int64_t(gridDim.x) * kNormWarps;
    const int64_t run = int64_t(warp) * gridDim.x + blockIdx.x;
    const int64_t first = all * run / runs;
    work.left = int32_t(all * (run + 1) / runs - first);
    work.t = first / work.groups;
    work.g = int32_t(first - work.t * work.groups);
  }
  Cursor ahead = work;
  uint8_t* const mine = ring + warp * kRing + lane * 16;
  const uint32_t mine_at = uint32_t(__cvta_generic_to_shared(mine));
  auto fetch = [&](int stage) {
    if (ahead.left > 0) {
      const int kind = ahead.g >= ahead.groups_q;
      const int h = (kind ? ahead.g - ahead.groups_q : ahead.g) * kPer + slot;
      if (h < a.heads[kind]) {
        const uint32_t dst = mine_at + stage * (kParts * 512);
        const T* x = static_cast<const T*>(a.x[kind]) + ahead.t * a.stride[kind] + h * kDim;
        copy16(dst, x + at.c0);
        copy16(dst + 512, x + at.c1);
        if (kBack) {
          const T* dy = static_cast<const T*>(a.dy[kind]) + (ahead.t * a.heads[kind] + h) * kDim;
          copy16(dst + 1024, dy + at.c0);
          copy16(dst + 1536, dy + at.c1);
        }
      }
      ahead.next();
    }
    copies_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) fetch(i);
  for (int i = threadIdx.x; i < 2 * kDim; i += kNormThreads)
    sw[i / kDim][i % kDim] = weight_at(a.w[i / kDim], a.w_type, i % kDim);
  __syncthreads();

  float acc[2][16] = {};
  float c[8], s[8];
  int64_t token = -1;
  int32_t pos = a.rot > 0 ? a.positions[min(work.t, a.T - 1)] : 0;
  int stage = 0;
#pragma unroll 1
  for (; work.left > 0; work.next()) {
    if (work.t != token) {
      token = work.t;
      angles<kDim, kInter>(a, pos, turns[warp], at, c, s);
      if (a.rot > 0) pos = a.positions[min(token + 1, a.T - 1)];  // the next token's
    }
    const int kind = work.g >= work.groups_q;
    const int h = (kind ? work.g - work.groups_q : work.g) * kPer + slot;
    const bool real = h < a.heads[kind];
    copies_wait<kDepth - 1>();
    const uint8_t* from = mine + stage * (kParts * 512);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 u = real ? *reinterpret_cast<const uint4*>(from) : zero;
    const uint4 v = real ? *reinterpret_cast<const uint4*>(from + 512) : zero;
    float x[16];
    unpack8<T>(u, x);
    unpack8<T>(v, x + 8);
    [[maybe_unused]] float d[16];
    if (kBack) {
      const uint4 du = real ? *reinterpret_cast<const uint4*>(from + 1024) : zero;
      const uint4 dv = real ? *reinterpret_cast<const uint4*>(from + 1536) : zero;
      unpack8<T>(du, d);
      unpack8<T>(dv, d + 8);
    }
    fetch(stage);
    stage = stage + 1 == kDepth ? 0 : stage + 1;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
    // (lanes without a head add nothing to the weights' gradients, for eps = 0 neither)
    const float mean = head_sum<kLanes>(ss) * (1.f / kDim);
    const float n = real ? rsqrtf(mean + a.eps) : 0.f;
    if (!kBack) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(
            &sw[kind][(i < 8 ? at.c0 + i : at.c1 + i - 8)]);
        x[i] *= n * w.x;
        x[i + 1] *= n * w.y;
        x[i + 2] *= n * w.z;
        x[i + 3] *= n * w.w;
      }
      rotate16<kInter, false>(x, c, s);
    } else {
      rotate16<kInter, true>(d, c, s);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= n;  // u
      if (kind == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[0][i] = fmaf(d[i], x[i], acc[0][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[1][i] = fmaf(d[i], x[i], acc[1][i]);
      }
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(
            &sw[kind][(i < 8 ? at.c0 + i : at.c1 + i - 8)]);
        d[i] *= w.x;
        d[i + 1] *= w.y;
        d[i + 2] *= w.z;
        d[i + 3] *= w.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = fmaf(d[i + e], x[i + e], dot);
      }
      const float m = head_sum<kLanes>(dot) * (1.f / kDim);  // mean(g w u)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = n * (d[i] - x[i] * m);
    }
    if (real) {
      T* y = static_cast<T*>(a.y[kind]) + (token * a.heads[kind] + h) * kDim;
      *reinterpret_cast<uint4*>(y + at.c0) = pack8<T>(x);
      *reinterpret_cast<uint4*>(y + at.c1) = pack8<T>(x + 8);
    }
  }
  if (!kBack) return;
  // the warp's heads, then the CTA's warps, in order; sums where the rings were
  copies_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);  // [warps][2][dim]
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = acc[kind][i];
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (slot == 0) sums[(warp * 2 + kind) * kDim + (i < 8 ? at.c0 + i : at.c1 + i - 8)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kDim; i += kNormThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kNormWarps; ++w) v += sums[w * 2 * kDim + i];
    a.part[int64_t(blockIdx.x) * 2 * kDim + i] = v;
  }
}

constexpr int kJoinThreads = 1024;
template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) k_norm_rope_join(const NormArgs a) {
  constexpr int kWays = kJoinThreads / (2 * kDim);
  __shared__ float sums[kWays][2 * kDim];
  const int col = threadIdx.x % (2 * kDim), way = threadIdx.x / (2 * kDim);
  grid_dep_wait();
  grid_dep_release();
  float v = 0.f;
#pragma unroll 8
  for (int p = way; p < a.parts; p += kWays) v += a.part[int64_t(p) * 2 * kDim + col];
  sums[way][col] = v;
  __syncthreads();
  if (way == 0) {
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kWays; ++w) v += sums[w][col];
    a.dw[col / kDim][col % kDim] = v;
  }
}

constexpr int kMaxParts = 160;  // CTAs: one an SM
size_t norm_workspace(int32_t dim) { return sizeof(float) * kMaxParts * 2 * size_t(dim); }

// Forward, or the gradient (a.parts: its CTAs).
template <typename T, int kDim, bool kInter, bool kBack>
cudaError_t launch_norm_as(NormArgs& a, cudaStream_t s) {
  auto kernel = k_norm_rope<T, kDim, kInter, kBack>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, kNormSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t per = 512 / kDim, sms = std::min(device_sm_count(), kMaxParts);
  const int64_t groups = (a.heads[0] + per - 1) / per + (a.heads[1] + per - 1) / per;
  a.parts = int32_t(std::min<int64_t>(sms, a.T * groups));
  return launch_k(true, kernel, dim3(unsigned(a.parts)), dim3(kNormThreads), kNormSmem, s, a);
}
template <typename T, int kDim>
cudaError_t launch_norm(NormArgs& a, bool inter, bool back, cudaStream_t s) {
  if (back)
    return inter ? launch_norm_as<T, kDim, true, true>(a, s)
                 : launch_norm_as<T, kDim, false, true>(a, s);
  return inter ? launch_norm_as<T, kDim, true, false>(a, s)
               : launch_norm_as<T, kDim, false, false>(a, s);
}
cudaError_t launch_norm_any(NormArgs& a, const msa_norm_rope_args* p, bool back, cudaStream_t s) {
  const bool inter = p->interleaved != 0;
  if (p->dtype == MSA_BF16)
    return p->head_dim == 128 ? launch_norm<__nv_bfloat16, 128>(a, inter, back, s)
                              : launch_norm<__nv_bfloat16, 64>(a, inter, back, s);
  return p->head_dim == 128 ? launch_norm<__half, 128>(a, inter, back, s)
                            : launch_norm<__half, 64>(a, inter, back, s);
}
template <int kDim>
cudaError_t launch_norm_join(const NormArgs& a, cudaStream_t s) {
  return launch_k(true, k_norm_rope_join<kDim>, dim3(1), dim3(kJoinThreads), 0, s, a);
}

msa_status check_norm(const msa_norm_rope_args* p, NormArgs* a) {
  if (!p || !p->q || !p->k || !p->q_weight || !p->k_weight) return MSA_ERR_INVALID_ARG;
  if (p->T < 1 || p->T > kMaxTokens || (p->head_dim != 64 && p->head_dim != 128) ||
      p->q_heads < 1 || p->q_heads > 1024 || p->k_heads < 1 || p->k_heads > 1024 ||
      (p->dtype != MSA_BF16 && p->dtype != MSA_F16) || p->weight_dtype < 0 ||
      p->weight_dtype > MSA_F32)
    return MSA_ERR_INVALID_ARG;
  if (p->q_stride < int64_t(p->q_heads) * p->head_dim || p->q_stride % 8 ||
      p->k_stride < int64_t(p->k_heads) * p->head_dim || p->k_stride % 8)
    return MSA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || p->eps > 1e30f) return MSA_ERR_INVALID_ARG;
  if (p->inv_freq && (!p->positions || p->rotary_dim < 16 || p->rotary_dim % 16 ||
                      p->rotary_dim > p->head_dim))
    return MSA_ERR_INVALID_ARG;
  const uintptr_t w = p->weight_dtype == MSA_F32 ? 3 : 1;
  if (!paged_aligned(p->q) || !paged_aligned(p->k) || !paged_aligned4(p->positions) ||
      !paged_aligned4(p->inv_freq) || (reinterpret_cast<uintptr_t>(p->q_weight) & w) ||
      (reinterpret_cast<uintptr_t>(p->k_weight) & w))
    return MSA_ERR_ALIGNMENT;
  *a = NormArgs{};
  a->x[0] = p->q;
  a->x[1] = p->k;
  a->stride[0] = p->q_stride;
  a->stride[1] = p->k_stride;
  a->w[0] = p->q_weight;
  a->w[1] = p->k_weight;
  a->positions = p->positions;
  a->inv_freq = p->inv_freq;
  a->T = p->T;
  a->heads[0] = p->q_heads;
  a->heads[1] = p->k_heads;
  a->rot = p->inv_freq ? p->rotary_dim : 0;
  a->w_type = p->weight_dtype;
  a->eps = p->eps;
  return MSA_OK;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_norm_rope(const msa_norm_rope_args* args, void* q_out, void* k_out,
                                    msa_stream_t stream) {
  NormArgs a;
  msa_status st = check_norm(args, &a);
  if (st != MSA_OK) return st;
  if (!q_out || !k_out) return MSA_ERR_INVALID_ARG;
  if ((q_out == args->q && args->q_stride != int64_t(args->q_heads) * args->head_dim) ||
      (k_out == args->k && args->k_stride != int64_t(args->k_heads) * args->head_dim))
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(q_out) || !paged_aligned(k_out)) return MSA_ERR_ALIGNMENT;
  st = check_device();
  if (st != MSA_OK) return st;
  a.y[0] = q_out;
  a.y[1] = k_out;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin("norm_rope", s);
  const cudaError_t e = launch_norm_any(a, args, false, s);
  launch_end("norm_rope", s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

extern "C" msa_status msa_norm_rope_workspace_bytes(int32_t head_dim, size_t* bytes) {
  if (!bytes || (head_dim != 64 && head_dim != 128)) return MSA_ERR_INVALID_ARG;
  *bytes = norm_workspace(head_dim);
  return MSA_OK;
}

extern "C" msa_status msa_norm_rope_backward(const msa_norm_rope_args* args, const void* dq_out,
                                             const void* dk_out, void* dq, void* dk,
                                             float* dq_weight, float* dk_weight, void* workspace,
                                             size_t workspace_bytes, msa_stream_t stream) {
  NormArgs a;
  msa_status st = check_norm(args, &a);
  if (st != MSA_OK) return st;
  if (!dq_out || !dk_out || !dq || !dk || !dq_weight || !dk_weight || !workspace)
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(dq_out) || !paged_aligned(dk_out) || !paged_aligned(dq) ||
      !paged_aligned(dk) || !paged_aligned4(dq_weight) || !paged_aligned4(dk_weight) ||
      !paged_aligned(workspace))
    return MSA_ERR_ALIGNMENT;
  if (workspace_bytes < norm_workspace(args->head_dim)) return MSA_ERR_WORKSPACE;
  st = check_device();
  if (st != MSA_OK) return st;
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.y[0] = dq;
  a.y[1] = dk;
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  a.part = static_cast<float*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin("norm_rope_back", s);
  cudaError_t e = launch_norm_any(a, args, true, s);
  launch_end("norm_rope_back", s);
  if (e != cudaSuccess) return MSA_ERR_CUDA;
  launch_begin("norm_rope_join", s);
  e = args->head_dim == 128 ? launch_norm_join<128>(a, s) : launch_norm_join<64>(a, s);
  launch_end("norm_rope_join", s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
