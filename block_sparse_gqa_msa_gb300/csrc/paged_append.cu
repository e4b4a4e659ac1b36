// paged_append.cu - new tokens' keys and values into the paged cache, keys
// and queries rotated by their positions on the way.
//
// Mathematics: channel pair (x, y) number i of a token at position p becomes
// (x cos a - y sin a, y cos a + x sin a), a = p * inv_freq[i].  The angle is
// formed and reduced to one turn in 64 bits (p reaches 2^31, where a 32-bit
// product has lost the angle), its sine and cosine and the rotation are 32
// bits, and each result is rounded once to the cache's type.
//
// The work is a copy: q, k, v read once, q_out, cache (and k_out) written
// once.  A token is one CTA, or up to six are where they are many and narrow
// (launch_append).  An item is 16 channels (the two halves of 8 pairs, or 16
// that are copied); every thread loads all its items before it looks for the
// token's row, position and page and before the angles are formed, so those
// three dependent loads hide behind the data's.
//
// Measured: 17029 prompt tokens, 64 query heads and 4 key heads of 128 bf16
// channels, 645 MB: 95 us, 6.8 TB/s, a plain copy's rate; with 8 query heads
// and one key head (92 MB) 23.7 us, 38.8 if each token were its own CTA.  One
// token: 2.4 us, 150 tokens with 80 heads (6 MB, 0.9 us at that rate): 3.8 us:
// the launch and the dependent loads.
#include "paged.cuh"

namespace msa {
namespace {

constexpr int kAppThreads = 192;
constexpr int kAppItems = 3;  // items a thread holds: 192 x 3 = 64 + 4 + 4 heads of 128 channels
constexpr int kAppResident = 5;  // CTAs of several tokens (64 registers a thread) that an SM holds
constexpr int kAppTokens = kAppThreads / 32;  // the most tokens of a CTA: a warp places one

struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  void *q_out, *k_out;
  PagedPool kc, vc;
  PagedTable table;
  const int32_t *offs, *start;
  const float* inv_freq;
  int64_t T;
  int32_t q_heads, kv_heads, rot;
  int32_t share;  // items of one CTA (a multiple of its threads), where it has one token
  int32_t group;  // tokens of one CTA, where it has several
};

// Sine and cosine of pos * f.  The turns are counted in 64 bits (an exact
// product up to position 2^29) and only their fraction is rounded to 32.
__device__ __forceinline__ float2 turn_of(int64_t pos, float f) {
  const double turns = double(pos) * double(f) * 0.15915494309189533577;  // 1 / (2 pi)
  float s, c;
  sincospif(float(2.0 * (turns - rint(turns))), &s, &c);
  return make_float2(c, s);
}

template <typename T, int kDim, bool kInter, int kTokens>
__global__ void __launch_bounds__(kAppThreads) k_paged_append(const AppendArgs a) {
  constexpr int kPer = kDim / 16;  // items of a head
  __shared__ __align__(16) float cs[kTokens][kDim / 2], sn[kTokens][kDim / 2];
  __shared__ int64_t where[kTokens];  // the token's position
  __shared__ int32_t where_page[kTokens];
  const int tid = threadIdx.x;
  const int each = (a.q_heads + 2 * a.kv_heads) * kPer;  // items of a token
  const int64_t t0 = kTokens == 1 ? blockIdx.x : int64_t(blockIdx.x) * a.group;
  const int tokens = kTokens == 1 ? 1 : int(min(int64_t(a.group), a.T - t0));
  const int first = kTokens == 1 ? blockIdx.y * a.share : 0;
  const int items = kTokens == 1 ? min(each, first + a.share) : tokens * each;
  grid_dep_wait();
  grid_dep_release();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    check_offsets(a.offs, a.table.rows, a.T, a.table.status);

  bool placed = false;
  int32_t page = -1;
  int64_t pos = 0;
  const int half = a.rot / 2;
  for (int base = first; base < items; base += kAppThreads * kAppItems) {
    // Items run over the key heads, the value heads, the query heads.
    uint4 x[kAppItems], y[kAppItems];
    int head[kAppItems], c0[kAppItems], c1[kAppItems], tok[kAppItems];
    bool turn[kAppItems];
#pragma unroll
    for (int i = 0; i < kAppItems; ++i) {
      const int it = base + i * kAppThreads + tid;
      if (it >= items) {
        head[i] = -1;
        continue;
      }
      tok[i] = kTokens == 1 ? 0 : it / each;
      const int own = it - tok[i] * each;
      head[i] = own / kPer;
      const int sub = own % kPer;
      const int64_t t = t0 + tok[i];
      const bool is_v = head[i] >= a.kv_heads && head[i] < 2 * a.kv_heads;
      turn[i] = !is_v && sub * 16 < a.rot;
      // the item's two runs of 8 channels
      if (turn[i] && !kInter) {
        c0[i] = sub * 8;
        c1[i] = sub * 8 + half;
      } else {
        c0[i] = sub * 16;
        c1[i] = sub * 16 + 8;
      }
      const T* src;
      if (head[i] < a.kv_heads)
        src = static_cast<const T*>(a.k) + t * a.k_stride + head[i] * kDim;
      else if (is_v)
        src = static_cast<const T*>(a.v) + t * a.v_stride + (head[i] - a.kv_heads) * kDim;
      else
        src = static_cast<const T*>(a.q) + t * a.q_stride + (head[i] - 2 * a.kv_heads) * kDim;
      x[i] = *reinterpret_cast<const uint4*>(src + c0[i]);
      y[i] = *reinterpret_cast<const uint4*>(src + c1[i]);
    }
    if (kTokens > 1) {  // one round of the loop: each of the first warps places a token
      const int w = tid / 32, lane = tid % 32;
      if (w < tokens) {
        const int64_t t = t0 + w;
        const int32_t r = find_row_warp(a.offs, a.table.rows, t);
        const int32_t o0 = a.offs[r], o1 = a.offs[r + 1];
        if (o0 >= 0 && t >= o0 && t < o1) {
          pos = int64_t(a.start[r]) + (t - o0);
          page = page_of(a.table, r, pos);
          for (int i = lane; i < half; i += 32) {
            const float2 turned = turn_of(pos, a.inv_freq[i]);
            cs[w][i] = turned.x;
            sn[w][i] = turned.y;
          }
        }
        if (lane == 0) {
          where[w] = pos;
          where_page[w] = page;
        }
      }
      __syncthreads();
    } else if (!placed) {
      placed = true;
      const int32_t r = find_row_warp(a.offs, a.table.rows, t0);
      const int32_t o0 = a.offs[r], o1 = a.offs[r + 1];
      if (o0 < 0 || t0 < o0 || t0 >= o1) return;  // padding: no row owns this token
      pos = int64_t(a.start[r]) + (t0 - o0);
      page = page_of(a.table, r, pos);
      if (page < 0) return;
      if (tid < half) {
        const float2 w = turn_of(pos, a.inv_freq[tid]);
        cs[0][tid] = w.x;
        sn[0][tid] = w.y;
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kAppItems; ++i) {
      if (head[i] < 0) continue;
      if (kTokens > 1) {
        pos = where[tok[i]];
        page = where_page[tok[i]];
        if (page < 0) continue;  // padding, or no page of the cache
      }
      const int64_t t = t0 + tok[i];
      const int64_t slot = pos & ((int64_t(1) << a.table.shift) - 1);
      if (turn[i]) {
        uint32_t* xw = reinterpret_cast<uint32_t*>(&x[i]);
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y[i]);
        // the item's first pair: channels (p, p + half) or (2 p, 2 p + 1)
        const int p = kInter ? c0[i] / 2 : c0[i];
        float cc[8], ss[8];
        *reinterpret_cast<float4*>(cc) = *reinterpret_cast<const float4*>(cs[tok[i]] + p);
        *reinterpret_cast<float4*>(cc + 4) = *reinterpret_cast<const float4*>(cs[tok[i]] + p + 4);
        *reinterpret_cast<float4*>(ss) = *reinterpret_cast<const float4*>(sn[tok[i]] + p);
        *reinterpret_cast<float4*>(ss + 4) = *reinterpret_cast<const float4*>(sn[tok[i]] + p + 4);
        if (kInter) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 u = Pair<T>::unpack(xw[w]), v = Pair<T>::unpack(yw[w]);
            xw[w] = Pair<T>::pack(u.x * cc[w] - u.y * ss[w], u.y * cc[w] + u.x * ss[w]);
            yw[w] = Pair<T>::pack(v.x * cc[w + 4] - v.y * ss[w + 4],
                                  v.y * cc[w + 4] + v.x * ss[w + 4]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 u = Pair<T>::unpack(xw[w]), v = Pair<T>::unpack(yw[w]);
            xw[w] = Pair<T>::pack(u.x * cc[2 * w] - v.x * ss[2 * w],
                                  u.y * cc[2 * w + 1] - v.y * ss[2 * w + 1]);
            yw[w] = Pair<T>::pack(v.x * cc[2 * w] + u.x * ss[2 * w],
                                  v.y * cc[2 * w + 1] + u.y * ss[2 * w + 1]);
          }
        }
      }
      T* dst;
      if (head[i] < a.kv_heads) {
        dst = static_cast<T*>(a.kc.base) + page * a.kc.page + slot * a.kc.token +
              head[i] * a.kc.head;
        if (a.k_out) {
          T* ko = static_cast<T*>(a.k_out) + (t * a.kv_heads + head[i]) * kDim;
          *reinterpret_cast<uint4*>(ko + c0[i]) = x[i];
          *reinterpret_cast<uint4*>(ko + c1[i]) = y[i];
        }
      } else if (head[i] < 2 * a.kv_heads) {
        dst = static_cast<T*>(a.vc.base) + page * a.vc.page + slot * a.vc.token +
              (head[i] - a.kv_heads) * a.vc.head;
      } else {
        dst = static_cast<T*>(a.q_out) + (t * a.q_heads + head[i] - 2 * a.kv_heads) * kDim;
      }
      *reinterpret_cast<uint4*>(dst + c0[i]) = x[i];
      *reinterpret_cast<uint4*>(dst + c1[i]) = y[i];
    }
  }
}

template <typename T, int kDim>
cudaError_t launch_append(AppendArgs a, bool inter, cudaStream_t s) {
  const int items = (a.q_heads + 2 * a.kv_heads) * (kDim / 16);
  // Few tokens: several CTAs a token, while there are SMs for them.
  const int64_t rounds = (items + kAppThreads - 1) / kAppThreads;
  int64_t slices = device_sm_count() / a.T;
  if (slices < 1) slices = 1;
  if (slices > rounds) slices = rounds;
  const int64_t each = (rounds + slices - 1) / slices;  // rounds of a CTA
  a.share = int32_t(each * kAppThreads);
  // Many tokens of few heads: as many to a CTA as its items hold, but no more
  // than bring all the CTAs to the SMs at once (one head of 64 channels: 4015
  // tokens 10.2 -> 4.7 us, 1000 tokens 4.5 -> 3.2; 3.9 against 4.6 us for 600
  // tokens of 10 heads of 128 if they were grouped as well).
  const int64_t wave = int64_t(device_sm_count()) * kAppResident;
  const int64_t group = std::min<int64_t>(
      std::min<int64_t>(kAppTokens, kAppThreads * kAppItems / items), (a.T + wave - 1) / wave);
  if (group > 1) {
    a.group = int32_t(group);
    const dim3 grid(unsigned((a.T + group - 1) / group));
    return inter ? launch_k(true, k_paged_append<T, kDim, true, kAppTokens>, grid,
                            dim3(kAppThreads), 0, s, a)
                 : launch_k(true, k_paged_append<T, kDim, false, kAppTokens>, grid,
                            dim3(kAppThreads), 0, s, a);
  }
  const dim3 grid(unsigned(a.T), unsigned((rounds + each - 1) / each));
  return inter
             ? launch_k(true, k_paged_append<T, kDim, true, 1>, grid, dim3(kAppThreads), 0, s, a)
             : launch_k(true, k_paged_append<T, kDim, false, 1>, grid, dim3(kAppThreads), 0, s, a);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_paged_append(const msa_paged_cache* cache, const msa_page_table* table,
                                       const int32_t* row_offsets, const int32_t* start_pos,
                                       int64_t T, const void* k, int64_t k_stride, const void* v,
                                       int64_t v_stride, const void* q, int64_t q_stride,
                                       int32_t q_heads, const float* inv_freq,
                                       int32_t rotary_dim, int32_t interleaved, void* q_out,
                                       void* k_out, msa_stream_t stream) {
  msa_status st = check_cache(cache);
  if (st != MSA_OK) return st;
  st = check_table(table, cache->page_size);
  if (st != MSA_OK) return st;
  if (!row_offsets || !start_pos || !k || !v || T < 1 || T > kMaxTokens)
    return MSA_ERR_INVALID_ARG;
  const int64_t kv_width = int64_t(cache->kv_heads) * cache->head_dim;
  if (k_stride < kv_width || k_stride % 8 || v_stride < kv_width || v_stride % 8)
    return MSA_ERR_INVALID_ARG;
  if (q) {
    if (!q_out || q_heads < 1 || q_heads > 1024 || q_stride % 8 ||
        q_stride < int64_t(q_heads) * cache->head_dim)
      return MSA_ERR_INVALID_ARG;
    if (q_out == q && q_stride != int64_t(q_heads) * cache->head_dim) return MSA_ERR_INVALID_ARG;
  } else if (q_out) {
    return MSA_ERR_INVALID_ARG;
  }
  if (inv_freq && (rotary_dim < 16 || rotary_dim % 16 || rotary_dim > cache->head_dim))
    return MSA_ERR_INVALID_ARG;
  if (!paged_aligned(k) || !paged_aligned(v) || !paged_aligned(q) || !paged_aligned(q_out) ||
      !paged_aligned(k_out) || !paged_aligned4(row_offsets) || !paged_aligned4(start_pos) ||
      !paged_aligned4(inv_freq))
    return MSA_ERR_ALIGNMENT;
  st = check_device();
  if (st != MSA_OK) return st;
  AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.k_out = k_out;
  a.kc = PagedPool{cache->k, cache->k_stride[0], cache->k_stride[1], cache->k_stride[2]};
  a.vc = PagedPool{cache->v, cache->v_stride[0], cache->v_stride[1], cache->v_stride[2]};
  a.table = table_args(table, cache->page_size, cache->num_pages, cache->status);
  a.offs = row_offsets;
  a.start = start_pos;
  a.inv_freq = inv_freq;
  a.T = T;
  a.q_heads = q ? q_heads : 0;
  a.kv_heads = cache->kv_heads;
  a.rot = inv_freq ? rotary_dim : 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = interleaved != 0;
  launch_begin("paged_append", s);
  cudaError_t e;
  if (cache->dtype == MSA_BF16)
    e = cache->head_dim == 128 ? launch_append<__nv_bfloat16, 128>(a, inter, s)
                               : launch_append<__nv_bfloat16, 64>(a, inter, s);
  else
    e = cache->head_dim == 128 ? launch_append<__half, 128>(a, inter, s)
                               : launch_append<__half, 64>(a, inter, s);
  launch_end("paged_append", s);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

extern "C" msa_status msa_paged_read_status(const int64_t* status, msa_stream_t stream) {
  if (!status) return MSA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(status) & 7u) return MSA_ERR_ALIGNMENT;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return MSA_ERR_CUDA;
  int64_t bits = 0;
  if (cudaMemcpy(&bits, status, sizeof bits, cudaMemcpyDeviceToHost) != cudaSuccess)
    return MSA_ERR_CUDA;
  for (int c = 1; c < 63; ++c)
    if (bits & (int64_t(1) << c)) return static_cast<msa_status>(c);
  return MSA_OK;
}
