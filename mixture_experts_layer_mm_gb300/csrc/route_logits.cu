// Routing from given router logits with what training the router needs: the
// top-k experts and their weights (as mm_route gives them), the per-expert
// counts, the balance loss, and the gradient of the logits.
//
//   p[t,:] = softmax(l[t,:]),  S(t) = the top_k largest (ties: lower id)
//   w[t,j] = p at the j-th id of S(t), with renorm divided by their sum
//   counts[e] = tokens whose S holds e,  n = tokens,  P[e] = sum_t p[t,e]
//   loss = E * sum_e (counts[e] / (n k)) * (P[e] / n)
//
// The counts are step functions of the logits, so the loss differentiates
// through p alone: dloss/dp[t,e] = c_e = E * counts[e] / (n^2 k).
//   dl[t,e] = p_e (a_e - sum_i p_i a_i), a = dloss * c + (dw at S, no renorm)
//   with renorm the weights are the softmax over S alone, which gives
//   dl[t, S_j] += w_j (dw_j - sum_i dw_i w_i).
// The two terms are formed separately: their own differences cancel, their
// sum does not.
//
// One warp takes one token; lane l holds experts l, l + 32, ... Both passes
// read each logit once. The sums over tokens stay in the lane that owns the
// expert, then go block by block through the caller's workspace in a fixed
// order, so every output is the same on every call.
#include <math.h>

#include "mm_device.cuh"
#include "mm_internal.h"

namespace mm {
namespace {

constexpr int kRlThreads = 512;
constexpr int kRlWarps = kRlThreads / 32;
constexpr uint32_t kFullMask = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return bf16_bits_to_f32(__ldg(p));
}
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
  return v;
}

// Logits of token t in l[q] (expert lane + 32 q), -INFINITY past E.
template <int Q, typename TL>
__device__ __forceinline__ void load_row(const TL* __restrict__ logits, uint32_t t, int E,
                                         float (&l)[Q]) {
  const int lane = threadIdx.x & 31;
  const TL* row = logits + (size_t)t * E + lane;
#pragma unroll
  for (int q = 0; q < Q; ++q) l[q] = lane + 32 * q < E ? load_logit(row + 32 * q) : -INFINITY;
}

// p = softmax(l). False (and p = 0) for a row without a logit above -inf.
template <int Q>
__device__ __forceinline__ bool softmax_row(const float (&l)[Q], float (&p)[Q]) {
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < Q; ++q) m = fmaxf(m, l[q]);
  m = warp_max(m);
  bool any = true;
  if (m == -INFINITY) {  // all -inf: no expert; a NaN among them: the row's p are NaN
    bool nan = false;
#pragma unroll
    for (int q = 0; q < Q; ++q) nan |= l[q] != l[q];
    any = __any_sync(kFullMask, nan);
  }
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    p[q] = any ? expf(l[q] - m) : 0.f;  // exp(-inf) = 0 past E
    s += p[q];
  }
  s = warp_sum(s);
  const float inv = any ? 1.f / s : 0.f;
#pragma unroll
  for (int q = 0; q < Q; ++q) p[q] *= inv;
  return any;
}

// The top_k largest of l as a bit set over q (bit q: expert lane + 32 q). A
// logit is compared as an order-preserving uint32 (-0 folded into +0), so
// one warp-wide maximum finds the value and one minimum the lowest id.
template <int Q>
__device__ __forceinline__ uint32_t select_topk(const float (&l)[Q], int E, int top_k) {
  const int lane = threadIdx.x & 31;
  uint32_t key[Q], sel = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const uint32_t b = __float_as_uint(l[q] + 0.0f);
    key[q] = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    if (lane + 32 * q >= E) key[q] = 0;  // below every logit (-inf maps to 0x007fffff)
    else if (key[q] == 0) key[q] = 1;    // a NaN with the lowest pattern
  }
  for (int r = 0; r < top_k; ++r) {
    uint32_t best = 0;
    int bq = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)  // strict '>' keeps the lower id of this lane
      if (key[q] > best) {
        best = key[q];
        bq = q;
      }
    const uint32_t top = __reduce_max_sync(kFullMask, best);
    const uint32_t id = best == top ? (uint32_t)(bq * 32 + lane) : 0xffffffffu;
    const uint32_t win = __reduce_min_sync(kFullMask, id);
    if (win == id) {
      sel |= 1u << bq;
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (q == bq) key[q] = 0;  // taken
    }
  }
  return sel;
}

struct RouteLogitsArgs {
  const uint8_t* mask;
  int32_t* ids;
  float* w;
  float* part_p;     // [gridDim.x][EP]
  int32_t* part_c;   // [gridDim.x][EP]
  int32_t* counts;   // [E]
  float* prob_sums;  // [E]
  float* loss;       // [1]
  int T, E, top_k, renorm;
};

// Sums over the rows of part_p / part_c in order, then the outputs over the
// whole batch. One block of kRlThreads; red: [kRlThreads] floats, redi ints.
template <int EP>
__device__ __forceinline__ void finish_batch(const float* part_p, const int32_t* part_c, int rows,
                                             const RouteLogitsArgs& a, float* red, int* redi) {
  constexpr int G = kRlThreads / EP;  // EP <= 256
  const int e = threadIdx.x % EP, g = threadIdx.x / EP;
  float p = 0.f;
  int c = 0;
#pragma unroll 8
  for (int r = g; r < rows; r += G) {
    p += part_p[(size_t)r * EP + e];
    c += part_c[(size_t)r * EP + e];
  }
  red[threadIdx.x] = p;
  redi[threadIdx.x] = c;
  __syncthreads();
  if (g == 0) {
    for (int i = 1; i < G; ++i) {
      p += red[i * EP + e];
      c += redi[i * EP + e];
    }
    if (e < a.E) {
      a.prob_sums[e] = p;
      a.counts[e] = c;
    }
  }
  __syncthreads();
  // sum_e counts = n k, and the loss (float products summed in a fixed tree).
  if (g == 0) {
    red[e] = e < a.E ? (float)c * p : 0.f;
    redi[e] = e < a.E ? c : 0;
  }
  __syncthreads();
#pragma unroll
  for (int o = EP / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) {
      red[threadIdx.x] += red[threadIdx.x + o];
      redi[threadIdx.x] += redi[threadIdx.x + o];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float nk = (float)redi[0], n = nk / (float)a.top_k;
    *a.loss = redi[0] > 0 ? (float)a.E * (red[0] / nk) / n : 0.f;
  }
}

template <int EP, typename TL>
__global__ void __launch_bounds__(kRlThreads) route_logits_kernel(const TL* __restrict__ logits,
                                                                  const RouteLogitsArgs a) {
  constexpr int Q = EP / 32;
  __shared__ float sp[kRlWarps * EP > kRlThreads ? kRlWarps * EP : kRlThreads];
  __shared__ int sc[kRlWarps * EP > kRlThreads ? kRlWarps * EP : kRlThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t stride = gridDim.x * kRlWarps, T = (uint32_t)a.T;  // t + stride < 2^32
  pdl_wait();
  pdl_trigger();
  float psum[Q];
  int cnt[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    psum[q] = 0.f;
    cnt[q] = 0;
  }
  float next[Q];
  uint32_t t = blockIdx.x * kRlWarps + warp;
  if (t < T) load_row<Q>(logits, t, a.E, next);
  for (; t < T; t += stride) {
    float l[Q], p[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = next[q];
    if (t + stride < T) load_row<Q>(logits, t + stride, a.E, next);
    const bool valid = softmax_row<Q>(l, p) && (a.mask == nullptr || a.mask[t] != 0);
    const uint32_t sel = select_topk<Q>(l, a.E, a.top_k);
    float total = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if ((sel >> q) & 1u) total += p[q];
    total = warp_sum(total);
    const float scale = !valid ? 0.f : a.renorm ? 1.f / total : 1.f;
    if (valid) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        psum[q] += p[q];
        cnt[q] += (int)((sel >> q) & 1u);
      }
    }
    // Ascending ids: slot = number of selected experts with a lower id.
    const uint32_t lt = (1u << lane) - 1u;
    int base = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const bool mine = (sel >> q) & 1u;
      const uint32_t bal = __ballot_sync(kFullMask, mine);
      if (mine) {
        const size_t at = (size_t)t * a.top_k + base + __popc(bal & lt);
        a.ids[at] = lane + 32 * q;
        a.w[at] = valid ? p[q] * scale : 0.f;
      }
      base += __popc(bal);
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    sp[warp * EP + lane + 32 * q] = psum[q];
    sc[warp * EP + lane + 32 * q] = cnt[q];
  }
  __syncthreads();
  float p = 0.f;
  int c = 0;
  if (threadIdx.x < EP) {
#pragma unroll
    for (int w = 0; w < kRlWarps; ++w) {
      p += sp[w * EP + threadIdx.x];
      c += sc[w * EP + threadIdx.x];
    }
  }
  if (gridDim.x > 1) {
    if (threadIdx.x < EP) {
      a.part_p[(size_t)blockIdx.x * EP + threadIdx.x] = p;
      a.part_c[(size_t)blockIdx.x * EP + threadIdx.x] = c;
    }
    return;
  }
  __syncthreads();
  __shared__ float one_p[EP];
  __shared__ int one_c[EP];
  if (threadIdx.x < EP) {
    one_p[threadIdx.x] = p;
    one_c[threadIdx.x] = c;
  }
  __syncthreads();
  finish_batch<EP>(one_p, one_c, 1, a, sp, sc);
}

template <int EP>
__global__ void __launch_bounds__(kRlThreads) route_logits_finish_kernel(int rows,
                                                                         const RouteLogitsArgs a) {
  __shared__ float red[kRlThreads];
  __shared__ int redi[kRlThreads];
  pdl_wait();
  finish_batch<EP>(a.part_p, a.part_c, rows, a, red, redi);
}

struct RouteLogitsBwdArgs {
  const uint8_t* mask;
  const int32_t* ids;
  const int32_t* counts;
  const float* dw;     // NULL: no gradient of the weights
  const float* dloss;  // NULL: no gradient of the loss
  int T, E, top_k, renorm;
};

template <int EP, typename TL>
__global__ void __launch_bounds__(kRlThreads) route_logits_backward_kernel(
    const TL* __restrict__ logits, TL* __restrict__ grad, const RouteLogitsBwdArgs a) {
  constexpr int Q = EP / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t stride = gridDim.x * kRlWarps, T = (uint32_t)a.T;  // t + stride < 2^32
  pdl_wait();
  pdl_trigger();
  // c_e = dloss * E * counts[e] / (n^2 k), with n k = sum of the counts.
  float c[Q];
  {
    float tot = 0.f;  // exact below 2^24, else off by 2^-24: far below the gradient's rounding
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      c[q] = lane + 32 * q < a.E ? (float)__ldg(a.counts + lane + 32 * q) : 0.f;
      tot += c[q];
    }
    tot = warp_sum(tot);
    const float g = a.dloss != nullptr ? __ldg(a.dloss) : 0.f;
    const float f = tot > 0.f ? g * (float)a.E / tot * ((float)a.top_k / tot) : 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) c[q] *= f;
  }
  float next[Q];
  uint32_t t = blockIdx.x * kRlWarps + warp;
  if (t < T) load_row<Q>(logits, t, a.E, next);
  for (; t < T; t += stride) {
    float l[Q], p[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = next[q];
    if (t + stride < T) load_row<Q>(logits, t + stride, a.E, next);
    const bool valid = softmax_row<Q>(l, p) && (a.mask == nullptr || a.mask[t] != 0);
    // dw and the selection, moved to the lanes that own the experts. An id
    // outside [0, E) or repeated takes no (further) part.
    float d[Q];
    uint32_t sel = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) d[q] = 0.f;
    if (a.dw != nullptr) {
      int id = -1;
      float dwj = 0.f;
      if (lane < a.top_k) {
        id = __ldg(a.ids + (size_t)t * a.top_k + lane);
        dwj = __ldg(a.dw + (size_t)t * a.top_k + lane);
      }
      for (int j = 0; j < a.top_k; ++j) {
        const int e = __shfl_sync(kFullMask, id, j);
        const float v = __shfl_sync(kFullMask, dwj, j);
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (e == lane + 32 * q && e < a.E && !((sel >> q) & 1u)) {
            sel |= 1u << q;
            d[q] = v;
          }
      }
    }
    float tot = 0.f, pd = 0.f, pc = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if ((sel >> q) & 1u) {
        tot += p[q];
        pd += p[q] * d[q];
      }
      pc += p[q] * c[q];
    }
    pc = warp_sum(pc);
    if (a.dw != nullptr) {
      pd = warp_sum(pd);
      if (a.renorm) tot = warp_sum(tot);
    }
    // renorm: w_j (dw_j - sum dw w) on the selected; else p (dw - sum dw p).
    const float inv = a.renorm && tot > 0.f ? 1.f / tot : 0.f;
    const float mean = a.renorm ? pd * inv : pd;
    TL* row = grad + (size_t)t * a.E + lane;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const bool mine = (sel >> q) & 1u;
      float g;
      if (a.renorm)
        g = mine ? p[q] * inv * (d[q] - mean) : 0.f;
      else
        g = p[q] * (d[q] - mean);
      g += p[q] * (c[q] - pc);
      if (lane + 32 * q < a.E) store_grad(row + 32 * q, valid ? g : 0.f);
    }
  }
}

template <int EP, typename TL>
cudaError_t forward_ep(const TL* logits, const RouteLogitsArgs& a, int blocks, cudaStream_t st) {
  cudaError_t e = launch_k(route_logits_kernel<EP, TL>, dim3(blocks), dim3(kRlThreads), 0, st,
                           false, logits, a);
  if (e != cudaSuccess || blocks == 1) return e;
  return launch_k(route_logits_finish_kernel<EP>, dim3(1), dim3(kRlThreads), 0, st, true, blocks,
                  a);
}

template <typename TL>
cudaError_t forward_t(const TL* logits, const RouteLogitsArgs& a, int blocks, cudaStream_t st) {
  if (a.E <= 32) return forward_ep<32>(logits, a, blocks, st);
  if (a.E <= 64) return forward_ep<64>(logits, a, blocks, st);
  if (a.E <= 128) return forward_ep<128>(logits, a, blocks, st);
  return forward_ep<256>(logits, a, blocks, st);
}

template <typename TL>
cudaError_t backward_t(const TL* logits, TL* grad, const RouteLogitsBwdArgs& a, int blocks,
                       cudaStream_t st) {
  const dim3 g(blocks), b(kRlThreads);
  if (a.E <= 32)
    return launch_k(route_logits_backward_kernel<32, TL>, g, b, 0, st, false, logits, grad, a);
  if (a.E <= 64)
    return launch_k(route_logits_backward_kernel<64, TL>, g, b, 0, st, false, logits, grad, a);
  if (a.E <= 128)
    return launch_k(route_logits_backward_kernel<128, TL>, g, b, 0, st, false, logits, grad, a);
  return launch_k(route_logits_backward_kernel<256, TL>, g, b, 0, st, false, logits, grad, a);
}

int ep_of(int E) { return E <= 32 ? 32 : E <= 64 ? 64 : E <= 128 ? 128 : 256; }

int blocks_for(int T, int num_sms) {
  const int want = (T + kRlWarps - 1) / kRlWarps;
  return want < 2 * num_sms ? want : 2 * num_sms;
}

}  // namespace

// Rows of partial sums the forward may write (one per block; the grid never
// exceeds 2 * 160 blocks).
constexpr int kRlMaxBlocks = 320;

long long route_logits_workspace(int T, int E) {
  if (T <= kRlWarps) return 0;
  const long long rows = (T + kRlWarps - 1) / kRlWarps;
  return (rows < kRlMaxBlocks ? rows : kRlMaxBlocks) * ep_of(E) * 8;
}

cudaError_t launch_route_logits(const void* logits, bool is_bf16, const uint8_t* mask, int T, int E,
                                int top_k, int renorm, int32_t* ids, float* w, int32_t* counts,
                                float* prob_sums, float* loss, void* workspace, int num_sms,
                                cudaStream_t st) {
  int blocks = T > 0 ? blocks_for(T, num_sms) : 1;
  if (blocks > kRlMaxBlocks) blocks = kRlMaxBlocks;
  const int EP = ep_of(E);
  RouteLogitsArgs a = {mask, ids, w, nullptr, nullptr, counts, prob_sums, loss, T, E, top_k, renorm};
  if (blocks > 1) {
    a.part_p = static_cast<float*>(workspace);
    a.part_c = reinterpret_cast<int32_t*>(a.part_p + (size_t)blocks * EP);
  }
  return is_bf16 ? forward_t(static_cast<const uint16_t*>(logits), a, blocks, st)
                 : forward_t(static_cast<const float*>(logits), a, blocks, st);
}

cudaError_t launch_route_logits_backward(const void* logits, bool is_bf16, const uint8_t* mask,
                                         const int32_t* ids, const int32_t* counts, const float* dw,
                                         const float* dloss, int T, int E, int top_k, int renorm,
                                         void* grad, int num_sms, cudaStream_t st) {
  const RouteLogitsBwdArgs a = {mask, ids, counts, dw, dloss, T, E, top_k, renorm};
  const int blocks = blocks_for(T, num_sms);
  return is_bf16 ? backward_t(static_cast<const uint16_t*>(logits), static_cast<uint16_t*>(grad), a,
                              blocks, st)
                 : backward_t(static_cast<const float*>(logits), static_cast<float*>(grad), a,
                              blocks, st);
}

}  // namespace mm
