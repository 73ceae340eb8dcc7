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
// One warp takes one token; lane l holds the Q = 1, 2, 4 or 8 consecutive
// experts from l Q on (one vector load). Both passes read each logit once. The
// sums over tokens stay in the lane that owns the expert, then go block by block
// through the caller's workspace in a fixed order, so every output is the same
// on every call. A lane adds kRlChain tokens' p at most in plain fp32; longer
// sums (2^31 tokens are 440,000 a lane) keep their roundings, and all others are
// added in pairs: a sum is off by some 25 half steps at most, whatever T.
//
// What bounds it: small batches are launches (64 tokens x 128 experts 3.7 us in a
// captured graph, 5.4 a call back to back; 4096 x 128 in bf16 forward and backward
// 11.3 us a call). 131072 x 256 fp32 logits take 80 us forward and 54 us backward,
// 134 and 268 MB: the forward issues some 540 instructions a token (selection and
// the exponentials, mostly of the half-rate kind), 75 % of the issue slots; the
// backward 290, at 5 TB/s.
#include <math.h>

#include "mm_device.cuh"
#include "mm_internal.h"

namespace mm {
namespace {

constexpr int kRlThreads = 512;
constexpr int kRlWarps = kRlThreads / 32;
// Small batches take one launch and no workspace: one block up to
// kRlOneBlockTokens, one cluster up to kRlClusterTokens, two tokens a warp at
// most. 128 experts, us a call in a captured graph: 64 tokens 3.7 in a cluster,
// 5.8 in one block; 128 tokens 3.9, 4.9 in two launches; 256 tokens 5.1 and 4.9,
// but 5.6 and 9.3 outside of a graph, where a launch costs the host as much as the
// kernel takes: the cluster up to there gives up a little in a graph for that.
constexpr int kRlOneBlockWarps = 32;
constexpr int kRlOneBlockTokens = 32;
constexpr uint32_t kRlClusterBlocks = 8;
constexpr int kRlClusterTokens = 2 * kRlClusterBlocks * kRlWarps;
constexpr uint32_t kFullMask = 0xffffffffu;
constexpr uint32_t kRlChain = 8;  // tokens between two additions to a lane's long sums

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return bf16_bits_to_f32(__ldg(p));
}
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }

// Q consecutive values as one access (p aligned to its size, up to 32 bytes).
template <int Q>
__device__ __forceinline__ void load_vec(const float* p, float (&l)[Q]) {
  if constexpr (Q == 1) {
    l[0] = __ldg(p);
  } else if constexpr (Q == 2) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    l[0] = v.x;
    l[1] = v.y;
  } else if constexpr (Q == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    l[0] = v.x;
    l[1] = v.y;
    l[2] = v.z;
    l[3] = v.w;
  } else {
    asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(l[0]), "=f"(l[1]), "=f"(l[2]), "=f"(l[3]), "=f"(l[4]), "=f"(l[5]), "=f"(l[6]),
          "=f"(l[7])
        : "l"(p));
  }
}
template <int Q>
__device__ __forceinline__ void load_vec(const uint16_t* p, float (&l)[Q]) {
  uint32_t w[(Q + 1) / 2];
  if constexpr (Q == 1) w[0] = __ldg(p);
  if constexpr (Q == 2) w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  if constexpr (Q == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x;
    w[1] = v.y;
  }
  if constexpr (Q == 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q)
    l[q] = __uint_as_float((q & 1) ? w[q / 2] & 0xFFFF0000u : w[q / 2] << 16);
}
template <int Q>
__device__ __forceinline__ void store_vec(float* p, const float (&g)[Q]) {
  if constexpr (Q == 1) *p = g[0];
  if constexpr (Q == 2) *reinterpret_cast<float2*>(p) = make_float2(g[0], g[1]);
  if constexpr (Q == 4) *reinterpret_cast<float4*>(p) = make_float4(g[0], g[1], g[2], g[3]);
  if constexpr (Q == 8)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(g[0]),
                 "f"(g[1]), "f"(g[2]), "f"(g[3]), "f"(g[4]), "f"(g[5]), "f"(g[6]), "f"(g[7])
                 : "memory");
}
template <int Q>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&g)[Q]) {
  if constexpr (Q == 1) {
    *p = f32_to_bf16_bits(g[0]);
  } else {
    uint32_t w[Q / 2];
#pragma unroll
    for (int i = 0; i < Q / 2; ++i)
      w[i] = (uint32_t)f32_to_bf16_bits(g[2 * i]) | ((uint32_t)f32_to_bf16_bits(g[2 * i + 1]) << 16);
    if constexpr (Q == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
    if constexpr (Q == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    if constexpr (Q == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Q values of a lane to shared memory, p aligned to 4 Q bytes or 16.
template <int Q>
__device__ __forceinline__ void stage(float* p, const float (&g)[Q]) {
  if constexpr (Q == 1) *p = g[0];
  if constexpr (Q == 2) *reinterpret_cast<float2*>(p) = make_float2(g[0], g[1]);
#pragma unroll
  for (int i = 0; i + 3 < Q; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]);
}

// a + b, and in b what its rounding left out (exact).
__device__ __forceinline__ float add_keep(float a, float& b) {
  const float s = a + b, bb = s - a;
  b = (a - (s - bb)) + (b - bb);
  return s;
}

// Sum of n values (a power of two) a stride apart, added in pairs.
template <int N>
__device__ __forceinline__ float pair_sum(const float* v, int stride) {
  if constexpr (N == 1) {
    return *v;
  } else {
    return pair_sum<N / 2>(v, stride) + pair_sum<N / 2>(v + N / 2 * stride, stride);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
  return v;
}

// Logits of token t: l[q] of expert lane Q + q, -INFINITY past E. vec: rows
// begin at multiples of Q values and E is one, so a lane's values are all in
// or all out and aligned.
template <int Q, typename TL>
__device__ __forceinline__ void load_row(const TL* __restrict__ logits, uint32_t t, int E, bool vec,
                                         float (&l)[Q]) {
  const int e0 = (threadIdx.x & 31) * Q;
  const TL* row = logits + (size_t)t * E + e0;
  if (vec) {
    if (e0 < E) {
      load_vec<Q>(row, l);
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) l[q] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = e0 + q < E ? load_logit(row + q) : -INFINITY;
  }
}

template <int Q, typename TL>
__device__ __forceinline__ void store_row(TL* row, int E, bool vec, const float (&g)[Q]) {
  const int e0 = (threadIdx.x & 31) * Q;
  if (vec) {
    if (e0 < E) store_vec<Q>(row + e0, g);
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (e0 + q < E) store_grad(row + e0 + q, g[q]);
  }
}

// Sum of v over the lanes below this one.
__device__ __forceinline__ int exclusive_sum(int v) {
  const int lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl += u;
  }
  return incl - v;
}

// Maximum over the warp; no input is a NaN.
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// e^x for x <= 0 (or NaN): 2^t with t = x log2(e) in two parts, the second what
// the first product and the constant's rounding leave out (both grow with |x|), so
// that the error stays at that of the hardware's 2^t (2^-22) and one rounding
// (2^-24) for any x. Below 2^-126: 0. Two values, or one.
__device__ __forceinline__ Pair exp_neg(Pair x) {
  constexpr double kLog2eExact = 1.44269504088896341;
  constexpr float kLog2e = (float)kLog2eExact, kLog2eRest = (float)(kLog2eExact - kLog2e);
  constexpr float kLn2 = 0.693147180559945309f;
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(-200.f));  // e^-200 is below 2^-126 too
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(-200.f));
  const Pair t = x * Pair{kLog2e, kLog2e};
  const Pair rest = fma2(x, Pair{-kLog2eRest, -kLog2eRest},
                         fma2(x, Pair{-kLog2e, -kLog2e}, t));  // negative
  Pair r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(t.y));
  return fma2(r, rest * Pair{-kLn2, -kLn2}, r);
}
__device__ __forceinline__ float exp_neg(float x) { return exp_neg(Pair{x, x}).x; }

// f of pairs (or, of a lane's one value, a pair of it) of a lane's Q values.
template <int Q, typename F>
__device__ __forceinline__ void each_pair(F f) {
#pragma unroll
  for (int q = 0; q < Q; q += 2) f(q, Q == 1 ? 0 : q + 1);
}

// p = exp(l - m) (not yet divided by the returned sum), m the row's largest
// logit that is not a NaN. A row without a logit above -inf has p = 0 and
// sum 0; one that holds a NaN or +inf has a NaN sum.
template <int Q>
__device__ __forceinline__ float exp_row(const float (&l)[Q], float m, float (&p)[Q]) {
  if (m == -INFINITY) {  // all -inf; or NaN among them
    bool nan = false;
#pragma unroll
    for (int q = 0; q < Q; ++q) nan |= l[q] != l[q];
    nan = __any_sync(kFullMask, nan);
#pragma unroll
    for (int q = 0; q < Q; ++q) p[q] = 0.f;
    return nan ? __uint_as_float(0x7fffffffu) : 0.f;
  }
  Pair s = {0.f, 0.f};
  each_pair<Q>([&](int a, int b) {
    const Pair e = exp_neg(Pair{l[a], l[b]} + Pair{-m, -m});  // 0 past E
    s = s + e;
    p[a] = e.x;
    p[b] = e.y;
  });
  return warp_sum(Q == 1 ? s.x : s.x + s.y);
}

// Descending order of Q values (compare-exchange networks of 1, 5 and 19
// steps; values only, no index travels with them).
__device__ __forceinline__ void order2(float& a, float& b) {
  const float hi = fmaxf(a, b);
  b = fminf(a, b);
  a = hi;
}
template <int Q>
__device__ __forceinline__ void sort_desc(float (&v)[Q]) {
  static_assert(Q == 1 || Q == 2 || Q == 4 || Q == 8, "networks below");
  if constexpr (Q == 2) order2(v[0], v[1]);
  if constexpr (Q == 4) {
    order2(v[0], v[1]); order2(v[2], v[3]);
    order2(v[0], v[2]); order2(v[1], v[3]);
    order2(v[1], v[2]);
  }
  if constexpr (Q == 8) {
    order2(v[0], v[1]); order2(v[2], v[3]); order2(v[4], v[5]); order2(v[6], v[7]);
    order2(v[0], v[2]); order2(v[1], v[3]); order2(v[4], v[6]); order2(v[5], v[7]);
    order2(v[1], v[2]); order2(v[5], v[6]); order2(v[0], v[4]); order2(v[3], v[7]);
    order2(v[1], v[5]); order2(v[2], v[6]);
    order2(v[1], v[4]); order2(v[3], v[6]);
    order2(v[2], v[4]); order2(v[3], v[5]);
    order2(v[3], v[4]);
  }
}

// The top_k largest of the row: bit q of the returned word for expert
// lane Q + q. Every lane sorts its values; then the warp takes the largest
// head, drops it from every lane that shows it, and so on until top_k values
// are gone: that head is the top_k-th largest value, and what is at or above
// it is the selection. Only when more values equal it than have room, or it is
// -inf, which NaN and the places past E rank as, do the ids below E decide: the
// lowest stay. m: the largest value.
template <int Q>
__device__ __forceinline__ uint32_t select_topk(const float (&l)[Q], int E, int top_k, float& m) {
  const int lane = threadIdx.x & 31;
  float v[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) v[q] = fmaxf(l[q], -INFINITY);  // a NaN ranks as -inf
  sort_desc<Q>(v);
  float top = redux_max(v[0]);
  m = top;
  int left = top_k;
  while (true) {
    const bool here = v[0] == top;
    left -= __popc(__ballot_sync(kFullMask, here));
    if (left <= 0) break;
    if (here) {
#pragma unroll
      for (int q = 0; q + 1 < Q; ++q) v[q] = v[q + 1];
      v[Q - 1] = -INFINITY;
    }
    top = redux_max(v[0]);
  }
  uint32_t sel = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (l[q] >= top) sel |= 1u << q;
  const uint32_t total = __reduce_add_sync(kFullMask, (uint32_t)__popc(sel));
  if (total != (uint32_t)top_k || top == -INFINITY) {
    uint32_t above = 0, equal = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (l[q] > top) above |= 1u << q;
      if (fmaxf(l[q], -INFINITY) == top && lane * Q + q < E) equal |= 1u << q;
    }
    int room = top_k - (int)__reduce_add_sync(kFullMask, (uint32_t)__popc(above));
    room -= exclusive_sum(__popc(equal));
    for (; room > 0 && equal != 0; --room) {
      const uint32_t low = equal & (0u - equal);
      above |= low;
      equal ^= low;
    }
    sel = above;
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
  int T, E, top_k, renorm, vec;
};

// The outputs over the whole batch from its sums, thread e < EP holding
// expert e's p and c. red, redi: [EP] shared each, free to overwrite. All
// threads of the block call this (it has barriers).
template <int EP>
__device__ __forceinline__ void write_batch(float p, int c, const RouteLogitsArgs& a, float* red,
                                            int* redi) {
  const int e = threadIdx.x;
  if (e < EP) {
    if (e < a.E) {
      a.prob_sums[e] = p;
      a.counts[e] = c;
    }
    red[e] = e < a.E ? (float)c * p : 0.f;
    redi[e] = e < a.E ? c : 0;
  }
  __syncthreads();
#pragma unroll
  for (int o = EP / 2; o > 0; o >>= 1) {
    if (e < o) {
      red[e] += red[e + o];
      redi[e] += redi[e + o];
    }
    __syncthreads();
  }
  if (e == 0) {  // sum_e counts = n k
    const float nk = (float)redi[0], n = nk / (float)a.top_k;
    *a.loss = redi[0] > 0 ? (float)a.E * (red[0] / nk) / n : 0.f;
  }
}

// CLUSTER: the grid is one cluster, whose first block adds the blocks' sums up.
template <int EP, int W, bool CLUSTER, typename TL>
__device__ __forceinline__ void route_logits_block(const TL* __restrict__ logits,
                                                   const RouteLogitsArgs& a) {
  constexpr int Q = EP / 32;
  __shared__ __align__(16) float sp[W * EP];  // a warp's p of its token; at the end its sums
  __shared__ int sc[EP], sid[W * 32];         // counts; a warp's selection, ascending
  // A warp's long sums; the small batches' warps have two tokens at most.
  constexpr bool kLong = !CLUSTER && W == kRlWarps;
  __shared__ __align__(16) float slong[kLong ? W * EP : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t stride = gridDim.x * W, T = (uint32_t)a.T;  // t + stride < 2^32
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < EP) sc[threadIdx.x] = 0;
  __syncthreads();
  float psum[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) psum[q] = 0.f;
  float* mine = &slong[kLong ? warp * EP + lane * Q : 0];
  if (kLong) stage<Q>(mine, psum);
  uint32_t chain = 0;
  float next[Q];
  uint32_t t = blockIdx.x * W + warp;
  if (t < T) load_row<Q>(logits, t, a.E, a.vec, next);
  for (; t < T; t += stride) {
    float l[Q], p[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = next[q];
    if (t + stride < T) load_row<Q>(logits, t + stride, a.E, a.vec, next);
    float m;
    const uint32_t sel = select_topk<Q>(l, a.E, a.top_k, m);
    const float sum = exp_row<Q>(l, m, p);
    const bool valid = sum != 0.f && (a.mask == nullptr || a.mask[t] != 0);
    // The selected in ascending order (place = number of selected with a lower
    // id) and all p go through shared memory, so that lane j has the j-th.
    __syncwarp();
    int at = exclusive_sum(__popc(sel));
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if ((sel >> q) & 1u) sid[warp * 32 + at++] = lane * Q + q;
    stage<Q>(&sp[warp * EP + lane * Q], p);
    __syncwarp();
    int id = 0;
    float pj = 0.f;
    if (lane < a.top_k) {
      id = sid[warp * 32 + lane];
      pj = sp[warp * EP + id];
    }
    // Weights of the selected: p / sum, or p over the selected p alone.
    float scale = 0.f;
    if (valid) {
      const float inv = 1.f / sum;
      scale = inv;
      if (a.renorm) {
        const float total = warp_sum(pj);
        scale = sum == sum ? 1.f / total : sum;  // a NaN in the row: all its weights
      }
      each_pair<Q>([&](int a, int b) {
        const Pair n = fma2(Pair{p[a], p[b]}, Pair{inv, inv}, Pair{psum[a], psum[b]});
        psum[a] = n.x;
        psum[b] = n.y;
      });
    }
    if (kLong && ++chain == kRlChain) {
      chain = 0;
      float l[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) l[q] = add_keep(mine[q], psum[q]);
      stage<Q>(mine, l);
    }
    if (lane < a.top_k) {
      a.ids[(size_t)t * a.top_k + lane] = id;
      a.w[(size_t)t * a.top_k + lane] = valid ? pj * scale : 0.f;
      if (valid) atomicAdd(&sc[id], 1);  // integers: any order
    }
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < Q; ++q) sp[warp * EP + lane * Q + q] = psum[q];
  __syncthreads();
  float p = 0.f;
  int c = 0;
  if (threadIdx.x < EP) {
    p = pair_sum<W>(&sp[threadIdx.x], EP);
    if (kLong) p += pair_sum<W>(&slong[threadIdx.x], EP);
    c = sc[threadIdx.x];
  }
  if constexpr (CLUSTER) {
    __syncthreads();  // sp has been read
    if (threadIdx.x < EP) sp[threadIdx.x] = p;
    cluster_barrier();
    if (blockIdx.x == 0 && threadIdx.x < EP) {
      float part[kRlClusterBlocks];
      c = 0;
#pragma unroll
      for (uint32_t r = 0; r < kRlClusterBlocks; ++r) {
        part[r] = load_peer(&sp[threadIdx.x], r);
        c += load_peer(&sc[threadIdx.x], r);
      }
      p = pair_sum<kRlClusterBlocks>(part, 1);
    }
    cluster_barrier();  // all sums have been read
    if (blockIdx.x != 0) return;
  } else if (gridDim.x > 1) {
    if (threadIdx.x < EP) {
      a.part_p[(size_t)blockIdx.x * EP + threadIdx.x] = p;
      a.part_c[(size_t)blockIdx.x * EP + threadIdx.x] = c;
    }
    return;
  }
  __syncthreads();
  write_batch<EP>(p, c, a, sp, sc);
}

template <int EP, int W, typename TL>
__global__ void __launch_bounds__(W * 32) route_logits_kernel(const TL* __restrict__ logits,
                                                              const RouteLogitsArgs a) {
  route_logits_block<EP, W, false>(logits, a);
}

template <int EP, typename TL>
__global__ void __cluster_dims__(kRlClusterBlocks, 1, 1) __launch_bounds__(kRlThreads)
    route_logits_cluster_kernel(const TL* __restrict__ logits, const RouteLogitsArgs a) {
  route_logits_block<EP, kRlWarps, true>(logits, a);
}

// The blocks' sums, added in a fixed order: EP / 4 threads a row take 4 experts
// each, kRlFinish / (EP / 4) rows at a time. A thread adds kRlBatch rows in pairs
// before it adds them to the others.
constexpr int kRlFinish = 1024, kRlBatch = 8;

template <int EP>
__global__ void __launch_bounds__(kRlFinish) route_logits_finish_kernel(int rows,
                                                                        const RouteLogitsArgs a) {
  constexpr int C = EP / 4, G = kRlFinish / C;
  __shared__ float4 ps[G][C];
  __shared__ int4 cs[G][C];
  const int c4 = threadIdx.x % C, g = threadIdx.x / C;
  pdl_wait();
  pdl_trigger();
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
  int4 c = make_int4(0, 0, 0, 0);
  const float4* pp = reinterpret_cast<const float4*>(a.part_p) + c4;
  const int4* pc = reinterpret_cast<const int4*>(a.part_c) + c4;
  for (int r0 = g; r0 < rows; r0 += kRlBatch * G) {
    float4 u[kRlBatch];
#pragma unroll
    for (int i = 0; i < kRlBatch; ++i) {
      const int r = r0 + i * G;
      u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        u[i] = pp[(size_t)r * C];
        const int4 v = pc[(size_t)r * C];
        c.x += v.x; c.y += v.y; c.z += v.z; c.w += v.w;
      }
    }
    const float* f = reinterpret_cast<const float*>(u);
    p.x += pair_sum<kRlBatch>(f, 4);
    p.y += pair_sum<kRlBatch>(f + 1, 4);
    p.z += pair_sum<kRlBatch>(f + 2, 4);
    p.w += pair_sum<kRlBatch>(f + 3, 4);
  }
  ps[g][c4] = p;
  cs[g][c4] = c;
  __syncthreads();
  float* pf = reinterpret_cast<float*>(ps);  // [G][EP]
  int* ci = reinterpret_cast<int*>(cs);
  float sum = 0.f;
  int cnt = 0;
  if (threadIdx.x < EP) {
    sum = pair_sum<G>(&pf[threadIdx.x], EP);
#pragma unroll
    for (int i = 0; i < G; ++i) cnt += ci[i * EP + threadIdx.x];
  }
  __syncthreads();
  write_batch<EP>(sum, cnt, a, pf, ci);
}

struct RouteLogitsBwdArgs {
  const uint8_t* mask;
  const int32_t* ids;
  const int32_t* counts;
  const float* dw;     // NULL: no gradient of the weights
  const float* dloss;  // NULL: no gradient of the loss
  int T, E, top_k, renorm, vec;
};

template <int EP, typename TL>
__global__ void __launch_bounds__(kRlThreads) route_logits_backward_kernel(
    const TL* __restrict__ logits, TL* __restrict__ grad, const RouteLogitsBwdArgs a) {
  constexpr int Q = EP / 32;
  __shared__ float c_s[EP];
  __shared__ __align__(16) float sp[kRlWarps * EP];  // a warp's p of its token
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
      c[q] = lane * Q + q < a.E ? (float)__ldg(a.counts + lane * Q + q) : 0.f;
      tot += c[q];
    }
    tot = warp_sum(tot);
    const float g = a.dloss != nullptr ? __ldg(a.dloss) : 0.f;
    const float f = tot > 0.f ? g * (float)a.E / tot * ((float)a.top_k / tot) : 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      c[q] *= f;
      if (warp == 0) c_s[lane * Q + q] = c[q];
    }
  }
  __syncthreads();
  // The next token's logits and selected are on their way meanwhile.
  float next[Q], next_d = 0.f;
  int next_id = -1;
  const bool slot = a.dw != nullptr && lane < a.top_k;
  auto load = [&](uint32_t t) {
    load_row<Q>(logits, t, a.E, a.vec, next);
    if (slot) {
      next_id = __ldg(a.ids + (size_t)t * a.top_k + lane);
      next_d = __ldg(a.dw + (size_t)t * a.top_k + lane);
    }
  };
  uint32_t t = blockIdx.x * kRlWarps + warp;
  if (t < T) load(t);
  for (; t < T; t += stride) {
    float l[Q], p[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = next[q];
    int id = next_id;
    float dj = next_d;
    if (t + stride < T) load(t + stride);
    float m = l[0];
#pragma unroll
    for (int q = 1; q < Q; ++q) m = fmaxf(m, l[q]);
    m = redux_max(fmaxf(m, -INFINITY));
    const float sum = exp_row<Q>(l, m, p);
    const bool valid = sum != 0.f && (a.mask == nullptr || a.mask[t] != 0);
    TL* row = grad + (size_t)t * a.E;
    if (!valid) {
#pragma unroll
      for (int q = 0; q < Q; ++q) p[q] = 0.f;
      store_row<Q>(row, a.E, a.vec, p);
      continue;
    }
    const float inv = 1.f / sum;
    Pair both = {0.f, 0.f};
    each_pair<Q>([&](int a, int b) {
      const Pair n = Pair{p[a], p[b]} * Pair{inv, inv};
      both = fma2(n, Pair{c[a], c[b]}, both);
      p[a] = n.x;
      p[b] = n.y;
    });
    const float pc = warp_sum(Q == 1 ? both.x : both.x + both.y);
    // The selected experts, one a lane. An id outside [0, E) or repeated within
    // the row takes no part.
    float pj = 0.f, sel_term = 0.f, mean = 0.f;
    if (a.dw != nullptr) {
      __syncwarp();
      stage<Q>(&sp[warp * EP + lane * Q], p);
      const uint32_t same = __match_any_sync(kFullMask, id);
      if (id < 0 || id >= a.E || (same & ((1u << lane) - 1u)) != 0) {
        id = -1;
        dj = 0.f;
      }
      __syncwarp();
      if (id >= 0) pj = sp[warp * EP + id];
      mean = warp_sum(pj * dj);
      if (a.renorm) {
        const float tot = warp_sum(pj);
        const float r = tot > 0.f ? 1.f / tot : 0.f;
        sel_term = pj * r * (dj - mean * r);
        mean = 0.f;  // off the selection the weights' gradient is zero
      } else {
        sel_term = pj * dj;
      }
    }
    const float shift = pc + mean;
    each_pair<Q>([&](int a, int b) {
      const Pair n = Pair{p[a], p[b]} * (Pair{c[a], c[b]} + Pair{-shift, -shift});
      p[a] = n.x;
      p[b] = n.y;
    });
    store_row<Q>(row, a.E, a.vec, p);
    if (a.dw != nullptr) {
      __syncwarp();  // the row's stores above come before these
      if (id >= 0) store_grad(row + id, sel_term + pj * (c_s[id] - shift));
    }
  }
}

template <int EP, typename TL>
cudaError_t forward_ep(const TL* logits, const RouteLogitsArgs& a, int blocks, cudaStream_t st) {
  if (blocks == 1)
    return launch_k(route_logits_kernel<EP, kRlOneBlockWarps, TL>, dim3(1),
                    dim3(kRlOneBlockWarps * 32), 0, st, true, logits, a);
  if (blocks == 0)
    return launch_k(route_logits_cluster_kernel<EP, TL>, dim3(kRlClusterBlocks), dim3(kRlThreads),
                    0, st, true, logits, a);
  cudaError_t e = launch_k(route_logits_kernel<EP, kRlWarps, TL>, dim3(blocks), dim3(kRlThreads), 0,
                           st, true, logits, a);
  if (e != cudaSuccess) return e;
  return launch_k(route_logits_finish_kernel<EP>, dim3(1), dim3(kRlFinish), 0, st, true, blocks,
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
    return launch_k(route_logits_backward_kernel<32, TL>, g, b, 0, st, true, logits, grad, a);
  if (a.E <= 64)
    return launch_k(route_logits_backward_kernel<64, TL>, g, b, 0, st, true, logits, grad, a);
  if (a.E <= 128)
    return launch_k(route_logits_backward_kernel<128, TL>, g, b, 0, st, true, logits, grad, a);
  return launch_k(route_logits_backward_kernel<256, TL>, g, b, 0, st, true, logits, grad, a);
}

int ep_of(int E) { return E <= 32 ? 32 : E <= 64 ? 64 : E <= 128 ? 128 : 256; }

// Rows of E values that lanes may take Q at a time.
bool rows_are_vectors(const void* p, int E, int size) {
  const int Q = ep_of(E) / 32, bytes = Q * size;  // up to 32
  return E % Q == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// As many blocks as run at once: two an SM with 4 or 8 experts a lane (52 and 63
// registers a thread), three with fewer (40). 131072 tokens forward, two and three:
// 128 experts 60.8 and 64.9 us, 64 experts 67.2 and 49.1, 32 experts 62.7 and 44.9.
int blocks_per_sm(int E) { return ep_of(E) >= 128 ? 2 : 3; }
// The backward's (57 registers with 8 experts a lane, 39 with 4). 131072 tokens, two
// and three: 128 experts 37.8 and 36.3 us, 64 experts 33.0 and 31.4.
int backward_blocks_per_sm(int E) { return ep_of(E) == 256 ? 2 : 3; }

int blocks_for(int T, int per_sm, int num_sms) {
  const long long want = ((long long)T + kRlWarps - 1) / kRlWarps;
  const int most = per_sm * num_sms;
  return (int)(want < most ? want : most);
}

}  // namespace

// Rows of partial sums the forward may write: one per block, of blocks on 160
// SMs at most.
static int max_blocks(int E) { return 160 * blocks_per_sm(E); }

long long route_logits_workspace(int T, int E) {
  if (T <= kRlClusterTokens) return 0;
  const long long rows = ((long long)T + kRlWarps - 1) / kRlWarps;
  return (rows < max_blocks(E) ? rows : max_blocks(E)) * ep_of(E) * 8;
}

cudaError_t launch_route_logits(const void* logits, bool is_bf16, const uint8_t* mask, int T, int E,
                                int top_k, int renorm, int32_t* ids, float* w, int32_t* counts,
                                float* prob_sums, float* loss, void* workspace, int num_sms,
                                cudaStream_t st) {
  int blocks = T <= kRlOneBlockTokens ? 1
               : T <= kRlClusterTokens ? 0 : blocks_for(T, blocks_per_sm(E), num_sms);
  if (blocks > max_blocks(E)) blocks = max_blocks(E);
  const int EP = ep_of(E);
  RouteLogitsArgs a = {mask, ids, w, nullptr, nullptr, counts, prob_sums, loss, T, E, top_k, renorm,
                       rows_are_vectors(logits, E, is_bf16 ? 2 : 4)};
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
  const RouteLogitsBwdArgs a = {mask, ids, counts, dw, dloss, T, E, top_k, renorm,
                                rows_are_vectors(logits, E, is_bf16 ? 2 : 4) &&
                                    rows_are_vectors(grad, E, is_bf16 ? 2 : 4)};
  const int blocks = blocks_for(T, backward_blocks_per_sm(E), num_sms);
  return is_bf16 ? backward_t(static_cast<const uint16_t*>(logits), static_cast<uint16_t*>(grad), a,
                              blocks, st)
                 : backward_t(static_cast<const float*>(logits), static_cast<float*>(grad), a,
                              blocks, st);
}

}  // namespace mm
