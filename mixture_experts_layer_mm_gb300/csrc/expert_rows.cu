// Token rows to their experts' segments and back.
//
//   group     places[t, j] = the row of slot (t, j) among the slots sorted by expert
//             (stable: an expert's slots in their order), offsets[e] = first row of e
//   dispatch  rows[places[t, j]] = x[t]                       (and the slots' weights)
//   combine   out[t] = sum_j w[t, j] rows[places[t, j]]       (and the rows' values)
//
// A slot without a row (its token is masked, its id is out of range) has place -1.
// Combine adds a token's rows in the order of its slots, in fp32, and rounds once:
// no atomics, the same on every call. Dispatch with combine without weights are each
// other's gradient.
//
// Group ranks slots by ballots: within a warp the lanes of one expert find each
// other by a match, warps and chunks of 1024 slots are joined by counts in shared
// memory. Up to 1024 slots are one block's, a slot a thread; up to kGroupCluster those of a
// cluster of eight, whose counts each block reads in the others' shared memory; beyond,
// blocks count their spans first and every block of the second launch adds up the counts
// before its own.
//
// Dispatch and combine move 16 bytes a thread, a block a token: dispatch reads a
// token's row once and writes it to its slots, combine has the loads of all slots in
// flight before it adds. Both are bound by memory: 4096 tokens of 2048 bf16 and 8 slots
// take 24.5 and 23.5 us (151 MB each, 6.2 and 6.4 TB/s) and their grouping 5.4; 64 tokens
// 2.0, 2.1 and 1.9.
#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "mm.h"
#include "mm_internal.h"
#include "mx_device.cuh"
#include "pair_device.cuh"

namespace mm {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kGrThreads = 1024, kGrWarps = kGrThreads / 32;
constexpr int kGroupCtas = 8;          // of a cluster
constexpr int kGroupChunks = 2;        // of kGrThreads slots, at most, in one of its blocks
constexpr int kGroupCluster = kGroupCtas * kGroupChunks * kGrThreads;
constexpr int kMaxSpans = 152;  // one block an SM

// Slots a block takes, in whole chunks of kGrThreads.
long long span_of(long long n) {
  const long long chunks = (n + kGrThreads - 1) / kGrThreads;
  return (chunks + kMaxSpans - 1) / kMaxSpans * kGrThreads;
}

struct GroupArgs {
  const int32_t* ids;
  const uint8_t* mask;  // [T] or NULL
  int32_t* places;
  int32_t* offsets;
  int32_t* counts;  // [blocks][E] slots of each expert in each span (group_place_kernel)
  unsigned* err;
  long long n, span;
  int k, E;
};

// The slot's expert; E if it has no row. bad: its id is out of range.
__device__ __forceinline__ int expert_of(const GroupArgs& a, long long f, bool& bad) {
  const int id = __ldcg(a.ids + f);
  if (a.mask != nullptr && __ldcg(a.mask + (unsigned)f / (unsigned)a.k) == 0) return a.E;
  if (id < 0 || id >= a.E) {
    bad = true;
    return a.E;
  }
  return id;
}

__global__ void __launch_bounds__(kGrThreads) group_count_kernel(const GroupArgs a) {
  __shared__ int hist[kMaxExperts];
  pdl_wait();
  pdl_trigger();
  for (int e = threadIdx.x; e < a.E; e += kGrThreads) hist[e] = 0;
  __syncthreads();
  const long long f0 = blockIdx.x * a.span, f1 = min(f0 + a.span, a.n);
  bool bad = false;
  for (long long f = f0 + threadIdx.x; f < f1; f += kGrThreads) {
    const int e = expert_of(a, f, bad);
    if (e < a.E) atomicAdd(&hist[e], 1);
  }
  if (bad) atomicOr(a.err, kDevErrBadIds);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kGrThreads)
    a.counts[(size_t)blockIdx.x * a.E + e] = hist[e];
}

__global__ void __launch_bounds__(kGrThreads) group_place_kernel(const GroupArgs a) {
  __shared__ int base[kMaxExperts + 1];   // next row of each expert
  __shared__ int total[kMaxExperts];
  __shared__ __align__(16) int warp_count[kGrWarps][kMaxExperts];
  __shared__ int warp_sum[kMaxExperts / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long f0 = blockIdx.x * a.span, f1 = min(f0 + a.span, a.n);
  pdl_wait();
  pdl_trigger();
  for (int e = tid; e < kMaxExperts; e += kGrThreads) base[e] = total[e] = 0;
  __syncthreads();
  // Counts of all spans, and of those before this one: an expert a thread, spans
  // in turn over the thread's groups. Whole numbers: the order of the sums is free.
  if (const int e = tid & (kMaxExperts - 1); e < a.E) {
    int before = 0, all = 0;
    for (int b = tid / kMaxExperts; b < (int)gridDim.x; b += kGrThreads / kMaxExperts) {
      const int c = __ldcg(a.counts + (size_t)b * a.E + e);
      all += c;
      before += b < (int)blockIdx.x ? c : 0;
    }
    if (all > 0) atomicAdd(&total[e], all);
    if (before > 0) atomicAdd(&base[e], before);
  }
  __syncthreads();
  // Exclusive sums of the totals over the experts, 256 in 8 warps.
  int sum = 0, mine = 0;
  if (warp < kMaxExperts / 32) {
    mine = total[tid];
    sum = exclusive_sum(mine);
    if (lane == 31) warp_sum[warp] = sum + mine;
  }
  __syncthreads();
  if (warp < kMaxExperts / 32) {
    for (int i = 0; i < warp; ++i) sum += warp_sum[i];
    base[tid] += sum;
    if (blockIdx.x == 0) {
      if (tid < a.E) a.offsets[tid] = sum;
      if (tid == a.E - 1) a.offsets[a.E] = sum + mine;
    }
  }
  for (long long c0 = f0; c0 < f1; c0 += kGrThreads) {
    for (int i = tid; i < kGrWarps * kMaxExperts; i += kGrThreads) (&warp_count[0][0])[i] = 0;
    __syncthreads();
    const long long f = c0 + tid;
    bool bad = false;
    const int e = f < f1 ? expert_of(a, f, bad) : a.E;
    const uint32_t same = __match_any_sync(kAll, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (rank == 0 && e < a.E) warp_count[warp][e] = __popc(same);
    __syncthreads();
    if (tid < a.E) {  // counts -> first row of each warp's slots
      int at = base[tid];
#pragma unroll 8
      for (int w = 0; w < kGrWarps; ++w) {
        const int c = warp_count[w][tid];
        warp_count[w][tid] = at;
        at += c;
      }
      base[tid] = at;
    }
    __syncthreads();
    if (f < f1) a.places[f] = e < a.E ? warp_count[warp][e] + rank : -1;
    __syncthreads();
  }
}

// A slot a thread, one block: the ids are read once (8 slots 1.5 us, 512 1.9, 1024 2.7;
// 2.4, 2.9 and 3.4 in group_place_kernel).
__global__ void __launch_bounds__(kGrThreads) group_few_kernel(const GroupArgs a) {
  __shared__ __align__(16) int warp_count[kGrWarps][kMaxExperts];
  __shared__ int warp_sum[kMaxExperts / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  for (int i = tid; i < warps * kMaxExperts / 4; i += blockDim.x)
    reinterpret_cast<int4*>(warp_count)[i] = make_int4(0, 0, 0, 0);
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  const int e = tid < a.n ? expert_of(a, tid, bad) : a.E;
  if (bad) atomicOr(a.err, kDevErrBadIds);
  const uint32_t same = __match_any_sync(kAll, e);
  const int rank = __popc(same & ((1u << lane) - 1u));
  __syncthreads();
  if (rank == 0 && e < a.E) warp_count[warp][e] = __popc(same);
  __syncthreads();
  int sum = 0, mine = 0;
  if (warp < kMaxExperts / 32) {
#pragma unroll 8
    for (int w = 0; w < warps; ++w) mine += warp_count[w][tid];
    sum = exclusive_sum(mine);
    if (lane == 31) warp_sum[warp] = sum + mine;
  }
  __syncthreads();
  if (warp < kMaxExperts / 32) {
    for (int i = 0; i < warp; ++i) sum += warp_sum[i];
    if (tid < a.E) a.offsets[tid] = sum;
    if (tid == a.E - 1) a.offsets[a.E] = sum + mine;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {  // counts -> first row of each warp's slots
      const int c = warp_count[w][tid];
      warp_count[w][tid] = sum;
      sum += c;
    }
  }
  __syncthreads();
  if (tid < a.n) a.places[tid] = e < a.E ? warp_count[warp][e] + rank : -1;
}

// One cluster, spans of up to kGroupChunks chunks a block (4096 slots 3.1 us, 8192 3.7 to
// 4.0, 16384 5.4; counting and placing in two launches 4.8, 5.2 and 5.1, and 3 us more of
// the host's time).
__global__ void __launch_bounds__(kGrThreads) group_cluster_kernel(const GroupArgs a) {
  __shared__ int hist[kMaxExperts];   // this block's slots of each expert
  __shared__ int base[kMaxExperts], total[kMaxExperts];
  __shared__ __align__(16) int warp_count[kGrWarps][kMaxExperts];
  __shared__ int warp_sum[kMaxExperts / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank_in = (int)pair_rank();
  const long long f0 = rank_in * a.span, f1 = min(f0 + a.span, a.n);
  const int warps = (int)min((a.span + 31) / 32, (long long)kGrWarps);  // of a chunk, in use
  if (tid < kMaxExperts) hist[tid] = base[tid] = total[tid] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  int e[kGroupChunks];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kGroupChunks; ++i) {
    const long long f = f0 + i * kGrThreads + tid;
    e[i] = f < f1 ? expert_of(a, f, bad) : a.E;
  }
#pragma unroll
  for (int i = 0; i < kGroupChunks; ++i)
    if (e[i] < a.E) atomicAdd(&hist[e[i]], 1);
  if (bad) atomicOr(a.err, kDevErrBadIds);
  __syncwarp();
  cluster_barrier();
  {
    // Whole numbers: the order of the sums is free.
    const int x = tid & (kMaxExperts - 1);
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kGroupCtas * kMaxExperts / kGrThreads; ++i) {
      const int r = tid / kMaxExperts + i * (kGrThreads / kMaxExperts);
      const int c = load_peer(&hist[x], r);
      all += c;
      before += r < rank_in ? c : 0;
    }
    if (all > 0) atomicAdd(&total[x], all);
    if (before > 0) atomicAdd(&base[x], before);
  }
  // (No block ends, or counts again, while another may still read its counts.)
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  __syncthreads();
  int sum = 0, mine = 0;
  if (warp < kMaxExperts / 32) {
    mine = total[tid];
    sum = exclusive_sum(mine);
    if (lane == 31) warp_sum[warp] = sum + mine;
  }
  __syncthreads();
  if (warp < kMaxExperts / 32) {
    for (int i = 0; i < warp; ++i) sum += warp_sum[i];
    base[tid] += sum;
    if (rank_in == 0) {
      if (tid < a.E) a.offsets[tid] = sum;
      if (tid == a.E - 1) a.offsets[a.E] = sum + mine;
    }
  }
#pragma unroll
  for (int i = 0; i < kGroupChunks; ++i) {
    const long long c0 = f0 + i * kGrThreads;
    if (c0 >= f1) break;
    for (int j = tid; j < warps * kMaxExperts / 4; j += kGrThreads)
      reinterpret_cast<int4*>(warp_count)[j] = make_int4(0, 0, 0, 0);
    __syncthreads();
    const uint32_t same = __match_any_sync(kAll, e[i]);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (rank == 0 && e[i] < a.E) warp_count[warp][e[i]] = __popc(same);
    __syncthreads();
    if (tid < a.E) {  // counts -> first row of each warp's slots
      int at = base[tid];
#pragma unroll 8
      for (int w = 0; w < warps; ++w) {
        const int c = warp_count[w][tid];
        warp_count[w][tid] = at;
        at += c;
      }
      base[tid] = at;
    }
    __syncthreads();
    if (c0 + tid < f1) a.places[c0 + tid] = e[i] < a.E ? warp_count[warp][e[i]] + rank : -1;
    __syncthreads();
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Column chunks of 16 bytes of a row.
__global__ void __launch_bounds__(256)
    dispatch_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ places,
                    const float* __restrict__ w, int k, int chunks, long long R,
                    uint4* __restrict__ rows, float* __restrict__ row_w, unsigned* err) {
  __shared__ int place_s[kMaxTopK];
  pdl_wait();
  pdl_trigger();
  const long long t = blockIdx.x;
  if ((int)threadIdx.x < k) {
    const long long f = t * k + threadIdx.x;
    int p = __ldcg(places + f);
    if (p < -1 || p >= R) {
      atomicOr(err, kDevErrBadIds);
      p = -1;
    }
    place_s[threadIdx.x] = p;
    if (p >= 0 && row_w != nullptr) row_w[p] = __ldcg(w + f);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    const uint4 v = __ldcg(x + t * chunks + c);
    for (int j = 0; j < k; ++j) {
      const int p = place_s[j];
      if (p >= 0) rows[(size_t)p * chunks + c] = v;
    }
  }
}

template <bool FP16>
__device__ __forceinline__ void add_row(float (&s)[8], const uint4& v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    if (FP16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      lo = f.x;
      hi = f.y;
    } else {
      lo = __uint_as_float(u[i] << 16);
      hi = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    s[2 * i] = __fmaf_rn(w, lo, s[2 * i]);
    s[2 * i + 1] = __fmaf_rn(w, hi, s[2 * i + 1]);
  }
}

// The token's slots with a row, in order, are in shared memory; U rows' loads are in
// flight at a time.
template <bool FP16, int U>
__global__ void __launch_bounds__(256, U == 8 ? 4 : 6)
    combine_kernel(const uint4* __restrict__ rows, const int32_t* __restrict__ places,
                   const float* __restrict__ w, const float* __restrict__ row_values, int k,
                   int chunks, long long R, uint4* __restrict__ out, float* __restrict__ values,
                   unsigned* err) {
  __shared__ int place_s[kMaxTopK];
  __shared__ float w_s[kMaxTopK];
  __shared__ int used_s;
  pdl_wait();
  pdl_trigger();
  const long long t = blockIdx.x;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int p = -1;
    float wt = 1.f;
    if (lane < k) {
      const long long f = t * k + lane;
      p = __ldcg(places + f);
      if (p < -1 || p >= R) {
        atomicOr(err, kDevErrBadIds);
        p = -1;
      }
      if (w != nullptr) wt = __ldcg(w + f);
      if (values != nullptr) values[f] = p >= 0 ? __ldcg(row_values + p) : 0.f;
    }
    const uint32_t has = __ballot_sync(kAll, p >= 0);
    if (p >= 0) {
      const int i = __popc(has & ((1u << lane) - 1u));
      place_s[i] = p;
      w_s[i] = wt;
    }
    if (lane == 0) used_s = __popc(has);
  }
  __syncthreads();
  const int used = used_s;
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    float s[8] = {};
    for (int j0 = 0; j0 < used; j0 += U) {
      uint4 v[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (j0 + j < used) v[j] = __ldcs(rows + (size_t)place_s[j0 + j] * chunks + c);
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (j0 + j < used) add_row<FP16>(s, v[j], w_s[j0 + j]);
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack16x2(s[2 * i], s[2 * i + 1], FP16);
    out[t * chunks + c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

dim3 row_threads(int chunks) { return dim3((unsigned)std::min(256, (chunks + 31) / 32 * 32)); }

}  // namespace

long long group_slots_workspace(long long n, int E) {
  return n <= kGroupCluster ? 0 : (n + span_of(n) - 1) / span_of(n) * E * 4;
}

cudaError_t launch_group_slots(const int32_t* ids, const uint8_t* mask, int T, int top_k, int E,
                               int32_t* places, int32_t* offsets, void* workspace, unsigned* err,
                               cudaStream_t st) {
  GroupArgs a = {};
  a.ids = ids;
  a.mask = mask;
  a.places = places;
  a.offsets = offsets;
  a.err = err;
  a.n = (long long)T * top_k;
  a.k = top_k;
  a.E = E;
  if (a.n <= kGrThreads) {
    const unsigned threads = std::max(kMaxExperts, ((int)a.n + 31) / 32 * 32);
    return launch_k(group_few_kernel, dim3(1), dim3(threads), 0, st, true, a);
  }
  if (a.n <= kGroupCluster) {
    a.span = ((a.n + kGroupCtas - 1) / kGroupCtas + 31) / 32 * 32;
    static std::atomic<int> resident[kMaxDevices];
    return launch_clusters(group_cluster_kernel, kGroupCtas, resident, kGrThreads, 0, 1, 152, st,
                           a);
  }
  a.span = span_of(a.n);
  a.counts = static_cast<int32_t*>(workspace);
  const dim3 grid((unsigned)((a.n + a.span - 1) / a.span));
  if (cudaError_t e = launch_k(group_count_kernel, grid, dim3(kGrThreads), 0, st, true, a);
      e != cudaSuccess)
    return e;
  return launch_k(group_place_kernel, grid, dim3(kGrThreads), 0, st, true, a);
}

cudaError_t launch_dispatch_rows(const void* x, const int32_t* places, const float* w, int T,
                                 int top_k, int H, long long R, void* rows, float* row_w,
                                 unsigned* err, cudaStream_t st) {
  const int chunks = H / 8;
  return launch_k(dispatch_kernel, dim3((unsigned)T), row_threads(chunks), 0, st, true,
                  static_cast<const uint4*>(x), places, w, top_k, chunks, R,
                  static_cast<uint4*>(rows), row_w, err);
}

cudaError_t launch_combine_rows(const void* rows, bool fp16, const int32_t* places, const float* w,
                                const float* row_values, int T, int top_k, int H, long long R,
                                void* out, float* values, unsigned* err, cudaStream_t st) {
  const int chunks = H / 8;
  auto k = top_k > 4 ? (fp16 ? combine_kernel<true, 8> : combine_kernel<false, 8>)
                     : (fp16 ? combine_kernel<true, 4> : combine_kernel<false, 4>);
  return launch_k(k, dim3((unsigned)T),
                  row_threads(chunks), 0, st, true, static_cast<const uint4*>(rows), places, w,
                  row_values, top_k, chunks, R, static_cast<uint4*>(out), values, err);
}

}  // namespace mm
