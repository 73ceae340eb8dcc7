// Matrix products grouped by expert, over ragged segments of rows (rows
// off[e] .. off[e + 1] - 1 belong to expert e), in the three forms a training
// step needs:
//
//   forward  y[r]  = W[e] x[r]              reduction over K
//   dx       dx[r] = W[e]^T dy[r]           reduction over N
//   dw       dW[e] = sum_r dy[r] x[r]^T     reduction over the segment's rows
//
// One kernel on SM pairs (tcgen05.mma.cta_group::2, M = 256: 128 rows of the
// accumulator in each CTA's tensor memory). What goes where:
//
//            M side (256 a tile)       N side                     reduction
//   forward  features n, W rows        up to 256 rows r           K, contiguous in both
//   dx       features k, W columns     up to 256 rows r           N, W's rows; contiguous in dy
//   dw       features n, dy columns    256 (128) features k       rows, of both
//
// The rows are the N side of forward and dx because its size goes in steps of
// 16: a segment is cut into near-equal chunks of at most 256 rows, and nothing
// is computed for rows it does not have. No operand is transposed in memory:
// where the reduction runs along a matrix's rows, its tile of 64 rows x 64
// columns (128 bytes a row, 128-byte swizzle) is an MN-major operand, and the
// MMA is told so.
//
// Edges. Columns beyond a matrix are zeros out of the copy, and so are W's
// rows beyond an expert's (W is a 3-D tensor to the copies). Rows beyond a
// segment belong to another expert: in forward and dx they give columns of the
// accumulator that nobody reads; in dw they would enter the sums, so the last
// stage of a segment is cut to whole steps of 16 rows, and the producer
// writes zeros over what is left of the last step (in both operands: 0 times
// another expert's infinity is NaN).
#include <algorithm>

#include <cuda_fp16.h>

#include "mm.h"
#include "mm_device.cuh"
#include "mm_internal.h"
#include "mx_device.cuh"
#include "pair_device.cuh"

namespace mm {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kGK = 64;                   // reduction per stage: 128 bytes of 16-bit values
constexpr int kGStages = 6;
constexpr int kGHalf = 128 * kGK * 2;     // 16 KB: one CTA's half of an operand's stage
constexpr int kGStageBytes = 2 * kGHalf;
constexpr int kGBox = 64 * kGK * 2;       // 8 KB: 64 x 64 values, one MN-major block
constexpr int kGMaxN = 256;
constexpr int kGEpiWarp0 = 1, kGEpiWarps = 8;
constexpr int kGProd0 = kGEpiWarp0 + kGEpiWarps;          // producers: one warp a slot
constexpr int kGThreads = (kGProd0 + kGStages) * 32;      // 480
constexpr int kGSmemBytes = kGStages * kGStageBytes + 1024;
constexpr uint32_t kGTmemCols = 2 * kGMaxN;               // two accumulators
// Rows of a segment that one fp32 accumulation of dw takes, where the result is
// fp32: the tensor cores cut what they add, and 512 rows leave 5e-7 of it.
constexpr int kGSliceRows = 512;

enum { kForward = 0, kDx = 1, kDw = 2 };

struct ProductArgs {
  const int32_t* offsets;  // [E + 1]
  void* out;
  unsigned* err;
  int E, R;
  int F;         // features on the M side: N (forward, dw), K (dx)
  int D;         // forward, dx: length of the reduction. dw: features on the N side
  int m_tiles;   // of 256 features of F
  int n_tiles;   // dw: tiles of bn features of D
  int bn;        // dw: 256 or 128
  int fp16;      // type of the inputs (else bf16)
  int out_fp32;  // dw
  int accumulate;
  int wide;      // rows of the result begin at multiples of 32 bytes
};

struct Segments {
  int off[kMaxExperts + 1];
  int first[kMaxExperts + 1];  // first chunk of each expert
  int size[kMaxExperts];       // rows per chunk
  int bad;
};

// One tile of forward or dx: chunk of rows, m-tile. Of dw: expert, m-tile, n-tile.
struct GTile {
  int e, m, n, row0, nrows;
};

template <int WAY>
__device__ __forceinline__ GTile tile_at(int tile, const ProductArgs& a, const Segments& S) {
  GTile t;
  if (WAY == kDw) {
    const int per = a.m_tiles * a.n_tiles;
    t.e = tile / per;
    const int i = tile - t.e * per;
    t.m = i / a.n_tiles;
    t.n = i - t.m * a.n_tiles;
    t.row0 = S.off[t.e];
    t.nrows = S.off[t.e + 1] - t.row0;
  } else {
    const int ch = tile / a.m_tiles;
    t.m = tile - ch * a.m_tiles;
    t.n = 0;
    int lo = 0, hi = a.E;  // first[lo] <= ch < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (S.first[mid] <= ch)
        lo = mid;
      else
        hi = mid;
    }
    t.e = lo;
    t.row0 = S.off[lo] + (ch - S.first[lo]) * S.size[lo];
    t.nrows = min(S.size[lo], S.off[lo + 1] - t.row0);
  }
  return t;
}

__device__ __forceinline__ uint16_t to16(float v, bool fp16) {
  return fp16 ? __half_as_ushort(__float2half_rn(v)) : f32_to_bf16_bits(v);
}
__device__ __forceinline__ uint32_t to16x2(float lo, float hi, bool fp16) {
  return (uint32_t)to16(lo, fp16) | ((uint32_t)to16(hi, fp16) << 16);
}
__device__ __forceinline__ float from16(uint32_t bits, bool fp16) {
  return fp16 ? __half2float(__ushort_as_half((unsigned short)bits)) : bf16_bits_to_f32(bits);
}

// 32 contiguous bytes, 32-byte aligned.
__device__ __forceinline__ void store_32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// n * 8 values of one row (n <= 4) to `out` (element 0 at `at`), added to what is
// there if `add`.
__device__ __forceinline__ void store_row(void* out, size_t at, int n8, const uint32_t (&v)[32],
                                          const ProductArgs& a, bool add) {
  if (a.out_fp32) {
    float* p = static_cast<float*>(out) + at;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (g >= n8) break;
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = v[8 * g + j];
      if (add) {
        const float4 x = *reinterpret_cast<const float4*>(p + 8 * g);
        const float4 y = *reinterpret_cast<const float4*>(p + 8 * g + 4);
        const float o[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(o[j] + __uint_as_float(w[j]));
      }
      if (a.wide) {
        store_32(p + 8 * g, w);
      } else {
        reinterpret_cast<uint4*>(p + 8 * g)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p + 8 * g)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    return;
  }
  uint16_t* p = static_cast<uint16_t*>(out) + at;
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float lo = __uint_as_float(v[2 * j]), hi = __uint_as_float(v[2 * j + 1]);
    if (add && j / 4 < n8) {
      const uint32_t o = reinterpret_cast<const uint32_t*>(p)[j];
      lo += from16(o & 0xFFFFu, a.fp16);
      hi += from16(o >> 16, a.fp16);
    }
    w[j] = to16x2(lo, hi, a.fp16);
  }
#pragma unroll
  for (int g = 0; g < 4; g += 2) {
    if (a.wide && g + 2 <= n8) {
      const uint32_t x[8] = {w[4 * g],     w[4 * g + 1], w[4 * g + 2], w[4 * g + 3],
                             w[4 * g + 4], w[4 * g + 5], w[4 * g + 6], w[4 * g + 7]};
      store_32(p + 8 * g, x);
    } else {
#pragma unroll
      for (int h = g; h < g + 2; ++h)
        if (h < n8)
          reinterpret_cast<uint4*>(p)[h] =
              make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
    }
  }
}

// tmB32: rows in boxes of 32 (forward, dx), for chunks that do not fill a box of 128.
template <int WAY>
__global__ void __launch_bounds__(kGThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmB32, const ProductArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[3 * kGStages + 5];
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ Segments S;

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int E = a.E;
  const uint32_t rank = pair_rank();  // 0 = leader (issues the MMAs)
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  uint64_t* full = bars;
  uint64_t* empty = full + kGStages;
  uint64_t* land = empty + kGStages;  // dw: this CTA's copies of a segment's last stage
  uint64_t* tfull = land + kGStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  if (tid == 0) {
    for (int s = 0; s < kGStages; ++s) {
      mbar_init(smem_u32(&full[s]), 2);   // each CTA's producer announces its own bytes
      mbar_init(smem_u32(&empty[s]), 1);  // the leader's MMA commit, multicast to both CTAs
      mbar_init(smem_u32(&land[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 2 * kGEpiWarps);
    }
    mbar_init(smem_u32(done), 1);
    abort_s = 0;
    S.bad = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (WAY != kDw) tma_prefetch_desc(&tmB32);
  }
  if (warp == 0) {
    tmem_alloc_pair(smem_u32(&tmem_base_s), kGTmemCols);
    tmem_relinquish_pair();
  }
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i <= E; i += kGThreads) S.off[i] = a.offsets[i];
  __syncthreads();
  // Offsets that fall or leave [0, R] are refused as a whole: no row is touched.
  for (int i = tid; i < E; i += kGThreads)
    if (S.off[i] < 0 || S.off[i + 1] < S.off[i] || S.off[i + 1] > a.R) S.bad = 1;
  __syncthreads();
  const bool bad = S.bad != 0;
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(a.err, kDevErrBadIds);
    __syncthreads();
    for (int i = tid; i <= E; i += kGThreads) S.off[i] = 0;
    __syncthreads();
  }
  int total;
  if (WAY == kDw) {
    total = bad ? 0 : E * a.m_tiles * a.n_tiles;
  } else {
    if (warp == 0) {  // chunks: ceil(rows / 256) near-equal ones for each expert
      const int per = (E + 31) / 32, e0 = lane * per;
      int sum = 0;
      for (int e = e0; e < min(e0 + per, E); ++e)
        sum += (S.off[e + 1] - S.off[e] + kGMaxN - 1) / kGMaxN;
      int run = exclusive_sum(sum);
      for (int e = e0; e < min(e0 + per, E); ++e) {
        const int L = S.off[e + 1] - S.off[e], n = (L + kGMaxN - 1) / kGMaxN;
        S.first[e] = run;
        S.size[e] = n > 0 ? ((L + n - 1) / n + 15) / 16 * 16 : 0;
        run += n;
      }
      if (lane == 31) S.first[E] = run;
    }
    __syncthreads();
    total = S.first[E] * a.m_tiles;
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers initialised, tensor memory allocated
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_s;
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t peer_abort = peer_addr(smem_u32(&abort_s), rank ^ 1u);
  auto fail = [&]() {
    *reinterpret_cast<volatile int*>(&abort_s) = 1;
    st_cluster_u32(peer_abort, 1u);
    atomicOr(a.err, kDevErrTimeout);
  };
  auto aborted = [&]() {
    return __any_sync(kAll, *reinterpret_cast<volatile int*>(&abort_s) != 0);
  };
  // The reduction of a tile in slices (dw with an fp32 result: of kGSliceRows rows).
  const int slice_rows = WAY == kDw && a.out_fp32 ? kGSliceRows : 0x7fffffff;
  auto slices = [&](const GTile& t) {
    return WAY != kDw ? 1 : a.out_fp32 ? (t.nrows + kGSliceRows - 1) / kGSliceRows
                                       : (t.nrows > 0 ? 1 : 0);
  };
  auto length = [&](const GTile& t, int s) {  // of slice s
    return WAY != kDw ? a.D : min(slice_rows, t.nrows - s * kGSliceRows);
  };

  if (warp >= kGProd0) {
    // ------------------------------------------------------- producers ---
    // One warp a ring slot: a warp's copies that signal another barrier than
    // its previous ones wait for those to land.
    const int slot = warp - kGProd0;
    const bool leader = elect_one();
    const uint32_t st = smem_base + slot * kGStageBytes;
    const uint32_t fb = peer_addr(smem_u32(&full[slot]), 0);  // the leader's barrier
    const uint32_t eb = smem_u32(&empty[slot]), lb = smem_u32(&land[slot]);
    const uint64_t pol_once = l2_policy_evict_first(), pol_normal = l2_policy_evict_normal(),
                   pol_keep = l2_policy_evict_last();
    uint32_t use = 0, landed = 0;
    int q = 0;  // stage counter modulo the ring
    bool ok = true;
    for (int tile = pair; tile < total && ok; tile += npairs) {
      if (aborted()) break;
      const GTile t = tile_at<WAY>(tile, a, S);
      const int nsl = slices(t);
      for (int sl = 0; sl < nsl && ok; ++sl) {
        const int len = length(t, sl), nk = (len + kGK - 1) / kGK;
        // forward, dx: this CTA's half of the rows
        const int nh = ((t.nrows + 15) & ~15) / 2;
        const int brow = t.row0 + (int)rank * nh;
        const int boxes = nh > 96 ? 1 : (nh + 31) / 32;
        const uint32_t b_bytes = WAY == kDw ? (uint32_t)(a.bn / 128) * kGBox
                                            : nh > 96 ? kGHalf : (uint32_t)boxes * 32 * kGK * 2;
        const uint64_t pol_w =
            WAY != kDw && S.first[t.e + 1] - S.first[t.e] > 1 ? pol_normal : pol_once;
        for (int kb = 0; kb < nk; ++kb) {
          const bool mine = q == slot;
          if (++q == kGStages) q = 0;
          if (!mine) continue;
          if (!warp_wait(eb, (use & 1u) ^ 1u)) {
            fail();
            ok = false;
            break;
          }
          const int left = len - kb * kGK;  // dw: rows of this stage, if fewer than 64
          const bool tail = WAY == kDw && left < kGK && (left & 15) != 0;
          const uint32_t bar = tail ? peer_addr(lb, rank) : fb;
          if (leader) {
            mbar_expect_tx_cluster(bar, kGHalf + b_bytes);
            if (WAY == kForward) {
              tma_load_3d_pair(st, &tmA, bar, kb * kGK, t.m * 256 + (int)rank * 128, t.e, pol_w);
            } else if (WAY == kDx) {
              const int f = t.m * 256 + (int)rank * 128;
              tma_load_3d_pair(st, &tmA, bar, f, kb * kGK, t.e, pol_w);
              tma_load_3d_pair(st + kGBox, &tmA, bar, f + 64, kb * kGK, t.e, pol_w);
            }
            if (WAY == kDw) {
              const int r = t.row0 + sl * kGSliceRows + kb * kGK;
              const int f = t.m * 256 + (int)rank * 128, c = t.n * a.bn + (int)rank * (a.bn / 2);
              tma_load_2d_pair(st, &tmA, bar, f, r, pol_keep);
              tma_load_2d_pair(st + kGBox, &tmA, bar, f + 64, r, pol_keep);
              tma_load_2d_pair(st + kGHalf, &tmB, bar, c, r, pol_keep);
              if (a.bn == 256)
                tma_load_2d_pair(st + kGHalf + kGBox, &tmB, bar, c + 64, r, pol_keep);
            } else if (nh > 96) {
              tma_load_2d_pair(st + kGHalf, &tmB, bar, kb * kGK, brow, pol_keep);
            } else {
              for (int j = 0; j < boxes; ++j)
                tma_load_2d_pair(st + kGHalf + j * (32 * kGK * 2), &tmB32, bar, kb * kGK,
                                 brow + 32 * j, pol_keep);
            }
          }
          __syncwarp();
          if (tail) {
            if (!warp_wait(lb, landed & 1u)) {
              fail();
              ok = false;
              break;
            }
            ++landed;
            // Rows [left, next multiple of 16) of the four (three) blocks: 128 bytes each.
            const int n = ((left + 15) & ~15) - left, blocks = 2 + a.bn / 128;
            for (int i = lane; i < blocks * n * 8; i += 32) {
              const int b = i / (n * 8), j = i - b * (n * 8);
              st_shared_zero16(st + b * kGBox + left * 128 + j * 16);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (leader) mbar_arrive_cluster(fb);
          }
          ++use;
        }
      }
    }
    if (!ok || aborted()) {
      // Copies issued just before the abort may still be landing in this CTA's
      // shared memory: a copy completes within microseconds.
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 50000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ---------------------------------------------- MMA issuer (leader) ---
    // The whole warp runs the loops, so that descriptors stay in uniform
    // registers; one elected lane issues.
    if (rank == 0) {
      const bool leader = elect_one();
      constexpr bool a_mn = WAY != kForward, b_mn = WAY == kDw;
      const uint32_t id0 = idesc_16(a.fp16 != 0, a_mn, b_mn);
      int s = 0;
      uint32_t ph = 0;
      uint32_t it = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        if (aborted()) break;
        const GTile t = tile_at<WAY>(tile, a, S);
        const int nsl = slices(t);
        const uint32_t idesc =
            id0 | idesc_shape(256, WAY == kDw ? a.bn : (t.nrows + 15) & ~15);
        for (int sl = 0; sl < nsl && ok; ++sl, ++it) {
          const int len = length(t, sl), nk = (len + kGK - 1) / kGK;
          const uint32_t b = it & 1u, use = it >> 1;
          if (!warp_wait_cluster(smem_u32(&tempty[b]), (use & 1u) ^ 1u)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + b * kGMaxN;
          for (int kb = 0; kb < nk; ++kb) {
            if (!warp_wait_cluster(smem_u32(&full[s]), ph)) {
              fail();
              ok = false;
              break;
            }
            tc_fence_after();
            if (leader) {
              const uint32_t st = smem_base + s * kGStageBytes;
              const uint64_t da = a_mn ? sdesc_mnmajor(st, kGBox) : sdesc_kmajor<128>(st);
              const uint64_t db = b_mn ? sdesc_mnmajor(st + kGHalf, kGBox)
                                       : sdesc_kmajor<128>(st + kGHalf);
              // 16 of the reduction: 32 bytes of a K-major row, 16 rows of an MN-major block.
              constexpr uint64_t ia = a_mn ? 16 * 128 / 16 : 2, ib = b_mn ? 16 * 128 / 16 : 2;
              const int steps = min(4, (len - kb * kGK + 15) / 16);
              if (steps == 4) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_pair_bf16(d, da + kk * ia, db + kk * ib, idesc, (kb | kk) != 0);
              } else {
                for (int kk = 0; kk < steps; ++kk)
                  umma_pair_bf16(d, da + kk * ia, db + kk * ib, idesc, (kb | kk) != 0);
              }
              umma_pair_commit(smem_u32(&empty[s]), 0x3);  // frees stage s in both CTAs
            }
            __syncwarp();
            if (++s == kGStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (!ok) break;
          if (leader) umma_pair_commit(smem_u32(&tfull[b]), 0x3);
          __syncwarp();
        }
      }
      // Every MMA issued above has finished before tensor memory is freed.
      if (leader) umma_pair_commit(smem_u32(done), 0x1);
      __syncwarp();
      if (!warp_wait(smem_u32(done), 0)) fail();
    }
  } else {
    // -------------------------------------------------------- epilogue ---
    const int q = warp & 3;                          // tensor-memory lane quarter of this warp
    const int side = (warp - kGEpiWarp0) >> 2;       // takes 32-column chunks side, side + 2, ...
    const uint32_t te[2] = {peer_addr(smem_u32(&tempty[0]), 0), peer_addr(smem_u32(&tempty[1]), 0)};
    uint32_t it = 0;
    bool ok = true;
    for (int tile = pair; tile < total && ok; tile += npairs) {
      if (aborted()) break;
      const GTile t = tile_at<WAY>(tile, a, S);
      const int f = t.m * 256 + (int)rank * 128 + q * 32 + lane;  // this lane's feature
      const int nsl = slices(t);
      if (WAY == kDw && nsl == 0 && !a.accumulate) {  // an expert without rows
        const uint32_t v[32] = {};
        for (int c0 = side * 32; c0 < a.bn; c0 += 64) {
          const int c = t.n * a.bn + c0, n8 = min(32, a.D - c) / 8;
          if (f < a.F && n8 > 0)
            store_row(a.out, ((size_t)t.e * a.F + f) * a.D + c, n8, v, a, false);
        }
      }
      for (int sl = 0; sl < nsl; ++sl, ++it) {
        const uint32_t b = it & 1u, use = it >> 1;
        if (!warp_wait_cluster(smem_u32(&tfull[b]), use & 1u)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + b * kGMaxN;
        const int cols = WAY == kDw ? a.bn : t.nrows;
        for (int c0 = side * 32; c0 < cols; c0 += 64) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tb + c0, v);
          tmem_wait_ld();
          if (WAY == kDw) {
            const int c = t.n * a.bn + c0, n8 = min(32, a.D - c) / 8;
            if (f < a.F && n8 > 0)
              store_row(a.out, ((size_t)t.e * a.F + f) * a.D + c, n8, v, a,
                        a.accumulate || sl > 0);
          } else if (f < a.F) {
            uint16_t* p = static_cast<uint16_t*>(a.out) + (size_t)(t.row0 + c0) * a.F + f;
            const int n = cols - c0;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < n) p[(size_t)j * a.F] = to16(__uint_as_float(v[j]), a.fp16);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(te[b]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs are done with tensor memory and with each other's barriers
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kGTmemCols);
  }
}

template <int WAY>
cudaError_t launch_way(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmB32,
                       const ProductArgs& a, long long max_tiles, int num_sms, cudaStream_t st) {
  static DeviceFlags attr_done;
  if (cudaError_t e = smem_attr_once(attr_done, product_kernel<WAY>, kGSmemBytes);
      e != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kGThreads, 1, 1);
  cfg.dynamicSmemBytes = kGSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Persistent pairs: as many as can be resident at once.
  static std::atomic<int> resident[kMaxDevices];
  const int dev = current_device();
  int pairs = resident[dev].load(std::memory_order_relaxed);
  if (pairs <= 0) {
    cfg.gridDim = dim3((unsigned)num_sms / 2 * 2, 1, 1);
    if (cudaOccupancyMaxActiveClusters(&pairs, product_kernel<WAY>, &cfg) != cudaSuccess ||
        pairs <= 0) {
      cudaGetLastError();
      pairs = num_sms / 2;
    }
    resident[dev].store(pairs, std::memory_order_relaxed);
  }
  if (max_tiles < pairs) pairs = (int)std::max(1LL, max_tiles);
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, product_kernel<WAY>, tmA, tmB, tmB32, a);
}

// A 2-D matrix [rows, cols] in boxes of 64 columns x box_rows rows, or W [E, rows,
// cols] likewise (E > 0).
bool make_map(CUtensorMap* m, const void* base, int E, int rows, int cols, uint32_t box_rows) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)E};
  const uint64_t strides[2] = {(uint64_t)cols * 2, (uint64_t)cols * rows * 2};
  const uint32_t box[3] = {kGK, box_rows, 1};
  return make_tensor_map_sw128(m, base, E > 0 ? 3 : 2, dims, strides, box);
}

}  // namespace

cudaError_t launch_grouped_product(bool transposed, const void* x, const void* w,
                                   const int32_t* offsets, int R, int E, int N, int K, bool fp16,
                                   void* out, int num_sms, unsigned* err, cudaStream_t st) {
  ProductArgs a = {};
  a.offsets = offsets;
  a.out = out;
  a.err = err;
  a.E = E;
  a.R = R;
  a.F = transposed ? K : N;
  a.D = transposed ? N : K;
  a.m_tiles = (a.F + 255) / 256;
  a.fp16 = fp16;
  CUtensorMap tmA, tmB, tmB32;
  if (!make_map(&tmA, w, E, N, K, transposed ? 64 : 128) || !make_map(&tmB, x, 0, R, a.D, 128) ||
      !make_map(&tmB32, x, 0, R, a.D, 32))
    return cudaErrorInvalidValue;
  const long long chunks = std::min<long long>(R, (long long)E + R / kGMaxN);
  return transposed
             ? launch_way<kDx>(tmA, tmB, tmB32, a, chunks * a.m_tiles, num_sms, st)
             : launch_way<kForward>(tmA, tmB, tmB32, a, chunks * a.m_tiles, num_sms, st);
}

cudaError_t launch_grouped_product_dw(const void* dy, const void* x, const int32_t* offsets, int R,
                                      int E, int N, int K, bool fp16, void* out, bool out_fp32,
                                      bool accumulate, int num_sms, unsigned* err,
                                      cudaStream_t st) {
  ProductArgs a = {};
  a.offsets = offsets;
  a.out = out;
  a.err = err;
  a.E = E;
  a.R = R;
  a.F = N;
  a.D = K;
  a.m_tiles = (N + 255) / 256;
  a.bn = K <= 128 ? 128 : 256;
  a.n_tiles = (K + a.bn - 1) / a.bn;
  a.fp16 = fp16;
  a.out_fp32 = out_fp32;
  a.accumulate = accumulate;
  a.wide = ((size_t)K * (out_fp32 ? 4 : 2)) % 32 == 0 && reinterpret_cast<uintptr_t>(out) % 32 == 0;
  CUtensorMap tmA, tmB;
  if (!make_map(&tmA, dy, 0, R, N, 64) || !make_map(&tmB, x, 0, R, K, 64))
    return cudaErrorInvalidValue;
  return launch_way<kDw>(tmA, tmB, tmB, a, (long long)E * a.m_tiles * a.n_tiles, num_sms, st);
}

}  // namespace mm
