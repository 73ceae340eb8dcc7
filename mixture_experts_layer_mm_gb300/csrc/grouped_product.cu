// Matrix products grouped by expert, over ragged segments of rows (rows
// off[e] .. off[e + 1] - 1 belong to expert e): the product and the gradient of
// its rows (the gradient of its weights is in grouped_product_dw.cu).
//
//   forward  y[r]  = W[e] x[r]              reduction over K
//   dx       dx[r] = W[e]^T dy[r]           reduction over N
//
// One kernel on SM pairs (tcgen05.mma.cta_group::2, M = 256: 128 rows of the
// accumulator in each CTA's tensor memory). What goes where:
//
//            M side (256 a tile)       N side             reduction
//   forward  features n, W's rows      up to 256 rows     K, contiguous in both
//   dx       features k, W's columns   up to 256 rows     N, W's rows; contiguous in dy
//
// The token rows are the N side because its size goes in steps of 16: a segment
// is cut into near-equal chunks of at most 256 rows (fewer where there would be too few
// tiles, see chunk_rows), and nothing is computed for rows it does not have. W is not
// transposed in memory: where the reduction runs along its rows, a tile of 64 rows x 64
// columns (128 bytes a row, 128-byte swizzle) is an MN-major operand, and the MMA is told so.
//
// Edges. Columns beyond a matrix are zeros out of the copy, and so are W's rows
// beyond an expert's (W is a 3-D tensor to the copies) in a box that has some of it. Rows
// beyond a segment belong to another expert; they give columns of the accumulator that
// nobody reads.
//
// What bounds it, on one GB300: 512 rows over 128 experts x 1536 x 2048 are the weights'
// bytes, 111 us (7.2 TB/s). 32768 rows of uneven load over them take 180 us forward, and
// dx of the down product (2048 x 768) 99; their bytes at the copy rate 154 and 87. The
// SMs take in 2.3 GB there, 13 TB/s out of L2: an expert of more than 256 rows reads its
// weights for each chunk (168 us with 256 rows each). 1024 rows an expert run at 1.75
// PFLOP/s. 5003 rows over 60 experts x 1000 x 1016 take 24 us, of 21, in 2.5 rounds of
// tiles. Rows whose bytes are no multiple of 128 cost each copy two lines for one: 28600
// rows over 40 x 1680 x 1344 take 90 us, x 1352 140. One row x 64 x 64 takes 3.3 us.
#include <algorithm>
#include <cmath>

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
static_assert(kMaxExperts <= kGThreads, "an expert a thread");
constexpr uint32_t kGTmemCols = 2 * kGMaxN;               // two accumulators

enum { kForward = 0, kDx = 1 };

struct ProductArgs {
  const int32_t* offsets;  // [E + 1]
  void* out;
  unsigned* err;
  int E, R;
  int F;         // features of the result: N (forward), K (dx)
  int D;         // length of the reduction
  int m_tiles;   // of 256 features
  int max_rows;  // of a chunk
  int fp16;      // type of the rows and weights (else bf16)
  int splits;    // product_few_kernel: CTAs of a cluster
};

struct Segments {
  int off[kMaxExperts + 1];
  int first[kMaxExperts + 1];  // first chunk of each expert
  int size[kMaxExperts];       // rows per chunk
  int sum[kMaxExperts / 32];   // chunks of 32 experts
};

struct GTile {
  int e, m, row0, nrows;
  bool one;  // the expert's only chunk
};

__device__ __forceinline__ GTile tile_at(int tile, const ProductArgs& a, const Segments& S) {
  GTile t;
  const int ch = tile / a.m_tiles;
  t.m = tile - ch * a.m_tiles;
  int lo = 0, hi = a.E;  // first[lo] <= ch < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (S.first[mid] <= ch)
      lo = mid;
    else
      hi = mid;
  }
  t.e = uniform(lo);
  const int first = uniform(S.first[t.e]), size = uniform(S.size[t.e]);
  t.one = uniform(S.first[t.e + 1]) - first == 1;
  t.row0 = uniform(S.off[t.e]) + (ch - first) * size;
  t.nrows = min(size, uniform(S.off[t.e + 1]) - t.row0);
  return t;
}

// Segments and their chunks (ceil(rows / max_rows) near-equal ones), an expert a thread of
// the block. Offsets that fall or leave [0, R] are refused as a whole: no row is touched.
// Returns the number of chunks.
__device__ __forceinline__ int scan_chunks(const ProductArgs& a, Segments& S) {
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, E = a.E;
  int n = 0, before = 0;
  bool bad = false;
  if (warp < kMaxExperts / 32) {
    if (tid < E) {
      const int o = a.offsets[tid], end = a.offsets[tid + 1], L = end - o;
      bad = o < 0 || end < o || end > a.R;
      if (!bad) n = (L + a.max_rows - 1) / a.max_rows;
      S.off[tid] = o;
      if (tid == E - 1) S.off[E] = end;
      S.size[tid] = n > 0 ? ((L + n - 1) / n + 15) / 16 * 16 : 0;
    }
    before = exclusive_sum(n);
    if (lane == 31) S.sum[warp] = before + n;
  }
  // (The vote tells the compiler that all lanes know the same, and with it how long their
  // loops are: without it a stage took 8 % longer.)
  bad = __any_sync(kAll, __syncthreads_or(bad));
  if (bad && tid == 0 && blockIdx.x == 0) atomicOr(a.err, kDevErrBadIds);
  int chunks = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 32; ++w) {
    if (w == warp) before += chunks;
    chunks += S.sum[w];
  }
  if (bad) chunks = 0;
  if (tid < E) S.first[tid] = before;
  if (tid == 0) S.first[E] = chunks;
  __syncthreads();
  return uniform(chunks);
}

// tmB32: the rows again, in boxes of 32, for chunks that do not fill a box of 128.
template <int WAY>
__global__ void __launch_bounds__(kGThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmB32, const ProductArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kGStages + 5];
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ Segments S;

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t rank = pair_rank();  // 0 = leader (issues the MMAs)
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  uint64_t* full = bars;
  uint64_t* empty = full + kGStages;
  uint64_t* tfull = empty + kGStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  if (tid == 0) {
    for (int s = 0; s < kGStages; ++s) {
      mbar_init(smem_u32(&full[s]), 2);   // each CTA's producer announces its own bytes
      mbar_init(smem_u32(&empty[s]), 1);  // the leader's MMA commit, multicast to both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 2 * kGEpiWarps);
    }
    mbar_init(smem_u32(done), 1);
    abort_s = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmB32);
  }
  if (warp == 0) {
    tmem_alloc_pair(smem_u32(&tmem_base_s), kGTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers initialised, tensor memory allocated
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const int total = scan_chunks(a, S) * a.m_tiles;
  const uint32_t tmem_base = uniform(tmem_base_s);
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
  const int nk = (a.D + kGK - 1) / kGK;

  if (warp >= kGProd0) {
    // ------------------------------------------------------- producers ---
    // One warp a ring slot: a warp's copies that signal another barrier than
    // its previous ones wait for those to land.
    const int slot = warp - kGProd0;
    const bool leader = elect_one();
    const uint32_t st = smem_base + slot * kGStageBytes;
    const uint32_t fb = peer_addr(smem_u32(&full[slot]), 0);  // the leader's barrier
    const uint32_t eb = smem_u32(&empty[slot]);
    const uint64_t pol_once = l2_policy_evict_first(), pol_normal = l2_policy_evict_normal(),
                   pol_keep = l2_policy_evict_last();
    uint32_t use = 0;  // fills of this slot so far
    int q = 0;         // stage counter modulo the ring
    bool ok = true;
    for (int tile = pair; tile < total && ok; tile += npairs) {
      if (aborted()) break;
      const GTile t = tile_at(tile, a, S);
      const int nh = ((t.nrows + 15) & ~15) / 2;  // this CTA's half of the rows
      const int brow = t.row0 + (int)rank * nh;
      const int boxes = (nh + 31) / 32;
      const int f = t.m * 256 + (int)rank * 128;
      // Boxes wholly beyond W's features are left out, nobody reads what they give: zeros
      // take a copy longer than values (22886 rows x 128 x 128: 12.1 us with, 7.3 without).
      const bool lower = f < a.F, upper = WAY == kForward ? lower : f + 64 < a.F;
      const uint32_t bytes = (upper ? kGHalf : lower ? kGBox : 0) +
                             (nh > 96 ? kGHalf : (uint32_t)boxes * 32 * kGK * 2);
      // W is read by every chunk of the expert, the rows by every m-tile.
      const uint64_t pol_w = t.one ? pol_once : pol_normal;
      for (int kb = 0; kb < nk; ++kb) {
        const bool mine = q == slot;
        if (++q == kGStages) q = 0;
        if (!mine) continue;
        if (!warp_wait(eb, (use & 1u) ^ 1u)) {
          fail();
          ok = false;
          break;
        }
        if (leader) {
          mbar_expect_tx_cluster(fb, bytes);
          if (WAY == kForward) {
            if (lower) tma_load_3d_pair(st, &tmA, fb, kb * kGK, f, t.e, pol_w);
          } else {
            if (lower) tma_load_3d_pair(st, &tmA, fb, f, kb * kGK, t.e, pol_w);
            if (upper) tma_load_3d_pair(st + kGBox, &tmA, fb, f + 64, kb * kGK, t.e, pol_w);
          }
          if (nh > 96) {
            tma_load_2d_pair(st + kGHalf, &tmB, fb, kb * kGK, brow, pol_keep);
          } else {
            for (int j = 0; j < boxes; ++j)
              tma_load_2d_pair(st + kGHalf + j * (32 * kGK * 2), &tmB32, fb, kb * kGK,
                               brow + 32 * j, pol_keep);
          }
        }
        __syncwarp();
        ++use;
      }
    }
    if (!ok || aborted()) {
      // Copies issued just before the abort may still be landing in this CTA's
      // shared memory: a copy completes within microseconds.
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 50000ull) {
      }
    } else if (use > 0 && !warp_wait(eb, (use - 1) & 1u)) {
      fail();  // (the peer's last arrival at this slot's barrier is in before the CTA ends)
    }
    __syncwarp();
  } else if (warp == 0) {
    // ---------------------------------------------- MMA issuer (leader) ---
    // The whole warp runs the loops, so that descriptors stay in uniform
    // registers; one elected lane issues.
    if (rank == 0) {
      const bool leader = elect_one();
      constexpr bool a_mn = WAY == kDx;
      const uint32_t id0 = idesc_16(a.fp16 != 0, a_mn, false);
      int s = 0;
      uint32_t ph = 0;
      uint32_t it = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs, ++it) {
        if (aborted()) break;
        const GTile t = tile_at(tile, a, S);
        const uint32_t idesc = id0 | idesc_shape(256, (t.nrows + 15) & ~15);
        const uint32_t b = it & 1u, use = it >> 1;
        if (!warp_wait_cluster(smem_u32(&tempty[b]), (use & 1u) ^ 1u)) {
          fail();
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
            const uint64_t db = sdesc_kmajor<128>(st + kGHalf);
            // 16 of the reduction: 32 bytes of a K-major row, 16 rows of an MN-major block.
            constexpr uint64_t ia = a_mn ? 16 * 128 / 16 : 2, ib = 2;
            const int steps = min(4, (a.D - kb * kGK + 15) / 16);
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
      // Every MMA issued above has finished before tensor memory is freed.
      if (leader) umma_pair_commit(smem_u32(done), 0x1);
      __syncwarp();
      if (!warp_wait(smem_u32(done), 0)) fail();
    }
  } else {
    // -------------------------------------------------------- epilogue ---
    const int q = warp & 3;                        // tensor-memory lane quarter of this warp
    const int side = (warp - kGEpiWarp0) >> 2;     // takes 32-column chunks side, side + 2, ...
    const uint32_t te0 = peer_addr(smem_u32(&tempty[0]), 0);
    const uint32_t te1 = peer_addr(smem_u32(&tempty[1]), 0);
    uint32_t it = 0;
    for (int tile = pair; tile < total; tile += npairs, ++it) {
      if (aborted()) break;
      const GTile t = tile_at(tile, a, S);
      const int f = t.m * 256 + (int)rank * 128 + q * 32 + lane;  // this lane's feature
      const uint32_t b = it & 1u, use = it >> 1;
      if (!warp_wait_cluster(smem_u32(&tfull[b]), use & 1u)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + b * kGMaxN;
      for (int c0 = side * 32; c0 < t.nrows; c0 += 64) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tb + c0, v);
        tmem_wait_ld();
        if (f < a.F) {
          uint16_t* p = static_cast<uint16_t*>(a.out) + (size_t)(t.row0 + c0) * a.F + f;
          const int n = t.nrows - c0;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t w = pack16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), a.fp16);
            if (j < n) p[(size_t)j * a.F] = (uint16_t)w;
            if (j + 1 < n) p[(size_t)(j + 1) * a.F] = (uint16_t)(w >> 16);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(b == 0 ? te0 : te1);
      __syncwarp();
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

// Few chunks of few rows: a cluster a tile of 128 features x up to 64 rows, whose CTAs take a
// share of the reduction each (a.splits of them) with MMAs of their own, M = 128. Their
// sums, fp32, go to the CTA of the row in the cluster, which adds them in the CTAs' order.
//
// An SM takes in 64 bytes a cycle, 140 ns for 128 x 64 weights, whatever the rows are: what
// bounds a tile is the weights' way into its SMs, and 2048 x 2048 of them are 16 SMs' in
// the form above.
constexpr int kFewRows = 64, kFewStages = 7;
constexpr int kFewBytes = kGHalf + kFewRows * kGK * 2;   // of a stage
constexpr int kFewProd0 = 5;                             // after the issuer, four epilogues
constexpr int kFewThreads = (kFewProd0 + kFewStages) * 32;
constexpr int kFewSums = kFewRows * 128 * 4;             // of all CTAs, for this one's rows
constexpr int kFewSmemBytes = kFewStages * kFewBytes + kFewSums + 1024;
static_assert(kMaxExperts <= kFewThreads, "an expert a thread");

template <int WAY>
__global__ void __launch_bounds__(kFewThreads, 1)
    product_few_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB32, const ProductArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kFewStages + 2];
  __shared__ uint32_t tmem_base_s;
  __shared__ Segments S;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int rank = uniform((int)pair_rank());
  uint64_t *full = bars, *empty = full + kFewStages, *tfull = empty + kFewStages,
           *got = tfull + 1;  // got: the sums of every CTA
  if (tid == 0) {
    for (int s = 0; s < kFewStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    mbar_init(smem_u32(got), 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB32);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_base_s), kFewRows);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_barrier();  // every CTA is there to be written to
  pdl_wait();
  pdl_trigger();
  const int total = scan_chunks(a, S) * a.m_tiles;
  const int tile = blockIdx.x / a.splits;
  const bool active = tile < total;
  const uint32_t tmem_base = uniform(tmem_base_s);
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sums = smem_base + kFewStages * kFewBytes;
  // This CTA's stages of the reduction.
  const int nk = (a.D + kGK - 1) / kGK, share = (nk + a.splits - 1) / a.splits;
  const int kb0 = min(rank * share, nk), cnt = min(share, nk - kb0);
  GTile t = {};
  int n = 0, own = 0;  // columns of the accumulator; of those, the rows of a CTA
  if (active) {
    t = tile_at(tile, a, S);
    n = (t.nrows + 15) & ~15;
    own = n / a.splits;
  }
  auto fail = [&]() { atomicOr(a.err, kDevErrTimeout); };

  if (!active) {
  } else if (warp >= kFewProd0) {
    // One warp a ring slot, as above.
    const int slot = warp - kFewProd0;
    const bool leader = elect_one();
    const uint32_t st = smem_base + slot * kFewBytes;
    const uint32_t fb = smem_u32(&full[slot]), eb = smem_u32(&empty[slot]);
    const uint64_t pol_w = t.one ? l2_policy_evict_first() : l2_policy_evict_normal(),
                   pol_keep = l2_policy_evict_last();
    const int f = t.m * 128, boxes = (n + 31) / 32;
    const bool upper = WAY == kForward || f + 64 < a.F;  // (see product_kernel)
    const uint32_t bytes = (upper ? kGHalf : kGBox) + (uint32_t)boxes * 32 * kGK * 2;
    bool ok = true;
    for (int j = slot, use = 0; j < cnt; j += kFewStages, ++use) {
      if (!warp_wait(eb, (use & 1) ^ 1)) {
        fail();
        ok = false;
        break;
      }
      const int k = (kb0 + j) * kGK;
      if (leader) {
        mbar_arrive_expect_tx(fb, bytes);
        if (WAY == kForward) {
          tma_load_3d(st, &tmA, fb, k, f, t.e, pol_w);
        } else {
          tma_load_3d(st, &tmA, fb, f, k, t.e, pol_w);
          if (upper) tma_load_3d(st + kGBox, &tmA, fb, f + 64, k, t.e, pol_w);
        }
        for (int i = 0; i < boxes; ++i)
          tma_load_2d(st + kGHalf + i * (32 * kGK * 2), &tmB32, fb, k, t.row0 + 32 * i, pol_keep);
      }
      __syncwarp();
    }
    if (!ok) {  // copies issued before may still be landing
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 50000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    const bool leader = elect_one();
    constexpr bool a_mn = WAY == kDx;
    const uint32_t idesc = idesc_16(a.fp16 != 0, a_mn, false) | idesc_shape(128, n);
    int s = 0;
    uint32_t ph = 0;
    for (int j = 0; j < cnt; ++j) {
      if (!warp_wait(smem_u32(&full[s]), ph)) {
        fail();
        break;
      }
      tc_fence_after();
      if (leader) {
        const uint32_t st = smem_base + s * kFewBytes;
        const uint64_t da = a_mn ? sdesc_mnmajor(st, kGBox) : sdesc_kmajor<128>(st);
        const uint64_t db = sdesc_kmajor<128>(st + kGHalf);
        constexpr uint64_t ia = a_mn ? 16 * 128 / 16 : 2, ib = 2;
        const int steps = min(4, (a.D - (kb0 + j) * kGK + 15) / 16);
        for (int kk = 0; kk < steps; ++kk)
          umma_bf16(tmem_base, da + kk * ia, db + kk * ib, idesc, (j | kk) != 0);
        umma_commit(smem_u32(&empty[s]));
      }
      __syncwarp();
      if (++s == kFewStages) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (leader) umma_commit(smem_u32(tfull));
    __syncwarp();
  } else {
    const int q = warp & 3;
    if (!warp_wait(smem_u32(tfull), 0)) fail();
    tc_fence_after();
    // Into the ring, which the MMAs are done with, as [row][feature], and from there to the
    // rows' CTAs in one copy each. (Stores to the other CTAs: 14 cycles for 32 values, 64
    // rows x 1024 x 2048 6.7 us.)
    const uint32_t mine = smem_base + (q * 32 + lane) * 4;
    for (int c0 = 0; c0 < n; c0 += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + c0, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c0 + j < n) st_shared_u32(mine + (c0 + j) * 512, cnt > 0 ? v[j] : 0u);
    }
    fence_proxy_async_smem();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (warp == 1) {
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(got), n * 512);
      __syncwarp();
      if (lane < a.splits)
        bulk_copy_peer(peer_addr(sums + rank * own * 512, lane), smem_base + lane * own * 512,
                       own * 512, peer_addr(smem_u32(got), lane));
    }
    __syncwarp();
  }

  if (active && !warp_wait_cluster(smem_u32(got), 0)) fail();
  // Eight features of a row a thread.
  for (int i = tid; i < own * 16; i += kFewThreads) {
    const int c = i >> 4, ch = i & 15, row = rank * own + c, f = t.m * 128 + ch * 8;
    if (row >= t.nrows || f >= a.F) continue;
    float v[8] = {};
    for (int s = 0; s < a.splits; ++s) {
      const float4* p = reinterpret_cast<const float4*>(
          smem_raw + (sums - smem_u32(smem_raw)) + ((s * own + c) * 128 + ch * 8) * 4);
      const float4 x = p[0], y = p[1];
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
      v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
    }
    uint4 o;
    o.x = pack16x2(v[0], v[1], a.fp16);
    o.y = pack16x2(v[2], v[3], a.fp16);
    o.z = pack16x2(v[4], v[5], a.fp16);
    o.w = pack16x2(v[6], v[7], a.fp16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (size_t)(t.row0 + row) * a.F + f) = o;
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // no CTA ends before the others have its sums
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kFewRows);
  }
}

template <int WAY>
cudaError_t launch_few(const CUtensorMap& tmA, const CUtensorMap& tmB32, const ProductArgs& a,
                       int clusters, cudaStream_t st) {
  static DeviceFlags attr_done;
  if (cudaError_t e = smem_attr_once(attr_done, product_few_kernel<WAY>, kFewSmemBytes);
      e != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * a.splits));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kFewSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, product_few_kernel<WAY>, tmA, tmB32, a);
}

// CTAs that share a tile's reduction: as many as the chip holds at once (12 clusters of
// eight, 36 of four; 16 of eight took 10.8 us where four took 6.3); 0: the form of pairs,
// where it takes less by these estimates, in us (a stage 0.14 and 0.2, the way of a row's
// sums 0.02). Measured, pairs and this: 1 row x 128 x 2048 7.6 and 4.4; 16 rows x 1024 x 2048
// 8.0 and 5.1, x 2048 x 2048 8.1 and 6.0; 64 rows 8.1 and 7.2.
int few_splits(long long clusters, int R, int D) {
  const int nk = (D + kGK - 1) / kGK, s = clusters <= 12 ? 8 : clusters <= 36 ? 4 : 0;
  if (s == 0) return 0;
  const double few = 3.9 + 0.2 * ((nk + s - 1) / s) + 0.02 * std::min(R, kFewRows);
  return few + 0.3 < 3.3 + 0.14 * nk ? s : 0;
}

template <int WAY>
cudaError_t launch_way(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmB32,
                       const ProductArgs& a, long long max_tiles, int num_sms, cudaStream_t st) {
  static DeviceFlags attr_done;
  if (cudaError_t e = smem_attr_once(attr_done, product_kernel<WAY>, kGSmemBytes);
      e != cudaSuccess)
    return e;
  static std::atomic<int> resident[kMaxDevices];
  return launch_clusters(product_kernel<WAY>, 2, resident, kGThreads, kGSmemBytes, max_tiles,
                         num_sms, st, tmA, tmB, tmB32, a);
}

// Rows of a chunk, at most 256: where the chip's 76 pairs take a tile or two each, as many
// chunks as they take then (uneven segments make half a chunk more each), of at least 64
// rows. (Every chunk reads the weights again, and below 64 rows a stage's MMAs take less
// than its waits: 512 rows x 2048 x 2048 14.3 us in chunks of 256, 9.1 of 64, 14.6 of 32;
// 600 rows 9.7 us in chunks of 80, 13.4 of 64, which make two rounds; 2500 x 1024 x 1024 8.5
// and 9.8; 22886 x 256 x 512, two rounds of 160 rows and of 256, 9.9 and 11.2.)
int chunk_rows(int R, int E, int m_tiles) {
  for (int rounds = 1; rounds <= 2; ++rounds) {
    const double chunks = rounds * 76 / m_tiles - 0.5 * (E - 1);
    if (chunks * kGMaxN >= R) return std::max(64, (int)std::ceil(R / chunks / 16) * 16);
  }
  return kGMaxN;
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
  a.max_rows = chunk_rows(R, E, a.m_tiles);
  a.fp16 = fp16;
  CUtensorMap tmA, tmB, tmB32;
  if (!make_map(&tmA, w, E, N, K, transposed ? 64 : 128) || !make_map(&tmB32, x, 0, R, a.D, 32))
    return cudaErrorInvalidValue;
  const long long few = std::min<long long>(R, (R + 63LL * E) / kFewRows) * ((a.F + 127) / 128);
  if (a.splits = few_splits(few, R, a.D); a.splits > 0) {
    a.m_tiles = (a.F + 127) / 128;
    a.max_rows = kFewRows;
    return transposed ? launch_few<kDx>(tmA, tmB32, a, (int)few, st)
                      : launch_few<kForward>(tmA, tmB32, a, (int)few, st);
  }
  // A CTA's half of a chunk has at most 96 rows where these say so: the large box goes
  // unused (describing it takes the host 0.3 us).
  tmB = tmB32;
  if (std::min(R, a.max_rows) > 192 && !make_map(&tmB, x, 0, R, a.D, 128))
    return cudaErrorInvalidValue;
  const long long chunks = std::min<long long>(R, (long long)E + R / a.max_rows);
  return transposed
             ? launch_way<kDx>(tmA, tmB, tmB32, a, chunks * a.m_tiles, num_sms, st)
             : launch_way<kForward>(tmA, tmB, tmB32, a, chunks * a.m_tiles, num_sms, st);
}

}  // namespace mm
