// The gradient of the experts' weights over ragged segments of rows:
//
//   dW[e] = sum over the rows r of expert e of dy[r] x[r]^T          [N, K]
//
// The reduction runs along the rows of both matrices, so both operands are
// MN-major: tiles of 64 rows x 64 columns (128 bytes a row, 128-byte swizzle) as
// they lie in memory, no transpose. A tile of the result is 256 features n x bn
// (256 or 128) features k, made by a cluster of two CTAs: each has 128 of the
// features n, its own accumulators, its own copies and its own MMAs (M = 128). A stage
// of 256 columns brings 48 KB into an SM, 32 of which the other CTA reads too: out of
// L2, since the two run side by side. (Half of that loaded by each CTA and handed to the
// other through distributed shared memory: 301 us where this takes 188.)
//
// Long segments take one MMA over the pair instead, as in grouped_product.cu (PAIR: M =
// 256, half of the other operand in each CTA, 32 KB of shared memory a stage for 48).
// Why not all: a segment of some 256 rows is four stages, 2000 cycles of MMAs, after
// which 64 KB leave each SM. Signals between the CTAs queue behind those stores (measured:
// 2.2 us from the last MMA to the pair's completion signal, 1.6 us back from the epilogue),
// and with two accumulators that is what 32768 rows x 128 experts x 1536 x 2048 wait for:
// 264 us, where the form of two MMAs takes 188. All of its signals stay within a CTA.
//
// Rows beyond a segment belong to another expert: the last stage is cut to whole
// steps of 16 rows, and where those hold rows of the next segment the issuing
// warp writes zeros over them, in both operands (0 times another expert's infinity is
// NaN). Columns beyond a matrix are zeros out of the copy. The results leave
// through shared memory as boxes of 32 rows x 128 bytes, which the copy cuts at the
// matrix's edges (stores out of registers, 32 bytes a lane in 32 rows: 245 us where
// boxes took 191).
//
// fp32 results (and parts, below) are made of kSliceRows rows of the segment at a time:
// the tensor cores cut what they add, and 512 rows leave 5e-7 of it where 4096 leave
// 4e-6. In tiles of 128 columns the slices are summed in the epilogue's registers; in
// tiles of 256, which do not fit there, they are added up in memory, each after the one
// before (20011 rows x 8 x 640 x 328: 41 us that way, 30 in registers; but 32768 x 128 x
// 1536 x 2048, where few segments have a second slice, 313 and 411). 16-bit results are
// one accumulation.
//
// Few tiles with long reductions are cut into parts of `part_rows` rows, whose fp32
// results go to the workspace and are summed in order by a second launch (the rule is
// at split_of).
//
// What bounds it, on one GB300: the case above takes 188 us with even segments and 207
// with uneven ones (154 at the copy rate of its bytes; 120 for its results alone). 2.4 GB
// of loads and 0.8 GB of stores pass between L2 and the SMs, 17 TB/s, and shared memory
// moves 512 KB a tile. Long segments run at 1.64 to 1.82 PFLOP/s (two MMAs: 1.5, bound by
// shared memory). Few narrow tiles wait for their ring: a slot's turn takes 1.2 us, longer
// where the rows are no whole number of lines (20011 rows x 8 experts x 640 x 328: 26 us, x
// 320 21).
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
constexpr int kRows = 64;                    // rows of the reduction a stage
constexpr int kBlock = kRows * 128;          // 8 KB: 64 rows x 64 columns
constexpr int kABytes = 2 * kBlock;          // this CTA's 128 features n
constexpr int kEpiWarp0 = 1, kEpiWarps = 8;
constexpr int kProd0 = kEpiWarp0 + kEpiWarps;  // producers: one warp a slot
constexpr int kStore = 32 * 128;             // 4 KB a warp: results on their way out
constexpr int kStaticBytes = 2000;           // at most: barriers, offsets, parts

// The ring. A slot's turn takes some 1.2 us, so the bytes in flight bound the rate where
// nothing else does: 24000 rows x 4 x 512 x 1024 take 30.2 us with 4 slots of the narrow
// tiles' stages, 24.7 with 6. (One producer warp a slot.)
template <int BN, bool PAIR>
struct Ring {
  static constexpr int kStages = BN == 256 && !PAIR ? 4 : 6;
  static constexpr int kBoxes = BN / 64 / (PAIR ? 2 : 1);  // of 64 features k, in one SM
  static constexpr int kStageBytes = kABytes + kBoxes * kBlock;
  static constexpr int kThreads = (kProd0 + kStages) * 32;
  static constexpr int kSmemBytes = kStages * kStageBytes + kEpiWarps * kStore + 1024;
  static_assert(kSmemBytes <= 227 * 1024 - kStaticBytes, "shared memory");
};
constexpr int kAccCols = 256;                // columns of an accumulator, of which there are two
constexpr int kSliceRows = 512;
constexpr int kCtas = 2;                     // of a cluster: 128 features n each
constexpr int kPairs = 76;                   // clusters on the chip, for the choice of parts

struct DwArgs {
  const int32_t* offsets;  // [E + 1]
  void* out;
  float* parts;            // [parts][N][K] (part_rows != 0)
  unsigned* err;
  int E, R, N, K;
  int m_tiles, n_tiles;
  int part_rows;           // 0: segments are whole
  int ahead;               // bring the rows of the cluster's next tile into L2 (ahead_of)
  int sum_values;          // of a block that sums parts: 1024, or 128 for many parts
  int fp16, out_fp32, accumulate;
};

// Parts of a segment of L rows (an expert without rows has one, of zeros).
__host__ __device__ __forceinline__ int parts_of(int L, int part_rows) {
  return part_rows == 0 || L <= part_rows ? 1 : (L + part_rows - 1) / part_rows;
}

// Offsets that fall or leave [0, R].
__device__ __forceinline__ bool bad_at(const int32_t* off, int e, int R) {
  return off[e] < 0 || off[e + 1] < off[e] || off[e + 1] > R;
}

// Exclusive sums of the experts' parts into first[0 .. E], by one warp.
__device__ __forceinline__ void scan_parts(const int32_t* off, int E, int part_rows,
                                           uint16_t* first) {
  const int lane = threadIdx.x & 31, per = (E + 31) / 32, e0 = lane * per;
  int sum = 0;
  for (int e = e0; e < min(e0 + per, E); ++e) sum += parts_of(off[e + 1] - off[e], part_rows);
  int run = exclusive_sum(sum);
  for (int e = e0; e < min(e0 + per, E); ++e) {
    first[e] = (uint16_t)run;
    run += parts_of(off[e + 1] - off[e], part_rows);
  }
  if (lane == 31) first[E] = (uint16_t)run;
}

struct Item {
  int e, m, n, row0, rows;
  int part;   // its place in the workspace, -1: the result itself
};

// BN: features k of a tile. PAIR: one MMA over the cluster. tmC: the result, tmP: the
// parts.
template <int BN, bool PAIR>
__global__ void __launch_bounds__(Ring<BN, PAIR>::kThreads, 1)
    dw_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmP,
              const DwArgs a) {
  using R = Ring<BN, PAIR>;
  constexpr int kStages = R::kStages, kStageBytes = R::kStageBytes, kThreads = R::kThreads;
  static_assert(!PAIR || BN == 256, "narrow tiles are made by each CTA for itself");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[(PAIR ? 3 : 2) * kStages + 5];
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ int32_t off_s[kMaxExperts + 1];
  __shared__ uint16_t first_s[kMaxExperts + 1];
  static_assert(sizeof(bars) + 12 + sizeof(off_s) + sizeof(first_s) <= kStaticBytes, "shared memory");

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int E = a.E;
  const uint32_t rank = pair_rank();
  const int pair = blockIdx.x / kCtas, npairs = gridDim.x / kCtas;

  uint64_t* full = bars;
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint64_t* land = done + 1;  // PAIR: this CTA's copies of a segment's last stage
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      // A CTA's copies and MMAs are its own. PAIR: the leader's barrier counts both CTAs'
      // copies, and its MMAs free the slots of both.
      mbar_init(smem_u32(&full[s]), PAIR ? kCtas : 1);
      mbar_init(smem_u32(&empty[s]), 1);
      if (PAIR) mbar_init(smem_u32(&land[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), PAIR ? kCtas * kEpiWarps : kEpiWarps);
    }
    mbar_init(smem_u32(done), 1);
    abort_s = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 0) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(&tmem_base_s), 2 * kAccCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&tmem_base_s), 2 * kAccCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers are initialised
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  for (int e = tid; e < E; e += kThreads) {
    off_s[e] = a.offsets[e];
    if (e == E - 1) off_s[E] = a.offsets[E];
    bad |= bad_at(a.offsets, e, a.R);
  }
  // Bad offsets are refused as a whole: nothing is written. (The vote tells the compiler
  // that all lanes know the same, and with it how long their loops are: without it a stage
  // took 10 % longer.)
  bad = __any_sync(kAll, __syncthreads_or(bad));
  if (bad && tid == 0 && blockIdx.x == 0) atomicOr(a.err, kDevErrBadIds);
  if (a.part_rows != 0) {
    if (warp == 0 && !bad) scan_parts(off_s, E, a.part_rows, first_s);
    __syncthreads();
  }
  const int per = a.m_tiles * a.n_tiles;
  const int total = bad ? 0 : (a.part_rows != 0 ? uniform(first_s[E]) : E) * per;
  const uint32_t tmem_base = uniform(tmem_base_s);
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto fail = [&]() {
    for (int r = 0; r < kCtas; ++r) st_cluster_u32(peer_addr(smem_u32(&abort_s), r), 1u);
    atomicOr(a.err, kDevErrTimeout);
  };
  constexpr uint16_t all = (1 << kCtas) - 1;
  auto aborted = [&]() {
    return __any_sync(kAll, *reinterpret_cast<volatile int*>(&abort_s) != 0);
  };
  auto item_at = [&](int i) {
    Item t;
    const int p = i / per, j = i - p * per;
    t.m = j / a.n_tiles;
    t.n = j - t.m * a.n_tiles;
    if (a.part_rows == 0) {
      t.e = p;
      t.row0 = uniform(off_s[p]);
      t.rows = uniform(off_s[p + 1]) - t.row0;
      t.part = -1;
    } else {
      int lo = 0, hi = E;  // first[lo] <= p < first[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_s[mid] <= p)
          lo = mid;
        else
          hi = mid;
      }
      t.e = uniform(lo);
      const int first = uniform(first_s[t.e]);
      t.row0 = uniform(off_s[t.e]) + (p - first) * a.part_rows;
      t.rows = min(a.part_rows, uniform(off_s[t.e + 1]) - t.row0);
      t.part = uniform(first_s[t.e + 1]) - first > 1 ? p : -1;
    }
    return t;
  };
  // Zeros over the rows of a stage from `left` up to the next multiple of 16, in every block:
  // 128 bytes each. Straight-line code: in loops it took a warp 900 cycles, 14 us of 224
  // for 32768 rows of uneven load.
  auto clear = [&](uint32_t st, int left) {
    const uint32_t z = st + (left + (lane >> 3)) * 128 + (lane & 7) * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)  // four rows at a time
      if ((left & 15) + (lane >> 3) + 4 * j < 16) {
#pragma unroll
        for (int k = 0; k < 2 + R::kBoxes; ++k) st_shared_zero16(z + k * kBlock + j * 512);
      }
    __syncwarp();
    fence_proxy_async_smem();
    __syncwarp();
  };
  // Slices of an item's reduction, and the rows of one.
  auto slice_rows = [&](const Item& t) {
    return a.out_fp32 || t.part >= 0 ? kSliceRows : 1 << 30;
  };
  auto slices = [&](const Item& t) {
    return t.rows == 0 ? 0 : (t.rows - 1) / slice_rows(t) + 1;
  };

  if (warp >= kProd0) {
    // ------------------------------------------------------- producers ---
    // One warp a ring slot: a warp's copies that signal another barrier than
    // its previous ones wait for those to land.
    const int slot = warp - kProd0;
    const bool leader = elect_one();
    const uint32_t st = smem_base + slot * kStageBytes;
    const uint32_t fb = PAIR ? peer_addr(smem_u32(&full[slot]), 0) : smem_u32(&full[slot]);
    const uint32_t eb = smem_u32(&empty[slot]), lb = smem_u32(&land[slot]);
    const uint64_t pol = l2_policy_evict_last();  // read by every tile of the expert
    constexpr uint32_t bytes = kABytes + R::kBoxes * kBlock;
    uint32_t use = 0, landed = 0;  // fills of this slot so far
    int q = 0;                     // stage counter modulo the ring
    bool ok = true;
    for (int i = pair; i < total && ok; i += npairs) {
      if (aborted()) break;
      const Item t = item_at(i);
      const int nsl = slices(t), step = slice_rows(t);
      const int f = (t.m * kCtas + (int)rank) * 128, c = t.n * BN + (PAIR ? (int)rank * (BN / 2) : 0);
      if (BN == 256 && !PAIR && a.ahead && i + npairs < total) {
        const Item u = item_at(i + npairs);
        const int uf = (u.m * kCtas + (int)rank) * 128, uc = u.n * BN + (int)rank * (BN / 2);
        if (leader) {
          // Boxes 2 * stage + column block, shared out among the tiles that read them.
          const int boxes = (u.rows + kRows - 1) / kRows * 2;
          for (int x = u.n + slot * a.n_tiles; x < boxes; x += kStages * a.n_tiles)
            if (uf + 64 * (x & 1) < a.N)
              tma_prefetch_2d(&tmA, uf + 64 * (x & 1), u.row0 + (x >> 1) * kRows, pol);
          for (int x = u.m + slot * a.m_tiles; x < boxes; x += kStages * a.m_tiles)
            if (uc + 64 * (x & 1) < a.K)
              tma_prefetch_2d(&tmB, uc + 64 * (x & 1), u.row0 + (x >> 1) * kRows, pol);
        }
        __syncwarp();
      }
      for (int sl = 0; sl < nsl && ok; ++sl) {
        const int len = min(step, t.rows - sl * step), nk = (len + kRows - 1) / kRows;
        for (int kb = 0; kb < nk; ++kb) {
          const bool mine = q == slot;
          if (++q == kStages) q = 0;
          if (!mine) continue;
          if (!warp_wait_cluster(eb, (use & 1u) ^ 1u)) {
            fail();
            ok = false;
            break;
          }
          const int r = t.row0 + sl * step + kb * kRows;
          if constexpr (PAIR) {
            const int left = len - kb * kRows;  // rows of this stage, if fewer than 64
            const bool tail = left < kRows && (left & 15) != 0;
            const uint32_t bar = tail ? peer_addr(lb, rank) : fb;
            if (leader) {
              mbar_expect_tx_cluster(bar, bytes);
              tma_load_2d_pair(st, &tmA, bar, f, r, pol);
              tma_load_2d_pair(st + kBlock, &tmA, bar, f + 64, r, pol);
#pragma unroll
              for (int b = 0; b < R::kBoxes; ++b)
                tma_load_2d_pair(st + kABytes + b * kBlock, &tmB, bar, c + 64 * b, r, pol);
            }
            __syncwarp();
            if (tail) {
              if (!warp_wait(lb, landed & 1u)) {
                fail();
                ok = false;
                break;
              }
              ++landed;
              clear(st, left);
              if (leader) mbar_arrive_cluster(fb);
              __syncwarp();
            }
          } else {
            if (leader) {
              mbar_arrive_expect_tx(fb, bytes);
              tma_load_2d(st, &tmA, fb, f, r, pol);
              tma_load_2d(st + kBlock, &tmA, fb, f + 64, r, pol);
#pragma unroll
              for (int b = 0; b < R::kBoxes; ++b)
                tma_load_2d(st + kABytes + b * kBlock, &tmB, fb, c + 64 * b, r, pol);
            }
            __syncwarp();
          }
          ++use;
        }
      }
    }
    if (!ok || aborted()) {
      // Copies issued just before the abort may still be landing in either CTA's
      // shared memory: a copy completes within microseconds.
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 50000ull) {
      }
    } else if (use > 0 && !warp_wait_cluster(eb, (use - 1) & 1u)) {
      fail();  // (the peer's last arrival at this slot's barrier is in before the CTA ends)
    }
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------- MMA issuer (PAIR: the leader's) ---
    // The whole warp runs the loops, so that descriptors stay in uniform
    // registers; one elected lane issues.
    if (!PAIR || rank == 0) {
      const bool leader = elect_one();
      const uint32_t idesc = idesc_16(a.fp16 != 0, true, true) | idesc_shape(PAIR ? 256 : 128, BN);
      auto wait = [](uint32_t bar, uint32_t parity) {
        return PAIR ? warp_wait_cluster(bar, parity) : warp_wait(bar, parity);
      };
      auto mma = [&](uint32_t d, uint64_t da, uint64_t db, bool more) {
        if (PAIR)
          umma_pair_bf16(d, da, db, idesc, more);
        else
          umma_bf16(d, da, db, idesc, more);
      };
      int s = 0;
      uint32_t ph = 0, it = 0;
      bool ok = true;
      for (int i = pair; i < total && ok; i += npairs) {
        if (aborted()) break;
        const Item t = item_at(i);
        const int nsl = slices(t), step = slice_rows(t);
        for (int sl = 0; sl < nsl && ok; ++sl, ++it) {
          const int len = min(step, t.rows - sl * step), nk = (len + kRows - 1) / kRows;
          const uint32_t b = it & 1u, use = it >> 1;
          if (!wait(smem_u32(&tempty[b]), (use & 1u) ^ 1u)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + b * kAccCols;
          for (int kb = 0; kb < nk; ++kb) {
            if (!wait(smem_u32(&full[s]), ph)) {
              fail();
              ok = false;
              break;
            }
            const uint32_t st = smem_base + s * kStageBytes;
            const int left = len - kb * kRows;  // rows of this stage, if fewer than 64
            // (The MMAs of the stages before run meanwhile. With PAIR the rows lie in both
            // CTAs, whose producers clear them.)
            if (!PAIR && left < kRows && (left & 15) != 0) clear(st, left);
            tc_fence_after();
            if (leader) {
              const uint64_t da = sdesc_mnmajor(st, kBlock), db = sdesc_mnmajor(st + kABytes, kBlock);
              const int steps = min(4, (left + 15) / 16);
              // 16 rows are 128 descriptor units of 16 bytes.
              if (steps == 4) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma(d, da + kk * 128, db + kk * 128, (kb | kk) != 0);
              } else {
                for (int kk = 0; kk < steps; ++kk)
                  mma(d, da + kk * 128, db + kk * 128, (kb | kk) != 0);
              }
              if (PAIR)
                umma_pair_commit(smem_u32(&empty[s]), all);
              else
                umma_commit(smem_u32(&empty[s]));
            }
            __syncwarp();
            if (++s == kStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (!ok) break;
          if (leader) {
            if (PAIR)
              umma_pair_commit(smem_u32(&tfull[b]), all);
            else
              umma_commit(smem_u32(&tfull[b]));
          }
          __syncwarp();
        }
      }
      // Every MMA issued above has finished before tensor memory is freed.
      if (leader) {
        if (PAIR)
          umma_pair_commit(smem_u32(done), 1);
        else
          umma_commit(smem_u32(done));
      }
      __syncwarp();
      if (!warp_wait(smem_u32(done), 0)) fail();
    }
  } else {
    // -------------------------------------------------------- epilogue ---
    const int q = warp & 3;                     // tensor-memory lane quarter of this warp
    const int side = (warp - kEpiWarp0) >> 2;   // takes every other box of 128 bytes of columns
    const uint32_t buf = smem_base + kStages * kStageBytes + (warp - kEpiWarp0) * kStore;
    uint32_t it = 0;
    bool ok = true;
    for (int i = pair; i < total && ok; i += npairs) {
      if (aborted()) break;
      const Item t = item_at(i);
      const int nsl = slices(t);
      const int f0 = (t.m * kCtas + (int)rank) * 128 + q * 32;  // this warp's 32 features n
      const int k0 = t.n * BN, k1 = min(k0 + BN, a.K);
      // 32 rows of 128 bytes at column c, through this warp's buffer in the 128-byte
      // swizzle; the copy cuts what lies beyond the matrix.
      auto put = [&](int c, bool add, const uint32_t* v) {
        if (f0 >= a.N || c >= k1) return;
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_16(buf + lane * 128 + ((j ^ (lane & 7)) << 4),
                       make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (t.part >= 0)
            tma_store_3d(&tmP, buf, c, f0, t.part);
          else if (add)
            tma_add_3d(&tmC, buf, c, f0, t.e);
          else
            tma_store_3d(&tmC, buf, c, f0, t.e);
          bulk_commit();
        }
        __syncwarp();
      };
      // Waits for slice number `it`'s accumulator (its address), and hands it back.
      auto take = [&]() {
        const uint32_t bar = smem_u32(&tfull[it & 1u]), parity = (it >> 1) & 1u;
        ok = PAIR ? warp_wait_cluster(bar, parity) : warp_wait(bar, parity);
        if (!ok) fail();
        tc_fence_after();
        return tmem_base + ((uint32_t)(q * 32) << 16) + (it & 1u) * kAccCols;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        const uint32_t bar = smem_u32(&tempty[it & 1u]);
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_cluster(peer_addr(bar, 0));
          else
            mbar_arrive(bar);
        }
        __syncwarp();
        ++it;
      };
      if (nsl == 0) {
        // An expert without rows: its warps share out its zeros in whole pieces, whatever the
        // matrix's width (39 rows x 128 experts x 1552 x 1880 137 us; in boxes, where rows of
        // no whole number of lines take two for one, 218).
        if (a.accumulate) continue;
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) st_shared_zero16(buf + j * 512 + lane * 16);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const long long size = (long long)a.N * a.K * (a.out_fp32 ? 4 : 2);
          char* out = static_cast<char*>(a.out) + t.e * size;
          const int tile = (t.m * a.n_tiles + t.n) * kCtas + (int)rank;
          long long i = (long long)(tile * kEpiWarps + warp - kEpiWarp0) * kStore;
          for (; i < size; i += (long long)per * kCtas * kEpiWarps * kStore)
            bulk_store(out + i, buf, (uint32_t)min(size - i, (long long)kStore));
          bulk_commit();
        }
        __syncwarp();
        continue;
      }
      if constexpr (BN == 128) {
        if (a.out_fp32 || t.part >= 0) {
          // 64 columns a warp, summed over the slices in registers.
          uint32_t sum[2][32] = {};
          for (int sl = 0; sl < nsl && ok; ++sl) {
            const uint32_t tb = take();
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(tb + side * 64 + h * 32, v);
              tmem_wait_ld();
              if (sl == 0) {
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[h][j] = v[j];
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  sum[h][j] = __float_as_uint(__uint_as_float(sum[h][j]) + __uint_as_float(v[j]));
              }
            }
            release();
          }
          if (!ok) break;
          const bool add = a.accumulate && t.part < 0;
          put(k0 + side * 64, add, sum[0]);
          put(k0 + side * 64 + 32, add, sum[1]);
          continue;
        }
      }
      if (BN == 256 && a.out_fp32) {
        for (int sl = 0; sl < nsl; ++sl) {
          const uint32_t tb = take();
          if (!ok) break;
          // A slice is added to the ones before it once they are in memory.
          if (sl > 0 && lane == 0) bulk_wait();
          __syncwarp();
          for (int c = side * 32; c < BN; c += 64) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tb + c, v);
            tmem_wait_ld();
            if (c + 64 >= BN) release();
            put(k0 + c, a.accumulate || sl > 0, v);
          }
        }
        continue;
      }
      const uint32_t tb = take();
      if (!ok) break;
      if (a.accumulate) {
        for (int c = side * 32; c < BN; c += 64) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tb + c, v);
          tmem_wait_ld();
          if (f0 + lane < a.N && k0 + c < k1)
            add_row(static_cast<uint16_t*>(a.out) + ((size_t)t.e * a.N + f0 + lane) * a.K + k0 + c,
                    min(32, k1 - k0 - c) / 8, v, a.fp16);
          __syncwarp();
        }
        release();
      } else {
        // Boxes of 64 columns: the accumulator is free again once they are in registers,
        // before they are written.
        uint32_t w[BN / 128][32];
#pragma unroll
        for (int h = 0; h < BN / 64; ++h) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tb + (h >> 1) * 128 + side * 64 + (h & 1) * 32, v);
          tmem_wait_ld();
          if (a.fp16) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[h >> 1][(h & 1) * 16 + j] =
                  f16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[h >> 1][(h & 1) * 16 + j] =
                  bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
          }
        }
        release();
#pragma unroll
        for (int h = 0; h < BN / 128; ++h) put(k0 + h * 128 + side * 64, false, w[h]);
      }
    }
    if (lane == 0) bulk_wait();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  pair_sync();  // neither CTA ends while the other's copies or signals may still reach it
  if (warp == 0) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, 2 * kAccCols);
    else
      tmem_dealloc(tmem_base, 2 * kAccCols);
  }
}

// out[e] (+)= the sum of the expert's parts, for experts with several. blockIdx.y:
// expert. Four values a thread: a block takes 1024 and a thread sums its values' parts
// in order; or, of many parts, 128, whose parts the eight warps take in turn, and their
// sums are added in the warps' order (with the product, 129 parts of 64 x 64: 20.1 us in
// the first way, 12.3 in the second; 3 parts of 1024 x 1024: 72 and 82).
__global__ void __launch_bounds__(256) sum_parts_kernel(const DwArgs a) {
  __shared__ int before_s[8];
  __shared__ float4 sum_s[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  // The parts of the experts before this one, an expert a thread.
  static_assert(kMaxExperts == 256, "an expert a thread");
  int before = 0, bad = 0;
  if ((int)threadIdx.x < a.E) {
    bad = bad_at(a.offsets, threadIdx.x, a.R);
    if ((int)threadIdx.x < e)
      before = parts_of(a.offsets[threadIdx.x + 1] - a.offsets[threadIdx.x], a.part_rows);
  }
  before = __reduce_add_sync(kAll, before);
  if (lane == 0) before_s[warp] = before;
  const int n_parts = parts_of(a.offsets[e + 1] - a.offsets[e], a.part_rows);
  if (__syncthreads_or(bad) || n_parts <= 1) return;
  int p0 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) p0 += before_s[i];
  const long long n = (long long)a.N * a.K, i0 = (long long)blockIdx.x * a.sum_values;
  const float* parts = a.parts + (size_t)p0 * n;
  auto finish = [&](long long i, float4 s) {
    const size_t o = (size_t)e * n + i;
    if (a.out_fp32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o);
      if (a.accumulate) {
        const float4 x = *d;
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
      }
      *d = s;
    } else {
      uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o);
      if (a.accumulate) {
        const uint2 x = *d;
        s.x += from16(x.x & 0xFFFFu, a.fp16), s.y += from16(x.x >> 16, a.fp16);
        s.z += from16(x.y & 0xFFFFu, a.fp16), s.w += from16(x.y >> 16, a.fp16);
      }
      *d = make_uint2(pack16x2(s.x, s.y, a.fp16), pack16x2(s.z, s.w, a.fp16));
    }
  };
  auto sum = [&](long long i, int k0, int step) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = k0; k < n_parts; k += step) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(parts + (size_t)k * n + i));
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    return s;
  };
  if (a.sum_values == 1024) {
    const long long i = i0 + threadIdx.x * 4;
    if (i < n) finish(i, sum(i, 0, 1));
    return;
  }
  const long long i = i0 + lane * 4;
  sum_s[warp][lane] = i < n ? sum(i, warp, 8) : make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  if (warp == 0 && i < n) {
    float4 s = sum_s[0][lane];
    for (int k = 1; k < 8; ++k) {
      const float4 x = sum_s[k][lane];
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    finish(i, s);
  }
}

bool make_map(CUtensorMap* m, const void* base, int rows, int cols) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, kRows};
  return make_tensor_map_sw128(m, base, 2, dims, strides, box);
}

template <int BN, bool PAIR>
cudaError_t launch_tiles(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC,
                         const CUtensorMap& tmP, const DwArgs& a, long long items, int num_sms,
                         cudaStream_t st) {
  static DeviceFlags attr_done;
  if (cudaError_t e = smem_attr_once(attr_done, dw_kernel<BN, PAIR>, Ring<BN, PAIR>::kSmemBytes);
      e != cudaSuccess)
    return e;
  static std::atomic<int> resident[kMaxDevices];
  return launch_clusters(dw_kernel<BN, PAIR>, kCtas, resident, Ring<BN, PAIR>::kThreads,
                         Ring<BN, PAIR>::kSmemBytes, items, num_sms, st, tmA, tmB, tmC, tmP, a);
}

struct Split {
  int m_tiles, n_tiles, bn;
  bool pair;
  int part_rows;        // 0: whole segments
  long long max_parts;  // of all experts
};

// The tiles' width and the parts of long segments, by sizes alone: the choice of least
// estimated time.
//
// A row costs a tile 5.1 ns on its cluster at 256 columns (24576 rows x 2048 x 2048: 125
// us), 4.6 with MMAs over the pair (115) and 3.2 at 128 (32768 x 64 x 64 in one piece:
// 95); where x's rows are no whole number of 128-byte lines, each copy's row takes two for
// one, which is 7 ns (x 2040: 178 us), 4.6 (119) and 4 (32768 x 64 x 72: 132). A tile takes
// 0.3 us beside its rows, and the clusters take tiles in turn. Segments are
// taken to be of equal length, the longest of several half as long again. Cut into parts,
// the tiles are more, but the parts' fp32 results go to memory and back at 4 bytes a ps, and
// a second launch sums them. Parts need the narrow tiles, and fp32 results where segments
// have several slices.
//
// MMAs over the pair, each of whose CTAs loads only its half of x, against two (16-bit
// results; us):
//   several tiles a cluster, from 512 rows a segment on (128 experts x 1536 x 2048, even and
//   uneven: 256 rows 251 / 249 and 188 / 207, 512 rows 278 / 338 and 317 / 341, 640 rows 322
//   / 415 and 389 / 404, 768 rows 370 / 429 and 448 / 470); from 224 on where x's copies
//   touch two lines a row (x 1536 x 2040: 192 rows 260 / 260 and 237 / 258, 256 rows 265 /
//   271 and 284 / 302; 60 x 1000 x 1016, 250 rows: 52.5 / 53.2 and 54.0 / 60.7), from 384
//   where dy's do (x 1528 x 2048: 256 rows 246 / 257 and 222 / 243, 384 rows 272 / 297 and
//   297 / 299);
//   one tile a cluster, from 8192 on (2048 x 2048: 4096 rows 24.9 and 24.5); where x's copies
//   do, from 1024 (x 2040: 512 rows 10.6 and 10.4, 1024 rows 13.3 and 14.2), dy's 2048
//   (2040 x 2048: 1024 rows 13.2 and 12.4, 2048 rows 18.1 and 18.3, 4096 rows 25 and 29).
// Not inlined: the reported size and the launch have to come to the same choice.
__attribute__((noinline)) Split split_of(int R, int E, int N, int K, bool out_fp32) {
  Split best = {};
  double least = 0;
  const double rows = (double)R / E;
  const bool odd_k = K % 64 != 0, odd_n = N % 64 != 0;
  for (const int bn : {256, 128}) {
    if (bn == 256 && out_fp32 && rows > kSliceRows) continue;
    const int m = (N + 255) / 256, n = (K + bn - 1) / bn;
    const double tiles = (double)E * m * n;
    const bool pair =
        bn == 256 && !out_fp32 && rows >= (tiles > kPairs ? (odd_k ? 224 : odd_n ? 384 : 512)
                                                          : (odd_k ? 1024 : odd_n ? 2048 : 8192));
    const double row = bn == 128 ? (odd_k ? 4.0 : 3.2) : pair ? 4.6 : odd_k ? 7.0 : 5.1;
    for (int parts = 1; parts <= (bn == 128 && R > 512 ? 128 : 1); ++parts) {
      Split s = {m, n, bn, pair, 0, E};
      double t = std::ceil(tiles * parts / kPairs) * (rows / parts * row + 300);
      if (parts == 1) {
        if (E > 1 && tiles < 4 * kPairs) t += 0.5 * rows * row;
      } else {
        const double len = std::max(256.0, rows / parts);
        s.part_rows = ((int)len + kRows - 1) / kRows * kRows;
        s.max_parts = (long long)E + R / s.part_rows;
        if (s.max_parts >= 65536 || s.max_parts * m * n >= (1LL << 31)) break;
        t += s.max_parts * (double)N * K * 8 / 4000 + 3000;
      }
      if (best.bn == 0 || t < least) {
        best = s;
        least = t;
      }
      if (rows / parts < 256) break;
    }
  }
  return best;
}

// Whether the tiles' rows go to L2 ahead, a tile before the copies that read them. Under
// the stream of results first reads take long, and many tiles wait for the same ones: with
// 128 experts x 1536 x 2048, 256 rows each, 191 us and 188 with this (uneven 210 and 207;
// 2048 x 768: 103 and 101, 114 and 111), 180 rows 168 and 167 (180 and 175); 128 rows 151 and
// 154. Rows that are in L2 already are only read twice: below its size no gain. Nor with fp32
// results or for longer segments, which are bound by their MMAs (384 rows: 263 and 263).
bool ahead_of(const Split& s, int R, int E, int N, int K, bool out_fp32) {
  return s.bn == 256 && !s.pair && !out_fp32 && R >= 160LL * E && R <= 320LL * E &&
         2LL * R * (N + K) > 96LL << 20;
}

}  // namespace

long long grouped_product_dw_workspace(int R, int E, int N, int K, bool out_fp32) {
  const Split s = split_of(R, E, N, K, out_fp32);
  return s.part_rows == 0 ? 0 : s.max_parts * N * K * 4;
}

cudaError_t launch_grouped_product_dw(const void* dy, const void* x, const int32_t* offsets, int R,
                                      int E, int N, int K, bool fp16, void* out, bool out_fp32,
                                      bool accumulate, void* workspace, int num_sms,
                                      unsigned* err, cudaStream_t st) {
  const Split s = split_of(R, E, N, K, out_fp32);
  DwArgs a = {};
  a.offsets = offsets;
  a.out = out;
  a.parts = static_cast<float*>(workspace);
  a.err = err;
  a.E = E;
  a.R = R;
  a.N = N;
  a.K = K;
  a.m_tiles = s.m_tiles;
  a.n_tiles = s.n_tiles;
  a.part_rows = s.part_rows;
  a.ahead = ahead_of(s, R, E, N, K, out_fp32);
  a.sum_values = s.max_parts > 8LL * E ? 128 : 1024;
  a.fp16 = fp16;
  a.out_fp32 = out_fp32;
  a.accumulate = accumulate;
  CUtensorMap tmA, tmB, tmC, tmP;
  const int dt = out_fp32 ? MM_DTYPE_FP32 : fp16 ? MM_DTYPE_FP16 : MM_DTYPE_BF16;
  if (!make_map(&tmA, dy, R, N) || !make_map(&tmB, x, R, K) ||
      !make_tensor_map_rows(&tmC, out, dt, E, N, K, 32))
    return cudaErrorInvalidValue;
  tmP = tmC;
  if (s.part_rows != 0 &&
      !make_tensor_map_rows(&tmP, workspace, MM_DTYPE_FP32, (uint64_t)s.max_parts, N, K, 32))
    return cudaErrorInvalidValue;
  const long long items = s.max_parts * s.m_tiles * s.n_tiles;
  auto launch = s.bn == 128 ? launch_tiles<128, false>
                : s.pair    ? launch_tiles<256, true> : launch_tiles<256, false>;
  if (cudaError_t e = launch(tmA, tmB, tmC, tmP, a, items, num_sms, st);
      e != cudaSuccess || s.part_rows == 0)
    return e;
  const long long blocks = ((long long)N * K + a.sum_values - 1) / a.sum_values;
  return launch_k(sum_parts_kernel, dim3((unsigned)blocks, (unsigned)E), dim3(256), 0, st, true, a);
}

}  // namespace mm
