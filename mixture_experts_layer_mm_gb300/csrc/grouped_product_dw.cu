// The gradient of the experts' weights over ragged segments of rows:
//
//   dW[e] = sum over the rows r of expert e of dy[r] x[r]^T          [N, K]
//
// The reduction runs along the rows of both matrices, so both operands are
// MN-major: tiles of 64 rows x 64 columns (128 bytes a row, 128-byte swizzle) as
// they lie in memory, no transpose. A tile of the result is 256 features n x bn
// (256 or 128) features k, made by a cluster of two CTAs: each has 128 of the
// features n, its own accumulators and its own MMAs (M = 128), and each loads half of
// the other operand for both (TMA multicast), so that a stage brings 32 KB into an
// SM instead of 48.
//
// Why no MMA over the pair, as in grouped_product.cu: a segment of some 256 rows is
// four stages, 2000 cycles of MMAs, after which 64 KB leave each SM. Signals between
// the CTAs queue behind those stores (measured: 2.2 us from the last MMA to the
// pair's completion signal, 1.6 us back from the epilogue), and with two accumulators
// that was what 32768 rows x 128 experts x 1536 x 2048 waited for: 237 us. Here
// the accumulators' signals stay within a CTA; only the ring's slots, which are
// filled ahead, are handed over between the two.
//
// Rows beyond a segment belong to another expert: the last stage is cut to whole
// steps of 16 rows, and where those hold rows of the next segment the issuing
// warp writes zeros over them, in both operands (0 times another expert's infinity is
// NaN). Columns beyond a matrix are zeros out of the copy. The results leave
// through shared memory as boxes of 32 rows x 128 bytes, which the copy cuts at the
// matrix's edges (stores out of registers, 32 bytes a lane in 32 rows: 302 us where
// boxes took 273).
//
// fp32 results (and parts) take kSliceRows rows of a segment at a time, each slice
// added to memory in fp32: the tensor cores cut what they add, and 512 rows leave 5e-7
// of it where 4096 leave 4e-6. 16-bit results are one accumulation.
//
// Few tiles with long reductions are cut into parts of `part_rows` rows, whose fp32 results go
// to the workspace and are summed in order by a second launch (the rule is at
// split_of).
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
constexpr int kRows = 64;                    // rows of the reduction a stage
constexpr int kBlock = kRows * 128;          // 8 KB: 64 rows x 64 columns
constexpr int kStages = 4;
constexpr int kABytes = 2 * kBlock;          // this CTA's 128 features n
constexpr int kStageBytes = kABytes + 4 * kBlock;  // and up to 256 features k
constexpr int kEpiWarp0 = 1, kEpiWarps = 8;
constexpr int kProd0 = kEpiWarp0 + kEpiWarps;      // producers: one warp a slot
constexpr int kThreads = (kProd0 + kStages) * 32;  // 416
constexpr int kStore = 32 * 128;             // 4 KB a warp: results on their way out
constexpr int kSmemBytes = kStages * kStageBytes + kEpiWarps * kStore + 1024;
constexpr int kStaticBytes = 2000;           // at most: barriers, offsets, parts
static_assert(kSmemBytes <= 227 * 1024 - kStaticBytes, "shared memory");
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
  int m_tiles, n_tiles, bn;
  int part_rows;           // 0: segments are whole
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

// tmC: the result, tmP: the parts.
__global__ void __launch_bounds__(kThreads, 1)
    dw_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmP,
              const DwArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s, bad_s;
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
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), kCtas);  // every CTA's MMAs: its copies fill all
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), kEpiWarps);
    }
    mbar_init(smem_u32(done), 1);
    abort_s = 0;
    bad_s = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_base_s), 2 * kAccCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i <= E; i += kThreads) off_s[i] = a.offsets[i];
  __syncthreads();
  // Bad offsets are refused as a whole: nothing is written.
  for (int e = tid; e < E; e += kThreads)
    if (bad_at(off_s, e, a.R)) bad_s = 1;
  __syncthreads();
  const bool bad = bad_s != 0;
  if (bad && tid == 0 && blockIdx.x == 0) atomicOr(a.err, kDevErrBadIds);
  if (warp == 0 && a.part_rows != 0 && !bad) scan_parts(off_s, E, a.part_rows, first_s);
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers are initialised
  tc_fence_after();
  const int per = a.m_tiles * a.n_tiles;
  const int total = bad ? 0 : (a.part_rows != 0 ? (int)first_s[E] : E) * per;
  const uint32_t tmem_base = tmem_base_s;
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
      t.row0 = off_s[p];
      t.rows = off_s[p + 1] - t.row0;
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
      t.e = lo;
      const int at = (p - first_s[lo]) * a.part_rows;
      t.row0 = off_s[lo] + at;
      t.rows = min(a.part_rows, off_s[lo + 1] - t.row0);
      t.part = first_s[lo + 1] - first_s[lo] > 1 ? p : -1;
    }
    return t;
  };
  // Slices of an item's reduction, and the rows of one.
  auto slice_rows = [&](const Item& t) { return a.out_fp32 || t.part >= 0 ? kSliceRows : 1 << 30; };
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
    const uint32_t fb = smem_u32(&full[slot]), eb = smem_u32(&empty[slot]);
    const uint64_t pol = l2_policy_evict_last();  // read by every tile of the expert
    const int boxes = a.bn / 64;                  // of 64 columns, loaded by the CTAs in turn
    const uint32_t bytes = kABytes + boxes * kBlock;
    uint32_t use = 0;  // fills of this slot so far
    int q = 0;  // stage counter modulo the ring
    bool ok = true;
    for (int i = pair; i < total && ok; i += npairs) {
      if (aborted()) break;
      const Item t = item_at(i);
      const int nsl = slices(t), step = slice_rows(t);
      const int f = (t.m * kCtas + (int)rank) * 128, c = t.n * a.bn;
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
          if (leader) {
            const int r = t.row0 + sl * step + kb * kRows;
            mbar_arrive_expect_tx(fb, bytes);
            tma_load_2d(st, &tmA, fb, f, r, pol);
            tma_load_2d(st + kBlock, &tmA, fb, f + 64, r, pol);
            for (int b = rank; b < boxes; b += kCtas)
              tma_load_2d_all(st + kABytes + b * kBlock, &tmB, fb, c + 64 * b, r, all, pol);
          }
          __syncwarp();
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
    // ------------------------------------------------------ MMA issuer ---
    // The whole warp runs the loops, so that descriptors stay in uniform
    // registers; one elected lane issues.
    const bool leader = elect_one();
    const uint32_t idesc = idesc_16(a.fp16 != 0, true, true) | idesc_shape(128, a.bn);
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
        if (!warp_wait(smem_u32(&tempty[b]), (use & 1u) ^ 1u)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + b * kAccCols;
        for (int kb = 0; kb < nk; ++kb) {
          if (!warp_wait(smem_u32(&full[s]), ph)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t st = smem_base + s * kStageBytes;
          const int left = len - kb * kRows;  // rows of this stage, if fewer than 64
          if (left < kRows && (left & 15) != 0) {
            // Rows [left, next multiple of 16) of every block: 128 bytes each. (The MMAs
            // of the stages before run meanwhile. Straight-line code: in loops it took the
            // warp 900 cycles, 14 us of 224 for 32768 rows of uneven load.)
            const uint32_t z = st + (left + (lane >> 3)) * 128 + (lane & 7) * 16;
#pragma unroll
            for (int j = 0; j < 4; ++j)  // four rows at a time
              if ((left & 15) + (lane >> 3) + 4 * j < 16) {
#pragma unroll
                for (int k = 0; k < 6; ++k)
                  if (k < 4 || a.bn == 256) st_shared_zero16(z + k * kBlock + j * 512);
              }
            __syncwarp();
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          if (leader) {
            const uint64_t da = sdesc_mnmajor(st, kBlock), db = sdesc_mnmajor(st + kABytes, kBlock);
            const int steps = min(4, (len - kb * kRows + 15) / 16);
            // 16 rows are 128 descriptor units of 16 bytes.
            if (steps == 4) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16(d, da + kk * 128, db + kk * 128, idesc, (kb | kk) != 0);
            } else {
              for (int kk = 0; kk < steps; ++kk)
                umma_bf16(d, da + kk * 128, db + kk * 128, idesc, (kb | kk) != 0);
            }
            umma_commit_all(smem_u32(&empty[s]), all);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        if (leader) umma_commit(smem_u32(&tfull[b]));
        __syncwarp();
      }
    }
    // Every MMA issued above has finished before tensor memory is freed.
    if (leader) umma_commit(smem_u32(done));
    __syncwarp();
    if (!warp_wait(smem_u32(done), 0)) fail();
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
      const int k0 = t.n * a.bn, k1 = min(k0 + a.bn, a.K);
      const bool fp32 = a.out_fp32 || t.part >= 0;
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
          if (t.part >= 0) {
            if (add)
              tma_add_3d(&tmP, buf, c, f0, t.part);
            else
              tma_store_3d(&tmP, buf, c, f0, t.part);
          } else if (add) {
            tma_add_3d(&tmC, buf, c, f0, t.e);
          } else {
            tma_store_3d(&tmC, buf, c, f0, t.e);
          }
          bulk_commit();
        }
        __syncwarp();
      };
      if (nsl == 0 && !a.accumulate) {  // an expert without rows
        const uint32_t zero[32] = {};
        for (int c = side * (fp32 ? 32 : 64); c < a.bn; c += fp32 ? 64 : 128)
          put(k0 + c, false, zero);
      }
      for (int sl = 0; sl < nsl; ++sl, ++it) {
        const uint32_t b = it & 1u, use = it >> 1;
        if (!warp_wait(smem_u32(&tfull[b]), use & 1u)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + b * kAccCols;
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&tempty[b]));
          __syncwarp();
        };
        if (fp32) {
          const bool add = sl > 0 || (a.accumulate && t.part < 0);
          // A slice is added to the ones before it once they are in memory.
          if (sl > 0 && lane == 0) bulk_wait();
          __syncwarp();
          for (int c = side * 32; c < a.bn; c += 64) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tb + c, v);
            tmem_wait_ld();
            if (c + 64 >= a.bn) release();
            put(k0 + c, add, v);
          }
        } else if (a.accumulate) {
          for (int c = side * 32; c < a.bn; c += 64) {
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
          // Two boxes of 64 columns (one, if bn is 128): the accumulator is free again
          // once they are in registers, before they are written.
          uint32_t w[2][32];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int c = (h >> 1) * 128 + side * 64 + (h & 1) * 32;
            if (c < a.bn) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(tb + c, v);
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
          }
          release();
          put(k0 + side * 64, false, w[0]);
          if (a.bn == 256) put(k0 + 128 + side * 64, false, w[1]);
        }
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
    tmem_dealloc(tmem_base, 2 * kAccCols);
  }
}

// out[e] (+)= the sum of the expert's parts, in order, for experts with several.
// blockIdx.y: expert; 8 values a thread.
__global__ void __launch_bounds__(256) sum_parts_kernel(const DwArgs a) {
  __shared__ int32_t off_s[kMaxExperts + 1];
  __shared__ uint16_t first_s[kMaxExperts + 1];
  __shared__ int bad_s;
  if (threadIdx.x == 0) bad_s = 0;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i <= a.E; i += 256) off_s[i] = a.offsets[i];
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 256)
    if (bad_at(off_s, e, a.R)) bad_s = 1;
  __syncthreads();
  if (bad_s) return;
  if (threadIdx.x < 32) scan_parts(off_s, a.E, a.part_rows, first_s);
  __syncthreads();
  const int e = blockIdx.y, p0 = first_s[e], p1 = first_s[e + 1];
  const long long n = (long long)a.N * a.K, i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
  if (p1 - p0 <= 1 || i >= n) return;
  float s[8] = {};
  const size_t o = (size_t)e * n + i;
  if (a.accumulate) {
    if (a.out_fp32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.out) + o);
      const float4 x = p[0], y = p[1];
      s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w, s[4] = y.x, s[5] = y.y, s[6] = y.z, s[7] = y.w;
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.out) + o);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[2 * j] = from16(w[j] & 0xFFFFu, a.fp16);
        s[2 * j + 1] = from16(w[j] >> 16, a.fp16);
      }
    }
  }
  const float* p = a.parts + (size_t)p0 * n + i;
#pragma unroll 4
  for (int k = p0; k < p1; ++k, p += n) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 y = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
    s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
  }
  if (a.out_fp32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o);
    d[0] = make_float4(s[0], s[1], s[2], s[3]);
    d[1] = make_float4(s[4], s[5], s[6], s[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o) =
        make_uint4(pack16x2(s[0], s[1], a.fp16), pack16x2(s[2], s[3], a.fp16),
                   pack16x2(s[4], s[5], a.fp16), pack16x2(s[6], s[7], a.fp16));
  }
}

bool make_map(CUtensorMap* m, const void* base, int rows, int cols) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, kRows};
  return make_tensor_map_sw128(m, base, 2, dims, strides, box);
}

struct Split {
  int m_tiles, n_tiles, bn;
  int part_rows;        // 0: whole segments
  long long max_parts;  // of all experts
};

// The tiles' width and the parts of long segments, by sizes alone.
//
// bn: 256, whose stages carry more MMAs for their bytes; 128 where that leaves less of
// a tile empty (up to 384 columns) or where the tiles of 256 fill less than half of the
// chip.
//
// Parts: a row costs a tile 4 (bn = 128: 2) ns on its cluster. Whole segments take the
// rows of the longest (1.5 times the mean, say) as often as the clusters go round; in
// parts, about two a cluster, the rows are spread over all of them, but the parts' fp32
// results go to memory and back at 4 bytes a ps and a second launch adds them up.
Split split_of(int R, int E, int N, int K) {
  Split s;
  s.m_tiles = (N + 255) / 256;
  const bool narrow = K <= 128 || (K > 256 && K <= 384) ||
                      (long long)E * s.m_tiles * ((K + 255) / 256) < kPairs / 2;
  s.bn = narrow ? 128 : 256;
  s.n_tiles = (K + s.bn - 1) / s.bn;
  const double per = (double)s.m_tiles * s.n_tiles, row = s.bn == 128 ? 2 : 4;
  const double rounds = std::max(1.0, E * per / kPairs);
  const double whole = rounds * 1.5 * R / E * row;
  const double want = std::max(256.0, R * per / (2 * kPairs));
  s.part_rows = 0;
  s.max_parts = E;
  if (want < R) {
    const int rows = ((int)want + kRows - 1) / kRows * kRows;
    const long long parts = (long long)E + R / rows;
    const double cut = R * per / kPairs * row + parts * (double)N * K * 8 / 4000 + 3000;
    if (cut < whole && parts < 65536 && parts * (long long)per < (1LL << 31)) {
      s.part_rows = rows;
      s.max_parts = parts;
    }
  }
  return s;
}

}  // namespace

long long grouped_product_dw_workspace(int R, int E, int N, int K) {
  const Split s = split_of(R, E, N, K);
  return s.part_rows == 0 ? 0 : s.max_parts * N * K * 4;
}

cudaError_t launch_grouped_product_dw(const void* dy, const void* x, const int32_t* offsets, int R,
                                      int E, int N, int K, bool fp16, void* out, bool out_fp32,
                                      bool accumulate, void* workspace, int num_sms,
                                      unsigned* err, cudaStream_t st) {
  const Split s = split_of(R, E, N, K);
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
  a.bn = s.bn;
  a.part_rows = s.part_rows;
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
  static DeviceFlags attr_done;
  if (cudaError_t e = smem_attr_once(attr_done, dw_kernel, kSmemBytes); e != cudaSuccess) return e;
  static std::atomic<int> resident[kMaxDevices];
  const long long items = s.max_parts * s.m_tiles * s.n_tiles;
  if (cudaError_t e = launch_clusters(dw_kernel, kCtas, resident, kThreads,
                                      kSmemBytes, items, num_sms, st, tmA, tmB, tmC, tmP, a);
      e != cudaSuccess || s.part_rows == 0)
    return e;
  const long long blocks = ((long long)N * K / 8 + 255) / 256;
  return launch_k(sum_parts_kernel, dim3((unsigned)blocks, (unsigned)E), dim3(256), 0, st, true, a);
}

}  // namespace mm
