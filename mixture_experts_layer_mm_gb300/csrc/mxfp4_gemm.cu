// Products of microscaled 4-bit matrices on the sm_103a tensor cores
// (tcgen05.mma kind::mxf4 with block scales, accumulators in tensor memory,
// operands staged by TMA). One kernel, three epilogues:
//
//   dense    C[r, n] = x_r . w_n                       (bf16 or fp32)
//   gate_up  act[r, i] = Q(silu(g) u), g = x_r . w_i (gate), u = x_r . w_i (up)
//            for the rows r of every expert's segment; Q: 4-bit blocks along i
//   down     y[r, h] = x_r . w_h (fp32)
//
// Orientation as in gemm.cu: the weight rows are the MMA's M side (128 rows
// an MMA), the token rows its N side (any multiple of 16 up to 128). A tile
// is (chunk of up to 128 rows of one segment, m-tile); a stage holds 256
// columns of two 128-row weight tiles (A0, A1) and of the chunk's rows (B),
// 128 bytes a row, plus their scale tiles. Segments begin at multiples of 128
// rows, so a chunk's scale bytes are whole tiles.
//
// The products of two e2m1 values and two powers of two are exact; the
// accumulation is in fp32 in tensor memory.
//
// gate_up's blocks run along the output columns, which are the lanes of tensor
// memory. The weight tile's rows are loaded in an order (row 4 a
// + j of a group of 32 at place 8 j + a) that gives a thread of a 16 x 256-bit
// tensor-memory load four consecutive columns of a token row: a block's maximum
// is three maxima in the thread and three exchanges for two rows at once, and
// results leave the thread as they are. (For gate_up at 4096 tokens a warp
// reduction for every column took 90 us, a transpose through shared memory, whose
// bandwidth the MMAs need, 63; this 62.) The activation is quantised from the fp32
// product and is rounded once; y stays fp32 (70 us for down, 268 MB of y).
//
// What bounds it, on one GB300: 8192 x 4096 x 4096 takes 56 us (4.9 PFLOP/s).
// One stage of a tile alone on the chip takes 580 cycles, its 8 MMAs and 8
// scale copies the tensor pipe's 576; with all SMs at work 640, as the 52 KB of
// a stage come at 80 bytes a cycle and SM, 14 TB/s out of L2. Few tiles (64 x
// 4096 x 4096, 6.8 us on 32 of the SMs) take in 416 KB a tile at some 90 bytes a
// cycle, 2.5 us; the launch, the prologue and the epilogue are the rest. Few rows
// per expert (64 tokens) are bound by the weights' bytes.
#include <algorithm>

#include "mm.h"
#include "mm_internal.h"
#include "mx_device.cuh"

namespace mm {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kBN = 128;   // token rows per chunk
constexpr int kStageK = 256;                // columns per stage (128 bytes a row)
constexpr int kTileBytes = 128 * 128;       // 128 rows of one stage
constexpr int kScaleStage = 2 * kMxTileBytes;  // scale bytes of 128 rows of one stage

// The ring of stages: NA weight tiles and the token rows a slot, then the scales
// of each. A ring of one weight tile a slot holds six.
template <int NA>
struct Ring {
  static constexpr int kStages = NA == 1 ? 6 : 4;
  static constexpr int kRowsAt = NA * kTileBytes;
  static constexpr int kScalesAt = kRowsAt + kTileBytes;
  static constexpr int kStride = (kScalesAt + (NA + 1) * kScaleStage + 1023) / 1024 * 1024;
  static constexpr int kSmemBytes = kStages * kStride + 1024;
  static_assert(kSmemBytes <= 227 * 1024 - 4096, "shared memory");
};

// Warp roles: 0, 1 = MMA issuers (D0, D1), 2-17 = epilogue, 18, 19 = producers
// (every other ring slot). There is one pair of accumulators (the scales take
// the columns a second pair would need), so the epilogue first empties tensor
// memory into registers, 16 warps with a 32 x 32 piece of D0 and of D1 each,
// hands it back to the MMA warps and then does its work.
constexpr int kEpiWarp0 = 2, kEpiWarps = 16;
constexpr int kProdWarp0 = kEpiWarp0 + kEpiWarps;
constexpr int kProdWarps = 2;
constexpr int kThreads = (kProdWarp0 + kProdWarps) * 32;  // 640: 96 registers a thread

// Tensor memory: D0 and D1 (128 columns each), then per ring slot and
// accumulator the scale columns of the slot's two halves of K: weights, token
// rows, 4 columns each (each issuer brings the token rows' own copy, so that
// neither depends on the other's order).
constexpr uint32_t kScaleCol0 = 2 * kBN, kScaleCols = 32;
constexpr uint32_t kTmemCols = 512;
static_assert(kScaleCol0 + Ring<1>::kStages * kScaleCols <= kTmemCols, "tensor memory");
static_assert(kScaleCol0 + Ring<2>::kStages * kScaleCols <= kTmemCols, "tensor memory");

enum { kDense = 0, kGateUp = 1, kDown = 2 };

struct MxGemmArgs {
  const int32_t* counts;   // [E] rows of each segment (NULL: `rows` each)
  const int32_t* ids;      // [n_ids] the slots' experts instead of counts (small batches)
  int n_ids, top_k;
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  void* out;               // dense: C; gate_up: act codes; down: y
  uint8_t* act_scales;     // gate_up: scales of act
  unsigned* err;
  int E, rows;    // rows: of the one segment of a dense product (else 0)
  int N, K;       // output columns (gate_up: intermediates), reduction
  int n_mtiles;
  int out_fp32;   // dense
};

// Whether a warp of this CTA gave up a wait (asked by a converged warp).
__device__ __forceinline__ bool stopped(const int* flag) {
  return __any_sync(kAll, *reinterpret_cast<const volatile int*>(flag) != 0);
}

__device__ __forceinline__ void stop(int* flag, unsigned* err) {
  *reinterpret_cast<volatile int*>(flag) = 1;
  atomicOr(err, kDevErrTimeout);
}

struct Tile {
  int e, m, row0, nrows;
};

// Exclusive sums of the segments' chunks, by one warp: lane l takes the experts
// from 8 l on (at most 256 in all). first[E] is the total; each count is
// replaced by the row behind the segment's last. lead (or NULL): what leads from
// a segment's rows to its rows of y, which lie without gaps between segments.
__device__ __forceinline__ void scan_chunks(int* cnt, int E, int* first, int* lead) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kMaxExperts / 32;
  int c[kPer], sum = 0, rows = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    c[i] = e < E ? (cnt[e] + kBN - 1) / kBN : 0;
    sum += c[i];
    rows += e < E ? cnt[e] : 0;
  }
  if (lead != nullptr) rows = exclusive_sum(rows);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += v;
  }
  int run = incl - sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    if (e < E) {
      if (lead != nullptr) {
        lead[e] = rows - run * kBN;
        rows += cnt[e];
      }
      first[e] = run;
      cnt[e] += run * kBN;
    }
    run += c[i];
  }
  if (lane == 31) first[E] = incl;
}

// The tiles of a CTA: blockIdx.x, then every gridDim.x-th, m-tiles within chunks.
// Chunks of a segment follow one another, and segments begin at whole chunks:
// chunk ch of the table is rows [128 ch, 128 ch + 128) of the token matrix. Every
// warp walks on its own; a step finds the chunk's expert from the last one on.
struct Walk {
  Tile t;
  int ch, dch, dm;

  __device__ __forceinline__ Walk(int n_mtiles, int E, const int* first, const int* end) {
    ch = blockIdx.x / n_mtiles;
    t.m = blockIdx.x - ch * n_mtiles;
    dch = gridDim.x / n_mtiles;
    dm = gridDim.x - dch * n_mtiles;
    t.e = 0;
    find(E, first, end);
  }
  __device__ __forceinline__ void step(int n_mtiles, int E, const int* first, const int* end) {
    ch += dch;
    t.m += dm;
    if (t.m >= n_mtiles) {
      t.m -= n_mtiles;
      ++ch;
    }
    find(E, first, end);
  }

 private:
  // The last expert whose first chunk is at or before ch (first is ascending).
  __device__ __forceinline__ void find(int E, const int* first, const int* end) {
    const int lane = threadIdx.x & 31;
    int e = t.e;
    while (true) {
      const int i = e + 1 + lane;
      const int n = __popc(__ballot_sync(kAll, i < E && first[i] <= ch));
      e += n;
      if (n < 32) break;
    }
    t.e = uniform(e);
    t.row0 = ch * kBN;
    t.nrows = min(kBN, uniform(end[t.e]) - t.row0);
  }
};

// The first two m-tile halves of a tile in the weight matrices: 128-row tile
// index (also of the scales) and code row of A0; A1 exists if has1.
struct WeightAt {
  int row0, row1;
  long long st0, st1;  // scale tile rows
  bool has1;
};

template <int MODE, int NA>
__device__ __forceinline__ WeightAt weights_of(const MxGemmArgs& a, const Tile& t) {
  WeightAt w;
  const int tiles = (a.N + 127) / 128;  // scale tile rows per weight matrix
  if (MODE == kGateUp) {  // two matrices per expert: gate, up
    w.row0 = 2 * t.e * a.N + t.m * 128;
    w.row1 = w.row0 + a.N;
    w.st0 = (long long)(2 * t.e) * tiles + t.m;
    w.st1 = w.st0 + tiles;
    w.has1 = true;
  } else {
    const int m = NA * t.m;
    w.row0 = t.e * a.N + m * 128;
    w.row1 = w.row0 + 128;
    w.st0 = (long long)t.e * tiles + m;
    w.st1 = w.st0 + 1;
    w.has1 = NA == 2 && m + 1 < tiles;
  }
  return w;
}

// What one thread of an epilogue warp holds of a 32 x 32 piece of an
// accumulator: output columns col + j (j < 4, consecutive thanks to the row
// order of the weight tile) of token rows row(g, c) = 8 g + 2 (lane % 4) + c.
struct Piece {
  uint32_t r[2][16];
  __device__ __forceinline__ float at(int j, int g, int c) const {
    return __uint_as_float(r[j >> 1][4 * g + 2 * (j & 1) + c]);
  }
  __device__ __forceinline__ Pair rows(int j, int g) const { return {at(j, g, 0), at(j, g, 1)}; }
  __device__ __forceinline__ void set(int j, int g, Pair v) {
    r[j >> 1][4 * g + 2 * (j & 1)] = __float_as_uint(v.x);
    r[j >> 1][4 * g + 2 * (j & 1) + 1] = __float_as_uint(v.y);
  }
};

__device__ __forceinline__ void load_piece(uint32_t taddr, Piece& p) {
  tmem_ld_16x256b_x4(taddr, p.r[0]);                // lanes 0-15 of the quarter
  tmem_ld_16x256b_x4(taddr + (16u << 16), p.r[1]);  // lanes 16-31
}

// Block exponents. A block is a token row of the piece, its 32 columns spread
// over the 8 lanes of one lane % 4. Each thread takes the largest magnitude of
// its 4 columns; the upper halves of two rows (c = 0, 1) go into one word, which
// orders them by exponent (255: an infinity or a NaN). The exchanges fold as
// they reduce: at each step a lane keeps half of its words and gives the other
// half away, so that lane 8 g + i ends with the two rows of word g, and the
// factors come back by one shuffle a word.
__device__ __forceinline__ void local_max(const Piece& p, uint32_t (&w)[4]) {
#pragma unroll
  for (int g = 0; g < 4; ++g)
    w[g] = __byte_perm(
        __float_as_uint(max_abs4(p.at(0, g, 0), p.at(1, g, 0), p.at(2, g, 0), p.at(3, g, 0))),
        __float_as_uint(max_abs4(p.at(0, g, 1), p.at(1, g, 1), p.at(2, g, 1), p.at(3, g, 1))),
        0x7632);  // upper halves, signs are 0
}

// Keeps `mine` of two words, gives the other to lane ^ o, takes the maximum.
__device__ __forceinline__ uint32_t fold(uint32_t low, uint32_t high, int o) {
  const bool up = threadIdx.x & o;
  return __vmaxu2(up ? high : low, __shfl_xor_sync(kAll, up ? low : high, o));
}

__device__ __forceinline__ uint32_t exponents(uint32_t w) { return (w >> 7) & 0x00FF00FFu; }

// mx_scale_byte of two exponents, and f with mx_inv_scale = 2^(f - 127) (0 for f = 0).
__device__ __forceinline__ uint32_t scale_pair(uint32_t e, uint32_t& f) {
  uint32_t s = __vmaxu2(e, 0x00020002u) - 0x00020002u;
  f = 0x00FE00FEu - s;
  const uint32_t bad = (e + 0x00010001u) & 0x01000100u;  // exponents of 255
  s += bad >> 7;                                          // 253 -> 255
  if (bad & 0xFFFFu) f &= 0xFFFF0000u;
  if (bad >> 16) f &= 0xFFFFu;
  return s;
}

// 2^(f - 127) of the two halves of a word, 0 for f = 0.
__device__ __forceinline__ Pair factors(uint32_t f) {
  return {__uint_as_float(f << 23), __uint_as_float((f << 7) & 0xFF800000u)};
}

// Issues one stage of one accumulator: the scale tiles of its `steps` / 2
// halves (weights, token rows) to tensor memory, then `steps` MMAs of K = 64.
// One thread. a_tile 0 or 1: A0 into D0, A1 into D1.
template <int NA>
__device__ __forceinline__ void issue_stage(uint32_t st, int a_tile, uint32_t tsc, uint32_t d,
                                            uint32_t idesc, bool accumulate, int steps) {
  const uint64_t da = sdesc_kmajor<128>(st + a_tile * kTileBytes);
  const uint64_t db = sdesc_kmajor<128>(st + Ring<NA>::kRowsAt);
  const uint64_t sa = sdesc_scales(st + Ring<NA>::kScalesAt + a_tile * kScaleStage);
  const uint64_t sb = sdesc_scales(st + Ring<NA>::kScalesAt + NA * kScaleStage);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (2 * h >= steps) break;
    // Descriptor addresses count 16-byte units.
    tmem_cp_scales(tsc + h * 8, sa + h * (kMxTileBytes / 16));
    tmem_cp_scales(tsc + h * 8 + 4, sb + h * (kMxTileBytes / 16));
  }
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    if (kk >= steps) break;
    const uint32_t col = tsc + (kk >> 1) * 8;
    umma_mxf4(d, da + kk * 2, db + kk * 2, idesc | idesc_mxf4_pair((kk & 1) * 2), col, col + 4,
              accumulate || kk != 0);
  }
}

// NA: weight tiles of 128 rows a tile (1: dense only).
template <int MODE, bool PERM, int NA>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
                   const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmX32,
                   const MxGemmArgs a) {
  static_assert(PERM || MODE == kDense, "blocks along the output columns need the row order");
  static_assert(NA == 2 || MODE == kDense, "the experts' epilogues take pairs");
  using R = Ring<NA>;
  constexpr int kStages = R::kStages, kStageStride = R::kStride;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 3];
  __shared__ uint32_t tmem_base_s;
  __shared__ int stop_s;
  __shared__ int cnt_s[kMaxExperts], first_s[kMaxExperts + 1];
  __shared__ int lead_s[MODE == kDown ? kMaxExperts : 1];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.E;
  uint64_t* full = bars;
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 1;
  uint64_t* done = tempty + 1;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), NA);  // one commit of each issuer that reads it
    }
    mbar_init(smem_u32(tfull), 2);
    mbar_init(smem_u32(tempty), kEpiWarps);
    mbar_init(smem_u32(done), 2);
    stop_s = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tmW);
    if (PERM) tma_prefetch_desc(&tmS);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmX32);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_s), kTmemCols);
    tmem_relinquish();
  }
  // With the slots' ids at hand (a small batch) the segments are counted here,
  // while the kernels before this one still run, and the first weights are
  // fetched; only the token rows wait for those kernels.
  const bool early = a.ids != nullptr;
  for (int i = tid; i < E; i += kThreads) cnt_s[i] = a.rows;
  if (early) {
    __syncthreads();
    for (int i = tid; i < a.n_ids; i += kThreads) {
      const int id = __ldg(a.ids + i);
      bool drop = id < 0 || id >= E;
      for (int j = i / a.top_k * a.top_k; j < i; ++j) drop |= __ldg(a.ids + j) == id;
      if (!drop) atomicAdd(&cnt_s[id], 1);
    }
  } else {
    pdl_wait();
    if (a.counts != nullptr)
      for (int i = tid; i < E; i += kThreads) cnt_s[i] = a.counts[i];
  }
  pdl_trigger();
  __syncthreads();
  // cnt_s: from here on the segments' ends
  if (warp == 0) scan_chunks(cnt_s, E, first_s, MODE == kDown ? lead_s : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int total = uniform(first_s[E]) * a.n_mtiles;
  if ((int)blockIdx.x >= total) {  // uniform across the CTA
    if (warp == 1) tmem_dealloc(tmem_base_s, kTmemCols);
    if (early) pdl_wait();  // this kernel's end must mean the end of those before it
    return;
  }

  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // All 512 columns are this CTA's, so they begin at column 0: a constant in
  // the MMA's operands. (Were it ever otherwise, nothing below would run.)
  constexpr uint32_t tmem_base = 0;
  if (tmem_base_s != tmem_base) {
    if (tid == 0) atomicOr(a.err, kDevErrTimeout);
    if (warp == 1) tmem_dealloc(tmem_base_s, kTmemCols);
    if (early) pdl_wait();
    return;
  }
  const int k_tiles = (a.K + 127) / 128;         // scale tiles per row
  const int nk = (a.K + kStageK - 1) / kStageK;  // stages per tile

  if (warp >= kProdWarp0) {
    // ---------------------------------------------------- producers (18, 19) ---
    // Warp 18 + p fills slots p and p + 2: filling one takes a thread some 400
    // cycles. As in the MMA warps, all lanes run the loop and one issues.
    const int first = warp - kProdWarp0;
    const bool leader = elect_one();
    const uint64_t pol_w = l2_policy_evict_normal();
    const uint64_t pol_x = l2_policy_evict_last();
    const uint32_t row_bytes = kStageK / 2;
    // Weights of stage kb into a slot, and the bytes they will count.
    auto weight_bytes = [&](const WeightAt& w, int kb) {
      const uint32_t sb = PERM ? kScaleStage  // a box is always whole
                               : min(2, k_tiles - 2 * kb) * kMxTileBytes;
      return (w.has1 ? 2u : 1u) * (kTileBytes + sb);
    };
    auto load_weights = [&](const WeightAt& w, int kb, uint32_t st, uint32_t fb) {
      const uint32_t sc = st + R::kScalesAt;
      const int kt = 2 * kb;  // first scale tile of the stage
      if (PERM) {
        tma_load_4d(st, &tmW, fb, kb * row_bytes, w.row0 / 32, pol_w);
        tma_load_4d(sc, &tmS, fb, 0, (int)(w.st0 * k_tiles) + kt, pol_w);
        if (w.has1) {
          tma_load_4d(st + kTileBytes, &tmW, fb, kb * row_bytes, w.row1 / 32, pol_w);
          tma_load_4d(sc + kScaleStage, &tmS, fb, 0, (int)(w.st1 * k_tiles) + kt, pol_w);
        }
      } else {
        const uint32_t sb = min(2, k_tiles - kt) * kMxTileBytes;
        tma_load_2d(st, &tmW, fb, kb * row_bytes, w.row0, pol_w);
        bulk_load(sc, a.w_scales + (w.st0 * k_tiles + kt) * kMxTileBytes, sb, fb);
        if (w.has1) {
          tma_load_2d(st + kTileBytes, &tmW, fb, kb * row_bytes, w.row1, pol_w);
          bulk_load(sc + kScaleStage, a.w_scales + (w.st1 * k_tiles + kt) * kMxTileBytes, sb, fb);
        }
      }
    };
    // Token rows of a stage: one box of 128, or up to three boxes of 32. Behind
    // the last rows of a dense product a box reads nothing (zeros), so there the
    // one box is always the cheaper (64 rows in two boxes: 7.9 us, in one: 6.9).
    auto row_boxes = [](const Tile& t) {
      return MODE == kDense || t.nrows > 96 ? 4 : (t.nrows + 31) / 32;
    };
    auto stage_bytes = [&](const Tile& t, const WeightAt& w, int kb) {
      return weight_bytes(w, kb) + (uint32_t)row_boxes(t) * 4096u +
             (uint32_t)min(2, k_tiles - 2 * kb) * kMxTileBytes;
    };
    auto load_rows = [&](const Tile& t, int kb, uint32_t st, uint32_t fb) {
      const int nbox = row_boxes(t), kt = 2 * kb;
      if (nbox == 4) {
        tma_load_2d(st + R::kRowsAt, &tmX, fb, kb * row_bytes, t.row0, pol_x);
      } else {
        for (int b = 0; b < nbox; ++b)
          tma_load_2d(st + R::kRowsAt + b * 4096, &tmX32, fb, kb * row_bytes, t.row0 + 32 * b,
                      pol_x);
      }
      bulk_load(st + R::kScalesAt + NA * kScaleStage,
                a.x_scales + ((long long)(t.row0 / 128) * k_tiles + kt) * kMxTileBytes,
                min(2, k_tiles - kt) * kMxTileBytes, fb);
    };
    Walk walk(a.n_mtiles, E, first_s, cnt_s);
    int fetched = 0;  // stages of the first tile whose weights are already on their way
    if (early) {
      const Tile& t = walk.t;
      const WeightAt w = weights_of<MODE, NA>(a, t);
      fetched = min(nk, kStages);
      if (leader) {
        for (int kb = first; kb < fetched; kb += kProdWarps) {
          const uint32_t fb = smem_u32(&full[kb]);
          mbar_arrive_expect_tx(fb, stage_bytes(t, w, kb));
          load_weights(w, kb, smem_base + kb * kStageStride, fb);
        }
      }
      __syncwarp();
      pdl_wait();
    }
    uint32_t ph = 1;  // parity of the empty barriers: the first fill waits for nothing
    int s = 0;
    bool ok = true;
    uint32_t fills[kStages / kProdWarps] = {};  // of this warp's slots
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      // (The stages begun above are completed in any case: their weights are on
      // their way, and a barrier's phase ends only with all of its bytes.)
      if (tile != (int)blockIdx.x) {
        if (stopped(&stop_s)) break;
        walk.step(a.n_mtiles, E, first_s, cnt_s);
      }
      const Tile& t = walk.t;
      const WeightAt w = weights_of<MODE, NA>(a, t);
      for (int kb = 0; kb < nk; ++kb) {
        const int slot = s;
        const uint32_t parity = ph;
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
        if (slot % kProdWarps != first) continue;
        const uint32_t st = smem_base + slot * kStageStride;
        const uint32_t fb = smem_u32(&full[slot]);
        const bool todo = kb >= fetched || tile != (int)blockIdx.x;
        if (todo && !warp_wait(smem_u32(&empty[slot]), parity)) {
          stop(&stop_s, a.err);
          ok = false;
          break;
        }
        if (leader) {
          if (todo) {
            mbar_arrive_expect_tx(fb, stage_bytes(t, w, kb));
            load_weights(w, kb, st, fb);
          }
          load_rows(t, kb, st, fb);
        }
        ++fills[slot / kProdWarps];
        __syncwarp();
      }
    }
    // No copy of this warp is in flight when the CTA ends, also where the warps that
    // read the slots have given up (a slot's last fill completes its barrier's phase
    // whether or not anybody reads it).
#pragma unroll
    for (int i = 0; i < kStages / kProdWarps; ++i)
      if (fills[i] > 0) warp_wait(smem_u32(&full[i * kProdWarps + first]), (fills[i] - 1) & 1u);
  } else if (warp < 2) {
    // ------------------------------------------------- MMA issuers (0, 1) ---
    // Warp 0 feeds D0, warp 1 D1; with one weight tile, D0 from the even and D1
    // from the odd stages, which the epilogue adds up. A tcgen05 instruction takes its thread about
    // 30 cycles and a stage's wait 200 more, together above the 60 cycles an
    // MMA of N = 128 takes to run, so one thread for both accumulators leaves
    // the tensor cores waiting (57 us for 8192 x 4096 x 4096, two: 54; with one
    // weight tile 8.3 and 7.5 for 128 x 4096 x 4096).
    // The whole warp runs the loops, so that addresses, descriptors and columns
    // are warp-uniform; one elected lane issues.
    const bool leader = elect_one();
    const uint32_t d = tmem_base + warp * kBN;
    int s = 0;
    uint32_t ph = 0, it = 0;
    Walk walk(a.n_mtiles, E, first_s, cnt_s);
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++it) {
      if (stopped(&stop_s)) break;
      if (it != 0) walk.step(a.n_mtiles, E, first_s, cnt_s);
      const Tile& t = walk.t;
      const bool work = NA == 1 || warp == 0 || weights_of<MODE, NA>(a, t).has1;
      if (!warp_wait(smem_u32(tempty), (it & 1u) ^ 1u)) {
        stop(&stop_s, a.err);
        break;
      }
      tc_fence_after();
      const uint32_t idesc = idesc_mxf4(128, (t.nrows + 15) & ~15);
      bool ok = true;
      for (int kb = 0; kb < nk; ++kb) {
        const int slot = s;
        const uint32_t parity = ph;
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
        if (NA == 1 && (kb & 1) != warp) continue;
        if (!warp_wait(smem_u32(&full[slot]), parity)) {
          stop(&stop_s, a.err);
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {
          const uint32_t st = smem_base + slot * kStageStride;
          // Each slot has scale columns of its own: the MMAs that read their
          // last contents were complete before the slot was filled again.
          const uint32_t tsc = tmem_base + kScaleCol0 + slot * kScaleCols + warp * (kScaleCols / 2);
          const int steps = min(4, (a.K - kb * kStageK + 63) / 64);
          const int a_tile = NA == 1 ? 0 : warp;
          const bool more = NA == 1 ? kb > 1 : kb > 0;
          if (work && steps == 4)
            issue_stage<NA>(st, a_tile, tsc, d, idesc, more, 4);
          else if (work)
            issue_stage<NA>(st, a_tile, tsc, d, idesc, more, steps);
          umma_commit(smem_u32(&empty[slot]));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (leader) umma_commit(smem_u32(tfull));
      __syncwarp();
    }
    // Every MMA issued above has finished before the CTA tears down.
    if (leader) umma_commit(smem_u32(done));
    __syncwarp();
    if (!warp_wait(smem_u32(done), 0)) stop(&stop_s, a.err);
  } else if (warp >= kEpiWarp0) {
    // ----------------------------------------------------- epilogue (2-17) --
    const int q = warp & 3;                    // tensor-memory lane quarter of this warp
    const int c0 = ((warp - kEpiWarp0) >> 2) * 32;  // first column (token row) of this warp
    uint32_t it = 0;
    Walk walk(a.n_mtiles, E, first_s, cnt_s);
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++it) {
      if (stopped(&stop_s)) break;
      if (it != 0) walk.step(a.n_mtiles, E, first_s, cnt_s);
      const Tile& t = walk.t;
      if (!warp_wait(smem_u32(tfull), it & 1u)) {
        stop(&stop_s, a.err);
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      if constexpr (PERM) {
        Piece p0, p1;
        if (c0 < t.nrows) {
          load_piece(tb + c0, p0);
          load_piece(tb + kBN + c0, p1);
          tmem_wait_ld();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(tempty));
        const int ncol = t.nrows - c0;  // token rows of this piece (may exceed 32)
        if (ncol <= 0) continue;
        const int lane4 = lane & 3, col4 = (lane >> 2) * 4;
        const long long row0 = t.row0 + c0 + 2 * lane4;
        const int left = ncol - 2 * lane4;  // row (g, c) is one of them if 8 g + c < left
        // The row whose bytes this lane holds after the folds, with c = lane / 4 % 2.
        const int own = 8 * (lane >> 3) + 2 * lane4 + ((lane >> 2) & 1);
        const int from = lane & 7;  // lane 8 g + from has word g
        if (MODE == kGateUp) {
          const int blk = t.m * 4 + q;       // block of 32 intermediates: this warp's lanes
          const bool real = blk * 32 < a.N;  // else the padding of the last scale tile
          uint8_t* codes = static_cast<uint8_t*>(a.out) + row0 * (a.N / 2) + (blk * 32 + col4) / 2;
          const int k_tiles_act = (a.N + 127) / 128;
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) p0.set(j, g, swiglu(p0.rows(j, g), p1.rows(j, g)));
          uint32_t w[4], f;
          local_max(p0, w);
          uint32_t k = fold(fold(w[0], w[2], 16), fold(w[1], w[3], 16), 8);
          k = __vmaxu2(k, __shfl_xor_sync(kAll, k, 4));
          const uint32_t sb = scale_pair(exponents(k), f);
          if (own < ncol)
            a.act_scales[mx_scale_offset(t.row0 + c0 + own, blk, k_tiles_act)] =
                real ? (uint8_t)(lane & 4 ? sb >> 16 : sb) : 0;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const Pair inv = factors(__shfl_sync(kAll, f, 8 * g + from));
            Pair x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = p0.rows(j, g) * inv;
            if (real && 8 * g < left)
              *reinterpret_cast<uint16_t*>(codes + (8 * g) * (size_t)(a.N / 2)) =
                  mx_pack4(x[0].x, x[1].x, x[2].x, x[3].x);
            if (real && 8 * g + 1 < left)
              *reinterpret_cast<uint16_t*>(codes + (8 * g + 1) * (size_t)(a.N / 2)) =
                  mx_pack4(x[0].y, x[1].y, x[2].y, x[3].y);
          }
        } else {
          const int n = t.m * (NA * 128) + q * 32;  // and n + 128 from the second accumulator
          const bool in0 = n < a.N, in1 = NA == 2 && n + 128 < a.N;
          if (NA == 1 && nk > 1) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int j = 0; j < 4; ++j) p0.set(j, g, p0.rows(j, g) + p1.rows(j, g));
          }
          const long long lead = MODE == kDown ? lead_s[t.e] : 0;
          const size_t at = (size_t)(row0 + lead) * a.N + n + col4;
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (8 * g + c >= left) continue;
              const size_t to = at + (8 * g + c) * (size_t)a.N;
              if (MODE == kDown || a.out_fp32) {
                float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.out) + to);
                if (in0) d[0] = make_float4(p0.at(0, g, c), p0.at(1, g, c), p0.at(2, g, c), p0.at(3, g, c));
                if (in1) d[32] = make_float4(p1.at(0, g, c), p1.at(1, g, c), p1.at(2, g, c), p1.at(3, g, c));
              } else {
                uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to);
                if (in0)
                  d[0] = make_uint2(bf16x2(p0.at(0, g, c), p0.at(1, g, c)),
                                    bf16x2(p0.at(2, g, c), p0.at(3, g, c)));
                if (in1)
                  d[32] = make_uint2(bf16x2(p1.at(0, g, c), p1.at(1, g, c)),
                                     bf16x2(p1.at(2, g, c), p1.at(3, g, c)));
              }
            }
        }
      } else {
        // Any N: lane = output column, one value of 32 token rows a lane.
        uint32_t d0[32], d1[32];
        if (c0 < t.nrows) {
          tmem_ld_32x32b_x32(tb + c0, d0);
          tmem_ld_32x32b_x32(tb + kBN + c0, d1);
          tmem_wait_ld();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(tempty));
        if (NA == 1 && nk > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            d0[j] = __float_as_uint(__uint_as_float(d0[j]) + __uint_as_float(d1[j]));
        }
        const int ncol = t.nrows - c0, n0 = t.m * (NA * 128) + q * 32 + lane;
        const bool in0 = n0 < a.N, in1 = NA == 2 && n0 + 128 < a.N;
        size_t at = (size_t)(t.row0 + c0) * a.N + n0;
#pragma unroll
        for (int j = 0; j < 32; ++j, at += a.N) {
          if (j >= ncol) break;
          const float x1 = __uint_as_float(d1[j]);
          const float x0 = __uint_as_float(d0[j]);
          if (a.out_fp32) {
            float* c = static_cast<float*>(a.out);
            if (in0) c[at] = x0;
            if (in1) c[at + 128] = x1;
          } else {
            uint16_t* c = static_cast<uint16_t*>(a.out);
            if (in0) c[at] = f32_to_bf16_bits(x0);
            if (in1) c[at + 128] = f32_to_bf16_bits(x1);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// w: w_rows rows of weight codes (scale_tiles tiles of 512 bytes); x: x_rows
// rows of token codes.
template <int MODE, bool PERM, int NA>
cudaError_t launch_mode(const uint8_t* w, long long w_rows, long long scale_tiles, const uint8_t* x,
                        long long x_rows, const MxGemmArgs& a, long long max_tiles, int num_sms,
                        bool after_prev, cudaStream_t st) {
  static DeviceFlags attr_done;
  if (cudaError_t e = smem_attr_once(attr_done, mx_gemm_kernel<MODE, PERM, NA>, Ring<NA>::kSmemBytes);
      e != cudaSuccess)
    return e;
  CUtensorMap tmW, tmS = {}, tmX, tmX32;
  const uint64_t K = (uint64_t)a.K;
  bool ok = make_tensor_map_codes(&tmX, x, (uint64_t)x_rows, K, 128) &&
            make_tensor_map_codes(&tmX32, x, (uint64_t)x_rows, K, 32);
  if (PERM) {
    // Shared-memory row p of a group of 32 takes weight row 4 (p % 8) + p / 8:
    // the boxes run over 8 rows a stride of 4 apart, 4 rows, 4 groups; the
    // scales' 16-byte rows likewise.
    const uint64_t wd[4] = {K / 2, 8, 4, (uint64_t)w_rows / 32};
    const uint64_t ws[3] = {2 * K, K / 2, 16 * K};
    const uint32_t wb[4] = {128, 8, 4, 4};
    const uint64_t sd[4] = {16, 8, 4, (uint64_t)scale_tiles};
    const uint64_t ss[3] = {64, 16, kMxTileBytes};
    const uint32_t sbx[4] = {16, 8, 4, 2};
    ok = ok && make_tensor_map_bytes_4d(&tmW, w, wd, ws, wb, true) &&
         make_tensor_map_bytes_4d(&tmS, a.w_scales, sd, ss, sbx, false);
  } else {
    ok = ok && make_tensor_map_codes(&tmW, w, (uint64_t)w_rows, K, 128);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int grid = (int)std::min<long long>(max_tiles, num_sms);
  return launch_k(mx_gemm_kernel<MODE, PERM, NA>, dim3(grid), dim3(kThreads), Ring<NA>::kSmemBytes, st,
                  after_prev, tmW, tmS, tmX, tmX32, a);
}

}  // namespace

cudaError_t launch_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                           const uint8_t* b_scales, int M, int N, int K, void* c, bool out_fp32,
                           int num_sms, unsigned* err, cudaStream_t st) {
  MxGemmArgs a = {};
  a.w_scales = b_scales;
  a.x_scales = a_scales;
  a.out = c;
  a.err = err;
  a.E = 1;
  a.rows = M;
  a.N = N;
  a.K = K;
  a.out_fp32 = out_fp32 ? 1 : 0;
  const long long chunks = (M + kBN - 1) / kBN;
  // Tiles of 128 output columns where they still leave every CTA at most one: an
  // SM takes in some 90 bytes a cycle, so with few tiles the bytes of a tile
  // count (64 x 4096 x 4096: 8.9 us with tiles of 256, 6.9 with 128; 1111 x 1000
  // x 2080: 10.6 and 7.9). (Not the experts' down product, whose CTAs
  // fetch weights beside those of gate_up: one token 15.2 -> 16.7 us.)
  const bool narrow = chunks * ((N + 127) / 128) <= num_sms;
  a.n_mtiles = narrow ? (N + 127) / 128 : (N + 255) / 256;
  const long long tiles = chunks * a.n_mtiles;
  const long long scale_tiles = (long long)mx_tiles(N) * mx_tiles(K);
  // With whole groups of 32 output columns a thread can have four of them and
  // store wide, but the boxes in that row order take longer to load. Where tiles
  // fill the SMs it pays for short reductions only (8192 x 4096, in that order and
  // without: K = 512 19.2 and 20.1 us, 1024 24.5 and 23.7, 2048 37.9 and 35.3, 4096
  // 59.9 and 54.8); few tiles are bound by latency (64 x 4096 x 4096: 8.9 and 9.6).
  const bool perm = N % 32 == 0 && (K < 1024 || narrow || tiles < num_sms);
  auto launch = perm ? (narrow ? launch_mode<kDense, true, 1> : launch_mode<kDense, true, 2>)
                     : (narrow ? launch_mode<kDense, false, 1> : launch_mode<kDense, false, 2>);
  return launch(b_codes, N, scale_tiles, a_codes, M, a, tiles, num_sms, true, st);
}

cudaError_t launch_mx_experts_gate_up(const uint8_t* xs, const uint8_t* xs_scales,
                                      const uint8_t* w, const uint8_t* w_scales,
                                      const int32_t* counts, const int32_t* ids, int T,
                                      int top_k, int E, int I, int H, long long capacity, long long max_chunks,
                                      uint8_t* act, uint8_t* act_scales, int num_sms,
                                      unsigned* err, bool after_prev, cudaStream_t st) {
  MxGemmArgs a = {};
  a.counts = counts;
  if (T * top_k <= kMxEarlyIds) {
    a.ids = ids;
    a.n_ids = T * top_k;
    a.top_k = top_k;
  }
  a.w_scales = w_scales;
  a.x_scales = xs_scales;
  a.out = act;
  a.act_scales = act_scales;
  a.err = err;
  a.E = E;
  a.N = I;
  a.K = H;
  a.n_mtiles = (I + 127) / 128;
  return launch_mode<kGateUp, true, 2>(w, 2LL * E * I, 2LL * E * mx_tiles(I) * mx_tiles(H), xs, capacity,
                                    a, max_chunks * a.n_mtiles, num_sms, after_prev, st);
}

cudaError_t launch_mx_experts_down(const uint8_t* act, const uint8_t* act_scales, const uint8_t* w,
                                   const uint8_t* w_scales, const int32_t* counts,
                                   const int32_t* ids, int T, int top_k, int E, int H, int I, long long capacity, long long max_chunks,
                                   float* y, int num_sms, unsigned* err, bool after_prev, cudaStream_t st) {
  MxGemmArgs a = {};
  a.counts = counts;
  if (T * top_k <= kMxEarlyIds) {
    a.ids = ids;
    a.n_ids = T * top_k;
    a.top_k = top_k;
  }
  a.w_scales = w_scales;
  a.x_scales = act_scales;
  a.out = y;
  a.err = err;
  a.E = E;
  a.N = H;
  a.K = I;
  a.n_mtiles = (H + 255) / 256;
  return launch_mode<kDown, true, 2>(w, (long long)E * H, (long long)E * mx_tiles(H) * mx_tiles(I), act,
                                  capacity, a, max_chunks * a.n_mtiles, num_sms, after_prev, st);
}

}  // namespace mm
