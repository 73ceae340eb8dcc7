// Microscaled 4-bit rows: quantisation, the way back, and the row passes of
// the 4-bit experts (the grouping, token rows quantised into their experts'
// segments, the weighted sum of a token's expert outputs). The format is in
// mx_device.cuh.
//
// Per block of 32: e = floor(log2 max|x|) - 2, scale byte e + 127, codes
// e2m1(x 2^-e) to nearest even, saturating at 6. x 2^-e is a product with a
// power of two and exact, except where it underflows, far below the border
// 0.25 of the code 0; so the one rounding is the conversion to e2m1.
//
// A lane takes 16 consecutive columns, two lanes a block; the lanes of a row
// are a power of two (all 32 from K = 512 on). One pass: a row is read once,
// its codes and scale bytes are written once, so the kernels are bound by
// memory: 256 x 768 x 2048 bf16 values take 164 us to quantise (1.02 GB, 6.2
// TB/s) and 145 us to decode (7.0 TB/s). At 4096 tokens of 2048 values, 8 slots
// each, the experts' grouping takes 7 us, the rows 15 (17 MB read, 35 MB
// written, 32768 atomics), the weighted sum 45 (268 MB of fp32 rows, 6.2 TB/s).
#include "mm.h"
#include "mm_internal.h"
#include "mx_device.cuh"

#include <cuda_fp16.h>

namespace mm {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kMxThreads = 256;
constexpr int kMxWarps = kMxThreads / 32;

struct Raw16f { uint4 r[4]; };  // 16 float32
struct Raw16h { uint4 r[2]; };  // 16 bf16 or fp16

template <int DT> struct MxIn;  // storage of 16 input values
template <> struct MxIn<MM_DTYPE_FP32> { using Raw = Raw16f; static constexpr int kBytes = 4; };
template <> struct MxIn<MM_DTYPE_BF16> { using Raw = Raw16h; static constexpr int kBytes = 2; };
template <> struct MxIn<MM_DTYPE_FP16> { using Raw = Raw16h; static constexpr int kBytes = 2; };

// 32 contiguous bytes a lane in one access: a warp moves 1 KB of whole lines,
// where two 16-byte accesses would each touch half of them. Needs 32-byte
// alignment; the kernels' WIDE variants are taken where the caller's buffer
// has it (rows are multiples of 64 bytes), the others use 16-byte accesses.
__device__ __forceinline__ void load32(const unsigned char* p, uint4& a, uint4& b) {
  asm("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
      : "l"(p));
}
__device__ __forceinline__ void store32(unsigned char* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

template <int DT, bool WIDE>
__device__ __forceinline__ void load16(const unsigned char* p, typename MxIn<DT>::Raw& raw) {
#pragma unroll
  for (int i = 0; i < MxIn<DT>::kBytes; i += 2) {
    if constexpr (WIDE) {
      load32(p + 16 * i, raw.r[i], raw.r[i + 1]);
    } else {
      raw.r[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
      raw.r[i + 1] = __ldg(reinterpret_cast<const uint4*>(p) + i + 1);
    }
  }
}

template <int DT>
__device__ __forceinline__ void zero16(typename MxIn<DT>::Raw& raw) {
#pragma unroll
  for (int i = 0; i < MxIn<DT>::kBytes; ++i) raw.r[i] = make_uint4(0u, 0u, 0u, 0u);
}

template <int DT>
__device__ __forceinline__ void unpack16(const typename MxIn<DT>::Raw& raw, float (&v)[16]) {
  if constexpr (DT == MM_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = __uint_as_float(raw.r[i].x);
      v[4 * i + 1] = __uint_as_float(raw.r[i].y);
      v[4 * i + 2] = __uint_as_float(raw.r[i].z);
      v[4 * i + 3] = __uint_as_float(raw.r[i].w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {raw.r[i].x, raw.r[i].y, raw.r[i].z, raw.r[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == MM_DTYPE_BF16) {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          v[8 * i + 2 * j] = f.x;
          v[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
  }
}

// Bits (float32) of the largest magnitude of 16 values. Sixteen-bit floats are
// compared two at a time as integers, which orders magnitudes (and puts
// infinity and NaN on top): half the instructions of comparing them unpacked.
template <int DT>
__device__ __forceinline__ uint32_t amax16(const typename MxIn<DT>::Raw& raw) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < MxIn<DT>::kBytes; ++i) {
    const uint32_t w[4] = {raw.r[i].x, raw.r[i].y, raw.r[i].z, raw.r[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = DT == MM_DTYPE_FP32 ? max(m, w[j] & 0x7fffffffu) : __vmaxu2(m, w[j] & 0x7fff7fffu);
  }
  if constexpr (DT == MM_DTYPE_FP32) return m;
  m = max(m >> 16, m & 0xFFFFu);
  if constexpr (DT == MM_DTYPE_BF16) return m << 16;
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}

// The 16 values of this lane, half a block: codes (8 bytes) and, in every
// lane of a group of 8, the four scale bytes of the group's 128 columns.
template <int DT>
__device__ __forceinline__ uint2 encode16(const typename MxIn<DT>::Raw& raw, uint32_t& scales4) {
  uint32_t amax = amax16<DT>(raw);
  amax = max(amax, __shfl_xor_sync(kAll, amax, 1));
  const uint32_t s = mx_scale_byte(amax);
  const float inv = mx_inv_scale(s);
  float v[16], a[8], b[8];
  unpack16<DT>(raw, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = v[i] * inv;
    b[i] = v[8 + i] * inv;
  }
  uint32_t q = s << (8 * ((threadIdx.x >> 1) & 3));
  q |= __shfl_xor_sync(kAll, q, 2);
  q |= __shfl_xor_sync(kAll, q, 4);
  scales4 = q;
  return make_uint2(mx_pack8(a), mx_pack8(b));
}

// A row handed to a group of 2^lanes_log2 lanes: columns
// [16 * lane, 16 * lane + 16) of every span of 16 << lanes_log2. Columns at or
// past K of the last scale tile give zero scale bytes and no codes. src NULL:
// a padding row (zero scale bytes only). All lanes of the warp call this.
template <int DT, bool WIDE, int U>
__device__ __forceinline__ void quantize_row(const unsigned char* src, int K, int lanes_log2,
                                             uint8_t* codes, uint8_t* scale_row, bool active) {
  const int lane = threadIdx.x & ((1 << lanes_log2) - 1);
  const int span = 16 << lanes_log2;
  const int kp = (K + kMxTile - 1) / kMxTile * kMxTile;
  for (int c0 = lane * 16; c0 - lane * 16 < kp; c0 += U * span) {
    typename MxIn<DT>::Raw raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * span;
      if (src != nullptr && c < K)
        load16<DT, WIDE>(src + (size_t)c * MxIn<DT>::kBytes, raw[u]);
      else
        zero16<DT>(raw[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * span;
      if (c - lane * 16 >= kp) break;  // the same for every lane of the group
      uint32_t s4;
      const uint2 code = encode16<DT>(raw[u], s4);
      if (active && c < K && src != nullptr)
        *reinterpret_cast<uint2*>(codes + c / 2) = code;
      if (active && (threadIdx.x & 7) == 0 && c < kp)
        *reinterpret_cast<uint32_t*>(scale_row + (size_t)(c / kMxTile) * kMxTileBytes) = s4;
    }
  }
}

// Lanes of a row (log2): enough for 16 columns a lane, at least the 8 of one
// scale tile (so that a group's four bytes come from one row).
__host__ __device__ __forceinline__ int row_lanes_log2(int K) {
  return K > 256 ? 5 : K > 128 ? 4 : 3;
}

template <int DT, bool WIDE>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const unsigned char* __restrict__ x,
                                                                 long long prows, int rows, int rp,
                                                                 int K, int lanes_log2,
                                                                 uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int per_warp = 32 >> lanes_log2;
  const long long row = ((long long)blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * per_warp +
                        ((threadIdx.x & 31) >> lanes_log2);
  const bool active = row < prows;
  const long long b = active ? row / rp : 0;
  const int r = active ? (int)(row - b * rp) : 0;
  const bool real = active && r < rows;
  const int kt = (int)mx_tiles(K);
  const size_t at = (size_t)(b * rows + r) * K;
  quantize_row<DT, WIDE, 4>(real ? x + at * MxIn<DT>::kBytes : nullptr, K, lanes_log2, codes + at / 2,
                      scales + (size_t)b * (rp / kMxTile) * kt * kMxTileBytes +
                          mx_scale_offset(r, 0, kt),
                      active);
}

// Two e2m1 of a byte as two floats.
__device__ __forceinline__ float2 decode2(uint32_t byte) {
  uint32_t h;
  asm("{ .reg .b8 b, z;\n\t"
      "mov.b16 {b, z}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b; }"
      : "=r"(h)
      : "h"((uint16_t)byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  return (uint32_t)f32_to_bf16_bits(a) | ((uint32_t)f32_to_bf16_bits(b) << 16);
}

// The 16 values of 8 code bytes under scale s, written as DT at dst.
template <int DT, bool WIDE>
__device__ __forceinline__ void decode16(uint2 code, float s, unsigned char* dst) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = decode2(((i < 4 ? code.x : code.y) >> (8 * (i & 3))) & 0xffu);
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
  uint32_t w[16];
  if constexpr (DT == MM_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (DT == MM_DTYPE_BF16) {
        w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      } else {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MxIn<DT>::kBytes; i += 2) {
    const uint4 lo = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    const uint4 hi = make_uint4(w[4 * i + 4], w[4 * i + 5], w[4 * i + 6], w[4 * i + 7]);
    if constexpr (WIDE) {
      store32(dst + 16 * i, lo, hi);
    } else {
      reinterpret_cast<uint4*>(dst)[i] = lo;
      reinterpret_cast<uint4*>(dst)[i + 1] = hi;
    }
  }
}

// One lane: 16 columns (8 code bytes, one scale byte) of one row, kU spans of
// the row loaded before any is written.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(kMxThreads) mx_dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long nrows, int rows,
    int K, int lanes_log2, unsigned char* __restrict__ out) {
  constexpr int kU = 4;
  pdl_wait();
  pdl_trigger();
  const int per_warp = 32 >> lanes_log2;
  const long long row = ((long long)blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * per_warp +
                        ((threadIdx.x & 31) >> lanes_log2);
  if (row >= nrows) return;
  const int lane = threadIdx.x & ((1 << lanes_log2) - 1);
  const long long b = row / rows;
  const int r = (int)(row - b * rows);
  const int kt = (int)mx_tiles(K), span = 16 << lanes_log2;
  const uint8_t* srow =
      scales + (size_t)b * mx_tiles(rows) * kt * kMxTileBytes + mx_scale_offset(r, 0, kt);
  const size_t at = (size_t)row * K;
  for (int c0 = lane * 16; c0 < K; c0 += kU * span) {
    uint2 code[kU];
    uint32_t s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = c0 + u * span;
      if (c < K) {
        code[u] = __ldg(reinterpret_cast<const uint2*>(codes + (at + c) / 2));
        s[u] = __ldg(srow + (size_t)(c / kMxTile) * kMxTileBytes + (c / kMxBlock) % 4);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = c0 + u * span;
      if (c < K) decode16<DT, WIDE>(code[u], mx_scale(s[u]), out + (at + c) * MxIn<DT>::kBytes);
    }
  }
}

// ---------------------------------------------- rows of the experts' segments
//
// Every expert's token rows lie in one segment that begins at a multiple of
// 128 rows. The order of the rows inside a segment does not matter (rows are
// independent, and a token's sum runs over its slots), so a row takes the next
// free place. A slot whose id is outside [0, E) or repeats an earlier one of its
// token is dropped and flagged, as in the layer's grouping.

// U spans of a token's row (columns c, c + span, ...) to all its places: `place`
// in lane j < top_k is the row of slot j (-1: dropped), scale_at its scale
// offset.
template <int U>
__device__ __forceinline__ void write_places(const Raw16h (&raw)[U], int c, int span, int H,
                                             int top_k, int place, uint8_t* codes, uint8_t* scales,
                                             size_t scale_at) {
  uint2 code[U];
  uint32_t s4[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    code[u] = encode16<MM_DTYPE_BF16>(raw[u], s4[u]);
  }
  const int hp = (int)mx_tiles(H) * kMxTile;
  for (int j = 0; j < top_k; ++j) {
    const int r = __shfl_sync(kAll, place, j);
    if (r < 0) continue;
    uint8_t* row = codes + (size_t)r * (H / 2);
    uint8_t* srow = scales + __shfl_sync(kAll, scale_at, j);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cu = c + u * span;
      if (cu < H) *reinterpret_cast<uint2*>(row + cu / 2) = code[u];
      if ((threadIdx.x & 7) == 0 && cu < hp)
        *reinterpret_cast<uint32_t*>(srow + (size_t)(cu / kMxTile) * kMxTileBytes) = s4[u];
    }
  }
}

struct MxPlaceArgs {
  const unsigned char* hidden;
  const int32_t* ids;
  int32_t* counts;   // [E]
  // [E * kMxCursorStep] (large batches) an expert's next free row, and what leads
  // from its rows to those without the segments' padding
  int32_t* cursor;
  int32_t* pos;      // [T * top_k] row of a slot without the padding, -1 if dropped
  uint8_t* codes;
  uint8_t* scales;
  unsigned* err;
  int T, E, top_k, H;
};

// First rows of the segments from the counts, and what leads from a segment's
// rows to those without padding, by one warp (lane l the experts from 8 l on).
__device__ __forceinline__ void scan_segments(const int* cnt, int E, int* off, int* lead) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kMaxExperts / 32;
  int c[kPer], rows = 0, padded = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    c[i] = e < E ? cnt[e] : 0;
    rows += c[i];
    padded += (c[i] + kMxBlockM - 1) / kMxBlockM * kMxBlockM;
  }
  rows = exclusive_sum(rows);
  padded = exclusive_sum(padded);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    if (e < E) {
      off[e] = padded;
      lead[e] = rows - padded;
    }
    rows += c[i];
    padded += (c[i] + kMxBlockM - 1) / kMxBlockM * kMxBlockM;
  }
}

// Up to kMxEarlyIds slots: one block a token, one launch. Every block counts
// all slots itself (a few thousand shared-memory adds) and ranks its token
// among the earlier ones, while its part of the row is on the way.
constexpr int kPlaceWarps = 4;

__global__ void __launch_bounds__(kPlaceWarps * 32) mx_place_small_kernel(const MxPlaceArgs a) {
  __shared__ int ids_s[kMxEarlyIds];
  __shared__ int tot[kMaxExperts], before[kMaxExperts], off[kMaxExperts], lead[kMaxExperts];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kNT = kPlaceWarps * 32;
  const int t = blockIdx.x, k = a.top_k, n = a.T * k;
  pdl_wait();
  pdl_trigger();
  const unsigned char* row = a.hidden + (size_t)t * a.H * 2;
  const int hp = (int)mx_tiles(a.H) * kMxTile;
  int c = tid * 16;
  Raw16h raw[1];
  zero16<MM_DTYPE_BF16>(raw[0]);
  if (c < a.H) load16<MM_DTYPE_BF16, false>(row + (size_t)c * 2, raw[0]);
  for (int i = tid; i < n; i += kNT) ids_s[i] = __ldg(a.ids + i);
  for (int e = tid; e < a.E; e += kNT) tot[e] = before[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < n; i += kNT) {
    const int id = ids_s[i], i0 = i / k * k;
    bool drop = id < 0 || id >= a.E;
    for (int j = i0; j < i && !drop; ++j) drop = ids_s[j] == id;
    bad |= drop;
    if (!drop) {
      atomicAdd(&tot[id], 1);
      if (i < t * k) atomicAdd(&before[id], 1);
    }
  }
  if (bad && t == 0) atomicOr(a.err, kDevErrBadIds);
  __syncthreads();
  if (warp == 0) scan_segments(tot, a.E, off, lead);
  __syncthreads();
  int place = -1;
  if (lane < k) {
    const int id = ids_s[t * k + lane];
    bool drop = id < 0 || id >= a.E;
    for (int j = 0; j < lane && !drop; ++j) drop = ids_s[t * k + j] == id;
    if (!drop) place = off[id] + before[id];
    if (warp == 0) a.pos[t * k + lane] = drop ? -1 : place + lead[id];
  }
  const size_t scale_at = place >= 0 ? mx_scale_offset(place, 0, (int)mx_tiles(a.H)) : 0;
  for (; c - lane * 16 < hp; c += kNT * 16) {
    write_places<1>(raw, c, 0, a.H, k, place, a.codes, a.scales, scale_at);
    zero16<MM_DTYPE_BF16>(raw[0]);
    if (c + kNT * 16 < a.H) load16<MM_DTYPE_BF16, false>(row + (size_t)(c + kNT * 16) * 2, raw[0]);
  }
}

// Larger batches: one cluster counts the slots, its first block adds the counts
// up and lays the segments out ...
constexpr int kGroupThreads = 1024;
constexpr int kGroupBlocks = 8;

__global__ void __cluster_dims__(kGroupBlocks, 1, 1) __launch_bounds__(kGroupThreads, 1)
    mx_group_kernel(const MxPlaceArgs a) {
  __shared__ int tot[kMaxExperts], sum[kMaxExperts], off[kMaxExperts], lead[kMaxExperts];
  const int tid = threadIdx.x;
  const uint32_t k = a.top_k;
  pdl_wait();
  pdl_trigger();
  for (int e = tid; e < a.E; e += kGroupThreads) tot[e] = 0;
  __syncthreads();
  bool bad = false;
  // A thread takes a token, eight slots at a time, all loaded before any is used.
  for (uint32_t t = blockIdx.x * kGroupThreads + tid; t < (uint32_t)a.T;
       t += kGroupBlocks * kGroupThreads) {
    const int32_t* row = a.ids + (size_t)t * k;
    for (uint32_t j0 = 0; j0 < k; j0 += 8) {
      int id[8];
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) id[j] = j0 + j < k ? __ldg(row + j0 + j) : 0;
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) {
        if (j0 + j >= k) break;
        bool drop = id[j] < 0 || id[j] >= a.E;
#pragma unroll
        for (uint32_t i = 0; i < j; ++i) drop |= id[i] == id[j];
        for (uint32_t i = 0; i < j0; ++i) drop |= __ldg(row + i) == id[j];
        bad |= drop;
        if (!drop) atomicAdd(&tot[id[j]], 1);
      }
    }
  }
  if (bad) atomicOr(a.err, kDevErrBadIds);
  cluster_barrier();
  if (blockIdx.x == 0) {
    for (int e = tid; e < a.E; e += kGroupThreads) {
      int v = 0;
#pragma unroll
      for (uint32_t r = 0; r < kGroupBlocks; ++r) v += load_peer(&tot[e], r);
      sum[e] = v;
    }
    __syncthreads();
    if (tid < 32) scan_segments(sum, a.E, off, lead);
    __syncthreads();
    for (int e = tid; e < a.E; e += kGroupThreads) {
      a.counts[e] = sum[e];
      a.cursor[e * kMxCursorStep] = off[e];
      a.cursor[e * kMxCursorStep + 1] = lead[e];
    }
  }
  cluster_barrier();  // no block ends while its counts are being read
}

// ... then one warp a token takes the next free rows and fills them. The
// token's row and ids are the caller's, so they are read before the wait.
__global__ void __launch_bounds__(kMxThreads) mx_place_kernel(const MxPlaceArgs a) {
  const int lane = threadIdx.x & 31, k = a.top_k;
  const int t = blockIdx.x * kMxWarps + (threadIdx.x >> 5);
  constexpr int U = 4, kSpan = 512;
  const unsigned char* row = a.hidden + (size_t)t * a.H * 2;
  const int hp = (int)mx_tiles(a.H) * kMxTile;
  Raw16h raw[U];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kSpan;
      if (c < a.H)
        load16<MM_DTYPE_BF16, false>(row + (size_t)c * 2, raw[u]);
      else
        zero16<MM_DTYPE_BF16>(raw[u]);
    }
  };
  int place = -1;
  if (t < a.T) {
    load(lane * 16);
    if (lane < k) place = __ldg(a.ids + (size_t)t * k + lane);
  }
  pdl_wait();
  pdl_trigger();
  if (t >= a.T) return;
  const uint32_t same = __match_any_sync(kAll, place);
  int pos = -1;
  if (place < 0 || place >= a.E || (same & ((1u << lane) - 1u)) != 0) {
    place = -1;
  } else {
    int32_t* cursor = a.cursor + place * kMxCursorStep;
    pos = __ldcg(cursor + 1);
    place = atomicAdd(cursor, 1);
    pos += place;
  }
  if (lane < k) a.pos[(size_t)t * k + lane] = pos;
  const size_t scale_at = place >= 0 ? mx_scale_offset(place, 0, (int)mx_tiles(a.H)) : 0;
  for (int c0 = lane * 16; c0 - lane * 16 < hp; c0 += U * kSpan) {
    if (c0 != lane * 16) load(c0);
    write_places<U>(raw, c0, kSpan, a.H, k, place, a.codes, a.scales, scale_at);
  }
}

// out[t] = bf16(sum_j w[t,j] y[pos[t k + j]]) in slot order, 8 columns a thread;
// dropped slots (pos < 0) have no row in y and add nothing. y is fp32: its values
// are terms of a sum that may cancel, and one column says nothing of another's
// range. J slots at a time: their rows first, then all their loads, then the sum.
template <int J>
__global__ void __launch_bounds__(kMxThreads) mx_combine_kernel(
    const float* __restrict__ y, const int32_t* __restrict__ pos, const float* __restrict__ w, int T,
    int top_k, int h8, uint4* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const long long i = (long long)blockIdx.x * kMxThreads + threadIdx.x;
  if (i >= (long long)T * h8) return;
  const int t = (int)(i / h8), h = (int)(i - (long long)t * h8);
  const size_t f0 = (size_t)t * top_k;
  float s[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) s[q] = 0.f;
  for (int j0 = 0; j0 < top_k; j0 += J) {
    int r[J];
    float wj[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool in = j0 + j < top_k;
      r[j] = in ? __ldg(pos + f0 + j0 + j) : -1;
      wj[j] = in ? __ldg(w + f0 + j0 + j) : 0.f;
    }
    uint4 v[J][2];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      v[j][0] = v[j][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r[j] >= 0)
        load32(reinterpret_cast<const unsigned char*>(y + ((size_t)r[j] * h8 + h) * 8), v[j][0],
               v[j][1]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (r[j] < 0) continue;  // a NaN or infinite weight of a dropped slot stays out
      const uint32_t p[8] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w,
                             v[j][1].x, v[j][1].y, v[j][1].z, v[j][1].w};
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += wj[j] * __uint_as_float(p[q]);
    }
  }
  out[i] = make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]),
                      pack_bf16x2(s[6], s[7]));
}

}  // namespace

namespace {

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

template <int DT>
cudaError_t quantize_t(const unsigned char* x, long long prows, int rows, int rp, int K, int ll,
                       uint8_t* codes, uint8_t* scales, dim3 grid, cudaStream_t st) {
  return launch_k(aligned32(x) ? mx_quantize_kernel<DT, true> : mx_quantize_kernel<DT, false>, grid,
                  dim3(kMxThreads), 0, st, true, x, prows, rows, rp, K, ll, codes, scales);
}

template <int DT>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, long long nrows, int rows,
                         int K, int ll, unsigned char* out, dim3 grid, cudaStream_t st) {
  return launch_k(aligned32(out) ? mx_dequantize_kernel<DT, true> : mx_dequantize_kernel<DT, false>,
                  grid, dim3(kMxThreads), 0, st, true, codes, scales, nrows, rows, K, ll, out);
}

}  // namespace

cudaError_t launch_mx_quantize(const void* x, int dtype, long long batch, int rows, int K,
                               uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const int rp = (int)(mx_tiles(rows) * kMxTile), ll = row_lanes_log2(K);
  const long long prows = batch * rp;
  const long long per_block = (long long)kMxWarps * (32 >> ll);
  const dim3 grid((unsigned)((prows + per_block - 1) / per_block));
  const unsigned char* p = static_cast<const unsigned char*>(x);
  if (dtype == MM_DTYPE_FP32)
    return quantize_t<MM_DTYPE_FP32>(p, prows, rows, rp, K, ll, codes, scales, grid, st);
  if (dtype == MM_DTYPE_BF16)
    return quantize_t<MM_DTYPE_BF16>(p, prows, rows, rp, K, ll, codes, scales, grid, st);
  return quantize_t<MM_DTYPE_FP16>(p, prows, rows, rp, K, ll, codes, scales, grid, st);
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, long long batch,
                                 int rows, int K, void* out, int dtype, cudaStream_t st) {
  const int ll = row_lanes_log2(K);
  const long long nrows = batch * rows;
  const long long per_block = (long long)kMxWarps * (32 >> ll);
  const dim3 grid((unsigned)((nrows + per_block - 1) / per_block));
  unsigned char* p = static_cast<unsigned char*>(out);
  if (dtype == MM_DTYPE_FP32)
    return dequantize_t<MM_DTYPE_FP32>(codes, scales, nrows, rows, K, ll, p, grid, st);
  if (dtype == MM_DTYPE_BF16)
    return dequantize_t<MM_DTYPE_BF16>(codes, scales, nrows, rows, K, ll, p, grid, st);
  return dequantize_t<MM_DTYPE_FP16>(codes, scales, nrows, rows, K, ll, p, grid, st);
}

cudaError_t launch_mx_place(const uint16_t* hidden, const int32_t* ids, int T, int top_k, int E,
                            int H, int32_t* counts, int32_t* cursor,
                            int32_t* pos, uint8_t* codes, uint8_t* scales, unsigned* err,
                            cudaStream_t st) {
  const MxPlaceArgs a = {reinterpret_cast<const unsigned char*>(hidden), ids, counts,
                         cursor, pos, codes, scales, err, T, E, top_k, H};
  if (T * top_k <= kMxEarlyIds)
    return launch_k(mx_place_small_kernel, dim3(T), dim3(kPlaceWarps * 32), 0, st, true, a);
  cudaError_t e = launch_k(mx_group_kernel, dim3(kGroupBlocks), dim3(kGroupThreads), 0, st, true, a);
  if (e != cudaSuccess) return e;
  return launch_k(mx_place_kernel, dim3((T + kMxWarps - 1) / kMxWarps), dim3(kMxThreads), 0, st,
                  true, a);
}

cudaError_t launch_mx_combine(const float* y, const int32_t* pos, const float* w, int T, int top_k,
                              int H, uint16_t* out, bool after_prev, cudaStream_t st) {
  // Eight slots' loads at once (all of a call at T = 1 / 64 / 4096: 15.3 / 60.1 /
  // 201 us; four at once 15.9 / 62.7 / 204, two 16.2 / 61.9 / 204).
  const long long blocks = ((long long)T * (H / 8) + kMxThreads - 1) / kMxThreads;
  return launch_k(mx_combine_kernel<8>, dim3((unsigned)blocks), dim3(kMxThreads), 0, st, after_prev,
                  y, pos, w, T, top_k, H / 8, reinterpret_cast<uint4*>(out));
}

}  // namespace mm
