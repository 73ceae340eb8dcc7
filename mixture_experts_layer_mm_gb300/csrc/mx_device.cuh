// Device helpers of the microscaled 4-bit kernels: e2m1 conversion, block
// exponents, the stored order of the scale bytes, and the block-scaled
// tcgen05 instructions.
//
// A block is 32 consecutive columns of a row. Its scale byte s stands for
// 2^(s - 127) (s = 255: NaN, the whole block), its values for 4-bit floats
// e2m1 (sign, 2 exponent bits, 1 mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6),
// two to a byte, the even column in the low nibble.
//
// Scale bytes lie in tiles of 128 rows x 128 columns (4 blocks), 512
// contiguous bytes each, tile (r / 128, k / 128) of a [rows, K] matrix at
// 512 * ((r / 128) * ceil(K / 128) + k / 128); inside a tile the byte of row
// r, block c is (r % 32) * 16 + (r % 128) / 32 * 4 + c % 4. That is the image
// the block-scaled MMA wants in tensor memory (32 lanes of 16 bytes, copied
// to each lane quarter), so a tile goes there by one bulk copy and one
// tcgen05.cp, whoever reads it.
#pragma once

#include "mm_device.cuh"

namespace mm {

constexpr int kMxBlock = 32;      // columns per scale
constexpr int kMxTile = 128;      // rows and columns per scale tile
constexpr int kMxTileBytes = 512;
// Most rows (of a batch, in whole tiles) and columns: loops that step past the
// end by less than 4096 stay within 31 bits.
constexpr long long kMxMaxExtent = (1LL << 31) - 4096;

__host__ __device__ constexpr long long mx_tiles(long long n) { return (n + kMxTile - 1) / kMxTile; }

// Offset of the scale byte of (row, block) inside one matrix.
__host__ __device__ __forceinline__ size_t mx_scale_offset(long long row, int block, int k_tiles) {
  return ((size_t)(row / kMxTile) * k_tiles + block / 4) * kMxTileBytes +
         (size_t)((row % 32) * 16 + (row % kMxTile) / 32 * 4 + block % 4);
}

// Scale byte of a block whose largest magnitude has these float32 bits:
// floor(log2 amax) - 2, kept at or above -127, so that amax / 2^e is in
// [4, 8) (6 < x < 8 saturate to 6). Infinity or NaN in the block: 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t be = amax_bits >> 23;  // biased exponent, 0 for subnormals
  return be == 255u ? 255u : be > 2u ? be - 2u : 0u;
}

// 2^(127 - s), the factor that brings a block under its scale; 0 for s = 255
// (the codes of a NaN block are zeros). Exact: s <= 252 otherwise.
__device__ __forceinline__ float mx_inv_scale(uint32_t s) {
  return s == 255u ? 0.f : __uint_as_float((254u - s) << 23);
}

// 2^(s - 127); NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return s == 0u ? __uint_as_float(0x00400000u)
                 : s == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(s << 23);
}

// Eight floats to e2m1 (nearest, ties to even, beyond 6 to 6), v[0] in the
// lowest nibble. A NaN only reaches this under the factor 0 of a NaN block
// and becomes whatever finite code the conversion gives it.
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{ .reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3}; }"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Four floats to e2m1 in 16 bits.
__device__ __forceinline__ uint16_t mx_pack4(float v0, float v1, float v2, float v3) {
  uint16_t r;
  asm("{ .reg .b8 b0, b1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "mov.b16 %0, {b0, b1}; }"
      : "=h"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return r;
}

// The largest magnitude, NaN if any value is one.
__device__ __forceinline__ float max_abs4(float a, float b, float c, float d) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(fabsf(d)));
  return r;
}

// g / (1 + e^-g) * u for two values, within 2^-20.5 of it: the hardware's 2^t
// (2^-22) and 1 / x (2^-23), with what the product t = -g log2(e) and that constant
// round off, which grows with |g|, made up for by a factor. Above g = 200 e^-g is 0
// whatever t is; where it is beyond 2^126 (g < -87.3) the quotient is 0 (silu is
// above -2e-36 there). An infinite or NaN g makes the block NaN.
__device__ __forceinline__ Pair swiglu(Pair g, Pair u) {
  constexpr double kLog2eExact = 1.44269504088896341;
  constexpr float kLog2e = (float)kLog2eExact, kLog2eRest = (float)(kLog2eExact - kLog2e);
  constexpr float kLn2 = 0.693147180559945309f;
  Pair x;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x.x) : "f"(g.x), "f"(200.f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x.y) : "f"(g.y), "f"(200.f));
  const Pair t = x * Pair{-kLog2e, -kLog2e};
  const Pair rest = fma2(x, Pair{kLog2eRest, kLog2eRest}, fma2(x, Pair{kLog2e, kLog2e}, t));
  const Pair f = fma2(rest, Pair{-kLn2, -kLn2}, Pair{1.f, 1.f});
  Pair e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  const Pair d = fma2(e, f, Pair{1.f, 1.f});
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return g * r * u;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  return (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

// Sum of v over the lanes below this one.
__device__ __forceinline__ int exclusive_sum(int v) {
  const int lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  return incl - v;
}

// ------------------------------------------------- warp-uniform control ---
//
// The warps that issue copies and MMAs keep everything those instructions
// take (addresses, descriptors, coordinates) in uniform registers. That needs
// control flow and values that the compiler can see to be the same in all
// lanes: a branch on a vote, a value out of a warp reduction.

// A value all lanes hold, as a warp-uniform one.
__device__ __forceinline__ int uniform(int v) {
  return (int)__reduce_max_sync(0xffffffffu, (unsigned)v);
}

// mbar_wait for a whole converged warp. Bounded: after 64 failed polls (each
// suspends for a bounded time) the clock is read, which costs as much as a
// pipeline stage, and the limit of mbar_wait applies.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitLimitNs)) return false;
  }
}

// ------------------------------------------------ block-scaled tcgen05 ---

// `bytes` contiguous bytes (a multiple of 16, both sides 16-byte aligned)
// into shared memory, counted on mbarrier `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// A box of a 4-D byte tensor at coordinates (c0, 0, 0, c3).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0,
                                            int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(0), "r"(c3), "l"(policy)
      : "memory");
}

// 16 lanes x 32 columns of tensor memory: registers 4 g + 2 h + c of thread l
// hold lane l / 4 + 8 h, column 8 g + 2 (l % 4) + c.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Shared-memory descriptor of one 512-byte scale tile: rows of 16 bytes, no
// swizzle, 8-row groups 128 bytes apart (bits 32-45), version 1 (bit 46).
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

// One scale tile (32 rows of 16 bytes) into 4 columns of tensor memory,
// repeated in the four lane quarters. Ordered before the tcgen05.mma that
// the same thread issues after it.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

// D[tmem] (+)= (A * scales_a) (B * scales_b)^T over K = 64, e2m1 operands
// packed two to a byte, one e8m0 scale per 32 columns, fp32 accumulate.
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                          uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %6, 0;"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
      " [%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf4: e2m1 A and B (1 at bits 7-9 and
// 10-12), N >> 3 at 17-22, e8m0 scales (bit 23), M >> 7 at 27-28; and the byte
// pair of a scale column that the MMA reads (0 or 2), at 4-5 for B, 29-30 for A.
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 7) << 27);
}
__device__ __forceinline__ uint32_t idesc_mxf4_pair(uint32_t pair) {
  return (pair << 4) | (pair << 29);
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

}  // namespace mm
