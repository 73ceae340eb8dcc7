// The SwiGLU between the experts' products in training, and its backward pass
// from pre-activations that were kept in 8 bits.
//
//   pack      a = g sigma(g) u of z = (g, u); z stored as 8-bit integers
//   backward  from the stored z' and the gradient da of a, with a weight w a row:
//               dg = w da u sigma(g) (1 + g (1 - sigma(g))),  du = w da g sigma(g)
//               a' = w g sigma(g) u   (again: it was not kept)
//               dw = sum_i da_i g_i sigma(g_i) u_i
//
// The 8 bits (as MXINT8 of the OCP microscaling formats, whose byte is six more: it is
// that of 64 steps, this one of one): blocks of 32 columns under one power of two, values q 2^(s - 127), q in [-127, 127], s - 127
// = floor(log2 max|z|) - 6 but at least -127. The largest value is 64 to 128
// steps, so a value is off by at most half a step, 2^-7 of the block's largest; for
// normally distributed values 0.9 % of their norm. (Floats of 4 significant bits in
// the same bytes, e4m3, leave 2.9 %.) Only a value above 127.5 steps is cut to 127.
// The scaling is exact, so the one rounding is that to an integer. A block with an
// infinity or a NaN: s = 255, and all of it NaN.
//
// A group of 4 to 256 lanes takes a row, 8 columns a lane and step: a block of 32
// is four lanes, its largest magnitude two exchanges; the sum for dw runs over a
// lane's steps and then over the lanes and warps, the same on every call. The kernels
// read and write every byte once and are bound by memory: 32768 rows of 768 bf16 take 34
// us to pack (203 MB, 5.9 TB/s; 190 instructions a step of 16 values, the ALU 65 % busy),
// 41 backward (253 MB, 6.2 TB/s), 23 back to bf16 (6.5 TB/s); 512 rows 1.7, 2.3 and 1.8.
#include <algorithm>

#include <cuda_fp16.h>

#include "mm.h"
#include "mm_internal.h"
#include "mx_device.cuh"

namespace mm {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kSwThreads = 256;
constexpr int kSwWarps = kSwThreads / 32;

template <bool FP16>
__device__ __forceinline__ Pair unpack2(uint32_t w) {
  if (FP16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return {f.x, f.y};
  }
  return {__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(Pair v) {
  return pack16x2(v.x, v.y, FP16);
}

// Largest magnitude (float32 bits) of 8 values of 16 bits: compared as integers, which
// puts infinity and NaN on top.
template <bool FP16>
__device__ __forceinline__ uint32_t amax8(const uint4& r) {
  uint32_t m = __vmaxu2(__vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu),
                        __vmaxu2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu));
  m = max(m >> 16, m & 0xFFFFu);
  return FP16 ? __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) : m << 16;
}

// Scale byte of a block: floor(log2 amax) - 6 + 127, at least 0; 255 for infinity and NaN.
__device__ __forceinline__ uint32_t i8_scale_byte(uint32_t amax_bits) {
  const uint32_t be = amax_bits >> 23;  // 0 for zero and subnormals
  return be == 255u ? 255u : be > 6u ? be - 6u : 0u;
}

// v 2^(127 - s) to the nearest integer (ties to even) within +-127, in the low byte.
// Adding 1.5 2^23 leaves integers as the last bit; the product is exact.
__device__ __forceinline__ uint32_t i8_code(float v, float inv) {
  constexpr float kMagic = 12582912.f;
  const float r = __fmaf_rn(v, inv, kMagic);
  return __float_as_uint(fminf(fmaxf(r, kMagic - 127.f), kMagic + 127.f));
}

// The codes of 8 values.
__device__ __forceinline__ uint2 i8_codes(const Pair (&v)[4], uint32_t s) {
  const float inv = mx_inv_scale(s);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = __byte_perm(i8_code(v[2 * i].x, inv), i8_code(v[2 * i].y, inv), 0x0040);
    const uint32_t b =
        __byte_perm(i8_code(v[2 * i + 1].x, inv), i8_code(v[2 * i + 1].y, inv), 0x0040);
    w[i] = s == 255u ? 0u : __byte_perm(a, b, 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

// Four codes times `scale`. A code + 128 in the last bits of 2^23 is a float.
__device__ __forceinline__ void i8_values(uint32_t codes, float scale, Pair& a, Pair& b) {
  constexpr float kBase = 8388608.f + 128.f;
  codes ^= 0x80808080u;
  auto one = [&](uint32_t sel) { return __uint_as_float(__byte_perm(codes, 0x4B000000u, sel)); };
  const Pair m = {-kBase, -kBase}, s = {scale, scale};
  a = (Pair{one(0x7440), one(0x7441)} + m) * s;
  b = (Pair{one(0x7442), one(0x7443)} + m) * s;
}

// Rows in use: all, or up to the last segment's end.
__device__ __forceinline__ int rows_used(const int32_t* end, int R) {
  return end != nullptr ? min(__ldcg(end), R) : R;
}

// A group's lane and row. LPR: lanes of a row, a power of two.
struct Place {
  int row, lane;
};
__device__ __forceinline__ Place place_of(int lpr_log2) {
  Place p;
  p.lane = threadIdx.x & ((1 << lpr_log2) - 1);
  p.row = blockIdx.x * (kSwThreads >> lpr_log2) + (threadIdx.x >> lpr_log2);
  return p;
}

// sigma(g) within 2^-20.5, by the hardware's 2^t and 1 / x, with what the product
// t = -g log2(e) and that constant round off made up for by a factor. Beyond 200
// either way the exponential is 0 or infinite, and sigma 1 or 0, whatever g is. Where sigma
// is below 2^-126 (g under -87.3) it is 0: g sigma is above -2e-36 there.
__device__ __forceinline__ Pair sigmoid(Pair g) {
  constexpr double kLog2eExact = 1.44269504088896341;
  constexpr float kLog2e = (float)kLog2eExact, kLog2eRest = (float)(kLog2eExact - kLog2e);
  constexpr float kLn2 = 0.693147180559945309f;
  Pair x, e, s;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x.x) : "f"(g.x), "f"(200.f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x.y) : "f"(g.y), "f"(200.f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.x) : "f"(x.x), "f"(-200.f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.y) : "f"(x.y), "f"(-200.f));
  const Pair t = x * Pair{-kLog2e, -kLog2e};
  const Pair off = fma2(x, Pair{kLog2eRest, kLog2eRest}, fma2(x, Pair{kLog2e, kLog2e}, t));
  const Pair f = fma2(off, Pair{-kLn2, -kLn2}, Pair{1.f, 1.f});
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  const Pair d = fma2(e, f, Pair{1.f, 1.f});
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
  return s;
}

// U: steps whose loads are in flight together.
template <bool FP16, int U>
__global__ void __launch_bounds__(kSwThreads)
    swiglu_pack_kernel(const uint16_t* __restrict__ z, const int32_t* __restrict__ end, int R,
                       int I, int lpr_log2, uint16_t* __restrict__ act, int8_t* __restrict__ codes,
                       uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const Place p = place_of(lpr_log2);
  const int step = 8 << lpr_log2;
  const bool used = p.row < rows_used(end, R);
  const size_t zr = (size_t)p.row * (2 * I);
  for (int c0 = p.lane * 8; __any_sync(kAll, c0 < I && used); c0 += U * step) {
    uint4 g[U], u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + i * step;
      g[i] = u[i] = make_uint4(0u, 0u, 0u, 0u);
      if (used && c < I) {
        g[i] = __ldcs(reinterpret_cast<const uint4*>(z + zr + c));
        u[i] = __ldcs(reinterpret_cast<const uint4*>(z + zr + I + c));
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + i * step;
      uint32_t mg = amax8<FP16>(g[i]), mu = amax8<FP16>(u[i]);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mg = max(mg, __shfl_xor_sync(kAll, mg, o));
        mu = max(mu, __shfl_xor_sync(kAll, mu, o));
      }
      if (!used || c >= I) continue;
      const uint32_t sg = i8_scale_byte(mg), su = i8_scale_byte(mu);
      const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
      const uint32_t uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      Pair gv[4], uv[4];
      uint32_t a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        gv[j] = unpack2<FP16>(gw[j]);
        uv[j] = unpack2<FP16>(uw[j]);
        a[j] = pack2<FP16>(gv[j] * sigmoid(gv[j]) * uv[j]);
      }
      *reinterpret_cast<uint4*>(act + (size_t)p.row * I + c) = make_uint4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<uint2*>(codes + zr + c) = i8_codes(gv, sg);
      *reinterpret_cast<uint2*>(codes + zr + I + c) = i8_codes(uv, su);
      if ((c & 31) == 0) {
        uint8_t* s = scales + (size_t)p.row * (I / 16) + c / 32;
        s[0] = (uint8_t)sg;
        s[I / 32] = (uint8_t)su;
      }
    }
  }
}

// U: steps whose loads are in flight together, see unpack_as.
template <bool FP16, int U>
__global__ void __launch_bounds__(kSwThreads, U == 1 ? 6 : U == 2 ? 4 : 2)
    swiglu_unpack_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                         const uint16_t* __restrict__ da, const float* __restrict__ row_w,
                         const int32_t* __restrict__ end, int R, int I, int lpr_log2,
                         uint16_t* __restrict__ dz, uint16_t* __restrict__ act,
                         float* __restrict__ d_row_w) {
  pdl_wait();
  pdl_trigger();
  const Place p = place_of(lpr_log2);
  const int step = 8 << lpr_log2;
  const bool used = p.row < rows_used(end, R);
  const size_t zr = (size_t)p.row * (2 * I), ar = (size_t)p.row * I;
  const uint8_t* sr = scales + (size_t)p.row * (I / 16);
  const float w = used && row_w != nullptr ? __ldcg(row_w + p.row) : 1.f;
  const Pair ww = {w, w};
  float dot = 0.f;
  for (int c0 = p.lane * 8; used && c0 < I; c0 += U * step) {
    uint2 gs[U], us[U];
    uint4 ds[U];
    uint32_t sg[U], su[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + i * step;
      if (c < I) {
        gs[i] = __ldcs(reinterpret_cast<const uint2*>(codes + zr + c));
        us[i] = __ldcs(reinterpret_cast<const uint2*>(codes + zr + I + c));
        ds[i] = __ldcs(reinterpret_cast<const uint4*>(da + ar + c));
        sg[i] = __ldcg(sr + c / 32);
        su[i] = __ldcg(sr + I / 32 + c / 32);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + i * step;
      if (c >= I) break;
      const float fg = mx_scale(sg[i]), fu = mx_scale(su[i]);
      Pair gv[4], uv[4];
      i8_values(gs[i].x, fg, gv[0], gv[1]);
      i8_values(gs[i].y, fg, gv[2], gv[3]);
      i8_values(us[i].x, fu, uv[0], uv[1]);
      i8_values(us[i].y, fu, uv[2], uv[3]);
      const uint32_t dw[4] = {ds[i].x, ds[i].y, ds[i].z, ds[i].w};
      uint32_t og[4], ou[4], oa[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Pair dv = unpack2<FP16>(dw[j]);
        const Pair s = sigmoid(gv[j]);
        const Pair silu = gv[j] * s, a = silu * uv[j], wd = ww * dv;
        // sigma (1 + g (1 - sigma)); 1 - sigma is off by 2^-23 where it is small, which
        // the sum with 1 leaves at g 2^-23.
        const Pair slope =
            s * fma2(gv[j], fma2(s, Pair{-1.f, -1.f}, Pair{1.f, 1.f}), Pair{1.f, 1.f});
        dot = __fmaf_rn(dv.x, a.x, dot);
        dot = __fmaf_rn(dv.y, a.y, dot);
        og[j] = pack2<FP16>(wd * uv[j] * slope);
        ou[j] = pack2<FP16>(wd * silu);
        oa[j] = pack2<FP16>(ww * a);
      }
      *reinterpret_cast<uint4*>(dz + zr + c) = make_uint4(og[0], og[1], og[2], og[3]);
      *reinterpret_cast<uint4*>(dz + zr + I + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
      *reinterpret_cast<uint4*>(act + ar + c) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    }
  }
  if (d_row_w != nullptr) {
    for (int o = min(1 << lpr_log2, 32) >> 1; o > 0; o >>= 1)
      dot += __shfl_xor_sync(kAll, dot, o);
    if (lpr_log2 > 5) {  // a row over several warps
      __shared__ float dot_s[kSwWarps];
      if ((threadIdx.x & 31) == 0) dot_s[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (p.lane == 0)
        for (int w = 1; w < 1 << (lpr_log2 - 5); ++w) dot += dot_s[(threadIdx.x >> 5) + w];
    }
    if (used && p.lane == 0) d_row_w[p.row] = dot;
  }
}

// 16 values a thread. DT: MM_DTYPE of the result.
template <int DT>
__global__ void __launch_bounds__(kSwThreads)
    i8_dequantize_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                         long long n16, void* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const long long i = (long long)blockIdx.x * kSwThreads + threadIdx.x;
  if (i >= n16) return;
  const uint4 q = __ldcs(reinterpret_cast<const uint4*>(codes) + i);
  const float f = mx_scale(__ldcg(scales + i / 2));
  Pair v[8];
  i8_values(q.x, f, v[0], v[1]);
  i8_values(q.y, f, v[2], v[3]);
  i8_values(q.z, f, v[4], v[5]);
  i8_values(q.w, f, v[6], v[7]);
  if (DT == MM_DTYPE_FP32) {
    float4* o = static_cast<float4*>(out) + 4 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
  } else {
    uint4* o = static_cast<uint4*>(out) + 2 * i;
    constexpr bool h = DT == MM_DTYPE_FP16;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o[j] = make_uint4(pack2<h>(v[4 * j]), pack2<h>(v[4 * j + 1]), pack2<h>(v[4 * j + 2]),
                        pack2<h>(v[4 * j + 3]));
  }
}

struct Shape {
  int lpr_log2, u;
  unsigned blocks;
};

// The lanes of a row: a power of two that covers it in one step, at most 32; 16 instead
// where that leaves fewer of them idle in the last step and the rows are many (352
// columns, 44 lanes' worth: three steps of 16 lanes, where 32 idle in 20 of 64 places).
// Up to the whole block where the rows are so few that `per_sm` blocks an SM hold them (us,
// pack and back: 512 x 768 2.1 -> 1.7 and 3.1 -> 2.3, 200 x 2048 4.4 -> 1.8 and 6.0 -> 2.4,
// 1 x 768 1.6 -> 1.1 and 2.5 -> 1.7): four for pack, two for back (with two and four,
// pack of 1000 x 2048 5.4 and 4.6, back of 1000 x 768 2.9 and 3.4).
Shape shape_of(int R, int I, int per_sm) {
  Shape s = {};
  const int n = I / 8;
  s.lpr_log2 = 2;
  while (s.lpr_log2 < 5 && (1 << s.lpr_log2) < n) ++s.lpr_log2;
  if (s.lpr_log2 == 5 && (n + 15) / 16 * 16 < (n + 31) / 32 * 32 && R >= 8192) s.lpr_log2 = 4;
  while (s.lpr_log2 >= 5 && 1 << s.lpr_log2 < std::min(n, kSwThreads) &&
         (long long)R << (s.lpr_log2 + 1) <= per_sm * 152 * kSwThreads)
    ++s.lpr_log2;
  s.u = std::min((n + (1 << s.lpr_log2) - 1) >> s.lpr_log2, 3);
  const int rows = kSwThreads >> s.lpr_log2;
  s.blocks = (unsigned)(((long long)R + rows - 1) / rows);
  return s;
}

template <bool FP16>
cudaError_t pack_as(const uint16_t* z, const int32_t* end, int R, int I, uint16_t* act,
                    int8_t* codes, uint8_t* scales, cudaStream_t st) {
  const Shape s = shape_of(R, I, 4);
  auto k = s.u == 1 ? swiglu_pack_kernel<FP16, 1>
         : s.u == 2 ? swiglu_pack_kernel<FP16, 2> : swiglu_pack_kernel<FP16, 3>;
  return launch_k(k, dim3(s.blocks), dim3(kSwThreads), 0, st, true, z, end, R, I, s.lpr_log2, act,
                  codes, scales);
}

template <bool FP16>
cudaError_t unpack_as(const int8_t* codes, const uint8_t* scales, const uint16_t* da,
                      const float* row_w, const int32_t* end, int R, int I, uint16_t* dz,
                      uint16_t* act, float* d_row_w, cudaStream_t st) {
  const Shape s = shape_of(R, I, 2);
  // Many rows want warps rather than loads a warp: 32768 x 768 take 40.6 us with six blocks
  // an SM and one step at a time, 44.5 with four and two, 52 with two and three. Where all
  // blocks are under way at once the loads count: two blocks an SM take as many steps as
  // fit (304 blocks of 768 columns 3.5 us, one at a time 4.0). Three leave room for three of
  // the next call's at one step, and none at two (456 blocks 5.1 and 6.2). Four take two
  // steps, which fill the SM, and so do up to 76 blocks more: a second round on half the
  // SMs takes less than one step at a time loses. One step and two, in us, by blocks:
  //                  480          608          626          650          684          720
  //     352 columns  5.33  4.31   5.44  4.31   5.44  5.03   5.35  5.03   5.25  5.12   5.44  5.23
  //     768          7.84  6.35   8.15  6.79   8.29  8.21   8.29  8.35   8.42  8.62   8.50  8.86
  //    1056         12.07  9.52  12.39  9.79  12.43 11.62  12.49 11.76  12.60 11.91  12.77 12.57
  //    2048         18.76 14.03  19.06 14.61  19.17 18.04  19.26 18.54  19.25 19.49  19.19 20.80
  const int per_sm = (int)((s.blocks + 151) / 152);
  const int u = per_sm <= 2 ? s.u : s.u > 1 && per_sm > 3 && s.blocks <= 4 * 152 + 76 ? 2 : 1;
  auto k = u == 1 ? swiglu_unpack_kernel<FP16, 1>
         : u == 2 ? swiglu_unpack_kernel<FP16, 2> : swiglu_unpack_kernel<FP16, 3>;
  return launch_k(k, dim3(s.blocks), dim3(kSwThreads), 0, st, true, codes, scales, da, row_w, end,
                  R, I, s.lpr_log2, dz, act, d_row_w);
}

}  // namespace

cudaError_t launch_swiglu_pack(const uint16_t* z, bool fp16, const int32_t* end, int R, int I,
                               uint16_t* act, int8_t* codes, uint8_t* scales, cudaStream_t st) {
  return fp16 ? pack_as<true>(z, end, R, I, act, codes, scales, st)
              : pack_as<false>(z, end, R, I, act, codes, scales, st);
}

cudaError_t launch_swiglu_pack_backward(const int8_t* codes, const uint8_t* scales,
                                        const uint16_t* da, bool fp16, const float* row_w,
                                        const int32_t* end, int R, int I, uint16_t* dz,
                                        uint16_t* act, float* d_row_w, cudaStream_t st) {
  return fp16 ? unpack_as<true>(codes, scales, da, row_w, end, R, I, dz, act, d_row_w, st)
              : unpack_as<false>(codes, scales, da, row_w, end, R, I, dz, act, d_row_w, st);
}

cudaError_t launch_i8_dequantize(const int8_t* codes, const uint8_t* scales, long long n,
                                 void* out, int dtype, cudaStream_t st) {
  const long long n16 = n / 16;
  auto k = dtype == MM_DTYPE_FP32   ? i8_dequantize_kernel<MM_DTYPE_FP32>
           : dtype == MM_DTYPE_BF16 ? i8_dequantize_kernel<MM_DTYPE_BF16>
                                    : i8_dequantize_kernel<MM_DTYPE_FP16>;
  return launch_k(k, dim3((unsigned)((n16 + kSwThreads - 1) / kSwThreads)), dim3(kSwThreads), 0, st,
                  true, codes, scales, n16, out);
}

}  // namespace mm
