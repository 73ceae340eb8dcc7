// The C ABI of include/mm.h, second part: routing from logits with its
// gradient, and the microscaled 4-bit operators. Argument checks and launch
// sequences only. Nothing here keeps a workspace: every call works in the
// memory its caller gives it, so calls (and captured graphs) with distinct
// workspaces never share any.
#include <algorithm>

#include "mm.h"
#include "mm_internal.h"
#include "mx_device.cuh"

namespace {

using namespace mm;

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MM_OK : MM_ERR_CUDA; }
inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

int check_logits(int dtype, int T, int E, int top_k) {
  if (T < 0 || E <= 0 || top_k <= 0) return MM_ERR_INVALID_ARG;
  if (dtype != MM_DTYPE_FP32 && dtype != MM_DTYPE_BF16)
    return dtype == MM_DTYPE_FP16 ? MM_ERR_UNSUPPORTED : MM_ERR_INVALID_ARG;
  if (E > kMaxExperts || top_k > kMaxTopK || top_k > E) return MM_ERR_UNSUPPORTED;
  if ((long long)T * top_k >= (1LL << 31)) return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

int check_mx(int batch, int rows, int K) {
  if (batch < 0 || rows < 0 || K <= 0) return MM_ERR_INVALID_ARG;
  if (K % kMxBlock != 0) return MM_ERR_UNSUPPORTED;
  // Row indices (of the padded scale rows too) and column indices are 32-bit.
  if ((long long)batch * mx_tiles(rows) * kMxTile > kMxMaxExtent || K > kMxMaxExtent)
    return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

bool is_dtype(int d) { return d == MM_DTYPE_FP32 || d == MM_DTYPE_BF16 || d == MM_DTYPE_FP16; }

// Workspace of the 4-bit experts.
struct ExpertsLayout {
  size_t counts, cursor, pos, xs, xs_scales, act, act_scales, y, total;
  long long capacity, max_chunks;
};

int experts_layout(int T, int H, int E, int I, int k, ExpertsLayout* out) {
  if (T < 0 || H <= 0 || E <= 0 || I <= 0 || k <= 0) return MM_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > kMaxTopK || k > E || H % 64 != 0 || I % 64 != 0)
    return MM_ERR_UNSUPPORTED;
  ExpertsLayout L;
  const long long Tk = (long long)T * k;
  const long long busy = std::min<long long>(E, Tk);  // segments that hold rows
  // Whole 128-row tiles: a segment is padded to them, and so is the buffer.
  L.capacity = Tk + busy * (kMxBlockM - 1);
  const long long rows = mx_tiles(L.capacity) * kMxTile;
  if (rows > kMxMaxExtent || 2LL * E * std::max(I, H) > kMxMaxExtent) return MM_ERR_UNSUPPORTED;
  L.max_chunks = busy + (Tk - busy) / kMxBlockM;
  if (L.max_chunks * ((std::max(I, H) + 127) / 128) >= (1LL << 31)) return MM_ERR_UNSUPPORTED;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += round256(bytes);
    return o;
  };
  L.counts = take((size_t)E * 4);
  L.cursor = take(Tk > kMxEarlyIds ? (size_t)E * kMxCursorStep * 4 : 0);  // else unused
  L.pos = take((size_t)Tk * 4);
  L.xs = take((size_t)rows * H / 2);
  L.xs_scales = take((size_t)(rows / kMxTile) * mx_tiles(H) * kMxTileBytes);
  L.act = take((size_t)rows * I / 2);
  L.act_scales = take((size_t)(rows / kMxTile) * mx_tiles(I) * kMxTileBytes);
  // One fp32 row a slot. Few slots in many segments: no less than two bytes a
  // value of every padded row and one for 32 values, which the reported size has
  // always counted.
  L.y = take(std::max((size_t)Tk * H * 4, (size_t)rows * (2 * (size_t)H + (H + 255) / 256 * 8)));
  L.total = off;
  *out = L;
  return MM_OK;
}

template <typename Tp>
Tp* at(void* base, size_t off) {
  return reinterpret_cast<Tp*>(static_cast<char*>(base) + off);
}

}  // namespace

extern "C" {

int64_t mm_route_logits_workspace_size(int T, int E) {
  if (check_logits(MM_DTYPE_FP32, T, E, 1) != MM_OK) return -1;
  return (int64_t)route_logits_workspace(T, E);
}

int mm_route_logits(const void* logits, int dtype, const uint8_t* token_mask, int T, int E,
                    int top_k, int renorm, int32_t* topk_ids, float* topk_w,
                    int32_t* expert_counts, float* prob_sums, float* loss, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int rc = check_logits(dtype, T, E, top_k);
  if (rc != MM_OK) return rc;
  if (!expert_counts || !prob_sums || !loss) return MM_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids || !topk_w)) return MM_ERR_INVALID_ARG;
  if (!aligned(logits, dtype == MM_DTYPE_FP32 ? 4 : 2) || !aligned(topk_ids, 4) ||
      !aligned(topk_w, 4) || !aligned(expert_counts, 4) || !aligned(prob_sums, 4) ||
      !aligned(loss, 4) || !aligned(workspace, 16))
    return MM_ERR_INVALID_ARG;
  const long long need = route_logits_workspace(T, E);
  if (need > 0 && !workspace) return MM_ERR_INVALID_ARG;
  if ((long long)workspace_bytes < need) return MM_ERR_NO_MEMORY;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_route_logits(logits, dtype == MM_DTYPE_BF16, token_mask, T, E, top_k,
                                         renorm, topk_ids, topk_w, expert_counts, prob_sums, loss,
                                         workspace, sms, static_cast<cudaStream_t>(stream)));
}

int mm_route_logits_backward(const void* logits, int dtype, const uint8_t* token_mask,
                             const int32_t* topk_ids, const int32_t* expert_counts,
                             const float* d_topk_w, const float* d_loss, int T, int E, int top_k,
                             int renorm, void* d_logits, void* stream) {
  int rc = check_logits(dtype, T, E, top_k);
  if (rc != MM_OK) return rc;
  if (T == 0) return MM_OK;  // nothing to read or write
  if (!logits || !topk_ids || !expert_counts || !d_logits) return MM_ERR_INVALID_ARG;
  const size_t el = dtype == MM_DTYPE_FP32 ? 4 : 2;
  if (!aligned(logits, el) || !aligned(d_logits, el) || !aligned(topk_ids, 4) ||
      !aligned(expert_counts, 4) || !aligned(d_topk_w, 4) || !aligned(d_loss, 4))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_route_logits_backward(
      logits, dtype == MM_DTYPE_BF16, token_mask, topk_ids, expert_counts, d_topk_w, d_loss, T, E,
      top_k, renorm, d_logits, sms, static_cast<cudaStream_t>(stream)));
}

int64_t mm_mxfp4_scales_size(int batch, int rows, int K) {
  if (check_mx(batch, rows, K) != MM_OK) return -1;
  return (int64_t)batch * mx_tiles(rows) * mx_tiles(K) * kMxTileBytes;
}

int mm_mxfp4_quantize(const void* x, int dtype, int batch, int rows, int K, uint8_t* codes,
                      uint8_t* scales, void* stream) {
  int rc = check_mx(batch, rows, K);
  if (rc != MM_OK) return rc;
  if (!is_dtype(dtype)) return MM_ERR_INVALID_ARG;
  if (batch == 0 || rows == 0) return MM_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_mx_quantize(x, dtype, batch, rows, K, codes, scales,
                                        static_cast<cudaStream_t>(stream)));
}

int mm_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int batch, int rows, int K,
                        void* out, int dtype, void* stream) {
  int rc = check_mx(batch, rows, K);
  if (rc != MM_OK) return rc;
  if (!is_dtype(dtype)) return MM_ERR_INVALID_ARG;
  if (batch == 0 || rows == 0) return MM_OK;
  if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_mx_dequantize(codes, scales, batch, rows, K, out, dtype,
                                          static_cast<cudaStream_t>(stream)));
}

int mm_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                  const uint8_t* b_scales, int M, int N, int K, void* c, int out_dtype,
                  void* stream) {
  int rc = check_mx(1, M, K);
  if (rc == MM_OK) rc = check_mx(1, N, K);
  if (rc != MM_OK) return rc;
  if (!is_dtype(out_dtype)) return MM_ERR_INVALID_ARG;
  if (out_dtype == MM_DTYPE_FP16) return MM_ERR_UNSUPPORTED;
  if (mx_tiles(M) * mx_tiles(N) >= (1LL << 31)) return MM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MM_OK;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !c) return MM_ERR_INVALID_ARG;
  if (!aligned(a_codes, 16) || !aligned(a_scales, 16) || !aligned(b_codes, 16) ||
      !aligned(b_scales, 16) || !aligned(c, 16))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_mx_gemm(a_codes, a_scales, b_codes, b_scales, M, N, K, c,
                                    out_dtype == MM_DTYPE_FP32, sms, status,
                                    static_cast<cudaStream_t>(stream)));
}

int64_t mm_moe_experts_mxfp4_workspace_size(int T, int H, int E, int I, int top_k) {
  ExpertsLayout L;
  return experts_layout(T, H, E, I, top_k, &L) == MM_OK ? (int64_t)L.total : -1;
}

int mm_moe_experts_mxfp4(const uint16_t* hidden, const int32_t* topk_ids, const float* topk_w,
                         const uint8_t* w_gate_up, const uint8_t* w_gate_up_scales,
                         const uint8_t* w_down, const uint8_t* w_down_scales, int T, int H, int E,
                         int I, int top_k, uint16_t* out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  ExpertsLayout L;
  int rc = experts_layout(T, H, E, I, top_k, &L);
  if (rc != MM_OK) return rc;
  if (T == 0) return MM_OK;  // nothing to read or write
  if (!hidden || !topk_ids || !topk_w || !w_gate_up || !w_gate_up_scales || !w_down ||
      !w_down_scales || !out || !workspace)
    return MM_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
      !aligned(w_gate_up, 16) || !aligned(w_gate_up_scales, 16) || !aligned(w_down, 16) ||
      !aligned(w_down_scales, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return MM_ERR_INVALID_ARG;
  if (workspace_bytes < L.total) return MM_ERR_NO_MEMORY;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t* counts = at<int32_t>(workspace, L.counts);
  uint8_t* xs = at<uint8_t>(workspace, L.xs);
  uint8_t* xs_scales = at<uint8_t>(workspace, L.xs_scales);
  uint8_t* act = at<uint8_t>(workspace, L.act);
  uint8_t* act_scales = at<uint8_t>(workspace, L.act_scales);
  int32_t* pos = at<int32_t>(workspace, L.pos);
  float* y = at<float>(workspace, L.y);
  const long long rows = mx_tiles(L.capacity) * kMxTile;
  cudaError_t e = launch_mx_place(hidden, topk_ids, T, top_k, E, H, counts,
                                  at<int32_t>(workspace, L.cursor), pos, xs, xs_scales,
                                  status, st);
  if (e == cudaSuccess)
    e = launch_mx_experts_gate_up(xs, xs_scales, w_gate_up, w_gate_up_scales, counts, topk_ids, T,
                                  top_k, E, I, H, rows, L.max_chunks, act, act_scales, sms, status, true, st);
  if (e == cudaSuccess)
    e = launch_mx_experts_down(act, act_scales, w_down, w_down_scales, counts, topk_ids, T,
                               top_k, E, H, I, rows, L.max_chunks, y, sms, status, true, st);
  if (e == cudaSuccess)
    e = launch_mx_combine(y, pos, topk_w, T, top_k, H, out, true, st);
  return cuda_status(e);
}

}  // extern "C"
