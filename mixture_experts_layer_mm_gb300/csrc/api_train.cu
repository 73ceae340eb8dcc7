// The C ABI of include/mm.h, third part: the operators that train the routed
// experts. Argument checks and launches only; every call works in the memory its
// caller gives it.
#include "mm.h"
#include "mm_internal.h"

namespace {

using namespace mm;

constexpr int kMaxRows = (int)((1LL << 31) - 4096);  // loops step past the end by less
constexpr int kMaxCols = 1 << 20;

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MM_OK : MM_ERR_CUDA; }
inline cudaStream_t on(void* stream) { return static_cast<cudaStream_t>(stream); }

// Types of rows: bf16 and fp16.
int check_dtype(int d) {
  if (d == MM_DTYPE_BF16 || d == MM_DTYPE_FP16) return MM_OK;
  return d == MM_DTYPE_FP32 ? MM_ERR_UNSUPPORTED : MM_ERR_INVALID_ARG;
}

int check_slots(int T, int top_k) {
  if (T < 0 || top_k <= 0) return MM_ERR_INVALID_ARG;
  if (top_k > kMaxTopK || (long long)T * top_k >= (1LL << 31)) return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

int check_rows(int T, int top_k, int H, int R) {
  if (H <= 0 || R < 0) return MM_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > kMaxCols) return MM_ERR_UNSUPPORTED;
  return check_slots(T, top_k);
}

int check_product(int dtype, int R, int E, int N, int K) {
  if (R < 0 || E <= 0 || N <= 0 || K <= 0) return MM_ERR_INVALID_ARG;
  if (const int rc = check_dtype(dtype); rc != MM_OK) return rc;
  if (E > kMaxExperts || N % 8 != 0 || K % 8 != 0 || N > kMaxCols || K > kMaxCols || R >= kMaxRows)
    return MM_ERR_UNSUPPORTED;
  // A matrix's bytes are a 40-bit stride of the copies; tiles are counted in 31 bits, and
  // loops step past the end by the clusters of a chip.
  if ((long long)N * K >= (1LL << 37)) return MM_ERR_UNSUPPORTED;
  const long long m = (N > K ? N : K) / 256 + 1;
  if ((R / 256LL + E) * m >= kMaxRows || E * (N / 256 + 1LL) * (K / 128 + 1LL) >= kMaxRows)
    return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

int check_swiglu(int R, int C) {
  if (R < 0 || C <= 0) return MM_ERR_INVALID_ARG;
  // (the product: blocks of 4096 values in a grid's 31 bits)
  if (C % 32 != 0 || C > kMaxCols || R > kMaxRows || (long long)R * C >= (1LL << 42))
    return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

}  // namespace

extern "C" {

int64_t mm_group_slots_workspace_size(int T, int top_k, int E) {
  if (check_slots(T, top_k) != MM_OK || E <= 0 || E > kMaxExperts) return -1;
  return (int64_t)group_slots_workspace((long long)T * top_k, E);
}

int mm_group_slots(const int32_t* topk_ids, const uint8_t* token_mask, int T, int top_k, int E,
                   int32_t* places, int32_t* offsets, void* workspace, size_t workspace_bytes,
                   void* stream) {
  int rc = check_slots(T, top_k);
  if (rc == MM_OK && E <= 0) rc = MM_ERR_INVALID_ARG;
  if (rc == MM_OK && E > kMaxExperts) rc = MM_ERR_UNSUPPORTED;
  if (rc != MM_OK) return rc;
  if (!offsets || (T > 0 && (!topk_ids || !places))) return MM_ERR_INVALID_ARG;
  if (!aligned(topk_ids, 4) || !aligned(places, 4) || !aligned(offsets, 4) ||
      !aligned(workspace, 16))
    return MM_ERR_INVALID_ARG;
  const long long need = group_slots_workspace((long long)T * top_k, E);
  if (need > 0 && !workspace) return MM_ERR_INVALID_ARG;
  if ((long long)workspace_bytes < need) return MM_ERR_NO_MEMORY;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_group_slots(topk_ids, token_mask, T, top_k, E, places, offsets,
                                        workspace, status, on(stream)));
}

int mm_dispatch_rows(const void* x, int dtype, const int32_t* places, const float* topk_w, int T,
                     int top_k, int H, int R, void* rows, float* row_w, void* stream) {
  int rc = check_rows(T, top_k, H, R);
  if (rc == MM_OK) rc = check_dtype(dtype);
  if (rc != MM_OK) return rc;
  if ((topk_w == nullptr) != (row_w == nullptr)) return MM_ERR_INVALID_ARG;
  if (T == 0) return MM_OK;
  if (!x || !places || (R > 0 && !rows) || !aligned(x, 16) || !aligned(rows, 16) ||
      !aligned(places, 4) || !aligned(topk_w, 4) || !aligned(row_w, 4))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(
      launch_dispatch_rows(x, places, topk_w, T, top_k, H, R, rows, row_w, status, on(stream)));
}

int mm_combine_rows(const void* rows, int dtype, const int32_t* places, const float* topk_w,
                    const float* row_values, int T, int top_k, int H, int R, void* out,
                    float* values, void* stream) {
  int rc = check_rows(T, top_k, H, R);
  if (rc == MM_OK) rc = check_dtype(dtype);
  if (rc != MM_OK) return rc;
  if (T == 0) return MM_OK;
  if (values != nullptr ? R > 0 && !row_values : row_values != nullptr) return MM_ERR_INVALID_ARG;
  if ((R > 0 && !rows) || !places || !out || !aligned(rows, 16) || !aligned(out, 16) ||
      !aligned(places, 4) || !aligned(topk_w, 4) || !aligned(row_values, 4) || !aligned(values, 4))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_combine_rows(rows, dtype == MM_DTYPE_FP16, places, topk_w, row_values,
                                         T, top_k, H, R, out, values, status, on(stream)));
}

static int product(bool transposed, const void* x, const void* w, int dtype,
                   const int32_t* offsets, int R, int E, int N, int K, void* out, void* stream) {
  int rc = check_product(dtype, R, E, N, K);
  if (rc != MM_OK) return rc;
  if (R == 0) return MM_OK;
  if (!x || !w || !offsets || !out || !aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) ||
      !aligned(offsets, 4))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_grouped_product(transposed, x, w, offsets, R, E, N, K,
                                            dtype == MM_DTYPE_FP16, out, sms, status, on(stream)));
}

int mm_grouped_product(const void* x, const void* w, int dtype, const int32_t* offsets, int R,
                       int E, int N, int K, void* y, void* stream) {
  return product(false, x, w, dtype, offsets, R, E, N, K, y, stream);
}

int mm_grouped_product_dx(const void* dy, const void* w, int dtype, const int32_t* offsets, int R,
                          int E, int N, int K, void* dx, void* stream) {
  return product(true, dy, w, dtype, offsets, R, E, N, K, dx, stream);
}

int64_t mm_grouped_product_dw_workspace_size(int R, int E, int N, int K, int dw_dtype) {
  if (check_product(MM_DTYPE_BF16, R, E, N, K) != MM_OK ||
      (dw_dtype != MM_DTYPE_FP32 && check_dtype(dw_dtype) != MM_OK))
    return -1;
  return R == 0 ? 0 : (int64_t)grouped_product_dw_workspace(R, E, N, K, dw_dtype == MM_DTYPE_FP32);
}

int mm_grouped_product_dw(const void* dy, const void* x, int dtype, const int32_t* offsets, int R,
                          int E, int N, int K, void* dw, int dw_dtype, int accumulate,
                          void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_product(dtype, R, E, N, K);
  if (rc != MM_OK) return rc;
  if (dw_dtype != MM_DTYPE_FP32 && dw_dtype != dtype)
    return check_dtype(dw_dtype) == MM_OK ? MM_ERR_UNSUPPORTED : MM_ERR_INVALID_ARG;
  if (!dw || !aligned(dw, 16)) return MM_ERR_INVALID_ARG;
  if (R > 0 && (!dy || !x || !offsets || !aligned(dy, 16) || !aligned(x, 16) ||
                !aligned(offsets, 4)))
    return MM_ERR_INVALID_ARG;
  if (R == 0) {
    if (accumulate) return MM_OK;
    const size_t bytes = (size_t)E * N * K * (dw_dtype == MM_DTYPE_FP32 ? 4 : 2);
    return cuda_status(cudaMemsetAsync(dw, 0, bytes, on(stream)));
  }
  const long long need = grouped_product_dw_workspace(R, E, N, K, dw_dtype == MM_DTYPE_FP32);
  if (!aligned(workspace, 16) || (need > 0 && !workspace)) return MM_ERR_INVALID_ARG;
  if ((long long)workspace_bytes < need) return MM_ERR_NO_MEMORY;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_grouped_product_dw(
      dy, x, offsets, R, E, N, K, dtype == MM_DTYPE_FP16, dw, dw_dtype == MM_DTYPE_FP32,
      accumulate != 0, workspace, sms, status, on(stream)));
}

int mm_swiglu_pack(const void* z, int dtype, const int32_t* rows_used, int R, int I, void* act,
                   int8_t* codes, uint8_t* scales, void* stream) {
  int rc = check_swiglu(R, I);
  if (rc == MM_OK && I > kMaxCols / 2) rc = MM_ERR_UNSUPPORTED;
  if (rc == MM_OK) rc = check_dtype(dtype);
  if (rc != MM_OK) return rc;
  if (R == 0) return MM_OK;
  if (!z || !act || !codes || !scales || !aligned(z, 16) || !aligned(act, 16) ||
      !aligned(codes, 16) || !aligned(rows_used, 4))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_swiglu_pack(static_cast<const uint16_t*>(z), dtype == MM_DTYPE_FP16,
                                        rows_used, R, I, static_cast<uint16_t*>(act), codes,
                                        scales, on(stream)));
}

int mm_swiglu_pack_backward(const int8_t* codes, const uint8_t* scales, const void* d_act,
                            int dtype, const float* row_w, const int32_t* rows_used, int R, int I,
                            void* dz, void* act, float* d_row_w, void* stream) {
  int rc = check_swiglu(R, I);
  if (rc == MM_OK && I > kMaxCols / 2) rc = MM_ERR_UNSUPPORTED;
  if (rc == MM_OK) rc = check_dtype(dtype);
  if (rc != MM_OK) return rc;
  if (R == 0) return MM_OK;
  if (!codes || !scales || !d_act || !dz || !act || !aligned(codes, 16) || !aligned(d_act, 16) ||
      !aligned(dz, 16) || !aligned(act, 16) || !aligned(row_w, 4) || !aligned(d_row_w, 4) ||
      !aligned(rows_used, 4))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_swiglu_pack_backward(
      codes, scales, static_cast<const uint16_t*>(d_act), dtype == MM_DTYPE_FP16, row_w, rows_used,
      R, I, static_cast<uint16_t*>(dz), static_cast<uint16_t*>(act), d_row_w, on(stream)));
}

int mm_mxint8_dequantize(const int8_t* codes, const uint8_t* scales, int rows, int K, void* out,
                         int dtype, void* stream) {
  int rc = check_swiglu(rows, K);
  if (rc != MM_OK) return rc;
  if (dtype != MM_DTYPE_FP32 && check_dtype(dtype) != MM_OK) return MM_ERR_INVALID_ARG;
  if (rows == 0) return MM_OK;
  if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(out, 16))
    return MM_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* status = nullptr;
  if ((rc = current_device_info(&sms, &status)) != MM_OK) return rc;
  return cuda_status(launch_i8_dequantize(codes, scales, (long long)rows * K, out, dtype,
                                          on(stream)));
}

}  // extern "C"
