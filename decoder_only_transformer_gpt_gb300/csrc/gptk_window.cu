// Entry points of sliding-window attention with sinks (include/gpt_kernels.h): argument checks, tensor maps, scratch.
#include "../../include/gpt_kernels.h"
#include "model.h"

#include <cuda_runtime.h>

using namespace gptgb;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int failed(const char* what, cudaError_t e) {
  cudaGetLastError();                                // reported here, and not again by the caller's next check
  set_detail(what, e);
  return e == cudaErrorMemoryAllocation ? GPT_ENOMEM : GPT_ECUDA;
}

int window_shape(int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t D, int32_t window, int32_t sinks) {
  if (B < 1 || T < 1 || H < 1 || Hkv < 1 || D < 1 || window < 1 || sinks < 0) return GPT_EINVAL;
  // the kernels number rows, heads and row elements with 32 bits
  if (T >= (1 << 30) || static_cast<int64_t>(B) * T > 0x7fffffffLL || static_cast<int64_t>(B) * H > 0x7fffffffLL ||
      (static_cast<int64_t>(H) + 2LL * Hkv) * D > 0x3fffffffLL)
    return GPT_EINVAL;
  if ((D != 32 && D != 64) || H % Hkv) return GPT_ECONFIG;
  return GPT_OK;
}

}  // namespace

extern "C" {

int gptk_attention_window(const void* qkv, void* y, float* lse2, int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t D,
                          int32_t window, int32_t sinks, void* stream) {
  if (!qkv || !y) return GPT_EINVAL;
  const int rc = window_shape(B, T, H, Hkv, D, window, sinks);
  if (rc != GPT_OK) return rc;
  if (!aligned16(qkv) || !aligned16(y)) return GPT_ECONFIG;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  CUtensorMap tm, tm_y;
  if (!make_tmap_qkv(&tm, qkv, B, T, (H + 2 * Hkv) * D, D) || !make_tmap_attn_out(&tm_y, y, B, T, H * D, D)) {
    set_detail_text("window attention tensor maps");
    return GPT_ECUDA;
  }
  const cudaError_t e = launch_attention_window_tc(tm, tm_y, B, T, H, Hkv, D, window, sinks, err, lse2,
                                                   reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GPT_OK : failed("window attention", e);
}

int gptk_attention_window_bwd(const void* qkv, const void* y, const void* dy, const float* lse2, void* dqkv, int32_t B,
                              int32_t T, int32_t H, int32_t Hkv, int32_t D, int32_t window, int32_t sinks, void* stream) {
  if (!qkv || !y || !dy || !lse2 || !dqkv) return GPT_EINVAL;
  const int rc = window_shape(B, T, H, Hkv, D, window, sinks);
  if (rc != GPT_OK) return rc;
  if (!aligned16(qkv) || !aligned16(y) || !aligned16(dy) || !aligned16(dqkv)) return GPT_ECONFIG;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int C = H * D, row = (H + 2 * Hkv) * D;
  const size_t M = static_cast<size_t>(B) * T;
  // scratch on the stream: the fp32 dQ accumulator, the rows' values, and the sums of key tiles that several CTAs share
  const size_t acc_b = (M * C * sizeof(float) + 255) / 256 * 256, row_b = attention_window_bwd_row_bytes(B, T, H);
  const size_t slab_b = attention_window_bwd_slab_bytes(B, T, H, Hkv, D, window, sinks);
  uint8_t* ws = nullptr;
  cudaError_t e = scratch_alloc(reinterpret_cast<void**>(&ws), acc_b + row_b + slab_b, s);
  if (e != cudaSuccess) return failed("window attention derivative scratch", e);
  float* dqacc = reinterpret_cast<float*>(ws);
  float* rows = reinterpret_cast<float*>(ws + acc_b);
  float* slabs = reinterpret_cast<float*>(ws + acc_b + row_b);
  CUtensorMap tq, tdy, tdkv, tdq;
  if (!(make_tmap_qkv(&tq, qkv, B, T, row, D) && make_tmap_qkv(&tdy, dy, B, T, C, D) &&
        make_tmap_attn_out(&tdkv, dqkv, B, T, row, D) && make_tmap_bt_f32(&tdq, dqacc, B, T, C))) {
    scratch_free(ws, s);
    set_detail_text("window attention derivative tensor maps");
    return GPT_ECUDA;
  }
  e = launch_attention_window_bwd_tc(tq, tdy, tdkv, tdq, y, dy, lse2, rows, dqacc, slabs, dqkv, B, T, H, Hkv, D, window, sinks,
                                     err, s);
  scratch_free(ws, s);
  return e == cudaSuccess ? GPT_OK : failed("window attention derivative", e);
}

}  // extern "C"
