// Entry points of the log probabilities (include/gpt_kernels.h): argument checks, then the kernels of k_logprobs.cu.
#include "../../include/gpt_kernels.h"
#include "model.h"

#include <cuda_runtime.h>

using namespace gptgb;

namespace {

int logprob_rows(LogprobRows* x, const void* logits, const int32_t* targets, int32_t M, int32_t V, int64_t ld,
                 int32_t dtype) {
  if (!logits || M < 1 || V < 1 || ld < V || (dtype & ~1)) return GPT_EINVAL;
  if (M > 0x7fffffff / 8 || V > 0x7fffffff - 65536) return GPT_EINVAL;      // the kernels' block and value numbers: 32 bits
  if (ld > (1LL << 60) / M) return GPT_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) & (dtype ? 1u : 3u)) return GPT_ECONFIG;
  *x = {logits, targets, M, V, ld, dtype};
  return GPT_OK;
}

int finish(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return GPT_OK;
  cudaGetLastError();                                // reported here, and not again by the caller's next check
  set_detail(what, e);
  return e == cudaErrorMemoryAllocation ? GPT_ENOMEM : GPT_ECUDA;
}

}  // namespace

extern "C" {

int gptk_logprobs(const void* logits, const int32_t* targets, float* logp, float* entropy, float* stats, int32_t* top_ids,
                  float* top_logp, int32_t M, int32_t V, int64_t ld, int32_t K, int32_t dtype, void* stream) {
  LogprobRows x;
  const int rc = logprob_rows(&x, logits, targets, M, V, ld, dtype);
  if (rc != GPT_OK) return rc;
  if ((targets != nullptr) != (logp != nullptr)) return GPT_EINVAL;
  if (K < 0 || K > 32 || K > V || (K > 0) != (top_ids != nullptr) || (K > 0) != (top_logp != nullptr)) return GPT_EINVAL;
  if (!logp && !entropy && !stats && !top_ids) return GPT_EINVAL;
  if (reinterpret_cast<uintptr_t>(stats) & 7u) return GPT_ECONFIG;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("log probabilities", launch_logprobs(x, logp, entropy, stats, top_ids, top_logp, K, err,
                                                     reinterpret_cast<cudaStream_t>(stream)));
}

int gptk_logprobs_bwd(const void* logits, const int32_t* targets, const float* stats, const float* entropy,
                      const float* dlogp, const float* dentropy, void* dlogits, int32_t M, int32_t V, int64_t ld,
                      int64_t dld, int32_t dtype, void* stream) {
  LogprobRows x;
  const int rc = logprob_rows(&x, logits, targets, M, V, ld, dtype);
  if (rc != GPT_OK) return rc;
  if (!stats || !dlogits || dld < V || dld > (1LL << 60) / M) return GPT_EINVAL;
  if ((targets != nullptr) != (dlogp != nullptr) || (entropy != nullptr) != (dentropy != nullptr)) return GPT_EINVAL;
  if (!dlogp && !dentropy) return GPT_EINVAL;
  if (dlogits == logits && dld != ld) return GPT_EINVAL;
  if ((reinterpret_cast<uintptr_t>(dlogits) & (dtype ? 1u : 3u)) || (reinterpret_cast<uintptr_t>(stats) & 7u)) return GPT_ECONFIG;
  return finish("gradient of log probabilities", launch_logprobs_bwd(x, stats, entropy, dlogp, dentropy, dlogits, dld,
                                                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
