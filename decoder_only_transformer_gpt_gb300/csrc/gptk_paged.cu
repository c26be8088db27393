// Entry points of the paged key/value cache (include/gpt_kernels.h): argument checks, then the kernels of
// k_paged.cu. Everything that the host can check is refused before any device call; page numbers and lengths
// live on the device and are checked there (an access they would lead out of bounds is skipped and recorded).
#include "../../include/gpt_kernels.h"
#include "model.h"

#include <cuda_runtime.h>

using namespace gptgb;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The checks that every paged call shares. GPT_OK fills *c.
int paged_cache(PagedCache* c, const void* pool, const float* weight, const int32_t* table, int32_t B, int32_t Hkv,
                int32_t D, int32_t pages, int32_t page, int32_t max_pages) {
  if (!pool || !table || B < 1 || Hkv < 1 || D < 1 || pages < 1 || max_pages < 1) return GPT_EINVAL;
  if (page < 8 || page > 256 || (page & (page - 1))) return GPT_EINVAL;
  if (static_cast<int64_t>(max_pages) * page > kPagedMaxRows) return GPT_EINVAL;
  if (B > kPagedMaxB || Hkv > 65535) return GPT_EINVAL;
  if ((D != 32 && D != 64) || !aligned16(pool)) return GPT_ECONFIG;
  int lg = 0;
  while ((1 << lg) < page) ++lg;
  c->pool = const_cast<void*>(pool);
  c->weight = const_cast<float*>(weight);
  c->table = table;
  c->pages = pages;
  c->page_log2 = lg;
  c->max_pages = max_pages;
  c->Hkv = Hkv;
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

int gptk_paged_store(const void* qkv, void* pool, float* weight, const int32_t* table, const int32_t* start,
                     const int32_t* count, int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t D, int32_t pages,
                     int32_t page, int32_t max_pages, void* stream) {
  if (!qkv || T < 0 || H < 1) return GPT_EINVAL;
  PagedCache c;
  const int rc = paged_cache(&c, pool, weight, table, B, Hkv, D, pages, page, max_pages);
  if (rc != GPT_OK) return rc;
  if (H % Hkv || !aligned16(qkv)) return GPT_ECONFIG;
  if ((static_cast<int64_t>(H) + 2LL * Hkv) * D > 0x3fffffffLL) return GPT_EINVAL;   // a row's elements: 32 bits
  if (T == 0) return GPT_OK;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("paged store", launch_paged_store(c, qkv, start, count, B, T, H, D, err,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

int gptk_paged_attention(const void* qkv, void* pool, float* weight, const int32_t* table, const int32_t* lens, void* y,
                         float* lse2, int32_t B, int32_t H, int32_t Hkv, int32_t D, int32_t pages, int32_t page,
                         int32_t max_pages, int32_t window, int32_t sinks, void* stream) {
  if (!qkv || !lens || !y || H < 1 || window < 0 || sinks < 0) return GPT_EINVAL;
  PagedCache c;
  const int rc = paged_cache(&c, pool, weight, table, B, Hkv, D, pages, page, max_pages);
  if (rc != GPT_OK) return rc;
  if (H % Hkv || H / Hkv > kPagedMaxGroup || !aligned16(qkv) || !aligned16(y)) return GPT_ECONFIG;
  // the units of 32 rows are numbered with 32 bits, and with 64 over all heads
  const int64_t units = static_cast<int64_t>(B) * ((static_cast<int64_t>(max_pages) * page + 31) / 32);
  if (units > 0x7fffffffLL || units * Hkv > (1LL << 40)) return GPT_EINVAL;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("paged attention", launch_paged_attention(c, qkv, lens, y, lse2, B, H, D, window, sinks, err,
                                                          reinterpret_cast<cudaStream_t>(stream)));
}

int gptk_paged_evict(void* pool, float* weight, const int32_t* table, const int32_t* lens, const int32_t* dst_table,
                     int32_t* new_lens, int32_t* kept, int32_t B, int32_t Hkv, int32_t D, int32_t pages, int32_t page,
                     int32_t max_pages, int32_t dst_max_pages, int32_t budget, int32_t sinks, int32_t recent,
                     void* stream) {
  if (!weight || !lens || !dst_table || !new_lens || !kept || new_lens == lens) return GPT_EINVAL;
  if (dst_max_pages < 1 || budget < 1 || budget > kPagedMaxRows || sinks < 0 || recent < 0) return GPT_EINVAL;
  if (static_cast<int64_t>(sinks) + recent > budget) return GPT_EINVAL;
  PagedCache c;
  const int rc = paged_cache(&c, pool, weight, table, B, Hkv, D, pages, page, max_pages);
  if (rc != GPT_OK) return rc;
  if (static_cast<int64_t>(dst_max_pages) * page < budget) return GPT_EINVAL;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("paged evict", launch_paged_evict(c, lens, dst_table, dst_max_pages, new_lens, kept, B, D, budget, sinks,
                                                  recent, err, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
