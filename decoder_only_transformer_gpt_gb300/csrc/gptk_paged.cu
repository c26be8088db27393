// Entry points of the paged key/value caches and the position rotation (include/gpt_kernels.h): argument checks, then the
// kernels of k_paged.cu, k_append.cu and k_paged4.cu. Everything that the host can check is refused before any device call;
// page numbers and lengths live on the device and are checked there (an access they would lead out of bounds is skipped and
// recorded).
#include "../../include/gpt_kernels.h"
#include "model.h"

#include <cuda_runtime.h>

#include <cmath>

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

// Fused rows and their rotation. GPT_OK fills *x.
int rotary_rows(RotaryRows* x, const void* qkv, void* out, const int32_t* pos, const uint64_t* turns, int32_t B, int32_t T,
                int32_t H, int32_t Hkv, int32_t D, int32_t rot, int32_t interleaved, int32_t inverse) {
  if ((!qkv && T) || B < 1 || T < 0 || H < 1 || Hkv < 1 || D < 1 || rot < 0) return GPT_EINVAL;   // (no rows: no address)
  if (static_cast<int64_t>(B) * T > 0x7fffffffLL) return GPT_EINVAL;
  if ((static_cast<int64_t>(H) + 2LL * Hkv) * D > 0x3fffffffLL) return GPT_EINVAL;   // a row's elements: 32 bits
  if ((rot > 0) != (turns != nullptr) || (interleaved & ~1) || (inverse & ~1)) return GPT_EINVAL;
  if ((D != 32 && D != 64) || H % Hkv || rot % 16 || rot > D || !aligned16(qkv) || !aligned16(out)) return GPT_ECONFIG;
  if (reinterpret_cast<uintptr_t>(turns) & 7u) return GPT_ECONFIG;
  *x = {qkv, out, pos, turns, B, T, H, Hkv, D, rot, interleaved, inverse};
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

int gptk_rotary_turns(const double* freq, uint64_t* turns, int32_t n) {
  if (!freq || !turns || n < 0) return GPT_EINVAL;
  // 1 / (2 pi) in two doubles, and the product with the first in two as well: turns to about 2^-100 of themselves
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  for (int32_t i = 0; i < n; ++i) {
    const double f = freq[i];
    if (!(std::fabs(f) <= 1e12)) return GPT_EINVAL;
    const volatile double product = f * hi;          // rounded here, whatever the compiler would join it with
    const double p = product, e = std::fma(f, hi, -p) + f * lo;
    const double frac = p - std::trunc(p);           // exact; below a turn either way
    const uint64_t whole = static_cast<uint64_t>(std::nearbyint(std::ldexp(std::fabs(frac), 64)));
    const int64_t rest = static_cast<int64_t>(std::nearbyint(std::ldexp(e, 64)));   // |e| <= 2^-16 turns
    turns[i] = (frac < 0 ? 0 - whole : whole) + static_cast<uint64_t>(rest);
  }
  return GPT_OK;
}

int gptk_rotary(const void* qkv, void* out, const int32_t* pos, const uint64_t* turns, int32_t B, int32_t T, int32_t H,
                int32_t Hkv, int32_t D, int32_t rot, int32_t interleaved, int32_t inverse, void* stream) {
  if ((!out && T) || !turns) return GPT_EINVAL;
  RotaryRows x;
  const int rc = rotary_rows(&x, qkv, out, pos, turns, B, T, H, Hkv, D, rot, interleaved, inverse);
  if (rc != GPT_OK) return rc;
  if (T == 0) return GPT_OK;
  return finish("rotary", launch_rotary(x, reinterpret_cast<cudaStream_t>(stream)));
}

int gptk_paged_append(const void* qkv, void* out, void* pool, float* weight, const int32_t* table, const int32_t* start,
                      const int32_t* count, const int32_t* pos, const uint64_t* turns, int32_t B, int32_t T, int32_t H,
                      int32_t Hkv, int32_t D, int32_t rot, int32_t interleaved, int32_t pages, int32_t page,
                      int32_t max_pages, void* stream) {
  RotaryRows x;
  int rc = rotary_rows(&x, qkv, out, pos, turns, B, T, H, Hkv, D, rot, interleaved, 0);
  if (rc != GPT_OK) return rc;
  PagedCache c;
  rc = paged_cache(&c, pool, weight, table, B, Hkv, D, pages, page, max_pages);
  if (rc != GPT_OK) return rc;
  if (T == 0) return GPT_OK;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("paged append", launch_paged_append(c, x, start, count, err, reinterpret_cast<cudaStream_t>(stream)));
}

int gptk_paged_append4(const void* qkv, void* out, void* codes, void* ranges, const int32_t* table, const int32_t* start,
                       const int32_t* count, const int32_t* pos, const uint64_t* turns, int32_t B, int32_t T, int32_t H,
                       int32_t Hkv, int32_t D, int32_t rot, int32_t interleaved, int32_t pages, int32_t page,
                       int32_t max_pages, void* stream) {
  if (!ranges) return GPT_EINVAL;
  RotaryRows x;
  int rc = rotary_rows(&x, qkv, out, pos, turns, B, T, H, Hkv, D, rot, interleaved, 0);
  if (rc != GPT_OK) return rc;
  PagedCache c;
  rc = paged_cache(&c, codes, nullptr, table, B, Hkv, D, pages, page, max_pages);
  if (rc != GPT_OK) return rc;
  if (!aligned16(ranges)) return GPT_ECONFIG;
  if (T == 0) return GPT_OK;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("paged append in 4 bits",
                launch_paged_append4(c, ranges, x, start, count, err, reinterpret_cast<cudaStream_t>(stream)));
}

int gptk_paged_load4(const void* codes, const void* ranges, const int32_t* table, const int32_t* start,
                     const int32_t* count, void* rows, int32_t B, int32_t T, int32_t Hkv, int32_t D, int32_t pages,
                     int32_t page, int32_t max_pages, void* stream) {
  if (!ranges || (!rows && T) || T < 0 || static_cast<int64_t>(B) * T > 0x7fffffffLL) return GPT_EINVAL;
  PagedCache c;
  const int rc = paged_cache(&c, codes, nullptr, table, B, Hkv, D, pages, page, max_pages);
  if (rc != GPT_OK) return rc;
  if (!aligned16(ranges) || !aligned16(rows)) return GPT_ECONFIG;
  if (T == 0) return GPT_OK;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("paged load of 4 bits", launch_paged_load4(c, ranges, start, count, rows, B, T, D, err,
                                                           reinterpret_cast<cudaStream_t>(stream)));
}

int gptk_paged_attention4(const void* qkv, const void* codes, const void* ranges, const int32_t* table,
                          const int32_t* lens, void* y, float* lse2, int32_t B, int32_t H, int32_t Hkv, int32_t D,
                          int32_t pages, int32_t page, int32_t max_pages, int32_t window, int32_t sinks, int32_t added,
                          void* stream) {
  if (!qkv || !ranges || !lens || !y || H < 1 || window < 0 || sinks < 0 || added < 0) return GPT_EINVAL;
  PagedCache c;
  const int rc = paged_cache(&c, codes, nullptr, table, B, Hkv, D, pages, page, max_pages);
  if (rc != GPT_OK) return rc;
  if (added > static_cast<int64_t>(max_pages) * page) return GPT_EINVAL;
  if ((static_cast<int64_t>(H) + 2LL * Hkv) * D > 0x3fffffffLL) return GPT_EINVAL;
  if (H % Hkv || H / Hkv > kPagedMaxGroup || !aligned16(qkv) || !aligned16(y) || !aligned16(ranges)) return GPT_ECONFIG;
  // the units of 32 rows are numbered with 32 bits, and with 64 over all heads
  const int64_t units = static_cast<int64_t>(B) * ((static_cast<int64_t>(max_pages) * page + 31) / 32);
  if (units > 0x7fffffffLL || units * Hkv > (1LL << 40)) return GPT_EINVAL;
  int* err = step_err_word();
  if (!err) return GPT_ENOMEM;
  return finish("paged attention over 4 bits",
                launch_paged_attention4(c, ranges, qkv, lens, added, y, lse2, B, H, D, window, sinks, err,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
