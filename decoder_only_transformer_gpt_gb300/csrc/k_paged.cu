// Paged key/value cache: storing rows, attention of one new token per sequence, eviction by summed weight.
//
// The cache is a pool of pages shared by all sequences, bf16 [pages][2][Hkv][page][D]: within a page the rows
// of one key head are contiguous (page * D * 2 bytes of keys, and the same of values), so a head's reader
// streams whole pages instead of one row out of every token's. Row r of sequence b lies in page
// table[b][r >> page_log2] at slot r & (page - 1). H query heads share Hkv key heads, G = H / Hkv each.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

#include <math.h>

namespace gptgb {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// The page of row r of sequence b, or -1 (recorded) when the table names a page outside the pool.
__device__ __forceinline__ int page_of(const PagedCache& c, const int32_t* trow, int r, int* err) {
  const int pg = __ldg(trow + (r >> c.page_log2));
  if (static_cast<unsigned>(pg) < static_cast<unsigned>(c.pages)) return pg;
  record_error(err, GPT_DEV_EPAGE);
  return -1;
}

// Offset (in rows of D elements) of a page's row for key head h; which = 0 keys, 1 values.
__device__ __forceinline__ size_t row_at(const PagedCache& c, int pg, int which, int h, int slot) {
  return ((((static_cast<size_t>(pg) * 2 + which) * c.Hkv + h) << c.page_log2) + slot);
}

__device__ __forceinline__ size_t weight_at(const PagedCache& c, int pg, int h, int slot) {
  return ((static_cast<size_t>(pg) * c.Hkv + h) << c.page_log2) + slot;
}

// The newest query (row n - 1) sees row r if r < sinks or n - 1 - r < window (window 0: every row).
// Seen rows in order are v = 0 .. seen_rows - 1: v < head ones at the start, then from `gap` rows on.
struct Seen {
  int head, gap, n;
};
__device__ __forceinline__ Seen seen_rows(int n, int window, int sinks) {
  Seen s;
  s.head = n;
  s.gap = 0;
  s.n = n;
  if (window > 0 && window < n) {
    const int first = n - window;                    // first row of the window
    s.head = min(sinks, first);
    s.gap = first - s.head;
    s.n = window + s.head;
  }
  return s;
}
__device__ __forceinline__ int seen_row(const Seen& s, int v) { return v < s.head ? v : v + s.gap; }

// ---------------------------------------------------------------- store

// One thread per 16 bytes of a token's keys and values. Bound by memory: 8 D bytes moved per row and key head.
template <int D>
__global__ void __launch_bounds__(256)
paged_store_kernel(PagedCache c, const uint4* __restrict__ qkv, const int32_t* __restrict__ start,
                   const int32_t* __restrict__ count, int T, int H, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int U = D / 8;                           // 16-byte units of a row
  const int b = blockIdx.y;
  const int per_tok = 2 * c.Hkv * U;
  const int n = count ? min(__ldg(count + b), T) : T;
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<long long>(n) * per_tok) return;
  const int t = static_cast<int>(i / per_tok), e = static_cast<int>(i - static_cast<long long>(t) * per_tok);
  const int which = e / (c.Hkv * U), h = (e / U) % c.Hkv, u = e % U;
  const long long r = (start ? static_cast<long long>(__ldg(start + b)) : 0) + t;
  if (r < 0 || r >= static_cast<long long>(c.max_pages) << c.page_log2) {
    record_error(err, GPT_DEV_EPAGE);
    return;
  }
  const int pg = page_of(c, c.table + static_cast<size_t>(b) * c.max_pages, static_cast<int>(r), err);
  if (pg < 0) return;
  const int slot = static_cast<int>(r) & ((1 << c.page_log2) - 1);
  const uint4 v = __ldg(qkv + (static_cast<size_t>(b) * T + t) * (H + 2 * c.Hkv) * U + H * U + e);
  reinterpret_cast<uint4*>(c.pool)[row_at(c, pg, which, h, slot) * U + u] = v;
  if (c.weight && which == 0 && u == 0) c.weight[weight_at(c, pg, h, slot)] = 0.0f;
}

// ---------------------------------------------------------------- attention of one new token

// One block per (key head, sequence); its G query heads one after the other. Warp w takes 32-row chunks
// w, w + 8, ..: lane = row for the scores, lane = D / 32 columns for the values; running maximum and sum per
// warp, warps merged in a fixed order. A last pass adds the weights (scores once more).
constexpr int kDecWarps = 8;

template <int D>
__global__ void __launch_bounds__(kDecWarps * 32)
paged_attention_kernel(PagedCache c, const __nv_bfloat16* __restrict__ qkv, const int32_t* __restrict__ lens,
                       __nv_bfloat16* __restrict__ y, float* __restrict__ lse2, int H, int window, int sinks,
                       float scale_log2, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int CPL = D / 32;
  __shared__ float sq[D];
  __shared__ float sm[kDecWarps], sl[kDecWarps], so[kDecWarps][D];
  const int h = blockIdx.x, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = H / c.Hkv;
  const int last = __ldg(lens + b);
  if (last < 0) return;
  if (last >= static_cast<long long>(c.max_pages) << c.page_log2) {
    if (threadIdx.x == 0) record_error(err, GPT_DEV_EPAGE);
    return;
  }
  const int pmask = (1 << c.page_log2) - 1;
  const int32_t* trow = c.table + static_cast<size_t>(b) * c.max_pages;
  __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(c.pool);
  const __nv_bfloat16* tok = qkv + static_cast<size_t>(b) * (H + 2 * c.Hkv) * D;
  if (threadIdx.x < 2 * D) {                         // the token's own row
    const int which = threadIdx.x / D, d = threadIdx.x % D;
    const int pg = page_of(c, trow, last, err);
    if (pg >= 0) pool[row_at(c, pg, which, h, last & pmask) * D + d] = tok[(H + which * c.Hkv + h) * D + d];
    if (pg >= 0 && c.weight && threadIdx.x == 0) c.weight[weight_at(c, pg, h, last & pmask)] = 0.0f;
  }
  __syncthreads();
  const Seen sn = seen_rows(last + 1, window, sinks);
  auto score = [&](int pg, int r) {
    const __nv_bfloat16* k = pool + row_at(c, pg, 0, h, r & pmask) * D;
    float s = 0.0f;
    for (int d = 0; d < D; ++d) s = fmaf(__bfloat162float(k[d]), sq[d], s);
    return s * scale_log2;
  };
  for (int g = 0; g < G; ++g) {
    const int head = h * G + g;
    if (threadIdx.x < D) sq[threadIdx.x] = __bfloat162float(tok[head * D + threadIdx.x]);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o[CPL] = {};
    for (int v0 = warp * 32; v0 < sn.n; v0 += kDecWarps * 32) {
      const int v = v0 + lane;
      int pg = -1, r = 0;
      if (v < sn.n) {
        r = seen_row(sn, v);
        pg = page_of(c, trow, r, err);
      }
      const float s = pg >= 0 ? score(pg, r) : -INFINITY;
      float mx = s;
      for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float mn = fmaxf(m, mx);
      if (mn == -INFINITY) continue;
      const float a = exp2f(m - mn), p = exp2f(s - mn);
      m = mn;
      float ps = p;
      for (int k = 16; k > 0; k >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, k);
      l = l * a + ps;
      for (int k = 0; k < CPL; ++k) o[k] *= a;
      for (int i = 0; i < 32; ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i);
        const int pgi = __shfl_sync(0xffffffffu, pg, i), ri = __shfl_sync(0xffffffffu, r, i);
        if (pgi < 0) continue;
        const __nv_bfloat16* u = pool + row_at(c, pgi, 1, h, ri & pmask) * D + lane * CPL;
        for (int k = 0; k < CPL; ++k) o[k] = fmaf(pi, __bfloat162float(u[k]), o[k]);
      }
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    for (int k = 0; k < CPL; ++k) so[warp][lane * CPL + k] = o[k];
    __syncthreads();
    float mt = -INFINITY, lt = 0.0f;
    for (int w = 0; w < kDecWarps; ++w) mt = fmaxf(mt, sm[w]);
    for (int w = 0; w < kDecWarps; ++w) lt += sm[w] == -INFINITY ? 0.0f : sl[w] * exp2f(sm[w] - mt);
    if (threadIdx.x < D) {
      float a = 0.0f;
      for (int w = 0; w < kDecWarps; ++w) a += sm[w] == -INFINITY ? 0.0f : so[w][threadIdx.x] * exp2f(sm[w] - mt);
      y[(static_cast<size_t>(b) * H + head) * D + threadIdx.x] = __float2bfloat16(lt > 0.0f ? a / lt : 0.0f);
    }
    const float lse = mt + log2f(lt);
    if (lse2 && threadIdx.x == 0) lse2[static_cast<size_t>(b) * H + head] = lse;
    if (c.weight && lt > 0.0f) {
      for (int v = threadIdx.x; v < sn.n; v += kDecWarps * 32) {
        const int r = seen_row(sn, v);
        const int pg = page_of(c, trow, r, err);
        // added atomically: sequences may share a page (the sum of a page of one sequence has a fixed order)
        if (pg >= 0) atomicAdd(c.weight + weight_at(c, pg, h, r & pmask), exp2f(score(pg, r) - lse));
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- eviction

// Order of weights as unsigned numbers: larger weight, larger number; NaN lowest; -0 equals +0.
__device__ __forceinline__ uint32_t weight_rank(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kEvThreads = 512;

// The inclusive prefix sum of x over the block, and the total.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, k);
    if (lane >= k) x += y;
  }
  __syncthreads();                                   // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kEvThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  *total = all;
  return x + before;
}

// One block per (key head, sequence). Selection: the rank of the smallest kept weight by four passes over 8 bits
// each (a histogram of the rows that agree so far); equal weights are kept from the lowest row on. Then the
// kept rows' numbers are written in order, and the rows move to the front: row i's source is at or behind i, so
// a chunk's rows are all read before any of them is written and no later chunk reads what this one wrote.
template <int D>
__global__ void __launch_bounds__(kEvThreads)
paged_evict_kernel(PagedCache c, const int32_t* __restrict__ lens, const int32_t* dst_table, int dst_max_pages,
                   int32_t* __restrict__ new_lens, int32_t* kept, int budget, int sinks, int recent, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int U = D / 8;
  __shared__ int hist[256], sums[kEvThreads / 32], pick[2];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int pmask = (1 << c.page_log2) - 1;
  const int32_t* trow = c.table + static_cast<size_t>(b) * c.max_pages;
  const int32_t* drow = dst_table + static_cast<size_t>(b) * dst_max_pages;
  int32_t* out = kept + (static_cast<size_t>(b) * c.Hkv + h) * budget;
  int n = __ldg(lens + b);
  if (n > static_cast<long long>(c.max_pages) << c.page_log2) {
    if (tid == 0) record_error(err, GPT_DEV_EPAGE);
    n = 0;
  }
  const int m = min(n, budget);                      // rows kept
  if (h == 0 && tid == 0) new_lens[b] = m;
  for (int i = max(m, 0) + tid; i < budget; i += kEvThreads) out[i] = -1;
  if (m <= 0) return;
  auto rank_of = [&](int r) -> uint32_t {
    const int pg = page_of(c, trow, r, err);
    return pg < 0 ? 0u : weight_rank(c.weight[weight_at(c, pg, h, r & pmask)]);
  };
  if (n <= budget) {
    for (int i = tid; i < m; i += kEvThreads) out[i] = i;
  } else {
    const int lo = sinks, hi = n - recent;           // rows chosen by weight: [lo, hi)
    int want = budget - sinks - recent;              // how many of them
    uint32_t prefix = 0;                             // the leading bits of the smallest kept rank
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
      for (int i = tid; i < 256; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      for (int r = lo + tid; r < hi; r += kEvThreads) {
        const uint32_t k = rank_of(r);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = want, d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        pick[0] = d;
        pick[1] = left;                              // still to take among those with this digit
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      want = pick[1];
      __syncthreads();
    }
    // want rows of rank == prefix are kept (the first ones), and every row of a higher rank
    const bool any = budget > sinks + recent;
    int ties = 0, base = 0;
    for (int r0 = 0; r0 < n; r0 += kEvThreads) {
      const int r = r0 + tid;
      bool keep = r < n && (r < lo || r >= hi), tie = false;
      if (r >= lo && r < hi && any) {
        const uint32_t k = rank_of(r);
        keep = k > prefix;
        tie = k == prefix;
      }
      int total;
      const int ti = block_scan(tie ? 1 : 0, sums, &total);
      if (tie) keep = ties + ti <= want;
      ties += total;
      const int at = block_scan(keep ? 1 : 0, sums, &total);
      if (keep) out[base + at - 1] = r;
      base += total;
    }
  }
  __syncthreads();                                   // out[] is read below by other threads of the block
  constexpr int RPB = kEvThreads / U;                // rows per chunk: one 16-byte unit per thread
  uint4* pool = static_cast<uint4*>(c.pool);
  for (int i0 = 0; i0 < m; i0 += RPB) {
    const int i = i0 + tid / U, u = tid % U;
    int src = -1, dst = -1, r = 0;
    uint4 kx, vx;
    float w = 0.0f;
    if (i < m) {
      r = out[i];
      src = page_of(c, trow, r, err);
      dst = page_of(c, drow, i, err);
      if (src >= 0) {
        kx = pool[row_at(c, src, 0, h, r & pmask) * U + u];
        vx = pool[row_at(c, src, 1, h, r & pmask) * U + u];
        if (u == 0) w = c.weight[weight_at(c, src, h, r & pmask)];
      }
    }
    __syncthreads();
    if (src >= 0 && dst >= 0) {
      pool[row_at(c, dst, 0, h, i & pmask) * U + u] = kx;
      pool[row_at(c, dst, 1, h, i & pmask) * U + u] = vx;
      if (u == 0) c.weight[weight_at(c, dst, h, i & pmask)] = w;
    }
  }
}

}  // namespace

cudaError_t launch_paged_store(const PagedCache& c, const void* qkv, const int32_t* start, const int32_t* count, int B,
                               int T, int H, int D, int* err, cudaStream_t s) {
  const long long units = static_cast<long long>(T) * 2 * c.Hkv * (D / 8);
  const long long blocks = (units + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(B));
  const uint4* x = static_cast<const uint4*>(qkv);
  if (D == 64) return launch_k(paged_store_kernel<64>, grid, dim3(256), 0, s, c, x, start, count, T, H, err);
  return launch_k(paged_store_kernel<32>, grid, dim3(256), 0, s, c, x, start, count, T, H, err);
}

cudaError_t launch_paged_attention(const PagedCache& c, const void* qkv, const int32_t* lens, void* y, float* lse2,
                                   int B, int H, int D, int window, int sinks, int* err, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(c.Hkv), static_cast<unsigned>(B));
  const float sc = kLog2e / sqrtf(static_cast<float>(D));
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(qkv);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(y);
  if (D == 64)
    return launch_k(paged_attention_kernel<64>, grid, dim3(kDecWarps * 32), 0, s, c, x, lens, o, lse2, H, window, sinks,
                    sc, err);
  return launch_k(paged_attention_kernel<32>, grid, dim3(kDecWarps * 32), 0, s, c, x, lens, o, lse2, H, window, sinks,
                  sc, err);
}

cudaError_t launch_paged_evict(const PagedCache& c, const int32_t* lens, const int32_t* dst_table, int dst_max_pages,
                               int32_t* new_lens, int32_t* kept, int B, int D, int budget, int sinks, int recent,
                               int* err, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(c.Hkv), static_cast<unsigned>(B));
  if (D == 64)
    return launch_k(paged_evict_kernel<64>, grid, dim3(kEvThreads), 0, s, c, lens, dst_table, dst_max_pages, new_lens,
                    kept, budget, sinks, recent, err);
  return launch_k(paged_evict_kernel<32>, grid, dim3(kEvThreads), 0, s, c, lens, dst_table, dst_max_pages, new_lens, kept,
                  budget, sinks, recent, err);
}

}  // namespace gptgb
