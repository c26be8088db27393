// Device helpers shared by the kernels of the paged key/value caches (16-bit rows: k_paged.cu, 4-bit rows: k_paged4.cu):
// where a row lies, which rows a query sees, the dealing of units to warps, and the warp's copies and products.
#pragma once

#include "common.cuh"

namespace gptgb {

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

// `total` units dealt to n warps (every warp gets one at least): the first `rem` warps take q + 1, the others q. Written
// so that a range's start costs a multiplication and a unit's warp one division, of 32 bits where the numbers allow: the
// joining blocks ask several times before their first load.
struct Deal {
  long long q;
  int n, rem;
  __device__ __forceinline__ Deal(long long total, int warps) {
    n = total < warps ? static_cast<int>(total) : warps;
    if (total <= 0x7fffffffLL) {
      q = n ? static_cast<int>(total) / n : 0;
    } else {
      q = total / n;
    }
    rem = static_cast<int>(total - q * n);
  }
  __device__ __forceinline__ long long start(int g) const { return g * q + min(g, rem); }
  __device__ __forceinline__ int warp_of(long long u) const {
    const long long split = rem * (q + 1);           // the first unit of the shorter ranges
    if (u < split) return u <= 0x7fffffffLL ? static_cast<int>(u) / static_cast<int>(q + 1) : static_cast<int>(u / (q + 1));
    const long long v = u - split;
    return rem + (v <= 0x7fffffffLL && q <= 0x7fffffffLL ? static_cast<int>(v) / static_cast<int>(q) : static_cast<int>(v / q));
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool copy) {
  const int n = copy ? 16 : 0;                       // 0: the 16 bytes are zeros, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace gptgb
