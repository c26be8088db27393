// Attention of one query row per sequence over the paged cache in 4 bits (layout: k_append.cu).
//
// A row stands for low + scale * code, so with Q = sum of a query's values
//   q . k_r = scale_r (q . code_r) + low_r Q,    sum_r p_r u_r = sum_r (p_r scale_r) code_r + sum_r p_r low_r,
// and codes enter the products as they are: a 4-bit code placed in a bf16 number's upper four mantissa bits, with the
// exponent of 16, is the number 16 + code: one shift and one logical operation make two operands. The 16 is taken back
// where it costs nothing: the score products start from -16 Q, and low - 16 scale stands for low in the second sum.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "paged.cuh"

#include <math.h>

namespace gptgb {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kUnit4 = 32;                // seen rows per unit

// Bound by reading the cache (D + 8 bytes per seen row and key head) and, nearly as much, by issuing instructions: a byte of
// codes takes a warp four times the unpacking and products of a byte of bf16. Work is dealt as in the 16-bit cache's
// kernel (k_paged.cu): units of 32 seen rows of one (sequence, key head, group of up to 16 query heads), equal contiguous
// ranges of the list of all units to every warp, partial results joined by a second kernel. What differs:
//  * The rows' order inside a unit and the values' order inside a product are free, so fragments are read from shared
//    memory as they lie there, without ldmatrix: a lane takes a quarter of a key row (8 bytes: its codes are the lane's
//    operands of four products), and of value rows the same byte column of four rows, two of which are interleaved by one
//    byte permutation into eight operands. Column 2 q + i of score tile j is row 16 (j / 2) + 8 (j % 2) + 4 i + q; output
//    tile i holds value 8 n + i (D = 64; 4 n + i for 32) in column n, so a lane ends with D / 4 consecutive values.
//  * 16 warps per SM with a ring of their own each.
template <int D, int QR>
struct Dec4Cfg {
  static constexpr int ROWB = D / 2;                              // bytes of a row's codes
  static constexpr int TILE = kUnit4 * ROWB;                      // keys, or values, of a unit
  static constexpr int RANGES = 2 * TILE;                         // offset of the pairs (key range, value range)
  static constexpr int QUERIES = RANGES + kUnit4 * 8;             // offset of the query rows (where a unit starts a segment)
  static constexpr int STAGE = QUERIES + QR * D * 2;
  static constexpr int STAGES = QR == 8 ? 4 : 3;
  static constexpr int WARP = STAGES * STAGE;
  static constexpr int WARPS = 16;
};

struct Dec4Scratch {
  int* prefix;        // [B + 1] units of the sequences before b, per head group
  float* o;           // [warps][2][QR][D] unnormalised partial outputs
  float2* ml;         // [warps][2][QR] their maxima (log2 units) and sums
};

struct Dec4Shape {
  int B, H, G, mg;    // mg: head groups of up to 16 per key head
  int window, sinks, added;
  float scale_log2;
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool copy) {
  const int n = copy ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// d = a b + c
__device__ __forceinline__ void mma_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%10, %10, %11, %11};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// Codes p of both halves of w as the bf16 pair (16 + low half's, 16 + high half's).
template <int p>
__device__ __forceinline__ uint32_t pair16(uint32_t w) {
  const uint32_t x = p == 0 ? w << 3 : w >> (4 * p - 3);
  return (x & 0x00780078u) | 0x41804180u;
}

__device__ __forceinline__ float scale_of(uint32_t range) { return __uint_as_float(range << 16); }
__device__ __forceinline__ float low_of(uint32_t range) { return __uint_as_float(range & 0xffff0000u); }

// The rows that a sequence's query sees, from its length (-1: none to compute).
__device__ __forceinline__ int rows_of(const PagedCache& c, const Dec4Shape& w, int len) {
  return len < 0 ? -1 : static_cast<long long>(len) + w.added > (static_cast<long long>(c.max_pages) << c.page_log2) ? -2
                                                                                                                      : len + w.added;
}

// A group's queries as the products' A operands, and the sum of each row's values.
// rows: QR rows of D bf16 at shared address sq (zeros behind the group).
template <int D, int QR>
__device__ __forceinline__ void take_queries(uint32_t (&f)[D / 16][4], float (&q)[2], uint32_t sq, int lane) {
  constexpr int C = D / 4;                           // values of a lane: its codes' places
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < C / 8; ++w) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (rh == 0 || QR == 16) x = lds128(sq + ((lane >> 2) + 8 * rh) * D * 2 + ((lane & 3) * C + 8 * w) * 2);
      const float2 a = unpack_bf16x2(x.x), b = unpack_bf16x2(x.y), c = unpack_bf16x2(x.z), d = unpack_bf16x2(x.w);
      sum += ((a.x + a.y) + (b.x + b.y)) + ((c.x + c.y) + (d.x + d.y));
      // pairs (0, 4), (1, 5), (2, 6), (3, 7): as a word of codes unpacks
      f[2 * w][rh] = __byte_perm(x.x, x.z, 0x5410);
      f[2 * w][2 + rh] = __byte_perm(x.x, x.z, 0x7632);
      f[2 * w + 1][rh] = __byte_perm(x.y, x.w, 0x5410);
      f[2 * w + 1][2 + rh] = __byte_perm(x.y, x.w, 0x7632);
    }
    sum += __shfl_xor_sync(kAll, sum, 1);
    sum += __shfl_xor_sync(kAll, sum, 2);
    q[rh] = sum;
  }
}

// Products q . code of the 32 key rows at sk: tile j, column 2 q + i is row 16 (j / 2) + 8 (j % 2) + 4 i + q.
template <int D>
__device__ __forceinline__ void code_scores(float (&s)[4][4], const uint32_t (&f)[D / 16][4], const float (&q)[2], uint32_t sk,
                                            int lane) {
  const int c = lane >> 2;
  const uint32_t at = sk + ((c & 1) * 4 + (c >> 1)) * (D / 2) + (lane & 3) * (D / 8);
  const float c0 = -16.0f * q[0], c1 = -16.0f * q[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[2];
    if constexpr (D == 64) {
      const uint2 x = lds64(at + 8 * j * (D / 2));
      w[0] = x.x;
      w[1] = x.y;
    } else {
      w[0] = lds32(at + 8 * j * (D / 2));
      w[1] = 0u;
    }
    mma_from(s[j], f[0], pair16<0>(w[0]), pair16<1>(w[0]), c0, c1);
    mma_16816(s[j], f[1], pair16<2>(w[0]), pair16<3>(w[0]));
    if constexpr (D == 64) {
      mma_16816(s[j], f[2], pair16<0>(w[1]), pair16<1>(w[1]));
      mma_16816(s[j], f[3], pair16<2>(w[1]), pair16<3>(w[1]));
    }
  }
}

// O += P (16 + code) for the 16 value rows at sv (rows of half a unit): a, b are the score tiles of eight each, now p times
// the rows' scales, in two bf16 parts as in k_paged.cu: of up to eight query heads the second part takes the operand's other
// eight rows.
template <int D, int RH>
__device__ __forceinline__ void add_codes(float (&o)[D / 8][4], const float (&a)[4], const float (&b)[4], uint32_t sv, int lane) {
  uint32_t p[4], q[4];
#pragma unroll
  for (int i = 0; i < 2 * RH; ++i) {                 // heads lane / 4 (i even) and lane / 4 + 8, columns of a, then of b
    const float x = i < RH ? a[2 * i] : b[2 * (i - RH)], y = i < RH ? a[2 * i + 1] : b[2 * (i - RH) + 1];
    const int at = RH == 2 ? i : 2 * i;
    p[at] = pack_bf16x2(x, y);
    const float2 f = unpack_bf16x2(p[at]);
    const uint32_t lo = pack_bf16x2(x - f.x, y - f.y);
    if (RH == 2) q[at] = lo;
    else p[at + 1] = lo;
  }
  constexpr int ROWB = D / 2;
  uint32_t x[2], y[2];                               // rows (0, 4) and (8, 12) + q: codes 0-3 and, of D = 64, 4-7 of a word
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t at = sv + (8 * h + (lane & 3)) * ROWB + (lane >> 2) * (D / 16);
    if constexpr (D == 64) {
      const uint32_t w0 = lds32(at), w1 = lds32(at + 4 * ROWB);
      x[h] = __byte_perm(w0, w1, 0x5410);
      y[h] = __byte_perm(w0, w1, 0x7632);
    } else {
      x[h] = lds16(at) | (lds16(at + 4 * ROWB) << 16);
      y[h] = 0u;
    }
  }
  auto step = [&](const uint32_t (&t)[4]) {
    mma_16816(o[0], t, pair16<0>(x[0]), pair16<0>(x[1]));
    mma_16816(o[1], t, pair16<1>(x[0]), pair16<1>(x[1]));
    mma_16816(o[2], t, pair16<2>(x[0]), pair16<2>(x[1]));
    mma_16816(o[3], t, pair16<3>(x[0]), pair16<3>(x[1]));
    if constexpr (D == 64) {
      mma_16816(o[4], t, pair16<0>(y[0]), pair16<0>(y[1]));
      mma_16816(o[5], t, pair16<1>(y[0]), pair16<1>(y[1]));
      mma_16816(o[6], t, pair16<2>(y[0]), pair16<2>(y[1]));
      mma_16816(o[7], t, pair16<3>(y[0]), pair16<3>(y[1]));
    }
  };
  step(p);
  if constexpr (RH == 2) step(q);
}

// The list position of a unit: sequence, head group (key head * mg + group), tile of the sequence's seen rows.
struct Unit4 {
  int b, hm, tile, nt;
  Seen seen;
};

template <int D, int QR>
__global__ void __launch_bounds__(512, 1)
paged4_split_kernel(PagedCache c, const uint32_t* __restrict__ ranges, const __nv_bfloat16* __restrict__ qkv,
                    const int32_t* __restrict__ lens, __nv_bfloat16* __restrict__ y, float* __restrict__ lse2, Dec4Shape w,
                    Dec4Scratch ws, int* err) {
  using Cfg = Dec4Cfg<D, QR>;
  constexpr int ROWB = Cfg::ROWB, UNITS = ROWB / 16, NT = D / 8, RH = QR == 16 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  int* s_prefix = reinterpret_cast<int*>(smem + nwarps * Cfg::WARP);     // [B + 1]
  int* s_rows = s_prefix + w.B + 1;                                      // [B]
  __shared__ int s_sum[16];
  pdl_wait();
  pdl_trigger();

  // units per sequence and their prefix sums (per head group)
  if (threadIdx.x == 0) s_prefix[0] = 0;
  int carry = 0;
  for (int b0 = 0; b0 < w.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int rows = 0, x = 0;
    if (b < w.B) {
      rows = rows_of(c, w, __ldg(lens + b));
      if (rows == -2) record_error(err, GPT_DEV_EPAGE);
      rows = max(rows, 0);
      x = (seen_rows(rows, w.window, w.sinks).n + kUnit4 - 1) / kUnit4;
      s_rows[b] = rows;
    }
    int incl = x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, k);
      if (lane >= k) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = carry;
    for (int i = 0; i < nwarps; ++i) {
      if (i < warp) before += s_sum[i];
      carry += s_sum[i];
    }
    if (b < w.B) s_prefix[b + 1] = before + incl;
    __syncthreads();
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= w.B; b += blockDim.x) ws.prefix[b] = s_prefix[b];

  const int HM = c.Hkv * w.mg;
  const long long total = static_cast<long long>(carry) * HM;
  const Deal deal(total, static_cast<int>(gridDim.x) * nwarps);
  const int gw = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  if (gw >= deal.n) return;                          // no barrier of the block follows
  const long long u0 = deal.start(gw);
  const int count = static_cast<int>(deal.start(gw + 1) - u0);

  const uint32_t ring = smem_u32(smem + warp * Cfg::WARP);
  const int row = w.H + 2 * c.Hkv;                   // heads of a token's row
  const int pmask = (1 << c.page_log2) - 1;
  const size_t vrows = static_cast<size_t>(c.Hkv) << c.page_log2;        // rows from a page's keys to its values
  const uint8_t* pool = static_cast<const uint8_t*>(c.pool);

  auto set_seq = [&](Unit4& x) {                     // the sequence's lengths (b has units)
    x.nt = s_prefix[x.b + 1] - s_prefix[x.b];
    x.seen = seen_rows(s_rows[x.b], w.window, w.sinks);
  };
  auto advance = [&](Unit4& x) {
    if (++x.tile < x.nt) return;
    x.tile = 0;
    if (++x.hm < HM) return;
    x.hm = 0;
    do ++x.b; while (x.b < w.B && s_prefix[x.b + 1] == s_prefix[x.b]);
    if (x.b < w.B) set_seq(x);
  };
  Unit4 at;                                          // the unit that is computed next
  {
    const int target = static_cast<int>(u0 / HM);    // the sequence with prefix[b] <= target < prefix[b + 1]
    int lo = 0, hi = w.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_prefix[mid + 1] > target) hi = mid;
      else lo = mid + 1;
    }
    at.b = lo;
    set_seq(at);
    const long long r = u0 - static_cast<long long>(s_prefix[lo]) * HM;
    at.hm = static_cast<int>(r / at.nt);
    at.tile = static_cast<int>(r - static_cast<long long>(at.hm) * at.nt);
  }
  // A lane copies of rows lane / 2 and 16 + lane / 2 of a unit: half `part` of their codes (all of the keys', or the values',
  // where D = 32) and the range of the key (part 0) or the value. Their pages are looked up one unit ahead.
  const int part = lane & 1;
  Unit4 next = at;                                   // the unit whose rows are copied next
  int pg[2];
  auto look_up = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = next.tile * kUnit4 + 16 * i + (lane >> 1);
      pg[i] = v < next.seen.n ? __ldg(c.table + static_cast<size_t>(next.b) * c.max_pages + (seen_row(next.seen, v) >> c.page_log2)) : -1;
    }
  };
  look_up();
  int issued = 0;
  auto issue = [&]() {                               // copies unit `next` into stage issued % STAGES, steps on
    const uint32_t st = ring + (issued % Cfg::STAGES) * Cfg::STAGE;
    const int kh = next.hm / w.mg, g0 = (next.hm - kh * w.mg) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = 16 * i + (lane >> 1), v = next.tile * kUnit4 + rr;
      const bool seen = v < next.seen.n, ok = seen && static_cast<unsigned>(pg[i]) < static_cast<unsigned>(c.pages);
      if (seen && !ok) record_error(err, GPT_DEV_EPAGE);
      const size_t key = ok ? row_at(c, pg[i], 0, kh, seen_row(next.seen, v) & pmask) : 0, value = key + (ok ? vrows : 0);
      if constexpr (UNITS == 2) {
        cp_async16(st + rr * ROWB + 16 * part, pool + key * ROWB + 16 * part, ok);
        cp_async16(st + Cfg::TILE + rr * ROWB + 16 * part, pool + value * ROWB + 16 * part, ok);
      } else {
        cp_async16(st + part * Cfg::TILE + rr * ROWB, pool + (part ? value : key) * ROWB, ok);
      }
      cp_async4(st + Cfg::RANGES + 8 * rr + 4 * part, ranges + (part ? value : key), ok);
    }
    if (issued == 0 || next.tile == 0) {             // a segment starts: its queries (rows past the group: zeros)
      const int gn = min(w.G - g0, 16);
      const __nv_bfloat16* tok = qkv + (static_cast<size_t>(next.b) * row + kh * w.G + g0) * D;
#pragma unroll
      for (int i = 0; i < QR * D / 256; ++i) {
        const int e = 32 * i + lane, rr = e / (D / 8), u = e % (D / 8);
        cp_async16(st + Cfg::QUERIES + e * 16, tok + static_cast<size_t>(min(rr, gn - 1)) * D + 8 * u, rr < gn);
      }
    }
    ++issued;
    if (issued < count) {
      advance(next);
      look_up();
    }
  };
#pragma unroll
  for (int s = 0; s < Cfg::STAGES - 1; ++s) {
    if (issued < count) issue();
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  float o[NT][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, off[2] = {0.0f, 0.0f};   // rows lane / 4 and lane / 4 + 8
  uint32_t qf[D / 16][4];
  float qsum[2] = {0.0f, 0.0f};
  int piece0 = 0;                                    // the segment's first unit in this warp's range
  const int qrow = lane >> 2, q4 = lane & 3;
  for (int n = 0; n < count; ++n) {
    if (issued < count) issue();
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(Cfg::STAGES - 1) : "memory");
    __syncwarp();
    const uint32_t st = ring + (n % Cfg::STAGES) * Cfg::STAGE;
    const int kh = at.hm / w.mg, g0 = (at.hm - kh * w.mg) * 16, gn = min(w.G - g0, 16);
    if (n == 0 || at.tile == 0) {
      piece0 = n;
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        m[rh] = -INFINITY;
        l[rh] = off[rh] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
      take_queries<D, QR>(qf, qsum, st + Cfg::QUERIES, lane);
    }
    float s[4][4];
    code_scores<D>(s, qf, qsum, st, lane);
    // scores scale (q . code) + low Q, in units of the softmax's base-2 exponent over scale_log2
    uint32_t vr[4][2];                               // the value rows' ranges
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint2 r = lds64(st + Cfg::RANGES + 8 * (16 * (j >> 1) + 8 * (j & 1) + 4 * i + q4));
        vr[j][i] = r.y;
        const float sc = scale_of(r.x), lo = low_of(r.x);
        s[j][i] = fmaf(sc, s[j][i], lo * qsum[0]);
        if (RH == 2) s[j][2 + i] = fmaf(sc, s[j][2 + i], lo * qsum[1]);
      }
    const int left = at.seen.n - at.tile * kUnit4;
    if (left < kUnit4) {                             // rows behind the last: not seen
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2 * RH; ++i)
          if (16 * (j >> 1) + 8 * (j & 1) + 4 * (i & 1) + q4 >= left) s[j][i] = -INFINITY;
    }
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
      float mx = fmax3(s[0][2 * rh], s[0][2 * rh + 1], s[1][2 * rh]);
      mx = fmax3(mx, s[1][2 * rh + 1], s[2][2 * rh]);
      mx = fmax3(mx, s[2][2 * rh + 1], s[3][2 * rh]);
      mx = fmaxf(mx, s[3][2 * rh + 1]) * w.scale_log2;
      mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
      mx = fmaxf(mx, m[rh]);
      const float ref = mx == -INFINITY ? 0.0f : mx;   // every score so far -inf: every term is 2^-inf
      const float a = ex2_approx(m[rh] - ref);
      m[rh] = mx;
      float sum = 0.0f, low = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p = ex2_approx(fmaf(s[j][2 * rh + i], w.scale_log2, -ref));
          const float sc = scale_of(vr[j][i]);
          sum += p;
          low = fmaf(p, fmaf(-16.0f, sc, low_of(vr[j][i])), low);
          s[j][2 * rh + i] = p * sc;
        }
      l[rh] = l[rh] * a + sum;
      off[rh] = off[rh] * a + low;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][2 * rh] *= a;
        o[j][2 * rh + 1] *= a;
        if (RH == 1) {                               // the second part's
          o[j][2] *= a;
          o[j][3] *= a;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) add_codes<D, RH>(o, s[2 * k], s[2 * k + 1], st + Cfg::TILE + 16 * k * ROWB, lane);
    const bool ends = at.tile == at.nt - 1;
    if (ends || n == count - 1) {                    // the piece is done
      const bool whole = ends && piece0 + at.nt == n + 1;   // it holds all of the segment's units
      const size_t slot = static_cast<size_t>(gw) * 2 + (piece0 == 0 ? 0 : 1);
#pragma unroll
      for (int rh = 0; rh < RH; ++rh) {
        float lt = l[rh], ot = off[rh];
        lt += __shfl_xor_sync(kAll, lt, 1);
        lt += __shfl_xor_sync(kAll, lt, 2);
        ot += __shfl_xor_sync(kAll, ot, 1);
        ot += __shfl_xor_sync(kAll, ot, 2);
        const int r = qrow + 8 * rh;
        if (r >= gn) continue;
        float v[D / 4];                              // values D / 4 q4 .. of the head
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) v[i * NT + j] = o[j][2 * rh + i] + (RH == 1 ? o[j][2 + i] : 0.0f) + ot;
        if (whole) {
          const size_t head = static_cast<size_t>(at.b) * w.H + kh * w.G + g0 + r;
          const float inv = 1.0f / lt;               // (a sum of 0, every score -inf, gives NaN)
          uint4* dst = reinterpret_cast<uint4*>(y + head * D + q4 * (D / 4));
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            dst[k] = make_uint4(pack_bf16x2(v[8 * k] * inv, v[8 * k + 1] * inv), pack_bf16x2(v[8 * k + 2] * inv, v[8 * k + 3] * inv),
                                pack_bf16x2(v[8 * k + 4] * inv, v[8 * k + 5] * inv), pack_bf16x2(v[8 * k + 6] * inv, v[8 * k + 7] * inv));
          if (q4 == 0 && lse2) lse2[head] = m[rh] + log2f(lt);
        } else {
          float4* dst = reinterpret_cast<float4*>(ws.o + (slot * QR + r) * D + q4 * (D / 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          if (q4 == 0) ws.ml[slot * QR + r] = make_float2(m[rh], lt);
        }
      }
    }
    advance(at);
    __syncwarp();                                    // the stage is read before it is filled again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Joins the partial results of a (sequence, key head) in a fixed order; sequences of no rows get zeros and -inf.
constexpr int kJoin4Threads = 256;

template <int D, int QR>
__global__ void __launch_bounds__(kJoin4Threads)
paged4_join_kernel(PagedCache c, const int32_t* __restrict__ lens, __nv_bfloat16* __restrict__ y, float* __restrict__ lse2,
                   Dec4Shape w, Dec4Scratch ws, int warps) {
  pdl_wait();
  pdl_trigger();
  constexpr int P = kJoin4Threads / D;               // rows, or shares of a row's pieces, side by side
  __shared__ float s_o[P][D], s_m[P], s_l[P];
  const int kh = blockIdx.x, b = blockIdx.y;
  const int HM = c.Hkv * w.mg, p0 = ws.prefix[b], nt = ws.prefix[b + 1] - p0;
  const long long total = static_cast<long long>(ws.prefix[w.B]) * HM;
  const int tid = threadIdx.x, d = tid % D, part = tid / D;
  if (nt == 0) {
    if (rows_of(c, w, __ldg(lens + b)) != 0) return;
    const size_t head0 = static_cast<size_t>(b) * w.H + kh * w.G;
    for (int i = tid; i < w.G * D; i += kJoin4Threads) y[head0 * D + i] = __float2bfloat16(0.0f);
    if (lse2)
      for (int i = tid; i < w.G; i += kJoin4Threads) lse2[head0 + i] = -INFINITY;
    return;
  }
  const Deal deal(total, warps);
  for (int mt = 0; mt < w.mg; ++mt) {
    const long long t0 = static_cast<long long>(p0) * HM + static_cast<long long>(kh * w.mg + mt) * nt, t1 = t0 + nt;
    const int g1 = deal.warp_of(t0), g2 = deal.warp_of(t1 - 1);   // the warps that hold the first unit and the last
    if (g1 == g2) continue;                          // one warp held it all and wrote the output
    const int gn = min(w.G - mt * 16, 16);
    const size_t head0 = static_cast<size_t>(b) * w.H + kh * w.G + mt * 16;
    // a piece is its warp's first (slot 0) unless its segment starts behind the warp's start: only g1's can
    const size_t slot1 = static_cast<size_t>(g1) * 2 + (deal.start(g1) == t0 ? 0 : 1);
    // the pieces of one or two rows are shared by the parts
    const int share = gn >= P ? 1 : (gn >= 2 && P >= 4 ? P / 2 : P);
    for (int r0 = 0; r0 < gn; r0 += P / share) {
      const int r = r0 + part / share, sub = part % share;
      float m = -INFINITY, l = 0.0f, acc = 0.0f;
      if (r < gn) {
#pragma unroll 4
        for (int g = g1 + sub; g <= g2; g += share) {
          const size_t sl = (g == g1 ? slot1 : static_cast<size_t>(g) * 2) * QR + r;
          const float2 x = ws.ml[sl];
          const float o = ws.o[sl * D + d];
          const float mn = fmaxf(m, x.x), ref = mn == -INFINITY ? 0.0f : mn;
          const float f = ex2_approx(m - ref), h = ex2_approx(x.x - ref);
          m = mn;
          l = l * f + x.y * h;
          acc = acc * f + o * h;
        }
      }
      s_o[part][d] = acc;
      if (d == 0) {
        s_m[part] = m;
        s_l[part] = l;
      }
      __syncthreads();
      if (sub == 0 && r < gn) {
        float mx = m;
        for (int k = 1; k < share; ++k) mx = fmaxf(mx, s_m[part + k]);
        const float ref = mx == -INFINITY ? 0.0f : mx;
        float lt = 0.0f, at = 0.0f;
        for (int k = 0; k < share; ++k) {
          const float f = ex2_approx(s_m[part + k] - ref);
          lt += s_l[part + k] * f;
          at += s_o[part + k][d] * f;
        }
        y[(head0 + r) * D + d] = __float2bfloat16(at / lt);
        if (d == 0 && lse2) lse2[head0 + r] = mx + log2f(lt);
      }
      __syncthreads();
    }
  }
}

template <int D, int QR>
cudaError_t launch_decode4(const PagedCache& c, const uint32_t* ranges, const __nv_bfloat16* qkv, const int32_t* lens,
                           __nv_bfloat16* y, float* lse2, const Dec4Shape& w, int* err, cudaStream_t s) {
  using Cfg = Dec4Cfg<D, QR>;
  static SmemLimit limit;
  int dev = 0, num_sms = 0;
  cudaError_t e = device_sms(&dev, &num_sms);
  if (e != cudaSuccess) return e;
  // one block per SM with as many warps (rings) as its shared memory holds beside the sequences' lengths, 16 at most
  const size_t head = (2 * static_cast<size_t>(w.B) + 1) * sizeof(int);
  const size_t room = 232448 - 256 - head;
  const int warps = room / Cfg::WARP < Cfg::WARPS ? static_cast<int>(room / Cfg::WARP) : Cfg::WARPS;
  const size_t smem = static_cast<size_t>(warps) * Cfg::WARP + head;
  e = limit.raise(paged4_split_kernel<D, QR>, dev, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int NW = num_sms * warps;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t pre_b = up((w.B + 1) * sizeof(int)), o_b = up(static_cast<size_t>(NW) * 2 * QR * D * sizeof(float)),
               ml_b = up(static_cast<size_t>(NW) * 2 * QR * sizeof(float2));
  uint8_t* p = nullptr;
  e = scratch_alloc(reinterpret_cast<void**>(&p), pre_b + o_b + ml_b, s);
  if (e != cudaSuccess) return e;
  Dec4Scratch ws;
  ws.prefix = reinterpret_cast<int*>(p);
  ws.o = reinterpret_cast<float*>(p + pre_b);
  ws.ml = reinterpret_cast<float2*>(p + pre_b + o_b);
  e = launch_k(paged4_split_kernel<D, QR>, dim3(num_sms), dim3(32 * warps), smem, s, c, ranges, qkv, lens, y, lse2, w, ws, err);
  if (e == cudaSuccess)
    e = launch_k(paged4_join_kernel<D, QR>, dim3(static_cast<unsigned>(c.Hkv), static_cast<unsigned>(w.B)), dim3(kJoin4Threads), 0,
                 s, c, lens, y, lse2, w, ws, NW);
  const cudaError_t f = scratch_free(p, s);
  return e != cudaSuccess ? e : f;
}

}  // namespace

cudaError_t launch_paged_attention4(const PagedCache& c, const void* ranges, const void* qkv, const int32_t* lens, int added,
                                    void* y, float* lse2, int B, int H, int D, int window, int sinks, int* err,
                                    cudaStream_t s) {
  Dec4Shape w;
  w.B = B;
  w.H = H;
  w.G = H / c.Hkv;
  w.mg = (w.G + 15) / 16;
  w.window = window;
  w.sinks = sinks;
  w.added = added;
  w.scale_log2 = kLog2e / sqrtf(static_cast<float>(D));
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(qkv);
  const uint32_t* r = static_cast<const uint32_t*>(ranges);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(y);
  // up to 8 query heads per key head need half of the 16 query rows in shared memory and registers
  if (D == 64)
    return w.G <= 8 ? launch_decode4<64, 8>(c, r, x, lens, o, lse2, w, err, s) : launch_decode4<64, 16>(c, r, x, lens, o, lse2, w, err, s);
  return w.G <= 8 ? launch_decode4<32, 8>(c, r, x, lens, o, lse2, w, err, s) : launch_decode4<32, 16>(c, r, x, lens, o, lse2, w, err, s);
}

}  // namespace gptgb
