// Attention of one query row per sequence over the paged cache in 4 bits (layout: k_append.cu).
//
// A row stands for low + scale * code, so with Q = sum of a query's values
//   q . k_r = scale_r (q . code_r) + low_r Q,
//   sum_r p_r u_r = sum_r (p_r scale_r) (code_r - 8) + sum_r p_r (low_r + 8 scale_r),
// and codes enter the products as the fp16 numbers that their bits are: in bits 0 to 3 of a half with nothing above them a
// code is the subnormal code 2^-24, in bits 4 to 7 it is code 2^-20, so a word of eight codes takes one shift and four logical
// operations. The powers of two are taken back with the keys' scales, with the queries (2^-4 for every other value) and in the
// finished sums. The 8 is taken from the sums after every unit, by products of their own with -8: 64 rows' codes then add
// up to no more than the fp32 sums can hold beside their centred values. (As 1024 + code and 64 + code, less 1032 and 72 by a
// packed subtraction, an operand register took two instructions, and the long case below 59.8 us instead of 54.9. In bf16 every
// register takes its own shift, and a code comes out as 16 + code: taking the 16 back from the finished sums left the outputs
// of 20,000 rows 1.8e-3 of their norm off, where their own rounding makes 1.6e-3.)
// fp16 has few exponents: queries enter it times a power of two, exactly (largest value in [2^14, 2^15); what is below 2^-34
// of that is lost), and p_r scale_r times 2^(15 - E), where 2^E is above every such term of its head so far, at the present
// reference of the softmax, and at most 2^9 times the largest. (With 2^E above the rows' scales instead, whatever their weight, one
// row of no weight but 2^36 times the others' size left nothing of their codes.) They enter in two parts, what fp16 holds of
// them and what it holds of the rest: 2^-20 of a term is lost, and 2^-30 of the largest for each part of the smallest. One part
// alone loses 2^-12 and is less work: 28.6 us with 8 heads on each of 4 key heads below, 44.8 with 12; but the 16-bit
// cache's attention holds them in two parts as well. References of the softmax start at a score and rise by whole numbers, so that
// raising one rescales the sums exactly; scores are in the softmax's base-2 units but for a power of two, so that the exponent of
// the largest is exactly 0: a row seen alone comes out as it is.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "paged.cuh"

#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

namespace gptgb {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// Bound by memory once all warps are under way (8 sequences of 20,000 rows more take 19.3 us, 7.2 TB/s), with about 570
// instructions for 64 rows of a key head close behind: a byte of codes takes a warp twice the unpacking and products of a byte
// of bf16, and the integer unit takes a warp's instruction only every other cycle. Measured: 16 sequences of 9,000 to 32,000
// rows x 12 heads 53.5 us (graph replays of two inputs 56.6), 5.3 TB/s, of which the first rows' chain of loads and the last units
// take 8 and the join 5; the rows of a 16-bit cache take 160. With 4 query heads on each of 4 key heads 29.5, with 8 31.9, with 12
// 51.8 (graph replays), whose instructions bound them. Work is dealt as in the 16-bit cache's kernel (k_paged.cu): units of 64 rows
// (32 for more than eight heads) of one (sequence, key head, group of up to 16 query heads), equal contiguous ranges of the list
// of all units to every warp, partial results joined by a second kernel. What differs:
//  * The rows' order inside a unit and the values' order inside a product are free, so fragments are read from shared
//    memory as they lie there, without ldmatrix: a lane takes a quarter of a key row (8 bytes: its codes are the lane's
//    operands of four products), and of value rows the same byte column of four rows, two of which are interleaved by one
//    byte permutation into eight operands. The cached rows, and the values, are the 16 rows of a product, the heads its eight
//    columns, so that one key head for each query head wastes half as much as with the heads as rows; the probabilities are
//    turned over by movmatrix. (tcgen05 takes its operands from shared memory: codes would have to be written there again as 16
//    bits, four times their bytes, for products of 128 rows of which one to sixteen are heads.)
//  * A row's scales and lowest values are made into fp32 factors once, by the lane of its number.
//  * Units are whole tiles of the sequence, so every eight rows of one lie in one page and start on a 16-byte boundary: the
//    tile's pages, one to a lane, are looked up once and counted in blocks of eight rows, and every lane copies 16 bytes at a
//    time (cp.async) into the warp's own ring. (A few bulk copies by as many lanes, counted by an mbarrier, cost more: each
//    lane's copy is issued by itself.) Rows of a tile that are not seen are masked: their codes are numbers whatever they
//    hold, their factors are set to 0.
template <int D, int QR>
struct Dec4Cfg {
  static constexpr int UNIT = QR == 16 ? 32 : 64;                 // rows of a unit
  static constexpr int ROWB = D / 2;                              // bytes of a row's codes
  static constexpr int TILE = UNIT * ROWB;                        // keys, or values, of a unit
  static constexpr int RANGES = 2 * TILE;                         // offset of the keys' ranges, then the values'
  static constexpr int QUERIES = RANGES + UNIT * 8;               // offset of the query rows (where a unit starts a segment)
  static constexpr int STAGE = QUERIES + QR * D * 2;
  static constexpr int FACTORS = 2 * STAGE;                      // the rows' factors: behind two stages
  // one head a key head: its scores of 64 rows, their weights in two fp16 parts, zeros for the products' other columns
  static constexpr int WARP = FACTORS + (QR == 1 ? 256 + 2 * 128 + 32 : UNIT * 16);
  // more than eight heads: with 16 warps their registers spill (16 x 9,000 to 32,000 rows, 48 heads on 4, 53.6 us, with 12 50.8;
  // one sequence of 200,000, 12 on one, 31.4 and 26.2)
  static constexpr int WARPS = QR == 16 ? 12 : 16;
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

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The largest of the lanes' values, in all of them (a NaN is passed over).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
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
__device__ __forceinline__ float4 lds128f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128f(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
// fp16 products: d = a b, and c += a b
__device__ __forceinline__ void mma16_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%10, %10, %10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void sts16(uint32_t a, float x) {   // as fp16, cut off
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(__half_as_ushort(__float2half_rz(x))) : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t cut_half2(float lo, float hi) {
  uint32_t v;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return v;
}
// What fp16 cuts off a number (below 2^-14 less than that); mask 0: the number itself.
constexpr uint32_t kHalfBits = 0xffffe000u;
__device__ __forceinline__ float rest_of(float x) { return x - __uint_as_float(__float_as_uint(x) & kHalfBits); }
// The same of two, as fp16.
__device__ __forceinline__ uint32_t cut_rest2(float lo, float hi, uint32_t mask) {
  const float2 r = add2_rn(make_float2(lo, hi), make_float2(__uint_as_float((__float_as_uint(lo) & mask) ^ 0x80000000u),
                                                            __uint_as_float((__float_as_uint(hi) & mask) ^ 0x80000000u)));
  return cut_half2(r.x, r.y);
}

// An 8 x 8 matrix of 16-bit numbers, a row of pairs to four lanes, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The eight codes of a word as fp16 pairs (code p, code p + 4): r0 and r2 times 2^-24, r1 and r3 times 2^-20.
__device__ __forceinline__ void unpack8(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, uint32_t w) {
  const uint32_t h = w >> 8;
  r0 = w & 0x000f000fu;
  r1 = w & 0x00f000f0u;
  r2 = h & 0x000f000fu;
  r3 = h & 0x00f000f0u;
}

__device__ __forceinline__ float scale_of(uint32_t range) { return __uint_as_float(range << 16); }
__device__ __forceinline__ float low_of(uint32_t range) { return __uint_as_float(range & 0xffff0000u); }
// 2^e for -126 <= e <= 127, and the e with 2^e <= x < 2^(e + 1) (of a normal number's size; -127 below)
__device__ __forceinline__ float exp2_of(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }

// A sequence's rows, from its length (-1: no sequence, -2: more than its table has room for).
__device__ __forceinline__ int rows_of(const PagedCache& c, const Dec4Shape& w, int len) {
  if (len < 0) return -1;
  return static_cast<long long>(len) + w.added > (static_cast<long long>(c.max_pages) << c.page_log2) ? -2 : len + w.added;
}

// A unit's products have the cached rows, or the value columns, as the 16 rows of their first operand, and eight query heads
// as the columns (twice for 9 to 16 heads): lane 4 n + q holds, of every tile of scores, rows n and n + 8 under heads 2 q and
// 2 q + 1. Row n of a tile is row 4 (n % 2) + n / 2 of its eight rows in the cache. Up to four heads stand in the columns twice, so
// that the products with the values take the first parts of their weights and the second ones at once (QR = 4).
__device__ __forceinline__ int row_in_eight(int n) { return (n & 1) * 4 + (n >> 1); }

// Eight heads' queries as second operands, times 2^(14 - e) for 2^e <= the head's largest value < 2^(e + 1). sum: the sums of heads
// 2 q and 2 q + 1, times that; c: the powers of two from a score to the softmax's base-2 exponent. load(row, i): values 8 i .. of one
// of the gn heads (none where gn <= 0); zeros behind them. TWICE: heads 0 to 3 are heads 4 to 7 too.
template <int D>
struct Queries {
  uint32_t f[D / 16][2];
  float sum[2], c[2];
  template <bool TWICE, typename Load>
  __device__ __forceinline__ void take(int gn, int lane, Load&& load) {
    constexpr int C = D / 4;                         // values of a lane: its codes' places
    const int head = TWICE ? (lane >> 2) & 3 : lane >> 2;
    float v[C], top = 0.0f, mine = 0.0f;
#pragma unroll
    for (int w = 0; w < C / 8; ++w) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (head < gn) x = load(head, (lane & 3) * (C / 8) + w);   // (no head behind the last one is read)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 p = unpack_bf16x2((&x.x)[k]);
        v[8 * w + 2 * k] = p.x;
        v[8 * w + 2 * k + 1] = p.y;
        top = fmax3(top, fabsf(p.x), fabsf(p.y));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
    const int e = max(exponent_of(top), -100);
    const float factor = exp2_of(14 - e), back = exp2_of(e - 14);
#pragma unroll
    for (int k = 0; k < C; ++k) {
      v[k] *= factor;
      mine += v[k];
    }
    mine += __shfl_xor_sync(kAll, mine, 1);
    mine += __shfl_xor_sync(kAll, mine, 2);
#pragma unroll
    for (int w = 0; w < C / 8; ++w) {                // pairs (0, 4), (1, 5), (2, 6), (3, 7): as a word of codes unpacks
      f[2 * w][0] = pack_half2(v[8 * w], v[8 * w + 4]);
      f[2 * w][1] = pack_half2(v[8 * w + 1] * 0.0625f, v[8 * w + 5] * 0.0625f);
      f[2 * w + 1][0] = pack_half2(v[8 * w + 2], v[8 * w + 6]);
      f[2 * w + 1][1] = pack_half2(v[8 * w + 3] * 0.0625f, v[8 * w + 7] * 0.0625f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] = __shfl_sync(kAll, mine, 8 * (lane & 3) + 4 * i);
      c[i] = __shfl_sync(kAll, back, 8 * (lane & 3) + 4 * i);
    }
  }
};

// Products q . code of 16 key rows, tile j of s; w: this lane's quarter of rows n and n + 8.
template <int D, int NQ, int NJ>
__device__ __forceinline__ void code_scores(float (&s)[NQ][NJ][4], int j, const Queries<D> (&q)[NQ],
                                            const uint32_t (&w)[2][D / 32]) {
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    uint32_t a[4], b[4];
    unpack8(a[0], a[2], b[0], b[2], w[0][k]);
    unpack8(a[1], a[3], b[1], b[3], w[1][k]);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      if (k == 0) mma16_new(s[i][j], a, q[i].f[0][0], q[i].f[0][1]);
      else mma16(s[i][j], a, q[i].f[2 * k][0], q[i].f[2 * k][1]);
      mma16(s[i][j], b, q[i].f[2 * k + 1][0], q[i].f[2 * k + 1][1]);
    }
  }
}

// O += (code - 8) P for 16 value rows; w: byte columns (of D = 64 words, else half words) of rows q, q + 4, q + 8, q + 12; p:
// probabilities times the rows' scales, as second operands. Tile t of O has values 8 n + 2 t and, in its lower half,
// 8 n + 2 t + 1 as rows (D = 32: 4 n + ..).
template <bool FIRST, int D, int NQ>
__device__ __forceinline__ void add_codes(float (&o)[NQ][D / 16][4], float (&eights)[NQ][4], const uint32_t (&p)[NQ][2],
                                          const uint32_t (&w)[4]) {
  const uint32_t less8[4] = {0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u};
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    if (FIRST) mma16_new(eights[i], less8, p[i][0], p[i][1]);
    else mma16(eights[i], less8, p[i][0], p[i][1]);
  }
  uint32_t x[2][2];                                  // codes 0-3 and, of D = 64, 4-7 of two rows each, side by side
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    x[0][h] = __byte_perm(w[2 * h], w[2 * h + 1], 0x5410);
    if (D == 64) x[1][h] = __byte_perm(w[2 * h], w[2 * h + 1], 0x7632);
  }
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    uint32_t a[4], b[4];
    unpack8(a[0], a[1], b[0], b[1], x[k][0]);
    unpack8(a[2], a[3], b[2], b[3], x[k][1]);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      mma16(o[i][2 * k], a, p[i][0], p[i][1]);
      mma16(o[i][2 * k + 1], b, p[i][0], p[i][1]);
    }
  }
}

// A head's terms, probabilities times their rows' scales, enter the products times 2^(15 - E), kLeast <= E. E is set anew where a
// term may pass it, kRoom above what that takes, so that rows of ordinary sizes rarely do, and where the reference has risen by more
// than kSlack since, which has made all earlier terms smaller: 2^E is at most 2^(1 + kRoom + kSlack) times the largest term.
constexpr int kLeast = -111, kRoom = 4, kSlack = 4;

// What a warp holds of a segment: up to QR heads of one key head. Lane 4 n + q has heads 8 i + 2 q and the next, and of every
// lane's rows its own share of the sums l and off; with one head (QR = 1) all lanes have rows of it.
template <int D, int QR>
struct Segment {
  static constexpr int NQ = (QR + 7) / 8, NT = D / 16;
  static constexpr bool ONE = QR == 1, TWICE = QR == 4;
  Queries<D> qs[NQ];
  float o[NQ][NT][4];                                // times `into`, as off is
  float m[NQ][2], l[NQ][2], off[NQ][2];              // m: the reference
  float into[NQ][2];                                 // 2^(15 - E): 2^E is above every term of the head, at m
  float due[NQ][2];                                  // the reference above which E has to be set anew
  float most;                                        // the largest of all heads' 2^(15 - E)

  template <typename Load>
  __device__ __forceinline__ void start(int gn, int lane, Load&& load) {
    most = exp2_of(15 - kLeast);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[i][k] = -INFINITY;
        l[i][k] = off[i][k] = 0.0f;
        into[i][k] = exp2_of(15 - kLeast);
        due[i][k] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][j][k] = 0.0f;
      qs[i].template take<TWICE>(gn - 8 * i, lane, [&](int r, int u) { return load(8 * i + r, u); });
    }
    if constexpr (ONE) {                             // every lane has rows of the one head
      qs[0].sum[0] = __shfl_sync(kAll, qs[0].sum[0], 0);
      qs[0].c[0] = __shfl_sync(kAll, qs[0].c[0], 0);
    }
  }

  __device__ __forceinline__ float reference(int i, int k) const {
    return m[i][k] == -INFINITY ? 0.0f : m[i][k];    // every score so far -inf: every term is 2^-inf
  }
  __device__ __forceinline__ void multiply(int i, int k, float a) {
    off[i][k] *= a;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      o[i][j][k] *= a;
      o[i][j][2 + k] *= a;
      if constexpr (ONE) {                           // the second parts' column
        o[i][j][1] *= a;
        o[i][j][3] *= a;
      }
    }
  }
  // Raises a head's reference for a largest score of mx. True: its E has to be set anew.
  __device__ __forceinline__ bool raise(int i, int k, float mx) {
    const float before = m[i][k];
    float up = 0.0f;
    if (mx > before) {                               // (rounded upwards: no score is above its reference)
      up = ceilf(__fsub_ru(mx, before));
      m[i][k] = before == -INFINITY ? mx : __fadd_ru(before, up);
    }
    const float a = exp2_of(-static_cast<int>(fminf(up, 127.0f)));
    l[i][k] *= a;
    multiply(i, k, a);
    return m[i][k] > due[i][k];
  }
  // Sets a head's E anew, where the unit's largest term is t.
  __device__ __forceinline__ void fit(int i, int k, float t) {
    const int e = 15 - exponent_of(into[i][k]), need = exponent_of(t);
    const int risen = static_cast<int>(fminf(fmaxf(m[i][k] - due[i][k] + kSlack, 0.0f), 100.0f));
    int up = max(e - risen, kLeast);
    if (need >= up) up = need + 1 + kRoom;
    multiply(i, k, exp2_of(max(e - up, -127)));
    into[i][k] = exp2_of(15 - up);
    due[i][k] = m[i][k] + kSlack;
  }
  __device__ __forceinline__ void fitted() {
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < NQ; ++i) x = fmax3(x, into[i][0], into[i][1]);
    most = warp_max(x);
  }

  // Adds a unit's -8 sum P to its sums of code P.
  __device__ __forceinline__ void centre(const float (&eights)[NQ][4]) {
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          if constexpr (ONE) {
            o[i][j][k] += eights[i][k] + eights[i][k + 1];
          } else {
            const float2 x = add2_rn(make_float2(o[i][j][k], o[i][j][k + 1]), make_float2(eights[i][k], eights[i][k + 1]));
            o[i][j][k] = x.x;
            o[i][j][k + 1] = x.y;
          }
        }
  }

  // 16 rows' products with their values: s, their probabilities times their scales, in two parts.
  template <bool FIRST, int NJ>
  __device__ __forceinline__ void add(const float (&s)[NQ][NJ][4], int j, float (&eights)[NQ][4], const uint32_t (&w)[4],
                                      int lane) {
    uint32_t p[NQ][2];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = s[i][j][2 * h], y = s[i][j][2 * h + 1];
        p[i][h] = transposed(TWICE ? cut_rest2(x, y, (lane & 2) ? kHalfBits : 0u) : cut_half2(x, y));
      }
    add_codes<FIRST, D, NQ>(o, eights, p, w);
    if constexpr (!TWICE) {
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) p[i][h] = transposed(cut_rest2(s[i][j][2 * h], s[i][j][2 * h + 1], kHalfBits));
      add_codes<false, D, NQ>(o, eights, p, w);
    }
  }

  // Scores of the tiles into probabilities times the rows' scales. factors: shared address of the rows' (key scale, key
  // lowest, both in base-2 units, value scale, value lowest + 8 value scale); large: one of the latter may pass a head's 2^E.
  template <int NJ>
  __device__ __forceinline__ void weigh(float (&s)[NQ][NJ][4], uint32_t factors, const uint32_t (&seen)[NJ / 2],
                                        uint32_t unseen, bool large, int lane) {
    const int n8 = lane >> 2;
    float2 vf[2 * NJ];                               // the value rows' factors, of rows 8 r + row_in_eight(n8)
#pragma unroll
    for (int r = 0; r < 2 * NJ; ++r) {
      const float4 f = lds128f(factors + 16 * (8 * r + row_in_eight(n8)));
      vf[r] = make_float2(f.z, f.w);
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float& x = s[i][r >> 1][2 * (r & 1) + k];
          x = fmaf(f.x, x, f.y * qs[i].sum[k]);
        }
    }
    if (unseen) {
#pragma unroll
      for (int r = 0; r < 2 * NJ; ++r)
        if (!((seen[r >> 2] >> (8 * (r & 3) + row_in_eight(n8))) & 1u))
#pragma unroll
          for (int i = 0; i < NQ; ++i) s[i][r >> 1][2 * (r & 1)] = s[i][r >> 1][2 * (r & 1) + 1] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float mx[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = s[i][0][k];
#pragma unroll
        for (int j = 0; j < NJ; ++j) x = j ? fmax3(x, s[i][j][k], s[i][j][2 + k]) : fmaxf(x, s[i][j][2 + k]);
        x *= qs[i].c[k];
        x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
        x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
        mx[k] = fmaxf(x, __shfl_xor_sync(kAll, x, 16));
      }
      bool anew = large;
      if (__any_sync(kAll, mx[0] > m[i][0] || mx[1] > m[i][1])) {   // a higher reference
        const bool x = raise(i, 0, mx[0]), y = raise(i, 1, mx[1]);
        anew = __any_sync(kAll, large || x || y);
      }
      const float2 c = make_float2(qs[i].c[0], qs[i].c[1]), less = make_float2(-reference(i, 0), -reference(i, 1));
      float2 sum = make_float2(l[i][0], l[i][1]);
#pragma unroll
      for (int r = 0; r < 2 * NJ; ++r) {
        float* x = &s[i][r >> 1][2 * (r & 1)];
        const float2 d = fma2_rn(make_float2(x[0], x[1]), c, less);
        x[0] = ex2_approx(d.x);
        x[1] = ex2_approx(d.y);
        sum = add2_rn(sum, make_float2(x[0], x[1]));
      }
      l[i][0] = sum.x;
      l[i][1] = sum.y;
      if (anew) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float t = 0.0f;
#pragma unroll
          for (int r = 0; r < 2 * NJ; ++r) t = fmaxf(t, s[i][r >> 1][2 * (r & 1) + k] * fmaxf(vf[r].x, fabsf(vf[r].y)));
          t = fmaxf(t, __shfl_xor_sync(kAll, t, 4));
          t = fmaxf(t, __shfl_xor_sync(kAll, t, 8));
          fit(i, k, fmaxf(t, __shfl_xor_sync(kAll, t, 16)));
        }
        fitted();
      }
#pragma unroll
      for (int r = 0; r < 2 * NJ; ++r) {
        float* x = &s[i][r >> 1][2 * (r & 1)];
        const float2 p = mul2_rn(make_float2(x[0], x[1]), make_float2(into[i][0], into[i][1]));
        off[i][0] = fmaf(p.x, vf[r].y, off[i][0]);
        off[i][1] = fmaf(p.y, vf[r].y, off[i][1]);
        const float2 t = mul2_rn(p, make_float2(vf[r].x, vf[r].x));
        x[0] = t.x;
        x[1] = t.y;
      }
    }
  }

  // The same of one head: s has the products in lanes 4 n, which go round the warp in shared memory (128 NH bytes at `room`),
  // 32 rows to a value of x and of the rows' factors; x becomes the rows' probabilities times their scales.
  template <int NH, int NJ>
  __device__ __forceinline__ void weigh_one(const float (&s)[1][NJ][4], float (&x)[NH], uint32_t room,
                                            const float (&ks)[NH], const float (&kl)[NH], const float (&vs)[NH],
                                            const float (&vl)[NH], const uint32_t (&seen)[NH], uint32_t unseen, bool large, int lane) {
    if ((lane & 3) == 0) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
        sts128f(room + NH * 4 * lane + 16 * h, s[0][2 * h][0], s[0][2 * h][2], s[0][2 * h + 1][0], s[0][2 * h + 1][2]);
    }
    __syncwarp();
    // row 8 v + i of the tile is value v of lane 4 n with row_in_eight(n) = i
    const uint32_t mine = room + NH * 16 * (2 * (lane & 3) + ((lane >> 2) & 1)) + 4 * (lane >> 3);
    float mx = -INFINITY;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      x[h] = fmaf(ks[h], __uint_as_float(lds32(mine + 16 * h)), kl[h] * qs[0].sum[0]);
      if (unseen && !((seen[h] >> lane) & 1u)) x[h] = -INFINITY;
      mx = fmaxf(mx, x[h]);
    }
    mx = warp_max(mx * qs[0].c[0]);
    bool anew = large;
    if (mx > m[0][0]) anew = raise(0, 0, mx) || large;   // a higher reference (the same for all lanes)
    const float ref = reference(0, 0);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      x[h] = ex2_approx(fmaf(x[h], qs[0].c[0], -ref));
      l[0][0] += x[h];
    }
    if (anew) {
      float t = 0.0f;
#pragma unroll
      for (int h = 0; h < NH; ++h) t = fmaxf(t, x[h] * fmaxf(vs[h], fabsf(vl[h])));
      fit(0, 0, warp_max(t));
      most = into[0][0];
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const float p = x[h] * into[0][0];
      off[0][0] = fmaf(p, vl[h], off[0][0]);
      x[h] = p * vs[h];
    }
  }

  // Heads whose values a lane has: NK of each eight, those of `head`. With every head in the columns twice a lane takes one of its
  // two, and gives the other's to the lane that has its other part.
  static constexpr int NK = TWICE ? 1 : 2;
  static __device__ __forceinline__ int head(int i, int k, int lane) {
    return TWICE ? 2 * (lane & 1) + ((lane >> 1) & 1) : 8 * i + 2 * (lane & 3) + k;
  }
  static __device__ __forceinline__ float of(const float (&x)[2], int k, int lane) { return TWICE ? (lane & 2 ? x[1] : x[0]) : x[k]; }
  __device__ __forceinline__ float maximum(int i, int k, int lane) const { return of(m[i], k, lane); }
  // Its values D / 8 n .., not divided by the sum, which is returned.
  __device__ __forceinline__ float values(int i, int k, int lane, float (&v)[D / 8]) const {
    float lt = of(l[i], k, lane), ot = of(off[i], k, lane);
#pragma unroll
    for (int x = ONE ? 1 : 4; x < 32; x <<= 1) {
      lt += __shfl_xor_sync(kAll, lt, x);
      ot += __shfl_xor_sync(kAll, ot, x);
    }
    const int e = -exponent_of(of(into[i], k, lane));
    const float back = exp2_of(e / 2), rest = exp2_of(e - e / 2);   // 1 / into in two steps
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = o[i][j][2 * h], b = o[i][j][2 * h + 1];
        if constexpr (ONE) x[h] = a + b;             // the two parts
        else if constexpr (TWICE) x[h] = (lane & 2 ? b : a) + __shfl_xor_sync(kAll, lane & 2 ? a : b, 2);
        else x[h] = k ? b : a;
      }
      v[2 * j] = fmaf(x[0], 16777216.0f, ot) * back * rest;   // 2^24 and 2^20
      v[2 * j + 1] = fmaf(x[1], 1048576.0f, ot) * back * rest;
    }
    return lt;
  }
};

// A row's probability times its scale as part of a second operand: lane q of head 0 takes of the rows 8 v the rows q and q + 4
// of every v, NV words of fp16 pairs at `weights`.
template <int NV>
__device__ __forceinline__ uint32_t weight_place(int row) {
  return 4 * (NV * (row & 3) + (row >> 3)) + 2 * ((row >> 2) & 1);
}

// The tiles of UNIT rows that hold the rows which a sequence's query sees, of n rows: v < head at the start, then from `gap`
// tiles on.
struct Tiles {
  int n, head, gap, count;
};
template <int UNIT>
__device__ __forceinline__ Tiles tiles_of(int n, int window, int sinks) {
  Tiles t;
  t.n = n;
  t.count = (n + UNIT - 1) / UNIT;
  t.head = t.count;
  t.gap = 0;
  if (window > 0 && window < n) {
    const int first = n - window, from = first / UNIT;   // the first row of the window, and its tile
    t.head = min((min(sinks, first) + UNIT - 1) / UNIT, from);
    t.gap = from - t.head;
    t.count -= t.gap;
  }
  return t;
}
template <int UNIT>
__device__ __forceinline__ int first_row(const Tiles& t, int v) { return (v < t.head ? v : v + t.gap) * UNIT; }

// A warp's part of a segment: tiles [t0, t1) of the rows that a sequence's query sees, of one key head and a group of its query
// heads.
struct Piece {
  int b, kh, mt, t0, t1;
  Tiles t;
};

template <int D, int QR>
__global__ void __launch_bounds__(32 * Dec4Cfg<D, QR>::WARPS, 1)
paged4_split_kernel(PagedCache c, const uint32_t* __restrict__ ranges, const __nv_bfloat16* __restrict__ qkv,
                    const int32_t* __restrict__ lens, __nv_bfloat16* __restrict__ y, float* __restrict__ lse2, Dec4Shape w,
                    Dec4Scratch ws, int* err) {
  using Cfg = Dec4Cfg<D, QR>;
  constexpr int ROWB = Cfg::ROWB, UNIT = Cfg::UNIT, NT = D / 16, NQ = (QR + 7) / 8, NJ = UNIT / 16, NH = UNIT / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  int* s_prefix = reinterpret_cast<int*>(smem + nwarps * Cfg::WARP);     // [B + 1]
  int* s_rows = s_prefix + w.B + 1;                                      // [B]
  __shared__ int s_sum[Cfg::WARPS];
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
      x = tiles_of<UNIT>(rows, w.window, w.sinks).count;
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

  int left = count;                                  // units behind the pieces made so far
  auto cut_piece = [&](Piece& x) {
    x.t1 = min(x.t.count, x.t0 + left);
    left -= x.t1 - x.t0;
  };
  auto next_piece = [&](Piece& x) {
    x.t0 = 0;
    if (++x.mt == w.mg) {
      x.mt = 0;
      if (++x.kh == c.Hkv) {
        x.kh = 0;
        do ++x.b; while (s_prefix[x.b + 1] == s_prefix[x.b]);   // (a sequence with units follows)
        x.t = tiles_of<UNIT>(s_rows[x.b], w.window, w.sinks);
      }
    }
    cut_piece(x);
  };
  Piece at;                                          // the piece that is computed
  {
    const int target = static_cast<int>(u0 / HM);    // the sequence with prefix[b] <= target < prefix[b + 1]
    int lo = 0, hi = w.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_prefix[mid + 1] > target) hi = mid;
      else lo = mid + 1;
    }
    at.b = lo;
    at.t = tiles_of<UNIT>(s_rows[lo], w.window, w.sinks);
    const long long r = u0 - static_cast<long long>(s_prefix[lo]) * HM;
    const int hm = static_cast<int>(r / at.t.count);
    at.kh = hm / w.mg;
    at.mt = hm - at.kh * w.mg;
    at.t0 = static_cast<int>(r - static_cast<long long>(hm) * at.t.count);
    cut_piece(at);
  }
  Piece next = at;                                   // and the one behind it
  bool more = left > 0;
  if (more) next_piece(next);
  // A copy of the warp takes 512 bytes: RPC rows' codes. Eight rows of a head lie side by side, and the pool is counted in
  // such blocks (32 bits: 2^32 of them are more than the memory holds): lanes below UNIT / 8 know those of the unit that is
  // copied next, and every lane copies 16 bytes of block `block` (of the first copy; RPC / 8 on for each further one). Of the
  // ranges it copies four rows' of the keys (lanes below UNIT / 4) or of the values.
  constexpr int RPC = 512 / ROWB, COPIES = UNIT / RPC, PER8 = ROWB / 2;   // PER8: lanes that copy a block's codes
  constexpr uint32_t kNoBlock = 0xffffffffu;
  const int block = lane / PER8, pmask = (1 << c.page_log2) - 1;
  const uint32_t page_blocks = static_cast<uint32_t>(c.Hkv) << (c.page_log2 - 2);   // of a page: keys, then values
  const uint8_t* kfrom = static_cast<const uint8_t*>(c.pool) + (lane % PER8) * 16;
  const uint8_t* vfrom = kfrom + static_cast<size_t>(page_blocks / 2) * (8 * ROWB);
  const int rrow = 4 * (lane % (UNIT / 4));
  const uint8_t* rfrom = reinterpret_cast<const uint8_t*>(ranges) + (lane / (UNIT / 4) ? page_blocks * 16 : 0u) + (rrow & 4) * 4;
  bool wanted = false;                               // whether this lane has eight rows of it, their page
  int pg = -1;
  uint32_t in_page = 0;                              // and their block in it
  auto look_up = [&](const Piece& x, int tile) {
    const int r = first_row<UNIT>(x.t, tile) + 8 * lane;
    // (no page of eight rows that are all out of sight: it need not exist)
    wanted = lane < UNIT / 8 && r < x.t.n && (w.window == 0 || r + 7 >= x.t.n - w.window || r < w.sinks);
    pg = wanted ? __ldg(c.table + static_cast<size_t>(x.b) * c.max_pages + (r >> c.page_log2)) : -1;
    in_page = ((static_cast<uint32_t>(x.kh) << c.page_log2) + (r & pmask)) >> 3;
  };
  // Returns the unit's eight rows whose page does not exist (a bit each): what stands in their place in the ring is not theirs.
  auto copy_rows = [&](uint32_t to) {
    const bool there = static_cast<unsigned>(pg) < static_cast<unsigned>(c.pages);
    const uint32_t blk = there ? static_cast<uint32_t>(pg) * page_blocks + in_page : kNoBlock;
    const uint32_t lost = __ballot_sync(kAll, wanted && !there);
    if (wanted && !there) record_error(err, GPT_DEV_EPAGE);
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const uint32_t mine = __shfl_sync(kAll, blk, block + i * (RPC / 8));
      if (mine != kNoBlock) {
        copy16(to + lane * 16 + i * 512, kfrom + static_cast<size_t>(mine) * (8 * ROWB));
        copy16(to + Cfg::TILE + lane * 16 + i * 512, vfrom + static_cast<size_t>(mine) * (8 * ROWB));
      }
    }
    const uint32_t mine = __shfl_sync(kAll, blk, rrow / 8);
    if (mine != kNoBlock && lane < UNIT / 2) copy16(to + Cfg::RANGES + lane * 16, rfrom + static_cast<size_t>(mine) * 32);
    return lost;
  };
  auto copy_queries = [&](const Piece& x, uint32_t to) {
    const int gn = min(w.G - x.mt * 16, 16);
    const __nv_bfloat16* tok = qkv + (static_cast<size_t>(x.b) * row + x.kh * w.G + x.mt * 16) * D;
#pragma unroll
    for (int i = 0; i < (QR * D + 255) / 256; ++i)
      if (32 * i + lane < gn * (D / 8)) copy16(to + Cfg::QUERIES + (32 * i + lane) * 16, tok + 8 * (32 * i + lane));
  };

  constexpr bool ONE = QR == 1;
  Segment<D, QR> g;
  const int n8 = lane >> 2, q4 = lane & 3;
  const uint32_t factors = ring + Cfg::FACTORS;
  if constexpr (ONE) {
    if (lane < 2) sts128f(factors + 256 + 2 * 128 + 16 * lane, 0.0f, 0.0f, 0.0f, 0.0f);
  }
  uint32_t st = ring, other = ring + Cfg::STAGE;     // the stage that is read, and the one that is filled meanwhile
  look_up(at, at.t0);
  uint32_t lost = copy_rows(st), lost_next = 0;      // of the stage that is read, and of the other
  copy_queries(at, st);
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (at.t0 + 1 < at.t1) look_up(at, at.t0 + 1);
  uint32_t slot0 = 0;                                // of the two places for partial results
  while (true) {
    for (int tile = at.t0; tile < at.t1; ++tile) {
      if (tile + 1 < at.t1) {
        lost_next = copy_rows(other);
        if (tile + 2 < at.t1) look_up(at, tile + 2);
        else if (more) look_up(next, 0);
      } else if (more) {
        if (at.t1 == at.t0 + 1) look_up(next, 0);      // (of pieces of one tile not before now)
        lost_next = copy_rows(other);
        copy_queries(next, other);
        if (next.t1 > 1) look_up(next, 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      if (tile == at.t0)
        g.start(min(w.G - at.mt * 16, 16), lane,
                [&](int r, int u) { return lds128(st + Cfg::QUERIES + (r * (D / 8) + u) * 16); });
      const int f = first_row<UNIT>(at.t, tile), after = at.t.n - w.window;   // the window's first row
      uint32_t seen[NH], unseen = 0u;                  // the tile's rows that are
      float ks[NH], kl[NH], vs[NH], vl[NH], size = 0.0f;   // the factors of rows `lane` and, of a unit of 64, 32 + lane
      {
        const bool cut = lost || f + UNIT > at.t.n || (w.window > 0 && f < after && f + UNIT > w.sinks);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const uint32_t kr = lds32(st + Cfg::RANGES + 4 * (32 * h + lane));
          uint32_t vr = lds32(st + Cfg::RANGES + 4 * (UNIT + 32 * h + lane));
          seen[h] = kAll;
          if (cut) {
            const int r = f + 32 * h + lane;
            const bool mine = r < at.t.n && (w.window == 0 || r >= after || r < w.sinks) &&
                              !((lost >> (4 * h + (lane >> 3))) & 1u);
            seen[h] = __ballot_sync(kAll, mine);
            if (!mine) vr = 0u;
          }
          unseen |= ~seen[h];
          ks[h] = scale_of(kr) * (16777216.0f * w.scale_log2);
          kl[h] = low_of(kr) * w.scale_log2;
          vs[h] = scale_of(vr);
          vl[h] = fmaf(8.0f, vs[h], low_of(vr));
          size = fmax3(size, vs[h], fabsf(vl[h]));
          if constexpr (!ONE) sts128f(factors + 16 * (32 * h + lane), ks[h], kl[h], vs[h], vl[h]);
        }
      }
      const bool large = __any_sync(kAll, size * g.most >= 32768.0f);
      float s[NQ][NJ][4], eights[NQ][4];
      const uint32_t krow = st + row_in_eight(n8) * ROWB + q4 * (D / 8), vcol = st + Cfg::TILE + q4 * ROWB + n8 * (D / 16);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t x[2][D / 32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (D == 64) {
            const uint2 u = lds64(krow + (16 * j + 8 * h) * ROWB);
            x[h][0] = u.x;
            x[h][1] = u.y;
          } else {
            x[h][0] = lds32(krow + (16 * j + 8 * h) * ROWB);
          }
        }
        code_scores<D, NQ, NJ>(s, j, g.qs, x);
      }
      auto value_words = [&](uint32_t (&x)[4], int j) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if constexpr (D == 64) x[h] = lds32(vcol + (16 * j + 4 * h) * ROWB);
          else x[h] = lds16(vcol + (16 * j + 4 * h) * ROWB);
        }
      };
      if constexpr (ONE) {
        float x[NH];
        g.weigh_one(s, x, factors, ks, kl, vs, vl, seen, unseen, large, lane);
        const uint32_t weights = factors + 256;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const uint32_t to = weights + weight_place<2 * NJ>(32 * h + lane);
          sts16(to, x[h]);
          sts16(to + 128, rest_of(x[h]));
        }
        __syncwarp();
        const uint32_t pa = weights + (n8 < 2 ? 128 * n8 + 32 * q4 : 256);   // the parts' columns; others: zeros
        const uint32_t step = n8 < 2 ? 16 : 0;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const uint4 w4 = lds128(pa + step * h);
          const uint32_t p0[1][2] = {{w4.x, w4.y}}, p1[1][2] = {{w4.z, w4.w}};
          uint32_t u[4];
          value_words(u, 2 * h);
          if (h == 0) add_codes<true, D, NQ>(g.o, eights, p0, u);
          else add_codes<false, D, NQ>(g.o, eights, p0, u);
          value_words(u, 2 * h + 1);
          add_codes<false, D, NQ>(g.o, eights, p1, u);
        }
      } else {
        __syncwarp();
        g.weigh(s, factors, seen, unseen, large, lane);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          uint32_t u[4];
          value_words(u, j);
          if (j == 0) g.template add<true>(s, j, eights, u, lane);
          else g.template add<false>(s, j, eights, u, lane);
        }
      }
      g.centre(eights);
      const uint32_t swap = st;
      st = other;
      other = swap;
      lost = lost_next;
      __syncwarp();                                    // the stage and the factors are read before they are filled again
    }
    const bool whole = at.t0 == 0 && at.t1 == at.t.count;   // the piece is the segment
    const size_t slot = static_cast<size_t>(gw) * 2 + slot0;
    const int gn = min(w.G - at.mt * 16, 16);
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int k = 0; k < g.NK; ++k) {
        float v[D / 8];                               // values D / 8 n8 .. of the head
        const float lt = g.values(i, k, lane, v), mx = g.maximum(i, k, lane);
        const int r = g.head(i, k, lane);
        if (r >= gn) continue;
        if (whole) {
          const size_t head = static_cast<size_t>(at.b) * w.H + at.kh * w.G + at.mt * 16 + r;
          const float inv = 1.0f / lt;                // (a sum of 0, every score -inf, gives NaN)
          uint32_t h[D / 16];
#pragma unroll
          for (int j = 0; j < NT; ++j) h[j] = pack_bf16x2(v[2 * j] * inv, v[2 * j + 1] * inv);
          if constexpr (D == 64) *reinterpret_cast<uint4*>(y + head * D + 8 * n8) = make_uint4(h[0], h[1], h[2], h[3]);
          else *reinterpret_cast<uint2*>(y + head * D + 4 * n8) = make_uint2(h[0], h[1]);
          if (n8 == 0 && lse2) lse2[head] = mx + log2f(lt);
        } else {
          float4* dst = reinterpret_cast<float4*>(ws.o + (slot * QR + r) * D + n8 * (D / 8));
#pragma unroll
          for (int x = 0; x < D / 32; ++x) dst[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
          if (n8 == 0) ws.ml[slot * QR + r] = make_float2(mx, lt);
        }
      }
    if (!more) break;
    at = next;
    slot0 = 1;
    more = left > 0;
    if (more) next_piece(next);
  }
}

// The same attention where the rows that can be seen fit the warps of one cluster, UPW units of 32 rows a warp: one launch, no
// scratch. Blocks behind a sequence's last unit leave at once. Codes and ranges go from the cache straight into the lanes
// that use them, all at once; each block adds up its warps' outputs in shared memory and pushes them to the block that joins
// that query row, and its maxima and sums to every block; one cluster barrier. Bound by latency.
template <int D, int QR>
__global__ void __launch_bounds__(256, QR == 16 ? 1 : 2)
paged4_short_kernel(PagedCache c, const uint32_t* __restrict__ ranges, const __nv_bfloat16* __restrict__ qkv,
                    const int32_t* __restrict__ lens, __nv_bfloat16* __restrict__ y, float* __restrict__ lse2, Dec4Shape w, int upw,
                    int* err) {
  constexpr int ROWB = D / 2, NQ = (QR + 7) / 8, UNIT = 32;
  constexpr bool ONE = QR == 1;
  __shared__ __align__(16) float s_own[8][QR][D];    // the warps' outputs
  __shared__ __align__(16) float s_factors[8][ONE ? 32 + 2 * 16 + 4 : UNIT * 4];
  __shared__ float2 s_ml[8][QR];                     // the warps' maxima and sums
  __shared__ float2 s_all[8][QR];                    // the blocks', pushed by each of them
  __shared__ float s_o[QR + 7][D];                   // pushed outputs: [row / NB * NB + block][D]
  auto cluster = cooperative_groups::this_cluster();
  const int NC = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n8 = lane >> 2, q4 = lane & 3;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // every block has started (awaited below)
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, hm = static_cast<int>(blockIdx.x) / NC;
  const int kh = hm / w.mg, g0 = (hm - kh * w.mg) * 16, gn = min(w.G - g0, 16);
  const int pmask = (1 << c.page_log2) - 1;
  const int32_t* trow = c.table + static_cast<size_t>(b) * c.max_pages;
  const __nv_bfloat16* tok = qkv + (static_cast<size_t>(b) * (w.H + 2 * c.Hkv) + kh * w.G + g0) * D;
  const size_t head0 = static_cast<size_t>(b) * w.H + kh * w.G + g0;
  const int len = __ldg(lens + b);
  // the first unit's pages, on their way before the length is known: right unless a window cuts
  const int guess = (rank * upw * 8 + warp) * UNIT;
  int page = __ldg(trow + min((guess + lane) >> c.page_log2, c.max_pages - 1));
  Segment<D, QR> g;
  g.start(gn, lane,
          [&](int r, int u) { return __ldg(reinterpret_cast<const uint4*>(tok + static_cast<size_t>(r) * D) + u); });
  const int n = rows_of(c, w, len);
  if (n <= 0) {                                      // (the same for the whole cluster)
    if (n == -2 && rank == 0 && tid == 0) record_error(err, GPT_DEV_EPAGE);
    if (n == 0 && rank == 0) {
      for (int i = tid; i < gn * D; i += 256) y[head0 * D + i] = __float2bfloat16(0.0f);
      if (lse2 && tid < gn) lse2[head0 + tid] = -INFINITY;
    }
    return;
  }
  const Tiles t = tiles_of<UNIT>(n, w.window, w.sinks);
  const int NB = (t.count + 8 * upw - 1) / (8 * upw);   // blocks that hold units
  if (rank >= NB) return;                            // (whole blocks: barriers wait for the others only)
  const size_t prows = static_cast<size_t>(2 * c.Hkv) << c.page_log2, vrows = prows / 2;
  const uint8_t* codes = static_cast<const uint8_t*>(c.pool);
  const uint32_t factors = smem_u32(&s_factors[warp][0]);
  if constexpr (ONE) {
    if (lane == 0) sts128f(factors + 256, 0.0f, 0.0f, 0.0f, 0.0f);
  }
  for (int u = 0; u < upw; ++u) {
    const int unit = (rank * upw + u) * 8 + warp;
    if (unit >= t.count) break;
    const int r0 = first_row<UNIT>(t, unit), mine = r0 + lane;
    if (r0 != guess) page = mine < n ? __ldg(trow + (mine >> c.page_log2)) : 0;
    const bool in_sight = mine < n && (w.window == 0 || mine >= n - w.window || mine < w.sinks);   // (others' pages need not exist)
    const bool is_seen = in_sight && static_cast<unsigned>(page) < static_cast<unsigned>(c.pages);
    if (in_sight && !is_seen) record_error(err, GPT_DEV_EPAGE);
    // eight rows lie in one page: theirs, from the lane of the first one
    const uint32_t have = __ballot_sync(kAll, is_seen);
    uint32_t kw[4][D / 32], vw[8];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const size_t row = static_cast<size_t>(static_cast<uint32_t>(__shfl_sync(kAll, page, 8 * r))) * prows +
                         (static_cast<size_t>(kh) << c.page_log2) + ((r0 + 8 * r) & pmask);
      const bool ok = (have >> (8 * r)) & 255u;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) kw[r][k] = 0u;
      vw[2 * r] = vw[2 * r + 1] = 0u;
      if (!ok) continue;
      const uint8_t* k8 = codes + (row + row_in_eight(n8)) * ROWB + q4 * (D / 8);
      const uint8_t* v8 = codes + (row + vrows + q4) * ROWB + n8 * (D / 16);
      if constexpr (D == 64) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(k8));
        kw[r][0] = x.x;
        kw[r][1] = x.y;
        vw[2 * r] = __ldg(reinterpret_cast<const uint32_t*>(v8));
        vw[2 * r + 1] = __ldg(reinterpret_cast<const uint32_t*>(v8 + 4 * ROWB));
      } else {
        kw[r][0] = __ldg(reinterpret_cast<const uint32_t*>(k8));
        vw[2 * r] = __ldg(reinterpret_cast<const uint16_t*>(v8));
        vw[2 * r + 1] = __ldg(reinterpret_cast<const uint16_t*>(v8 + 4 * ROWB));
      }
    }
    uint32_t kr = 0u, vr = 0u;                       // row `lane`'s ranges
    if (is_seen) {
      const size_t row = static_cast<size_t>(static_cast<uint32_t>(page)) * prows + (static_cast<size_t>(kh) << c.page_log2) +
                         (mine & pmask);
      kr = __ldg(ranges + row);
      vr = __ldg(ranges + row + vrows);
    }
    const uint32_t seen[1] = {have};
    float ks[1] = {scale_of(kr) * (16777216.0f * w.scale_log2)}, kl[1] = {low_of(kr) * w.scale_log2}, vs[1] = {scale_of(vr)};
    float vl[1] = {fmaf(8.0f, vs[0], low_of(vr))};
    const bool large = __any_sync(kAll, fmaxf(vs[0], fabsf(vl[0])) * g.most >= 32768.0f);
    float s[NQ][2][4], eights[NQ][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t x[2][D / 32];
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        x[0][k] = kw[2 * j][k];
        x[1][k] = kw[2 * j + 1][k];
      }
      code_scores<D, NQ, 2>(s, j, g.qs, x);
    }
    if constexpr (ONE) {
      float x[1];
      g.weigh_one(s, x, factors, ks, kl, vs, vl, seen, ~seen[0], large, lane);
      const uint32_t to = factors + 128 + weight_place<4>(lane);
      sts16(to, x[0]);
      sts16(to + 64, rest_of(x[0]));
      __syncwarp();
      const uint4 w4 = lds128(factors + 128 + (n8 < 2 ? 64 * n8 + 16 * q4 : 128));   // the parts' columns; others: zeros
      const uint32_t p0[1][2] = {{w4.x, w4.y}}, p1[1][2] = {{w4.z, w4.w}};
      const uint32_t u0[4] = {vw[0], vw[1], vw[2], vw[3]}, u1[4] = {vw[4], vw[5], vw[6], vw[7]};
      add_codes<true, D, NQ>(g.o, eights, p0, u0);
      add_codes<false, D, NQ>(g.o, eights, p1, u1);
    } else {
      sts128f(factors + 16 * lane, ks[0], kl[0], vs[0], vl[0]);
      __syncwarp();
      g.weigh(s, factors, seen, ~seen[0], large, lane);
      const uint32_t u0[4] = {vw[0], vw[1], vw[2], vw[3]}, u1[4] = {vw[4], vw[5], vw[6], vw[7]};
      g.template add<true>(s, 0, eights, u0, lane);
      g.template add<false>(s, 1, eights, u1, lane);
    }
    g.centre(eights);
    __syncwarp();                                    // the factors are read before they are written again
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i)
#pragma unroll
    for (int k = 0; k < g.NK; ++k) {
      float v[D / 8];
      const float lt = g.values(i, k, lane, v);
      const int r = g.head(i, k, lane);
      if (r >= gn) continue;
#pragma unroll
      for (int x = 0; x < D / 32; ++x)
        *reinterpret_cast<float4*>(&s_own[warp][r][n8 * (D / 8) + 4 * x]) = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
      if (n8 == 0) s_ml[warp][r] = make_float2(g.maximum(i, k, lane), lt);
    }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  // this block's maximum, sum and output of each row, to the blocks that want them
  for (int i = tid; i < gn * D; i += 256) {
    const int r = i / D, d = i % D;
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, s_ml[k][r].x);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float lt = 0.0f, acc = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = ex2_approx(s_ml[k][r].x - ref);
      lt += s_ml[k][r].y * f;
      acc += s_own[k][r][d] * f;
    }
    cluster.map_shared_rank(&s_o[0][0], r % NB)[(r / NB * NB + rank) * D + d] = acc;
    if (d < NB) cluster.map_shared_rank(&s_all[0][0], d)[rank * QR + r] = make_float2(mx, lt);
  }
  cluster.sync();
  for (int i = tid; i < (gn + NB - 1) / NB * D; i += 256) {
    const int r = i / D * NB + rank, d = i % D;
    if (r >= gn) continue;
    float mx = -INFINITY;
    for (int k = 0; k < NB; ++k) mx = fmaxf(mx, s_all[k][r].x);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float lt = 0.0f, acc = 0.0f;
    for (int k = 0; k < NB; ++k) {
      const float f = ex2_approx(s_all[k][r].x - ref);
      lt += s_all[k][r].y * f;
      acc += s_o[r / NB * NB + k][d] * f;
    }
    y[(head0 + r) * D + d] = __float2bfloat16(acc / lt);
    if (d == 0 && lse2) lse2[head0 + r] = mx + log2f(lt);
  }
}

// Joins the partial results of a (sequence, query head) in a fixed order, D / 4 threads to a piece, four pieces of a thread on
// their way at once; sequences of no rows get zeros and -inf. (A block for all heads of a key head, one after another, took 126
// of 133 us for one sequence of 4,000 rows, 16 heads on one.) Bound by latency: the lists' start, then the pieces.
constexpr int kJoin4Pieces = 4;

template <int D, int QR>
__global__ void __launch_bounds__(1024)
paged4_join_kernel(PagedCache c, const int32_t* __restrict__ lens, __nv_bfloat16* __restrict__ y, float* __restrict__ lse2,
                   Dec4Shape w, Dec4Scratch ws, int warps) {
  pdl_wait();
  pdl_trigger();
  constexpr int LANES = D / 4;
  __shared__ __align__(16) float s_o[32][D];
  __shared__ float s_m[32], s_l[32];
  const int P = static_cast<int>(blockDim.x) / LANES, W = static_cast<int>(blockDim.x) / 32;
  const int b = blockIdx.y, h = blockIdx.x, kh = h / w.G, mt = (h - kh * w.G) / 16, r = (h - kh * w.G) % 16;
  const int HM = c.Hkv * w.mg, p0 = ws.prefix[b], nt = ws.prefix[b + 1] - p0;
  const long long total = static_cast<long long>(ws.prefix[w.B]) * HM;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, d4 = tid % LANES, part = tid / LANES;
  const size_t head = static_cast<size_t>(b) * w.H + h;
  if (nt == 0) {
    if (rows_of(c, w, __ldg(lens + b)) != 0) return;
    if (tid < D) y[head * D + tid] = __float2bfloat16(0.0f);
    if (tid == 0 && lse2) lse2[head] = -INFINITY;
    return;
  }
  const Deal deal(total, warps);
  const long long t0 = static_cast<long long>(p0) * HM + static_cast<long long>(kh * w.mg + mt) * nt, t1 = t0 + nt;
  const int g1 = deal.warp_of(t0), g2 = deal.warp_of(t1 - 1);   // the warps that hold the first unit and the last
  if (g1 == g2) return;                              // one warp held it all and wrote the output
  // a piece is its warp's first (slot 0) unless its segment starts behind the warp's start: only g1's can
  const size_t slot1 = static_cast<size_t>(g1) * 2 + (deal.start(g1) == t0 ? 0 : 1);
  float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](float m2, float l2, const float4& o2) {
    const float mn = fmaxf(m, m2), ref = mn == -INFINITY ? 0.0f : mn;
    const float f = ex2_approx(m - ref), e = ex2_approx(m2 - ref);
    m = mn;
    l = l * f + l2 * e;
    acc[0] = acc[0] * f + o2.x * e;
    acc[1] = acc[1] * f + o2.y * e;
    acc[2] = acc[2] * f + o2.z * e;
    acc[3] = acc[3] * f + o2.w * e;
  };
  for (int g0 = g1 + part; g0 <= g2; g0 += kJoin4Pieces * P) {
    float2 x[kJoin4Pieces];
    float4 o[kJoin4Pieces];
#pragma unroll
    for (int k = 0; k < kJoin4Pieces; ++k) {
      const int g = g0 + k * P;
      x[k] = make_float2(-INFINITY, 0.0f);
      o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (g <= g2) {
        const size_t sl = (g == g1 ? slot1 : static_cast<size_t>(g) * 2) * QR + r;
        x[k] = ws.ml[sl];
        o[k] = *reinterpret_cast<const float4*>(ws.o + sl * D + 4 * d4);
      }
    }
#pragma unroll
    for (int k = 0; k < kJoin4Pieces; ++k) add(x[k].x, x[k].y, o[k]);
  }
#pragma unroll
  for (int k = LANES; k < 32; k <<= 1) {             // the parts of a warp
    const float m2 = __shfl_xor_sync(kAll, m, k), l2 = __shfl_xor_sync(kAll, l, k);
    const float4 o2 = make_float4(__shfl_xor_sync(kAll, acc[0], k), __shfl_xor_sync(kAll, acc[1], k),
                                  __shfl_xor_sync(kAll, acc[2], k), __shfl_xor_sync(kAll, acc[3], k));
    add(m2, l2, o2);
  }
  if (lane < LANES) {
    *reinterpret_cast<float4*>(&s_o[warp][4 * d4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
  }
  __syncthreads();
  if (tid >= D) return;
  float mx = -INFINITY;
#pragma unroll 8
  for (int k = 0; k < W; ++k) mx = fmaxf(mx, s_m[k]);
  const float ref = mx == -INFINITY ? 0.0f : mx;
  float lt = 0.0f, at = 0.0f;
#pragma unroll 8
  for (int k = 0; k < W; ++k) {
    const float f = ex2_approx(s_m[k] - ref);
    lt += s_l[k] * f;
    at += s_o[k][tid] * f;
  }
  y[head * D + tid] = __float2bfloat16(at / lt);
  if (tid == 0 && lse2) lse2[head] = mx + log2f(lt);
}

template <int D, int QR>
cudaError_t launch_decode4(const PagedCache& c, const uint32_t* ranges, const __nv_bfloat16* qkv, const int32_t* lens,
                           __nv_bfloat16* y, float* lse2, const Dec4Shape& w, int* err, cudaStream_t s) {
  using Cfg = Dec4Cfg<D, QR>;
  static SmemLimit limit;
  int dev = 0, num_sms = 0;
  cudaError_t e = device_sms(&dev, &num_sms);
  if (e != cudaSuccess) return e;
  // Few rows in sight: one launch of clusters, eight blocks at most, with as many units a warp as that takes. It pays while
  // there are not many more blocks than run at once (of more than eight heads on one, whose blocks take more registers, one an
  // SM), and not many units behind each other. Graph replays, against the general form: 12 heads, 12 sequences of 1,000 rows 8.7
  // and 9.7 us, 14 11.5 and 11.4, 32 22.6 and 14.1; 4 of 4,000 rows 10.7 and 11.3, 8 16.2 and 12.7; one of 12,000 9.8 and 10.3, of
  // 16,000 11.3 and 11.3; 16 heads on 4, 32 of 1,000 9.7 and 11.3, 48 14.0 and 12.9, 16 of 4,000 12.9 and 13.9; 32 heads on 4, 32 of 1,000
  // 10.9 and 12.8, 16 of 4,000 14.5 and 14.8; 48 heads on 4, 16 of 1,000 11.5 and 13.4, 24 16.7 and 15.0, 8 of 2,000 16.2 and 14.3, 4 of
  // 4,000 14.2 and 15.3, 8 of 4,000 21.2 and 16.1.
  long long units = ((static_cast<long long>(c.max_pages) << c.page_log2) + 31) / 32;
  if (w.window > 0) {
    const long long cut = (w.window + 31LL) / 32 + 1 + (w.sinks + 31LL) / 32;
    if (cut < units) units = cut;
  }
  const long long lists = static_cast<long long>(w.B) * c.Hkv * w.mg;
  if (units <= 384) {
    int nc = 1;
    while (nc < 8 && nc * 8 < units) nc *= 2;
    const int upw = static_cast<int>((units + 8 * nc - 1) / (8 * nc));
    const long long blocks = nc * lists, most = QR < 16 ? 4 : nc < 8 ? 2 : 1;
    if (blocks <= most * num_sms && blocks * upw <= (QR < 16 ? 7LL : 2LL) * num_sms) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(nc) * c.Hkv * w.mg, static_cast<unsigned>(w.B));
      cfg.blockDim = dim3(256);
      cfg.stream = s;
      cudaLaunchAttribute attr[2];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim = {static_cast<unsigned>(nc), 1, 1};
      cfg.attrs = attr;
      cfg.numAttrs = 2;
      return cudaLaunchKernelEx(&cfg, paged4_short_kernel<D, QR>, c, ranges, qkv, lens, y, lse2, w, upw, err);
    }
  }
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
  // Blocks of 1,024 threads join where each has an SM and there are more pieces to a list than 256 take at once (graph replays,
  // against 256): 12 heads on one, 200,000 rows 28.6 and 67.0 us; 16 x 20,000 rows, 4 key heads 23.5 and 24.5; but 192 lists of
  // 13 pieces 53.1 and 50.7, 384 of 76 33.5 and 29.2.
  const int join_threads = static_cast<long long>(w.B) * w.H <= num_sms && lists * (1024 / D) < NW ? 1024 : 256;
  if (e == cudaSuccess)
    e = launch_k(paged4_join_kernel<D, QR>, dim3(static_cast<unsigned>(w.H), static_cast<unsigned>(w.B)), dim3(join_threads), 0, s,
                 c, lens, y, lse2, w, ws, NW);
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
  // Up to four heads on a key head have a form of their own, whose columns hold each of them twice (16 x 9,000 to 32,000 rows, 16
  // heads on 4, 28.5 us, with the form for eight 31.2; 16 x up to 1,023 5.3 and 5.6).
  auto launch = launch_decode4<64, 16>;
  if (w.G == 1) launch = D == 64 ? launch_decode4<64, 1> : launch_decode4<32, 1>;
  else if (w.G <= 4) launch = D == 64 ? launch_decode4<64, 4> : launch_decode4<32, 4>;
  else if (w.G <= 8) launch = D == 64 ? launch_decode4<64, 8> : launch_decode4<32, 8>;
  else if (D == 32) launch = launch_decode4<32, 16>;
  return launch(c, r, x, lens, o, lse2, w, err, s);
}

}  // namespace gptgb
