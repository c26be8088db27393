// Paged key/value cache: storing rows, attention of one new token per sequence, eviction by summed weight.
//
// The cache is a pool of pages shared by all sequences, bf16 [pages][2][Hkv][page][D]: within a page the rows
// of one key head are contiguous (page * D * 2 bytes of keys, and the same of values), so a head's reader
// streams whole pages instead of one row out of every token's. Row r of sequence b lies in page
// table[b][r >> page_log2] at slot r & (page - 1). H query heads share Hkv key heads, G = H / Hkv each.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "paged.cuh"

#include <cooperative_groups.h>
#include <math.h>

namespace gptgb {

namespace {

// ---------------------------------------------------------------- store

// Bound by memory: 8 D bytes moved per row and key head. A block takes 16 tokens of a sequence: their places are
// looked up once into shared memory, then its threads walk the tokens' 16-byte units, four copies in flight each (16
// prompts of up to 1,024 tokens x 12 heads: 15.8 us, 4.9 TB/s; with one copy per thread 17.4, with twelve 18).
constexpr int kStoreTokens = 16;

template <int D>
__global__ void __launch_bounds__(256)
paged_store_kernel(PagedCache c, const uint4* __restrict__ qkv, const int32_t* __restrict__ start,
                   const int32_t* __restrict__ count, int T, int H, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int U = D / 8;                           // 16-byte units of a row
  __shared__ long long s_row[kStoreTokens];          // row (of D elements) of the token's key of head 0; -1: nowhere
  __shared__ long long s_weight[kStoreTokens];
  const int b = blockIdx.y, t0 = blockIdx.x * kStoreTokens;
  const int n = (count ? min(max(__ldg(count + b), 0), T) : T) - t0;  // tokens from t0 on; a count below 0 is 0
  if (n <= 0) return;
  if (threadIdx.x < kStoreTokens) {
    long long row = -1, weight = 0;
    if (threadIdx.x < n) {
      const long long r = (start ? static_cast<long long>(__ldg(start + b)) : 0) + t0 + threadIdx.x;
      if (r < 0 || r >= static_cast<long long>(c.max_pages) << c.page_log2) {
        record_error(err, GPT_DEV_EPAGE);
      } else {
        const int pg = page_of(c, c.table + static_cast<size_t>(b) * c.max_pages, static_cast<int>(r), err);
        const int slot = static_cast<int>(r) & ((1 << c.page_log2) - 1);
        if (pg >= 0) {
          row = static_cast<long long>(row_at(c, pg, 0, 0, slot));
          weight = static_cast<long long>(weight_at(c, pg, 0, slot));
        }
      }
    }
    s_row[threadIdx.x] = row;
    s_weight[threadIdx.x] = weight;
  }
  __syncthreads();
  const int per_tok = 2 * c.Hkv * U, all = min(n, kStoreTokens) * per_tok;
  const uint4* src = qkv + (static_cast<size_t>(b) * T + t0) * (H + 2 * c.Hkv) * U + static_cast<size_t>(H) * U;
  uint4* pool = reinterpret_cast<uint4*>(c.pool);
  constexpr int K = 4;
  for (int i0 = threadIdx.x; i0 < all; i0 += K * 256) {
    uint4 v[K];
    long long dst[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = i0 + k * 256, t = i / per_tok, e = i - t * per_tok;   // e: (keys or values, head, unit)
      dst[k] = -1;
      if (i < all && s_row[t] >= 0) {
        v[k] = __ldg(src + static_cast<size_t>(t) * (H + 2 * c.Hkv) * U + e);
        dst[k] = (s_row[t] + (static_cast<long long>(e / U) << c.page_log2)) * U + e % U;
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (dst[k] >= 0) pool[dst[k]] = v[k];
  }
  if (c.weight)
    for (int i = threadIdx.x; i < min(n, kStoreTokens) * c.Hkv; i += 256) {
      const int t = i / c.Hkv, h = i - t * c.Hkv;
      if (s_row[t] >= 0) c.weight[s_weight[t] + (static_cast<long long>(h) << c.page_log2)] = 0.0f;
    }
}

// ---------------------------------------------------------------- attention of one new token
//
// Bound by reading the cache: 4 D bytes per seen row and key head, once. What the design does for that:
//  * Work is cut by rows, not by sequences. A unit is 32 consecutive seen rows of one (sequence, key head, group of
//    up to 16 query heads); all units form one list (sequence-major) and every warp of the grid takes an equal
//    contiguous range of it, so ragged lengths, one long sequence or a single one all load the machine evenly. A warp
//    that holds all units of a (sequence, head group) writes its output; the others write a partial result (maximum,
//    sum, unnormalised output), at most two per warp, which a second kernel joins in a fixed order.
//  * A warp streams its units through its own ring of kStages stages of shared memory (cp.async, 16 bytes a lane,
//    whole rows), with no barrier across warps; the page numbers of a unit are loaded two units before its rows. Rows
//    are found through the table one by one, so windows, sinks and pages may end anywhere in a unit. Rows that are
//    not seen are not read (their shared memory is filled with zeros).
//  * The scores and the product with the values are mma.sync m16n8k16 with the query heads of the group as the 16
//    rows: with at most 16 rows of queries per key head the tensor core's rate does not matter (a tcgen05 tile
//    would have 128), but shared keys and values are unpacked once for all heads. P enters that product in two bf16
//    parts; scores, maxima, sums and outputs stay fp32.
// Measured: 16 sequences of 9,000 to 32,000 rows x 12 heads 160 us, 6.3 TB/s. Units of 16 rows were slower (16 sequences
// of up to 1,023 rows, as this form was then: 15.6 against 14.5 us).
constexpr int kStages = 3;
constexpr int kUnit = 32;                 // seen rows per unit

template <int D, int QR>
struct DecCfg {
  static constexpr int ROWB = D * 2;
  static constexpr int U = D / 8;                                 // 16-byte units per row
  static constexpr int TILE = kUnit * ROWB;                       // keys, or values, of a unit
  static constexpr int STAGE = 2 * TILE + QR * ROWB;              // + the query rows where a unit starts a segment
  static constexpr int WARP = kStages * STAGE + 128;              // + the stages' row masks
};

// Where the partial results of a launch lie (device scratch).
struct DecScratch {
  int* prefix;        // [B + 1] units of the sequences before b, per head group
  float* o;           // [warps][2][QR][D] unnormalised partial outputs
  float2* ml;         // [warps][2][QR] their maxima (log2 units) and sums
  float* lse;         // [B][H] log2-sum-exp of segments held by one warp
  float* score;       // [B][H][score_ld] scores in log2 units by seen row, or nullptr (no weights wanted)
  int score_ld;
};

struct DecShape {
  int B, H, G, mg;    // mg: head groups of up to 16 per key head
  int window, sinks;
  float scale_log2;
};

// Byte offset of 16-byte unit u of row r in a tile of rows of D bf16, permuted within 128 bytes so that the eight
// rows of an ldmatrix fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int u) {
  return D == 64 ? r * 128 + ((u ^ (r & 7)) << 4) : r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
}

// O += P U for 16 cached rows (a, b: the score tiles of eight each, now probabilities; u0: their first value row's place in
// shared memory), P in two bf16 parts: hi is p rounded, lo is p - hi rounded, so p - hi - lo is at most 2^-16 of p (one
// part alone made the outputs' error 2.0e-3 of their norm where their own rounding makes 1.6e-3). Of up to eight query
// heads lo takes the operand's other eight rows, its products o[][2] and o[][3] (joined_parts adds them): the second
// product of their own took 16 sequences of up to 1,023 rows from 10.6 to 11.7 us. Of 9 to 16 heads it is a product of its
// own (16 sequences of 9,000 to 32,000 rows, 12 key heads of 16 heads: 185 us, with one part 168).
template <int D, int RH>
__device__ __forceinline__ void add_values(float (&o)[D / 8][4], const float (&a)[4], const float (&b)[4], uint32_t u0, int lane) {
  uint32_t p[4], q[4];
#pragma unroll
  for (int i = 0; i < 2 * RH; ++i) {                 // heads lane / 4 (i even) and lane / 4 + 8, columns of a, then of b
    const float x = i < RH ? a[2 * i] : b[2 * (i - RH)], y = i < RH ? a[2 * i + 1] : b[2 * (i - RH) + 1];
    const int at = RH == 2 ? i : 2 * i;              // a: registers 0 and 1, b: 2 and 3
    p[at] = pack_bf16x2(x, y);
    const float2 f = unpack_bf16x2(p[at]);
    const uint32_t lo = pack_bf16x2(x - f.x, y - f.y);
    if (RH == 2) q[at] = lo;
    else p[at + 1] = lo;
  }
  uint32_t f[D / 16][4];
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    ldmatrix4_trans(f[j], u0 + tile_at<D>(lane & 15, 2 * j + (lane >> 4)));
    mma_16816(o[2 * j], p, f[j][0], f[j][1]);
    mma_16816(o[2 * j + 1], p, f[j][2], f[j][3]);
  }
  if constexpr (RH == 2) {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      mma_16816(o[2 * j], q, f[j][0], f[j][1]);
      mma_16816(o[2 * j + 1], q, f[j][2], f[j][3]);
    }
  }
}
template <int NT, int RH>
__device__ __forceinline__ void joined_parts(float (&o)[NT][4]) {
  if constexpr (RH == 1) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      o[j][0] += o[j][2];
      o[j][1] += o[j][3];
    }
  }
}

// The list position of a unit: sequence, head group (key head * mg + group), tile of the sequence's seen rows.
struct Unit {
  int b, hm, tile, nt, last;
  Seen seen;
};

template <int D, int QR>
__global__ void __launch_bounds__(256, 1)
paged_split_kernel(PagedCache c, const __nv_bfloat16* __restrict__ qkv, const int32_t* __restrict__ lens,
                   __nv_bfloat16* __restrict__ y, float* __restrict__ lse2, DecShape w, DecScratch ws, int* err) {
  using Cfg = DecCfg<D, QR>;
  constexpr int U = Cfg::U;
  constexpr int RPI = 32 / U;                        // rows per copy instruction of a warp
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  int* s_prefix = reinterpret_cast<int*>(smem + nwarps * Cfg::WARP);     // [B + 1]
  int* s_len = s_prefix + w.B + 1;                                       // [B]
  __shared__ int s_sum[8];
  pdl_wait();
  pdl_trigger();

  // units per sequence and their prefix sums (per head group)
  const long long cap = static_cast<long long>(c.max_pages) << c.page_log2;
  if (threadIdx.x == 0) s_prefix[0] = 0;
  int carry = 0;
  for (int b0 = 0; b0 < w.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int last = -1, x = 0;
    if (b < w.B) {
      last = __ldg(lens + b);
      if (last >= cap) {
        record_error(err, GPT_DEV_EPAGE);
        last = -1;
      }
      if (last >= 0) x = (seen_rows(last + 1, w.window, w.sinks).n + kUnit - 1) / kUnit;
      s_len[b] = last;
    }
    int incl = x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, k);
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

  uint8_t* ring = smem + warp * Cfg::WARP;
  const uint32_t ring_a = smem_u32(ring);
  volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(ring + kStages * Cfg::STAGE);
  const int row = w.H + 2 * c.Hkv;                   // heads of a token's row
  const int pmask = (1 << c.page_log2) - 1;
  const size_t vstep = (static_cast<size_t>(c.Hkv) << c.page_log2) * D;   // from a page's keys to its values
  const __nv_bfloat16* pool = static_cast<const __nv_bfloat16*>(c.pool);

  auto set_seq = [&](Unit& x) {                      // the sequence's lengths (b has units)
    x.nt = s_prefix[x.b + 1] - s_prefix[x.b];
    x.last = s_len[x.b];
    x.seen = seen_rows(x.last + 1, w.window, w.sinks);
  };
  auto advance = [&](Unit& x) {
    if (++x.tile < x.nt) return;
    x.tile = 0;
    if (++x.hm < HM) return;
    x.hm = 0;
    do ++x.b; while (x.b < w.B && s_prefix[x.b + 1] == s_prefix[x.b]);
    if (x.b < w.B) set_seq(x);
  };
  Unit at;                                           // the unit that is computed next
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
  Unit next = at, ahead = at;                        // the unit whose rows are copied next, and the one after it
  auto look_up = [&](const Unit& x) -> int {         // the page of its row, this lane
    const int v = x.tile * kUnit + lane;
    return v < x.seen.n ? __ldg(c.table + static_cast<size_t>(x.b) * c.max_pages + (seen_row(x.seen, v) >> c.page_log2)) : -1;
  };
  int page = look_up(next), page_ahead = -1;
  int issued = 0;
  if (count > 1) {
    advance(ahead);
    page_ahead = look_up(ahead);
  }
  auto issue = [&]() {                               // copies unit `next` into stage issued % kStages, steps on
    const int st = issued % kStages;
    const uint32_t sk = ring_a + st * Cfg::STAGE, sv = sk + Cfg::TILE, sq = sv + Cfg::TILE;
    const int kh = next.hm / w.mg, g0 = (next.hm - kh * w.mg) * 16;
    const int v = next.tile * kUnit + lane, r = seen_row(next.seen, v);
    const __nv_bfloat16* tok = qkv + static_cast<size_t>(next.b) * row * D;
    const __nv_bfloat16* kp = pool;
    size_t dv = vstep;
    bool ok = v < next.seen.n;
    if (ok && r == next.last) {                      // the new token's own row comes from qkv
      kp = tok + static_cast<size_t>(w.H + kh) * D;
      dv = static_cast<size_t>(c.Hkv) * D;
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.pages)) record_error(err, GPT_DEV_EPAGE);
    } else if (ok) {
      if (static_cast<unsigned>(page) < static_cast<unsigned>(c.pages)) {
        kp = pool + row_at(c, page, 0, kh, r & pmask) * D;
      } else {
        ok = false;
        record_error(err, GPT_DEV_EPAGE);
      }
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) masks[st] = mask;
    const unsigned long long ka = reinterpret_cast<unsigned long long>(kp);
    const unsigned long long va = reinterpret_cast<unsigned long long>(kp + (ok ? dv : 0));
    const int u = lane % U;
#pragma unroll
    for (int i = 0; i < kUnit / RPI; ++i) {
      const int rr = i * RPI + lane / U;
      const bool have = (mask >> rr) & 1u;
      const unsigned long long k = __shfl_sync(0xffffffffu, ka, rr), x = __shfl_sync(0xffffffffu, va, rr);
      cp_async16(sk + tile_at<D>(rr, u), reinterpret_cast<const uint8_t*>(k) + 16 * u, have);
      cp_async16(sv + tile_at<D>(rr, u), reinterpret_cast<const uint8_t*>(x) + 16 * u, have);
    }
    if (issued == 0 || next.tile == 0) {             // a segment starts: its queries (rows past the group: zeros)
      const int gn = min(w.G - g0, 16);
#pragma unroll
      for (int i = 0; i < (QR + RPI - 1) / RPI; ++i) {
        const int rr = i * RPI + lane / U;
        if (rr < QR)
          cp_async16(sq + tile_at<D>(rr, u), tok + static_cast<size_t>(kh * w.G + g0 + min(rr, gn - 1)) * D + 8 * u, rr < gn);
      }
    }
    ++issued;
    next = ahead;
    page = page_ahead;
    if (issued + 1 < count) {
      advance(ahead);
      page_ahead = look_up(ahead);
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (issued < count) issue();
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  constexpr int NT = D / 8;                          // 8-column output tiles
  float o[NT][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};   // rows lane / 4 and lane / 4 + 8
  uint32_t qf[D / 16][4];
  int piece0 = 0;                                    // the segment's first unit in this warp's range
  const int qrow = lane >> 2, qcol = 2 * (lane & 3);
  for (int n = 0; n < count; ++n) {
    if (issued < count) issue();
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const int st = n % kStages;
    const uint32_t sk = ring_a + st * Cfg::STAGE, sv = sk + Cfg::TILE, sq = sv + Cfg::TILE;
    const uint32_t mask = masks[st];
    const int kh = at.hm / w.mg, g0 = (at.hm - kh * w.mg) * 16, gn = min(w.G - g0, 16);
    if (n == 0 || at.tile == 0) {
      piece0 = n;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.0f;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
      // A operand: matrices rows 0-7 / 8-15 (units 2 k, 2 k + 1 of the 16 columns)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        if constexpr (QR == 16) {
          uint32_t f[4];
          ldmatrix4(f, sq + tile_at<D>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)));
          qf[k][0] = f[0]; qf[k][1] = f[1]; qf[k][2] = f[2]; qf[k][3] = f[3];
        } else {
          if ((k & 1) == 0) {                        // units 2 k .. 2 k + 3 of rows 0-7: two steps at once
            uint32_t f[4];
            ldmatrix4(f, sq + tile_at<D>(lane & 7, 2 * k + (lane >> 3)));
            qf[k][0] = f[0]; qf[k][1] = 0u; qf[k][2] = f[1]; qf[k][3] = 0u;
            qf[k + 1][0] = f[2]; qf[k + 1][1] = 0u; qf[k + 1][2] = f[3]; qf[k + 1][3] = 0u;
          }
        }
      }
    }
    // scores of 32 rows: four 8-column tiles
    float s[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][i] = 0.0f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint32_t f[4];
        ldmatrix4(f, sk + tile_at<D>(8 * j + (lane & 7), 4 * k + (lane >> 3)));
        mma_16816(s[j], qf[2 * k], f[0], f[1]);
        mma_16816(s[j], qf[2 * k + 1], f[2], f[3]);
      }
    }
    constexpr int RH = QR == 16 ? 2 : 1;             // row halves in use
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2 * RH; ++i)
        s[j][i] = (mask >> (8 * j + qcol + (i & 1))) & 1u ? s[j][i] * w.scale_log2 : -INFINITY;
    if (ws.score != nullptr) {
#pragma unroll
      for (int rh = 0; rh < RH; ++rh) {
        const int g = g0 + qrow + 8 * rh;
        if (qrow + 8 * rh < gn) {
          float* dst = ws.score + (static_cast<size_t>(at.b) * w.H + kh * w.G + g) * ws.score_ld + at.tile * kUnit + qcol;
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(s[j][2 * rh], s[j][2 * rh + 1]);
        }
      }
    }
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
      float mx = m[rh];
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = fmax3(mx, s[j][2 * rh], s[j][2 * rh + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float ref = mx == -INFINITY ? 0.0f : mx;   // nothing seen so far (bad pages): every term is 2^-inf
      const float a = ex2_approx(m[rh] - ref);
      m[rh] = mx;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j][2 * rh] = ex2_approx(s[j][2 * rh] - ref);
        s[j][2 * rh + 1] = ex2_approx(s[j][2 * rh + 1] - ref);
        sum += s[j][2 * rh] + s[j][2 * rh + 1];
      }
      l[rh] = l[rh] * a + sum;
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
    // O += P U: two steps of 16 rows (a step's offset keeps tile_at's permutation: it is a multiple of eight rows)
#pragma unroll
    for (int k = 0; k < 2; ++k) add_values<D, RH>(o, s[2 * k], s[2 * k + 1], sv + 16 * k * Cfg::ROWB, lane);
    const bool ends = at.tile == at.nt - 1;
    if (ends && g0 == 0) {                           // the sequence's newest row: into the cache
      const int pg = __ldg(c.table + static_cast<size_t>(at.b) * c.max_pages + (at.last >> c.page_log2));
      if (static_cast<unsigned>(pg) < static_cast<unsigned>(c.pages) && lane < 2 * U) {
        const int which = lane / U, u = lane % U;
        const __nv_bfloat16* src = qkv + (static_cast<size_t>(at.b) * row + w.H + which * c.Hkv + kh) * D;
        reinterpret_cast<uint4*>(c.pool)[row_at(c, pg, which, kh, at.last & pmask) * U + u] =
            __ldg(reinterpret_cast<const uint4*>(src) + u);
        if (c.weight && lane == 0) c.weight[weight_at(c, pg, kh, at.last & pmask)] = 0.0f;   // summed up by the join
      }
    }
    if (ends || n == count - 1) {                    // the piece is done
      const bool whole = ends && piece0 + at.nt == n + 1;   // it holds all of the segment's units
      const size_t slot = static_cast<size_t>(gw) * 2 + (piece0 == 0 ? 0 : 1);
      joined_parts<NT, RH>(o);
#pragma unroll
      for (int rh = 0; rh < RH; ++rh) {
        float lt = l[rh];
        lt += __shfl_xor_sync(0xffffffffu, lt, 1);
        lt += __shfl_xor_sync(0xffffffffu, lt, 2);
        const int r = qrow + 8 * rh;
        if (r >= gn) continue;
        if (whole) {
          const size_t head = static_cast<size_t>(at.b) * w.H + kh * w.G + g0 + r;
          const float inv = 1.0f / lt;               // (a sum of 0, every score -inf, gives NaN)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *reinterpret_cast<uint32_t*>(y + head * D + 8 * j + qcol) = pack_bf16x2(o[j][2 * rh] * inv, o[j][2 * rh + 1] * inv);
          if ((lane & 3) == 0) {
            const float v = m[rh] + log2f(lt);
            ws.lse[head] = v;
            if (lse2) lse2[head] = v;
          }
        } else {
          float* dst = ws.o + (slot * QR + r) * D + qcol;
#pragma unroll
          for (int j = 0; j < NT; ++j) *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(o[j][2 * rh], o[j][2 * rh + 1]);
          if ((lane & 3) == 0) ws.ml[slot * QR + r] = make_float2(m[rh], lt);
        }
      }
    }
    advance(at);
    __syncwarp();                                    // the stage is read before it is filled again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The same attention where the rows that can be seen fit the warps of one cluster (UPW units per warp): one launch, no
// scratch. A block takes 8 UPW consecutive units, and blocks behind the last leave at once (the table's room
// is the most a sequence can hold, not what it holds); a warp's rows are all copied at once and
// it holds its scores in registers, so there is one maximum and no rescaling, and the attention weights follow from the
// registers once the cluster's maxima and sums are known. Each block adds up its warps' outputs in shared memory and
// pushes them to the block that joins that query row, and its maxima and sums to every block; one cluster barrier.
// Bound by latency: the length and the page numbers, then the rows, then the barrier: 4.0 us for 600 rows x 12 heads,
// where the two launches of the general form take 7.0.
template <int D, int QR, int UPW>
struct ShortCfg {
  static constexpr int TILE = kUnit * D * 2;
  static constexpr int WARP = UPW * 2 * TILE;
  static constexpr int SMEM = 8 * WARP;
};

template <int D, int QR, int UPW>
__global__ void __launch_bounds__(256, UPW == 1 ? 3 : 1)
paged_short_kernel(PagedCache c, const __nv_bfloat16* __restrict__ qkv, const int32_t* __restrict__ lens,
                   __nv_bfloat16* __restrict__ y, float* __restrict__ lse2, DecShape w, int* err) {
  using Cfg = ShortCfg<D, QR, UPW>;
  constexpr int U = D / 8, RPI = 32 / U, NT = D / 8, RH = QR == 16 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[8][QR];                     // the warps' maxima and sums
  __shared__ float2 s_all[8][QR];                    // the blocks', pushed by each of them
  __shared__ float s_o[QR + 7][D];                   // pushed outputs: [row / NB * NB + block][D]
  auto cluster = cooperative_groups::this_cluster();
  const int NC = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // every block has started (awaited below)
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, hm = static_cast<int>(blockIdx.x) / NC;
  const int kh = hm / w.mg, g0 = (hm - kh * w.mg) * 16, gn = min(w.G - g0, 16);
  const int row = w.H + 2 * c.Hkv, pmask = (1 << c.page_log2) - 1;
  const int32_t* trow = c.table + static_cast<size_t>(b) * c.max_pages;
  const __nv_bfloat16* tok = qkv + static_cast<size_t>(b) * row * D;
  int last = __ldg(lens + b);
  int page[UPW];                                     // on its way before the length is known: right unless a window cuts
#pragma unroll
  for (int j = 0; j < UPW; ++j)
    page[j] = __ldg(trow + min((((rank * UPW + j) * 8 + warp) * kUnit + lane) >> c.page_log2, c.max_pages - 1));
  const int qrow = lane >> 2, qcol = 2 * (lane & 3);
  uint32_t qf[D / 16][4];                            // A operand: the group's queries, zeros behind them
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = qrow + 8 * (i & 1);
      qf[k][i] = (i & 1) < RH && r < gn
          ? __ldg(reinterpret_cast<const uint32_t*>(tok + static_cast<size_t>(kh * w.G + g0 + r) * D + 16 * k + 8 * (i >> 1) + qcol))
          : 0u;
    }
  if (last >= static_cast<long long>(c.max_pages) << c.page_log2) {
    if (tid == 0) record_error(err, GPT_DEV_EPAGE);
    last = -1;
  }
  const Seen seen = seen_rows(last + 1, w.window, w.sinks);
  const int NB = (seen.n + 8 * UPW * kUnit - 1) / (8 * UPW * kUnit);   // blocks that hold units
  if (rank >= NB) return;                            // (whole blocks: barriers wait for the others only)
  uint8_t* ring = smem + warp * Cfg::WARP;
  const uint32_t ring_a = smem_u32(ring);
  const size_t vstep = (static_cast<size_t>(c.Hkv) << c.page_log2) * D;
  const __nv_bfloat16* pool = static_cast<const __nv_bfloat16*>(c.pool);
  uint32_t mask[UPW];
#pragma unroll
  for (int j = 0; j < UPW; ++j) {
    const int v = ((rank * UPW + j) * 8 + warp) * kUnit + lane, r = seen_row(seen, v);
    bool ok = v < seen.n;
    if (ok && r != v) page[j] = __ldg(trow + (r >> c.page_log2));
    const __nv_bfloat16* kp = pool;
    size_t dv = vstep;
    if (ok && static_cast<unsigned>(page[j]) >= static_cast<unsigned>(c.pages)) record_error(err, GPT_DEV_EPAGE);
    if (ok && r == last) {                           // the new token's own row comes from qkv
      kp = tok + static_cast<size_t>(w.H + kh) * D;
      dv = static_cast<size_t>(c.Hkv) * D;
    } else {
      ok = ok && static_cast<unsigned>(page[j]) < static_cast<unsigned>(c.pages);
      if (ok) kp = pool + row_at(c, page[j], 0, kh, r & pmask) * D;
    }
    mask[j] = __ballot_sync(0xffffffffu, ok);
    const unsigned long long ka = reinterpret_cast<unsigned long long>(kp);
    const unsigned long long va = reinterpret_cast<unsigned long long>(kp + (ok ? dv : 0));
    const uint32_t sk = ring_a + j * 2 * Cfg::TILE, sv = sk + Cfg::TILE;
    const int u = lane % U;
    if (mask[j])
#pragma unroll
      for (int i = 0; i < kUnit / RPI; ++i) {
        const int rr = i * RPI + lane / U;
        const bool have = (mask[j] >> rr) & 1u;
        const unsigned long long k = __shfl_sync(0xffffffffu, ka, rr), x = __shfl_sync(0xffffffffu, va, rr);
        cp_async16(sk + tile_at<D>(rr, u), reinterpret_cast<const uint8_t*>(k) + 16 * u, have);
        cp_async16(sv + tile_at<D>(rr, u), reinterpret_cast<const uint8_t*>(x) + 16 * u, have);
      }
  }
  // the newest row into the cache, by the warp whose unit holds it
  const int ntail = (seen.n - 1) / kUnit;            // its unit
  if (g0 == 0 && ntail / (8 * UPW) == rank && ntail % 8 == warp) {
    const int pg = __ldg(trow + (last >> c.page_log2));
    if (static_cast<unsigned>(pg) < static_cast<unsigned>(c.pages) && lane < 2 * U) {
      const int which = lane / U, u = lane % U;
      reinterpret_cast<uint4*>(c.pool)[row_at(c, pg, which, kh, last & pmask) * U + u] =
          __ldg(reinterpret_cast<const uint4*>(tok + static_cast<size_t>(w.H + which * c.Hkv + kh) * D) + u);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();

  float s[4 * UPW][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
#pragma unroll
  for (int t = 0; t < UPW; ++t) {
    const uint32_t sk = ring_a + t * 2 * Cfg::TILE;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float (&x)[4] = s[4 * t + j];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = 0.0f;
      if (mask[t])
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t f[4];
          ldmatrix4(f, sk + tile_at<D>(8 * j + (lane & 7), 4 * k + (lane >> 3)));
          mma_16816(x, qf[2 * k], f[0], f[1]);
          mma_16816(x, qf[2 * k + 1], f[2], f[3]);
        }
#pragma unroll
      for (int i = 0; i < 2 * RH; ++i) {
        x[i] = (mask[t] >> (8 * j + qcol + (i & 1))) & 1u ? x[i] * w.scale_log2 : -INFINITY;
        m[i >> 1] = fmaxf(m[i >> 1], x[i]);
      }
    }
  }
#pragma unroll
  for (int rh = 0; rh < RH; ++rh) {
    m[rh] = fmaxf(m[rh], __shfl_xor_sync(0xffffffffu, m[rh], 1));
    m[rh] = fmaxf(m[rh], __shfl_xor_sync(0xffffffffu, m[rh], 2));
    const float ref = m[rh] == -INFINITY ? 0.0f : m[rh];   // nothing seen: every term is 2^-inf
#pragma unroll
    for (int j = 0; j < 4 * UPW; ++j) {
      s[j][2 * rh] = ex2_approx(s[j][2 * rh] - ref);
      s[j][2 * rh + 1] = ex2_approx(s[j][2 * rh + 1] - ref);
      l[rh] += s[j][2 * rh] + s[j][2 * rh + 1];
    }
    l[rh] += __shfl_xor_sync(0xffffffffu, l[rh], 1);
    l[rh] += __shfl_xor_sync(0xffffffffu, l[rh], 2);
  }
#pragma unroll
  for (int k = 0; k < 2 * UPW; ++k) {
    if (!mask[k >> 1]) continue;
    const uint32_t sv = ring_a + (k >> 1) * 2 * Cfg::TILE + Cfg::TILE;
    add_values<D, RH>(o, s[2 * k], s[2 * k + 1], sv + 16 * (k & 1) * D * 2, lane);
  }
  joined_parts<NT, RH>(o);
  __syncwarp();                                      // the warp's tiles are read: its outputs take their place
  float* own = reinterpret_cast<float*>(ring);       // [QR][D]
#pragma unroll
  for (int rh = 0; rh < RH; ++rh) {
    const int r = qrow + 8 * rh;
    if (r >= gn) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<float2*>(own + r * D + 8 * j + qcol) = make_float2(o[j][2 * rh], o[j][2 * rh + 1]);
    if ((lane & 3) == 0) s_ml[warp][r] = make_float2(m[rh], l[rh]);
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
      acc += reinterpret_cast<const float*>(smem + k * Cfg::WARP)[r * D + d] * f;
    }
    cluster.map_shared_rank(&s_o[0][0], r % NB)[(r / NB * NB + rank) * D + d] = acc;
    if (d < NB) cluster.map_shared_rank(&s_all[0][0], d)[rank * QR + r] = make_float2(mx, lt);
  }
  cluster.sync();
  auto joined = [&](int r, float* sum) -> float {    // a row's maximum and sum over all blocks
    float mx = -INFINITY;
    for (int k = 0; k < NB; ++k) mx = fmaxf(mx, s_all[k][r].x);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float lt = 0.0f;
    for (int k = 0; k < NB; ++k) lt += s_all[k][r].y * ex2_approx(s_all[k][r].x - ref);
    *sum = lt;
    return mx;
  };
  for (int i = tid; i < (gn + NB - 1) / NB * D; i += 256) {
    const int r = i / D * NB + rank, d = i % D;
    if (r >= gn) continue;
    float lt;
    const float mx = joined(r, &lt), ref = mx == -INFINITY ? 0.0f : mx;
    float acc = 0.0f;
    for (int k = 0; k < NB; ++k) acc += s_o[r / NB * NB + k][d] * ex2_approx(s_all[k][r].x - ref);
    const size_t head = static_cast<size_t>(b) * w.H + kh * w.G + g0 + r;
    y[head * D + d] = __float2bfloat16(acc / lt);
    if (d == 0 && lse2) lse2[head] = mx + log2f(lt);
  }
  if (!c.weight) return;
  // the weights: a row's probabilities summed over the group's heads, one row per lane
  float f[2] = {0.0f, 0.0f};
#pragma unroll
  for (int rh = 0; rh < RH; ++rh)
    if (qrow + 8 * rh < gn) {
      float lt;
      const float mx = joined(qrow + 8 * rh, &lt);
      f[rh] = ex2_approx(m[rh] - mx) / lt;
    }
#pragma unroll
  for (int t = 0; t < UPW; ++t) {
    if (!mask[t]) continue;
    float mine = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = qrow < gn ? s[4 * t + j][i] * f[0] : 0.0f;   // (rows behind the group may hold NaN)
        if (RH == 2 && qrow + 8 < gn) x += s[4 * t + j][2 + i] * f[1];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (qrow == 2 * j + i) mine = x;
      }
    const int at = 8 * (qrow >> 1) + qcol + (qrow & 1), v = ((rank * UPW + t) * 8 + warp) * kUnit + at, r = seen_row(seen, v);
    const int pg = __shfl_sync(0xffffffffu, page[t], at);
    if (v >= seen.n || static_cast<unsigned>(pg) >= static_cast<unsigned>(c.pages)) continue;
    float* dst = c.weight + weight_at(c, pg, kh, r & pmask);
    if (r == last) *dst = mine;
    else atomicAdd(dst, mine);                       // sequences may share a page
  }
}

// Joins the partial results of a (sequence, key head), and adds the attention weights of its seen rows: block
// (key head, z, sequence) takes rows z kJoinRows, + kJoinRows, then on in steps of the grid; blocks z > 0 only that.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 1024;

template <int D, int QR>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(PagedCache c, const int32_t* __restrict__ lens, __nv_bfloat16* __restrict__ y, float* __restrict__ lse2,
                  DecShape w, DecScratch ws, int warps, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int P = kJoinThreads / D;                // rows, or shares of a row's pieces, side by side
  constexpr int K = kJoinRows / kJoinThreads;
  __shared__ float s_lse[kPagedMaxGroup];
  __shared__ float s_o[P][D], s_m[P], s_l[P];
  const int kh = blockIdx.x, b = blockIdx.z;
  const int p0 = ws.prefix[b], nt = ws.prefix[b + 1] - p0, last = __ldg(lens + b);
  const long long total = static_cast<long long>(ws.prefix[w.B]) * (c.Hkv * w.mg);
  if (nt == 0 || (blockIdx.y > 0 && static_cast<long long>(blockIdx.y) * kJoinRows >= static_cast<long long>(nt) * kUnit)) return;
  const int HM = c.Hkv * w.mg;
  const Deal deal(total, warps);
  const int tid = threadIdx.x, d = tid % D, part = tid / D;
  const Seen sn = seen_rows(last + 1, w.window, w.sinks);
  const int pmask = (1 << c.page_log2) - 1;
  const int32_t* trow = c.table + static_cast<size_t>(b) * c.max_pages;
  const float* score = ws.score ? ws.score + (static_cast<size_t>(b) * w.H + kh * w.G) * ws.score_ld : nullptr;
  const long long v0 = static_cast<long long>(blockIdx.y) * kJoinRows;
  // the pages, and the first head's scores, of the rows whose weights this block adds to: on their way early
  int pg[K];
  float sc[K];
  auto fetch = [&](long long first) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long v = min(first + tid + k * kJoinThreads, static_cast<long long>(sn.n) - 1);
      pg[k] = __ldg(trow + (seen_row(sn, static_cast<int>(v)) >> c.page_log2));
      sc[k] = score[v];
    }
  };
  if (score) fetch(v0);
  for (int mt = 0; mt < w.mg; ++mt) {
    const long long t0 = static_cast<long long>(p0) * HM + static_cast<long long>(kh * w.mg + mt) * nt, t1 = t0 + nt;
    const int g1 = deal.warp_of(t0), g2 = deal.warp_of(t1 - 1);   // the warps that hold the first unit and the last
    const int gn = min(w.G - mt * 16, 16);
    const size_t head0 = static_cast<size_t>(b) * w.H + kh * w.G + mt * 16;
    // a piece is its warp's first (slot 0) unless its segment starts behind the warp's start: only g1's can
    const size_t slot1 = static_cast<size_t>(g1) * 2 + (deal.start(g1) == t0 ? 0 : 1);
    if (g1 == g2) {                                  // one warp held it all and wrote the output
      if (tid < gn) s_lse[mt * 16 + tid] = ws.lse[head0 + tid];
      __syncthreads();
      continue;
    }
    // maxima, sums and outputs in one walk over the pieces; the pieces of one or two rows are shared by the parts
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
        if (blockIdx.y == 0) y[(head0 + r) * D + d] = __float2bfloat16(at / lt);
        if (d == 0) {
          const float lse = mx + log2f(lt);
          s_lse[mt * 16 + r] = lse;
          if (lse2 && blockIdx.y == 0) lse2[head0 + r] = lse;
        }
      }
      __syncthreads();
    }
  }
  if (!score) return;
  for (long long first = v0; first < sn.n; first += static_cast<long long>(gridDim.y) * kJoinRows) {
    if (first != v0) fetch(first);
    float sum[K];
#pragma unroll
    for (int k = 0; k < K; ++k) sum[k] = exp2f(sc[k] - s_lse[0]);
    for (int r = 1; r < w.G; ++r) {
      const float lse = s_lse[r];
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (first + tid + k * kJoinThreads < sn.n)
          sum[k] += exp2f(score[static_cast<size_t>(r) * ws.score_ld + first + tid + k * kJoinThreads] - lse);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (first + tid + k * kJoinThreads >= sn.n) continue;
      const int row = seen_row(sn, static_cast<int>(first) + tid + k * kJoinThreads);
      // atomic: sequences may share a page (each adds to a row once, so a page of one sequence has one order)
      if (static_cast<unsigned>(pg[k]) < static_cast<unsigned>(c.pages))
        atomicAdd(c.weight + weight_at(c, pg[k], kh, row & pmask), sum[k]);
      else record_error(err, GPT_DEV_EPAGE);
    }
  }
}

// ---------------------------------------------------------------- eviction

// Order of weights as unsigned numbers: larger weight, larger number; NaN lowest; -0 equals +0.
__device__ __forceinline__ uint32_t weight_rank(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One kernel chooses the rows of each (sequence, key head), and for short lists copies them too; for the others a second
// one does. The choice: a cluster of NC blocks holds the weights between the sinks and the recent rows as ranks in shared
// memory, a stretch each (read once, through the table, all loads independent; a list that does not fit is read again by
// each pass). Up to three passes over 11, 11 and 10 bits find the rank of the smallest kept weight: a histogram of the
// rows that agree so far, summed over the blocks, whose bins are scanned from the top; a bin that is kept whole ends them.
// Then every warp counts its stretch of rows, and places them behind the stretches before it. Equal weights are kept
// from the lowest row on.
// Bound by issuing about 200 instructions a row and by the passes' barriers, so long lists are spread over four SMs
// (10,000 to 20,000 rows, 48 lists: 24 us with one block of 1024 threads each; in clusters of eight both kernels took
// 65 us against 32), and lists of up to 4,096 rows are not (500 to 1,024 rows, 192 lists: clusters of two 28 against
// 18.5). Measured: 4 x 12 lists of 10,000 to 20,000 rows to 2,500 28 us, 16 x 12 of 500 to 1,024 to 512 15 us. Clusters
// of four that copy as well were slower than the second launch (25.2 against 23.6 us, graph replays).
constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;

// Copies the m kept rows (s_keep) of one key head and sequence by the block that chose them: a batch of rows is read
// whole before any of it is written, as row i comes from a row at or behind i (no later batch reads what one wrote).
template <int D>
__device__ __forceinline__ void copy_kept(const PagedCache& c, const int32_t* trow, const int32_t* drow, const int* s_keep,
                                          int m, int h, int* err) {
  constexpr int U = D / 8, ROWS = kEvThreads / U, K = 4;
  const int u = threadIdx.x % U, pmask = (1 << c.page_log2) - 1;
  uint4* pool = static_cast<uint4*>(c.pool);
  const size_t vstep = (static_cast<size_t>(c.Hkv) << c.page_log2) * U;
  for (int i0 = threadIdx.x / U; i0 - static_cast<int>(threadIdx.x) / U < m; i0 += ROWS * K) {
    uint4 kx[K], vx[K];
    float wx[K];
    int src[K], dst[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = min(i0 + k * ROWS, m - 1);
      src[k] = __ldg(trow + (s_keep[i] >> c.page_log2));
      dst[k] = __ldg(drow + (i >> c.page_log2));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = i0 + k * ROWS, slot = s_keep[min(i, m - 1)] & pmask;
      const bool ok = static_cast<unsigned>(src[k]) < static_cast<unsigned>(c.pages) &&
                      static_cast<unsigned>(dst[k]) < static_cast<unsigned>(c.pages);
      if (!ok) record_error(err, GPT_DEV_EPAGE);
      if (!ok || i >= m) dst[k] = -1;                // nothing to write; the loads go to page 0
      const int pg = ok ? src[k] : 0;
      const uint4* from = pool + row_at(c, pg, 0, h, slot) * U + u;
      kx[k] = from[0];
      vx[k] = from[vstep];
      wx[k] = c.weight[weight_at(c, pg, h, slot)];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (dst[k] < 0) continue;
      const int slot = (i0 + k * ROWS) & pmask;
      uint4* to = pool + row_at(c, dst[k], 0, h, slot) * U + u;
      to[0] = kx[k];
      to[vstep] = vx[k];
      if (u == 0) c.weight[weight_at(c, dst[k], h, slot)] = wx[k];
    }
  }
}

// D = 0: the chosen rows are named in `kept` for the kernel that moves them; else the block moves them itself.
template <int NC, int D>
__global__ void __launch_bounds__(kEvThreads, 2)
paged_choose_kernel(PagedCache c, const int32_t* __restrict__ lens, int32_t* __restrict__ new_lens,
                    int32_t* __restrict__ kept, const int32_t* __restrict__ dst_table, int dst_max_pages, int budget,
                    int sinks, int recent, int room, int* err) {
  namespace cg = cooperative_groups;
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t s_rank[];               // [room] ranks of this block's stretch, then the kept rows
  int* s_keep = reinterpret_cast<int*>(s_rank + room);
  __shared__ __align__(16) int hists[3][kEvBins];    // one per pass: another block may still read the last one's
  __shared__ int s_sum[kEvWarps], s_tie[kEvWarps], pick[3], s_total[2];
  const int part = NC == 1 ? 0 : static_cast<int>(blockIdx.x % NC), h = static_cast<int>(blockIdx.x / NC), b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pmask = (1 << c.page_log2) - 1;
  const int32_t* trow = c.table + static_cast<size_t>(b) * c.max_pages;
  int32_t* out = kept + (static_cast<size_t>(b) * c.Hkv + h) * budget;
  auto sync_all = [&]() {
    if constexpr (NC == 1) __syncthreads();
    else cg::this_cluster().sync();
  };
  int n = __ldg(lens + b);
  if (n > static_cast<long long>(c.max_pages) << c.page_log2) {
    if (tid == 0) record_error(err, GPT_DEV_EPAGE);
    n = 0;
  }
  const int m = min(n, budget);                      // rows kept
  const int me = part * kEvThreads + tid;            // thread of the cluster
  if (h == 0 && me == 0) new_lens[b] = m;
  for (int i = max(m, 0) + me; i < budget; i += NC * kEvThreads) out[i] = -1;
  const int32_t* drow = dst_table + static_cast<size_t>(b) * dst_max_pages;
  auto keep_row = [&](int i, int r) {
    out[i] = r;
    if constexpr (D > 0) s_keep[i] = r;
  };
  auto finish = [&]() {
    if constexpr (D > 0) {
      __syncthreads();
      copy_kept<D>(c, trow, drow, s_keep, m, h, err);
    }
  };
  if (n <= budget) {                                 // (the same for the whole cluster)
    for (int i = me; i < m; i += NC * kEvThreads) keep_row(i, i);
    if (n > 0) finish();
    return;
  }
  const int lo = sinks, mid = n - recent - sinks;    // rows chosen by weight: lo .. lo + mid - 1
  for (int i = me; i < sinks; i += NC * kEvThreads) keep_row(i, i);
  for (int i = me; i < recent; i += NC * kEvThreads) keep_row(budget - recent + i, n - recent + i);
  int want = budget - sinks - recent;                // how many of them
  if (want == 0) return finish();
  const int each = ((mid + NC - 1) / NC + 31) / 32 * 32;
  const int base = min(mid, part * each), size = min(mid - base, each);   // this block's stretch
  const bool fits = each <= room;
  auto load = [&](int i) -> uint32_t {
    const int r = lo + base + i, pg = page_of(c, trow, r, err);
    return pg < 0 ? 0u : weight_rank(__ldg(c.weight + weight_at(c, pg, h, r & pmask)));
  };
  for (int i = tid; i < 3 * kEvBins; i += kEvThreads) hists[0][i] = 0;
  __syncthreads();
  if (fits) {
    // K pages, then K weights in flight per thread: bad pages are looked at behind the loads (a branch between them
    // had every load wait for the one before)
    constexpr int K = 8;
    for (int i0 = tid; i0 < size; i0 += K * kEvThreads) {
      int pg[K];
      float wt[K];
#pragma unroll
      for (int j = 0; j < K; ++j) pg[j] = __ldg(trow + ((lo + base + min(i0 + j * kEvThreads, size - 1)) >> c.page_log2));
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int p = static_cast<unsigned>(pg[j]) < static_cast<unsigned>(c.pages) ? pg[j] : 0;
        wt[j] = __ldg(c.weight + weight_at(c, p, h, (lo + base + min(i0 + j * kEvThreads, size - 1)) & pmask));
      }
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (i0 + j * kEvThreads >= size) break;
        const bool ok = static_cast<unsigned>(pg[j]) < static_cast<unsigned>(c.pages);
        if (!ok) record_error(err, GPT_DEV_EPAGE);
        const uint32_t k = ok ? weight_rank(wt[j]) : 0u;
        s_rank[i0 + j * kEvThreads] = k;
        atomicAdd(&hists[0][k >> 21], 1);            // the first pass
      }
    }
  } else {
    for (int i = tid; i < size; i += kEvThreads) atomicAdd(&hists[0][load(i) >> 21], 1);
  }
  uint32_t prefix = 0;                               // the leading bits of the smallest kept rank
  int low = 32;                                      // bits below them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass == 2 ? 10 : 11, shift = low - bits;
    int* hist = hists[pass];
    if (pass > 0) {
      for (int i = tid; i < size; i += kEvThreads) {
        const uint32_t k = fits ? s_rank[i] : load(i);
        if ((k >> low) == (prefix >> low)) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1);
      }
    }
    sync_all();                                      // every block's histogram is complete
    // the bin where the count from the top reaches `want`: thread t sums bins 4 t .. 4 t + 3
    constexpr int BPT = kEvBins / kEvThreads;
    static_assert(BPT == 4, "one 16-byte load per histogram");
    int c4[BPT] = {};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int* other = NC == 1 ? hist : cg::this_cluster().map_shared_rank(hist, k);
      const int4 x = *reinterpret_cast<const int4*>(other + tid * BPT);
      c4[0] += x.x;
      c4[1] += x.y;
      c4[2] += x.z;
      c4[3] += x.w;
    }
    const int own = c4[0] + c4[1] + c4[2] + c4[3];
    int above = own;                                 // counts of this and the later lanes
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int v = __shfl_down_sync(0xffffffffu, above, k);
      if (lane + k < 32) above += v;
    }
    if (lane == 0) s_sum[warp] = above;
    __syncthreads();
    for (int w = warp + 1; w < kEvWarps; ++w) above += s_sum[w];
    above -= own;                                    // rows in bins behind this thread's
    if (above < want && above + own >= want) {       // one thread of each block
      int left = want - above, j = BPT - 1;
#pragma unroll
      for (int k = BPT - 1; k > 0; --k)
        if (j == k && c4[k] < left) { left -= c4[k]; --j; }
      pick[0] = tid * BPT + j;
      pick[1] = left;                                // still to take among the rows of that bin
      int bin = c4[0];
#pragma unroll
      for (int k = 1; k < BPT; ++k)
        if (j == k) bin = c4[k];
      pick[2] = bin;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(pick[0]) << shift;
    want = pick[1];
    low = shift;
    if (want == pick[2]) break;                      // all of that bin are kept: no need to order them
  }
  // kept: every row whose leading bits are above prefix and the first `want` where they are equal
  prefix >>= low;
  const int per = ((size + kEvWarps - 1) / kEvWarps + 31) / 32 * 32;   // rows of a warp's stretch
  const int first = min(size, warp * per), end = min(size, first + per);
  int sure = 0, ties = 0;
  for (int i0 = first; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < end ? (fits ? s_rank[i] : load(i)) : 0u;
    sure += __popc(__ballot_sync(0xffffffffu, i < end && (k >> low) > prefix));
    ties += __popc(__ballot_sync(0xffffffffu, i < end && (k >> low) == prefix));
  }
  __syncthreads();
  if (lane == 0) {
    s_sum[warp] = sure;
    s_tie[warp] = ties;
  }
  __syncthreads();
  int at = 0, seen_ties = 0, all = 0, all_ties = 0;
  for (int w = 0; w < kEvWarps; ++w) {
    if (w == warp) {
      at = all;
      seen_ties = all_ties;
    }
    all += s_sum[w];
    all_ties += s_tie[w];
  }
  if constexpr (NC > 1) {
    if (tid == 0) {
      s_total[0] = all;
      s_total[1] = all_ties;
    }
    sync_all();
    for (int k = 0; k < part; ++k) {
      const int* other = cg::this_cluster().map_shared_rank(s_total, k);
      at += other[0];
      seen_ties += other[1];
    }
  }
  at += lo + min(seen_ties, want);                   // sinks, rows kept before, and the kept ties among them
  for (int i0 = first; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < end ? (fits ? s_rank[i] : load(i)) : 0u;
    const uint32_t tie = __ballot_sync(0xffffffffu, i < end && (k >> low) == prefix), below = (1u << lane) - 1u;
    const bool keep = i < end && ((k >> low) > prefix || ((k >> low) == prefix && seen_ties + __popc(tie & below) < want));
    const uint32_t mask = __ballot_sync(0xffffffffu, keep);
    if (keep) keep_row(at + __popc(mask & below), lo + base + i);
    at += __popc(mask);
    seen_ties += __popc(tie);
  }
  if constexpr (NC > 1) sync_all();                  // no block leaves while another reads its totals
  finish();
}

// Moves the kept rows of one (sequence, key head), a cluster of blocks each: 8 D bytes per row, bound by memory. Row i
// comes from a row at or behind i, so in place a chunk's rows are all read before any of them is written (a cluster
// barrier between), and no later chunk reads what this one wrote. Into other pages no order is needed, and each of the
// list's clusters takes its share of the chunks (in place the first cluster takes all).
constexpr int kMoveBlocks = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoveDepth = 2;

template <int D>
__global__ void __cluster_dims__(kMoveBlocks, 1, 1) __launch_bounds__(kMoveThreads)
paged_move_kernel(PagedCache c, const int32_t* __restrict__ dst_table, int dst_max_pages, const int32_t* __restrict__ kept,
                  int budget, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int U = D / 8;
  constexpr int ROWS = kMoveThreads / U;             // rows a block copies at once
  constexpr int K = kMoveDepth;                      // times that, in flight
  constexpr int CHUNK = kMoveBlocks * ROWS * K;
  const int h = blockIdx.y, b = blockIdx.z, u = threadIdx.x % U;
  const int part = static_cast<int>(blockIdx.x) % kMoveBlocks, share = static_cast<int>(blockIdx.x) / kMoveBlocks;
  const int pmask = (1 << c.page_log2) - 1;
  const int32_t* trow = c.table + static_cast<size_t>(b) * c.max_pages;
  const int32_t* drow = dst_table + static_cast<size_t>(b) * dst_max_pages;
  const int32_t* rows = kept + (static_cast<size_t>(b) * c.Hkv + h) * budget;
  const bool in_place = __ldg(trow) == __ldg(drow);
  if (in_place && share > 0) return;                 // (the whole cluster)
  const long long step = in_place ? CHUNK : static_cast<long long>(gridDim.x / kMoveBlocks) * CHUNK;
  uint4* pool = static_cast<uint4*>(c.pool);
  const size_t vstep = (static_cast<size_t>(c.Hkv) << c.page_log2) * U;   // from a page's keys to its values
  int r[K], src[K], dst[K];
  auto look_up = [&](int i0) {                       // the chunk's row numbers, then their pages, K in flight
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = i0 + (k * kMoveBlocks + part) * ROWS + threadIdx.x / U;
      r[k] = i < budget ? __ldg(rows + i) : -1;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = i0 + (k * kMoveBlocks + part) * ROWS + threadIdx.x / U;
      src[k] = __ldg(trow + (max(r[k], 0) >> c.page_log2));
      dst[k] = __ldg(drow + (min(i, budget - 1) >> c.page_log2));
    }
  };
  if (share * static_cast<long long>(CHUNK) >= budget) return;
  look_up(share * CHUNK);
  for (long long first = share * static_cast<long long>(CHUNK); first < budget; first += step) {
    const int i0 = static_cast<int>(first);
    if (__ldg(rows + i0) < 0) break;                 // behind the last row (the same for the whole cluster)
    uint4 kx[K], vx[K];
    float wx[K];
    size_t to[K], wto[K];
    bool go[K];
    // page 0 stands in for a bad page until the check behind the loads
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = i0 + (k * kMoveBlocks + part) * ROWS + threadIdx.x / U;
      const bool ok = static_cast<unsigned>(src[k]) < static_cast<unsigned>(c.pages);
      const int pg = ok ? src[k] : 0, slot = max(r[k], 0) & pmask;
      const uint4* from = pool + row_at(c, pg, 0, h, slot) * U + u;
      if (r[k] >= 0) {
        kx[k] = from[0];
        vx[k] = from[vstep];
        if (u == 0) wx[k] = c.weight[weight_at(c, pg, h, slot)];
      }
      go[k] = r[k] >= 0 && ok && static_cast<unsigned>(dst[k]) < static_cast<unsigned>(c.pages);
      if (r[k] >= 0 && !go[k]) record_error(err, GPT_DEV_EPAGE);
      to[k] = row_at(c, go[k] ? dst[k] : 0, 0, h, i & pmask) * U + u;
      wto[k] = weight_at(c, go[k] ? dst[k] : 0, h, i & pmask);
    }
    if (first + step < budget) look_up(static_cast<int>(first + step));   // while the rows travel
    if (in_place) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!go[k]) continue;
      pool[to[k]] = kx[k];
      pool[to[k] + vstep] = vx[k];
      if (u == 0) c.weight[wto[k]] = wx[k];
    }
  }
}

}  // namespace

cudaError_t launch_paged_store(const PagedCache& c, const void* qkv, const int32_t* start, const int32_t* count, int B,
                               int T, int H, int D, int* err, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((T - 1) / kStoreTokens + 1), static_cast<unsigned>(B));
  const uint4* x = static_cast<const uint4*>(qkv);
  if (D == 64) return launch_k(paged_store_kernel<64>, grid, dim3(256), 0, s, c, x, start, count, T, H, err);
  return launch_k(paged_store_kernel<32>, grid, dim3(256), 0, s, c, x, start, count, T, H, err);
}

namespace {

template <int D, int QR, int UPW>
cudaError_t launch_short(const PagedCache& c, const __nv_bfloat16* qkv, const int32_t* lens, __nv_bfloat16* y, float* lse2,
                         const DecShape& w, int nc, int dev, int* err, cudaStream_t s) {
  static SmemLimit limit;
  constexpr int smem = ShortCfg<D, QR, UPW>::SMEM;
  const cudaError_t e = limit.raise(paged_short_kernel<D, QR, UPW>, dev, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(nc) * c.Hkv * w.mg, static_cast<unsigned>(w.B));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(nc), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, paged_short_kernel<D, QR, UPW>, c, qkv, lens, y, lse2, w, err);
}

template <int D, int QR>
cudaError_t launch_decode(const PagedCache& c, const __nv_bfloat16* qkv, const int32_t* lens, __nv_bfloat16* y, float* lse2,
                          DecShape w, int* err, cudaStream_t s) {
  using Cfg = DecCfg<D, QR>;
  static SmemLimit limit;
  int dev = 0, num_sms = 0;
  cudaError_t e = device_sms(&dev, &num_sms);
  if (e != cudaSuccess) return e;
  long long seen_max = static_cast<long long>(c.max_pages) << c.page_log2;
  if (w.window > 0 && static_cast<long long>(w.window) + w.sinks < seen_max) seen_max = w.window + w.sinks;
  // Few rows in sight: one launch of clusters (8 NC warps of UPW units). It pays for blocks that a short sequence leaves
  // idle, so it is taken up to 12 blocks per SM with one unit per warp (2,048 rows; 12 heads, graph replays: 16 sequences of
  // up to 1,023 rows 10.2 against 13.1 us, of up to 2,047 15.9 against 16.9; 64 sequences of up to 1,023, 20 blocks per
  // SM, 32.5 against 30.1), and with two units while all blocks run at once (one per SM; 4,095 rows: one sequence 5.1
  // against 13.2 us, four of them, 2.5 blocks per SM, 16.4 against 14.5).
  const long long units = (seen_max + kUnit - 1) / kUnit, lists = static_cast<long long>(w.B) * c.Hkv * w.mg;
  if (units <= 128 && (!c.weight || w.mg == 1)) {
    int nc = 1;
    while (nc < 8 && nc * 8 < units) nc *= 2;
    if (units <= 64 && nc * lists <= 12LL * num_sms) return launch_short<D, QR, 1>(c, qkv, lens, y, lse2, w, nc, dev, err, s);
    if (units > 64 && nc * lists <= num_sms) return launch_short<D, QR, 2>(c, qkv, lens, y, lse2, w, nc, dev, err, s);
  }
  // one block per SM with as many warps (rings) as its shared memory holds beside the sequences' lengths, 8 at most
  const size_t head = (2 * static_cast<size_t>(w.B) + 1) * sizeof(int);
  const size_t room = 232448 - 256 - head;
  const int warps = room / Cfg::WARP < 8 ? static_cast<int>(room / Cfg::WARP) : 8;
  const size_t smem = static_cast<size_t>(warps) * Cfg::WARP + head;
  e = limit.raise(paged_split_kernel<D, QR>, dev, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int NW = num_sms * warps;
  const int score_ld = static_cast<int>((seen_max + kUnit - 1) / kUnit * kUnit);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t pre_b = up((w.B + 1) * sizeof(int)), o_b = up(static_cast<size_t>(NW) * 2 * QR * D * sizeof(float)),
               ml_b = up(static_cast<size_t>(NW) * 2 * QR * sizeof(float2)), lse_b = up(static_cast<size_t>(w.B) * w.H * sizeof(float)),
               sc_b = c.weight ? static_cast<size_t>(w.B) * w.H * score_ld * sizeof(float) : 0;
  uint8_t* p = nullptr;
  e = scratch_alloc(reinterpret_cast<void**>(&p), pre_b + o_b + ml_b + lse_b + sc_b, s);
  if (e != cudaSuccess) return e;
  DecScratch ws;
  ws.prefix = reinterpret_cast<int*>(p);
  ws.o = reinterpret_cast<float*>(p + pre_b);
  ws.ml = reinterpret_cast<float2*>(p + pre_b + o_b);
  ws.lse = reinterpret_cast<float*>(p + pre_b + o_b + ml_b);
  ws.score = c.weight ? reinterpret_cast<float*>(p + pre_b + o_b + ml_b + lse_b) : nullptr;
  ws.score_ld = score_ld;
  e = launch_k(paged_split_kernel<D, QR>, dim3(num_sms), dim3(32 * warps), smem, s, c, qkv, lens, y, lse2, w, ws, err);
  if (e == cudaSuccess) {
    const long long chunks = c.weight ? (seen_max + kJoinRows - 1) / kJoinRows : 1;
    e = launch_k(paged_join_kernel<D, QR>,
                 dim3(static_cast<unsigned>(c.Hkv), static_cast<unsigned>(chunks < 65535 ? chunks : 65535), static_cast<unsigned>(w.B)),
                 dim3(kJoinThreads), 0, s, c, lens, y, lse2, w, ws, NW, err);
  }
  const cudaError_t f = scratch_free(p, s);
  return e != cudaSuccess ? e : f;
}

}  // namespace

cudaError_t launch_paged_attention(const PagedCache& c, const void* qkv, const int32_t* lens, void* y, float* lse2,
                                   int B, int H, int D, int window, int sinks, int* err, cudaStream_t s) {
  DecShape w;
  w.B = B;
  w.H = H;
  w.G = H / c.Hkv;
  w.mg = (w.G + 15) / 16;
  w.window = window;
  w.sinks = sinks;
  w.scale_log2 = kLog2e / sqrtf(static_cast<float>(D));
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(qkv);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(y);
  // up to 8 query heads per key head need half of the 16 query rows in shared memory and registers
  if (D == 64)
    return w.G <= 8 ? launch_decode<64, 8>(c, x, lens, o, lse2, w, err, s) : launch_decode<64, 16>(c, x, lens, o, lse2, w, err, s);
  return w.G <= 8 ? launch_decode<32, 8>(c, x, lens, o, lse2, w, err, s) : launch_decode<32, 16>(c, x, lens, o, lse2, w, err, s);
}

cudaError_t launch_paged_evict(const PagedCache& c, const int32_t* lens, const int32_t* dst_table, int dst_max_pages,
                               int32_t* new_lens, int32_t* kept, int B, int D, int budget, int sinks, int recent,
                               int* err, cudaStream_t s) {
  // one block per list up to 4,096 rows, clusters of four for longer lists; ranks for the longest stretch that the
  // table allows, as far as shared memory goes
  const long long all = static_cast<long long>(c.max_pages) << c.page_log2, rows = all - sinks - recent;
  const int nc = rows <= 4096 ? 1 : 4;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  // One launch where the choosing blocks copy as well: a block copies 256 rows in about 1.9 us, a second launch takes 2.5
  // and then has the whole machine. 64 sequences x 12 heads of up to 1,024 rows to 512: 44.6 us in one, 53.3 in two
  // launches, 16 sequences 12.8 and 13.3; 48 lists to 512 rows 8.5 and 9.3, to 900 rows 12.1 and 11.0; 12 lists to 128
  // rows 6.3 and 6.5, to 512 rows 8.4 and 6.6.
  const long long lists = static_cast<long long>(B) * c.Hkv;
  const int held = static_cast<int>(budget < all ? budget : all);      // rows that a list can keep
  const bool one = nc == 1 && held <= 4096 && (lists >= sms || held <= 14 * lists);
  const long long most = (232448 - 28672) / 4, stretch = rows < 0 ? 0 : ((rows + nc - 1) / nc + 31) / 32 * 32;
  const int room = static_cast<int>(stretch < most ? stretch : most);
  const int form = nc == 4 ? 0 : !one ? 1 : D == 64 ? 2 : 3;
  const int smem = 4 * (room + (one ? held : 0));
  auto choose = form == 0 ? paged_choose_kernel<4, 0> : form == 1 ? paged_choose_kernel<1, 0>
      : form == 2 ? paged_choose_kernel<1, 64> : paged_choose_kernel<1, 32>;
  static SmemLimit limit[4];
  e = limit[form].raise(choose, dev, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c.Hkv) * nc, static_cast<unsigned>(B));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(nc), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, choose, c, lens, new_lens, kept, dst_table, dst_max_pages, budget, sinks, recent, room, err);
  if (e != cudaSuccess || one) return e;
  const int chunk = kMoveBlocks * (kMoveThreads / (D / 8)) * kMoveDepth, chunks = (budget - 1) / chunk + 1;
  const dim3 grid(static_cast<unsigned>(kMoveBlocks * (chunks < 8 ? chunks : 8)), static_cast<unsigned>(c.Hkv),
                  static_cast<unsigned>(B));
  if (D == 64)
    return launch_k(paged_move_kernel<64>, grid, dim3(kMoveThreads), 0, s, c, dst_table, dst_max_pages,
                    static_cast<const int32_t*>(kept), budget, err);
  return launch_k(paged_move_kernel<32>, grid, dim3(kMoveThreads), 0, s, c, dst_table, dst_max_pages,
                  static_cast<const int32_t*>(kept), budget, err);
}

}  // namespace gptgb
