// Sliding-window attention with sinks on tcgen05 for sm_103a (prompt form).
//
// Query t sees key s if s <= t and (t - s < W or s < S): the last W keys and the sequence's first S ("sinks").
// y = softmax(Q K^T / sqrt(D)) U over the seen keys, per (batch b, head h); H query heads share Hkv key heads.
// Q, K, U are read straight out of the fused projection's rows [B, T, (H + 2 Hkv) D] through a 3-D TMA map (a
// head is a column offset) and the merged heads y [B, T, H D] are stored by TMA.
//
// The work follows the window: a 128-row query tile reads the key tiles from its first row's window start to its
// diagonal, and the tiles that hold sinks, so work and traffic grow with T (W + S), not T^2 / 2. The kernel is
// bound by the softmax warps, not by the tensor core: a 128-key tile takes them about 2,000 cycles, of which the
// exponentials are 1,024 (one per score on a quarter-rate unit, two warps per scheduler) and the rest waits between
// dependent instructions and for tensor memory; the tile's two products take 540. So a warp leaves out the 32-key
// parts of a tile of which its rows see nothing (beyond the diagonal, before the window, after the sinks), masks only
// tiles that a border crosses, takes few sinks (up to 16) as one step of 16 keys, and works 32 keys at a time with the
// next scores on their way out of tensor memory meanwhile.
// Measured (calls back to back): 12,001 tokens, 25 heads on 5, D 64, W 1500: 126 us, 860 TFLOP/s; 16 x 1,024 tokens,
// 12 heads, W 256: 35 us, 2.9 TB/s of rows.
//
// Pipeline (one persistent CTA per SM, 352 threads): as in the full causal kernel, a work item is one (b, h) and a
// PAIR of consecutive query tiles that share one stream of 128-key tiles, K and U through a four-stage TMA ring each; two
// softmax groups of four warps (thread = query row = TMEM lane) own one query tile each and run out of phase.
// Where the pairs would leave SMs without work an item is one query tile. Items are dealt statically, the long
// ones first, forwards and backwards in turn (item r of CTA c: r grid + c, or r grid + grid - 1 - c for odd r):
// all items but a sequence's first few cost the same, and no work counter has to be cleared before the launch.
//
// The score tiles of both groups form ONE sequence: list entry i of the item, group 0's tile then group 1's,
// leaving out what a group does not see. Score number k goes to TMEM buffer k % 3. One warp issues
// S(k + 3) = Q K^T into buffer k % 3 once the P U of number k has completed; another waits for the probabilities
// P(k) (written by the owning group over the first 64 columns of the buffer as bf16 pairs; one hand-over per tile:
// two, a 64-key half each, cost more in waits than their earlier start gave) and issues O_g += P(k) U_j with the A
// operand in tensor memory.
//
// An item's key tiles come from the diagonal down, the sinks last, so that every row sees a key of its first tile.
//
// Softmax: per row one running reference m and sum. The reference starts as the score of the warp's first diagonal key
// where all its rows see that (W >= 32), else as the exact maximum of the first half tile in which the row sees a key;
// it is raised only when a half tile's sum passes 2^16 and the maximum grew by more than 2^8, and by a whole number, so that
// sum, output and the tile's rounded probabilities are rescaled by a power of two, which is exact. Sums are fp32; P is
// rounded to bf16 once, for the second product (the type the tensor core multiplies), which costs at most 2^-8 of
// sum a |u|.
//
// Taken back, at the 12,001 tokens above as they were then: tiles of 64 keys in six score buffers (157 us against 151),
// a third softmax group (194 against 151), more registers for the softmax warps by setmaxnreg (207 against 185).
//
// Tensor memory (512 columns): score buffers at 0, 128, 256; O_g at 384 + 64 g.
// Warps: 0 TMA producer; 1 TMEM allocator and P U issuer; 2-5 softmax group 0; 6-9 group 1; 10 score issuer.
#include "attn_window.cuh"
#include "kernels.h"
#include "launch.h"

#include <math.h>

namespace gptgb {

namespace {

constexpr int BQ = kAttnBQ;       // query rows per tile
constexpr int BKV = 128;          // keys per tile
constexpr int THREADS = 352;
constexpr int TMEM_COLS = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;    // rescale O only when the max grows by more than this
constexpr float kSumLimit = 65536.0f;   // recompute a tile against its exact max past this sum
constexpr int NS = 4;                   // ring depth of K and of U
constexpr int NSB = 3;                  // score buffers
constexpr uint32_t kColO = 128 * NSB;   // O_g at kColO + 64 g
constexpr int SR = 4;                   // items announced ahead by the producer
constexpr int CH = 64;                  // keys that a softmax warp handles at a time
constexpr int kFewSinks = 16;           // sinks that are taken as one step of 16 keys
constexpr int kConsumers = 10;          // warps that read each announced item: 2 MMA issuers + 8 softmax

template <int D>
struct AttnCfg {
  static constexpr int ROWB = D * 2;                               // bytes per row of a Q/K/U tile
  static constexpr uint32_t SWZ = (ROWB == 128) ? SWZ_128B : SWZ_64B;
  static constexpr int TILE = BQ * ROWB;
  static constexpr int STG = 32 * ROWB;                            // one warp's 32 output rows
  static constexpr int OFF_Q = 0;                                    // [buffer][group] query tiles
  static constexpr int OFF_K = 4 * TILE;                             // NS stages
  static constexpr int OFF_U = OFF_K + NS * TILE;                    // NS stages
  static constexpr int OFF_STG = OFF_U + NS * TILE;                  // 8 warps' output staging
  static constexpr int OFF_BAR = OFF_STG + 8 * STG;
  // at least 120 KB so that two CTAs (2 x 512 TMEM columns) never share an SM
  static constexpr int SMEM = (OFF_BAR + 512 > 120 * 1024) ? OFF_BAR + 512 : 120 * 1024;
  static_assert(D == 32 || D == 64, "head width");
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct __align__(16) AttnBars {
  uint64_t q_empty[2];      // every S of the item that used Q buffer k has been computed
  uint64_t k_full[NS];      // ring stage holds K_j (and, for an item's first tile, its query tiles)
  uint64_t k_empty[NS];     // every S of that tile has been computed
  uint64_t u_full[NS];      // ring stage holds U_j
  uint64_t u_empty[NS];     // every P U of that tile has been computed
  uint64_t s_full[2][NSB];  // score buffer b holds a new score tile of group g (that group's uses of b, in order)
  uint64_t p_full[NSB];     // score buffer b holds that tile's probabilities (4 warps)
  uint64_t pv_done[NSB];    // the P U that read buffer b has completed (the buffer may take new scores)
  uint64_t drain[2];        // the issuing warps' own MMAs have completed (exit)
  uint64_t item_full[SR];   // slot r % SR holds this CTA's r-th item (from the producer)
  uint64_t item_empty[SR];  // every other warp has read it
  __align__(16) int item[SR][8];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(AttnBars) <= 512, "barrier block");


// The products of one step by one elected lane of the converged warp: a single election for all of them (and the
// commit), as the issuing warps' own instructions are part of every score buffer's round.
template <int D>
__device__ __forceinline__ void issue_s(uint32_t tS, uint64_t q_desc, uint64_t k_desc, uint64_t* full) {
  constexpr uint32_t idesc = idesc_bf16_f32(BQ, BKV, false);
  // K-major: a K step of 16 bf16 is 32 bytes (2 descriptor units) along the swizzled row
  if constexpr (D == 64) {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 b2, %2, 4;\n\t"
        "add.s64 a3, %1, 6;\n\tadd.s64 b3, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}\n"
        :: "r"(tS), "l"(q_desc), "l"(k_desc), "r"(idesc), "r"(smem_u32(full)) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a1, b1;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}\n"
        :: "r"(tS), "l"(q_desc), "l"(k_desc), "r"(idesc), "r"(smem_u32(full)) : "memory");
  }
}

// O += P_h U_h for keys [64 h, 64 h + 64) of a tile: P lies in TMEM over the first 64
// columns of its score buffer (two bf16 per column, row = lane; keys 64 h.. at column 32 h; a K step of 16 keys: 8
// columns), U is MN-major in shared memory (D contiguous per key; a K step: 16 rows, D * 2 descriptor units).
template <int D>
__device__ __forceinline__ void issue_pv_half(uint32_t tO, uint32_t tP, uint64_t u_desc, int h, bool accumulate) {
  using Cfg = AttnCfg<D>;
  constexpr uint32_t idesc = idesc_bf16_f32(BQ, D, true);     // U is MN-major (D contiguous)
  asm volatile(
      "{\n\t.reg .pred e, f, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, %5;\n\tadd.s64 b2, b1, %5;\n\tadd.s64 b3, b2, %5;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}\n"
      :: "r"(tO), "r"(tP + 32 * h), "l"(desc_add(u_desc, 64 * h * Cfg::ROWB)), "r"(idesc), "r"(accumulate ? 1u : 0u),
         "n"(16 * Cfg::ROWB / 16) : "memory");
}

// The same for the first 16 keys of a tile alone (those after the sinks of a sink tile have no probability).
template <int D>
__device__ __forceinline__ void issue_pv_sinks(uint32_t tO, uint32_t tP, uint64_t u_desc, bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(BQ, D, true);
  asm volatile(
      "{\n\t.reg .pred e, f;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 f, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t}\n"
      :: "r"(tO), "r"(tP), "l"(u_desc), "r"(idesc), "r"(accumulate ? 1u : 0u) : "memory");
}

// What a launch computes, and how its items are cut.
struct WinShape {
  int T, H, G, window, sinks;   // G query heads per key head; window >= 1
  int BH, n_qtiles;
  int per_item;                 // query tiles per item: 2 or 1
  int n_groups;                 // items per (b, h)
  int n_items;
  int sink_tiles;               // key tiles that hold a sink
};

// Item r of this CTA, or -1.
__device__ __forceinline__ int item_of(const WinShape& w, int r) {
  const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  const long long i = static_cast<long long>(r) * g + ((r & 1) ? g - 1 - c : c);
  return i < w.n_items ? static_cast<int>(i) : -1;
}

// One item: query tiles qt0 (group 0) and, if `two`, qt0 + 1 (group 1), and the list of key tiles they share: entries
// [0, m) are the tiles of the window from the last diagonal (tile `top`) down to the window start of qt0's first row,
// entries [m, m + a) the sink tiles before those. Group 0 takes all but the other's diagonal; group 1 takes all but
// entry m - 1 where `skip` (its own window starts one tile later and that tile holds no sink).
struct Item {
  int b, h, qt0, a, top, m, n;
  int two, skip;
  __device__ __forceinline__ int tile(int i) const { return i < m ? top - i : a - 1 - (i - m); }
  __device__ __forceinline__ int first0() const { return two; }
  __device__ __forceinline__ bool has1(int i) const { return two && !(skip && i == m - 1); }
  // position of (entry i, group g) in the item's score sequence, and the sequence's length
  __device__ __forceinline__ int number(int i, int g) const {
    return max(i + g - two, 0) + (two ? i - (skip && i >= m ? 1 : 0) : 0);
  }
  __device__ __forceinline__ int total() const { return number(n, 0); }
};

__device__ __forceinline__ Item decode_item(const WinShape& w, int item) {
  Item x;
  const int p = w.n_groups - 1 - item / w.BH;
  const int bh = item % w.BH;
  x.b = bh / w.H;
  x.h = bh % w.H;
  x.qt0 = w.per_item * p;
  x.two = w.per_item == 2 && x.qt0 + 1 < w.n_qtiles;
  const int first = x.qt0 * BQ - w.window + 1;       // window start of the first row (window < 2^30: no overflow)
  const int j0 = first > 0 ? first / BKV : 0;
  x.a = min(w.sink_tiles, j0);
  const int j1 = first + BQ > 0 ? (first + BQ) / BKV : 0;
  x.skip = x.two && j1 > j0 && j0 >= w.sink_tiles;
  x.top = x.qt0 + x.two;
  x.m = x.top - j0 + 1;
  x.n = x.m + x.a;
  return x;
}

// The CTA's r-th item from the producer, which decodes it (a chain of divisions that the other warps would wait for)
// and announces it through a ring of SR slots; n = 0 ends the list.
__device__ __forceinline__ bool next_item(AttnBars* bars, int r, Item& x, volatile int* abort_flag, int* err, int lane) {
  const int slot = r % SR;
  if (!mbar_wait_warp(&bars->item_full[slot], static_cast<uint32_t>(r / SR) & 1u, abort_flag, err)) return false;
  const int4* v = reinterpret_cast<const int4*>(bars->item[slot]);
  const int4 p = v[0], q = v[1];
  x.b = p.x;
  x.h = p.y;
  x.qt0 = p.z;
  x.a = p.w;
  x.top = q.x;
  x.m = q.y;
  x.n = q.z;
  x.two = q.w & 1;
  x.skip = q.w >> 1;
  __syncwarp();
  if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
  return x.n > 0;
}

__device__ __forceinline__ void load_chunk(uint32_t col, uint32_t (&v)[64]) {
  tmem_ld_32x32b_x64(col, v);
  tmem_ld_wait();
}
// The two rare steps of a softmax warp, out of line: inlined they took the registers and the instruction cache of the
// loop that turns scores into probabilities.

// Row references: the exact maximum of a chunk's seen keys becomes the reference of a row that had none. A reference that
// it passes by more than 2^8 rises by the next whole number of steps (to the rounding of the fp32 sum, as that of a score
// of its size); the running sum, the output so far (unless the item starts here) and the tile's probabilities so far (n_p
// columns of 16 at tS) are rescaled, by a power of two. `prev`: the group's previous score tile.
struct RowRef {
  float mr, l;
  bool ok;
};
template <int D>
__device__ __noinline__ RowRef raise_reference(AttnBars* bars, uint32_t tSc, uint32_t tS, uint32_t tO, int n_p, float mr,
                                               float l, float scale_log2, uint32_t seen0, uint32_t seen1, bool first,
                                               uint32_t prev, volatile int* abort_flag, int* err) {
  uint32_t v[CH];
  load_chunk(tSc, v);
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < CH; i += 2) {
    const uint32_t seen = i < 32 ? seen0 : seen1;
    mx[(i >> 1) & 3] = fmax3(mx[(i >> 1) & 3], (seen >> (i & 31)) & 1u ? __uint_as_float(v[i]) : -INFINITY,
                             (seen >> ((i + 1) & 31)) & 1u ? __uint_as_float(v[i + 1]) : -INFINITY);
  }
  const float m_max = fmaxf(mr, fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * scale_log2);
  const bool fresh = mr == -INFINITY;                // l and the row's outputs are zero
  const bool need = m_max > mr + kRescaleLog2;       // (true for a fresh row that sees a key here)
  const float up = need && !fresh ? ceilf(m_max - mr) : 0.0f;
  const float alpha = up > 126.0f ? 0.0f : __int_as_float((127 - static_cast<int>(up)) << 23);   // 2^-up
  RowRef out = {!need ? mr : fresh ? m_max : mr + up, l * alpha, true};
  if (__any_sync(0xffffffffu, need && !fresh)) {
    if (!first) {
      // every earlier P U of the group has completed
      if (!mbar_wait_warp(&bars->pv_done[prev % NSB], (prev / NSB) & 1u, abort_flag, err)) {
        out.ok = false;
        return out;
      }
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        uint32_t o[16];
        tmem_ld_32x32b_x16(tO + c * 16, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
        tmem_st_32x32b_x16(tO + c * 16, o);
      }
    }
    tmem_st_wait();
#pragma unroll 1
    for (int c = 0; c < n_p; ++c) {
      uint32_t q[16];
      tmem_ld_32x32b_x16(tS + 16 * c, q);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = unpack_bf16x2(q[i]);
        q[i] = pack_bf16x2(f.x * alpha, f.y * alpha);
      }
      tmem_st_32x32b_x16(tS + 16 * c, q);
    }
    tmem_st_wait();
  }
  return out;
}

// An item's output: this warp's 32 rows, normalised, staged and stored by TMA; the rows' log-sum-exp (`lse` nullable).
template <int D>
__device__ __noinline__ bool write_rows(AttnBars* bars, uint32_t prev, uint32_t tO, uint8_t* stg, const CUtensorMap* tm_y,
                                        int col, int row, int b, float l, float m, float* lse, volatile int* abort_flag,
                                        int* err) {
  using Cfg = AttnCfg<D>;
  const int lane = threadIdx.x & 31;
  if (!mbar_wait_warp(&bars->pv_done[prev % NSB], (prev / NSB) & 1u, abort_flag, err)) return false;
  tc_fence_after();
  const float inv = 1.0f / l;
  if (lane == 0) bulk_wait_read_all();               // this warp's previous store has read its staging box
  __syncwarp();
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(tO + 32 * c, o);
    tmem_ld_wait();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint4 v;
      v.x = pack_bf16x2(__uint_as_float(o[8 * u + 0]) * inv, __uint_as_float(o[8 * u + 1]) * inv);
      v.y = pack_bf16x2(__uint_as_float(o[8 * u + 2]) * inv, __uint_as_float(o[8 * u + 3]) * inv);
      v.z = pack_bf16x2(__uint_as_float(o[8 * u + 4]) * inv, __uint_as_float(o[8 * u + 5]) * inv);
      v.w = pack_bf16x2(__uint_as_float(o[8 * u + 6]) * inv, __uint_as_float(o[8 * u + 7]) * inv);
      *reinterpret_cast<uint4*>(stg + lane * Cfg::ROWB + (swz_unit(Cfg::ROWB, lane, 4 * c + u) << 4)) = v;
    }
  }
  tc_fence_before();                                 // the accumulator may be overwritten after this
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(tm_y, stg, col, row, b);
    bulk_commit();
  }
  if (lse != nullptr) *lse = m + log2f(l);
  return true;
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
attn_window_tc_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_y,
                      const WinShape w, float scale_log2, int* err, float* lse2) {
  using Cfg = AttnCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  AttnBars* bars = reinterpret_cast<AttnBars*>(smem_raw + Cfg::OFF_BAR);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((smem_u32(smem_raw) & 1023u) != 0) {           // the swizzle atoms need 1024-byte alignment
    if (threadIdx.x == 0) record_error(err, GPT_DEV_EALIGN);
    return;
  }
  uint8_t* sQ = smem_raw + Cfg::OFF_Q;
  uint8_t* sK = smem_raw + Cfg::OFF_K;
  uint8_t* sU = smem_raw + Cfg::OFF_U;
  volatile int* abort_flag = &bars->abort_flag;

  const int T = w.T, H = w.H;
  const int kcol = H * D, ucol = (H + H / w.G) * D;    // first key and value columns of a row

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_empty[0], 1);
    mbar_init(&bars->q_empty[1], 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->u_full[i], 1);
      mbar_init(&bars->u_empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&bars->s_full[0][i], 1);
      mbar_init(&bars->s_full[1][i], 1);
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->pv_done[i], 1);
    }
    mbar_init(&bars->drain[0], 1);
    mbar_init(&bars->drain[1], 1);
    for (int i = 0; i < SR; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], kConsumers);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm);
    tma_prefetch_desc(&tm_y);
  }
  if (warp == 1) tmem_alloc(&bars->tmem_base, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  pdl_wait();                       // qkv written by the previous kernel is now visible
  pdl_trigger();

  if (warp == 0) {
    // ------------------------------------------------ producer of items and copies
    if (lane == 0) {
      uint32_t pos = 0, u_pos = 0;                   // K and U tiles loaded so far (ring positions)
      int ux = 0, u_row = 0, ub = 0;                 // where the next U lies
      // U one tile behind K: its stage is released later, and K's copy does not wait for that
      auto load_u = [&]() -> bool {
        const int s = u_pos % NS;
        if (!mbar_wait(&bars->u_empty[s], ((u_pos / NS) & 1u) ^ 1u, abort_flag, err)) return false;
        mbar_arrive_expect_tx(&bars->u_full[s], Cfg::TILE);
        tma_load_3d(sU + s * Cfg::TILE, &tm, &bars->u_full[s], ux, u_row, ub);
        ++u_pos;
        return true;
      };
      bool ok = true;
      for (int r = 0; ok; ++r) {
        const int item = item_of(w, r);
        const int slot = r % SR;
        if (r >= SR && !mbar_wait(&bars->item_empty[slot], static_cast<uint32_t>(r / SR - 1) & 1u, abort_flag, err)) break;
        Item x = {};
        if (item >= 0) x = decode_item(w, item);
        int4* v = reinterpret_cast<int4*>(bars->item[slot]);
        v[0] = make_int4(x.b, x.h, x.qt0, x.a);
        v[1] = make_int4(x.top, x.m, x.n, x.two | (x.skip << 1));
        mbar_arrive(&bars->item_full[slot]);
        if (item < 0) break;
        const int kh = x.h / w.G;                    // key head
        const int qb = r & 1;                        // Q buffer of this item; its previous user was item r - 2
        if (r >= 2 && !mbar_wait(&bars->q_empty[qb], static_cast<uint32_t>((r >> 1) - 1) & 1u, abort_flag, err)) break;
        for (int i = 0; i < x.n; ++i) {
          const int s = pos % NS;
          if (!mbar_wait(&bars->k_empty[s], ((pos / NS) & 1u) ^ 1u, abort_flag, err)) { ok = false; break; }
          // the item's query tiles complete on the barrier of its first K tile
          const int nq = (i == 0) ? (x.two ? 2 : 1) : 0;
          const int row = x.tile(i) * BKV;
          mbar_arrive_expect_tx(&bars->k_full[s], (1 + nq) * Cfg::TILE);
          if (nq > 0) tma_load_3d(sQ + (2 * qb) * Cfg::TILE, &tm, &bars->k_full[s], x.h * D, x.qt0 * BQ, x.b);
          if (nq > 1) tma_load_3d(sQ + (2 * qb + 1) * Cfg::TILE, &tm, &bars->k_full[s], x.h * D, (x.qt0 + 1) * BQ, x.b);
          tma_load_3d(sK + s * Cfg::TILE, &tm, &bars->k_full[s], kcol + kh * D, row, x.b);
          ++pos;
          if (pos > 1 && !load_u()) { ok = false; break; }
          ux = ucol + kh * D;
          u_row = row;
          ub = x.b;
        }
      }
      if (ok && u_pos < pos) load_u();
      // never leave with copies in flight into this CTA's shared memory: the last ones into each stage
      for (uint32_t q = pos > NS ? pos - NS : 0; q < pos; ++q) mbar_wait_drain(&bars->k_full[q % NS], (q / NS) & 1u);
      for (uint32_t q = u_pos > NS ? u_pos - NS : 0; q < u_pos; ++q) mbar_wait_drain(&bars->u_full[q % NS], (q / NS) & 1u);
    }
  } else if (warp == 1 || warp == 10) {
    // ------------------------------------------------ MMA issuers (whole warp; one elected lane issues)
    // Two warps on different sub-partitions share the issue work, each walking the same
    // sequence of score numbers: warp 1 waits for P(k) and issues O_g += P(k) U_j; warp 10
    // issues S(k) = Q K_j^T into buffer k % 3 once the P U of number k - 3 (which read that
    // buffer) has completed. K's ring stage is released by the tile's last S, U's by its last P U,
    // which comes up to two tiles later: with one stage for both, K's loads had that much less time
    // (64 x 1,024 tokens, 12 heads, W 256: 118 us against 109).
    {
      const bool pv_warp = warp == 1;
      // base descriptors: Q and K K-major (8-row groups ROWB*8 apart), U MN-major (K-direction
      // 8-row groups ROWB*8 apart)
      const uint64_t dq0 = smem_desc(smem_u32(sQ), 16, 8 * Cfg::ROWB, Cfg::SWZ);
      const uint64_t dk0 = smem_desc(smem_u32(sK), 16, 8 * Cfg::ROWB, Cfg::SWZ);
      const uint64_t du0 = smem_desc(smem_u32(sU), Cfg::TILE, 8 * Cfg::ROWB, Cfg::SWZ);
      Item x;
      uint32_t b = 0;                                // buffer of number k (k % 3)
      uint32_t bits = 0;                             // phase per buffer of the barrier this warp waits on
      uint32_t pos = 0;                              // ring position
      bool ok = true;
      if (pv_warp) {
        for (int r = 0; ok && next_item(bars, r, x, abort_flag, err, lane); ++r) {
          for (int i = 0; i < x.n && ok; ++i, ++pos) {
            const uint32_t st = pos % NS;
            if (!mbar_wait_warp(&bars->u_full[st], (pos / NS) & 1u, abort_flag, err)) { ok = false; break; }
            const uint64_t du = desc_add(du0, st * Cfg::TILE);
            const int g_end = x.has1(i) ? 2 : 1;
#pragma unroll 1
            for (int g = i >= x.first0() ? 0 : 1; g < g_end; ++g) {
              const uint32_t tOg = tmem_base + kColO + 64 * g, tP = tmem_base + 128 * b;
              const bool more = i > (g ? 0 : x.first0());
              if (!mbar_wait_warp(&bars->p_full[b], (bits >> b) & 1u, abort_flag, err)) { ok = false; break; }
              bits ^= 1u << b;
              tc_fence_after();
              if (i >= x.m && w.sinks <= kFewSinks) {
                issue_pv_sinks<D>(tOg, tP, du, more);
              } else {
                issue_pv_half<D>(tOg, tP, du, 0, more);
                issue_pv_half<D>(tOg, tP, du, 1, true);
              }
              tc_commit_warp(&bars->pv_done[b]);
              b = b == NSB - 1 ? 0 : b + 1;
            }
            if (ok) tc_commit_warp(&bars->u_empty[st]);
          }
        }
      } else {
        uint32_t n = 0;                              // scores so far, up to NSB
        for (int r = 0; ok && next_item(bars, r, x, abort_flag, err, lane); ++r) {
          const uint32_t qb = static_cast<uint32_t>(r) & 1u;
          for (int i = 0; i < x.n && ok; ++i, ++pos) {
            const uint32_t st = pos % NS;
            if (!mbar_wait_warp(&bars->k_full[st], (pos / NS) & 1u, abort_flag, err)) { ok = false; break; }
            const uint64_t dk = desc_add(dk0, st * Cfg::TILE);
            const int g_end = x.has1(i) ? 2 : 1;
#pragma unroll 1
            for (int g = i >= x.first0() ? 0 : 1; g < g_end; ++g) {
              if (n == NSB) {                        // the P U that read this buffer has completed
                if (!mbar_wait_warp(&bars->pv_done[b], (bits >> b) & 1u, abort_flag, err)) { ok = false; break; }
                bits ^= 1u << b;
              } else {
                ++n;
              }
              tc_fence_after();
              issue_s<D>(tmem_base + 128 * b, desc_add(dq0, (2 * qb + g) * Cfg::TILE), dk, &bars->s_full[g][b]);
              b = b == NSB - 1 ? 0 : b + 1;
            }
            if (ok) tc_commit_warp(&bars->k_empty[st]);
          }
          if (ok) tc_commit_warp(&bars->q_empty[qb]);   // every S of the item has read its Q
        }
      }
      uint64_t* dr = &bars->drain[pv_warp ? 0 : 1];
      tc_commit_warp(dr);
      mbar_wait_drain(dr, 0);
    }
  } else {
    // ------------------------------------------------ softmax (group g owns query tile qt0 + g)
    const int g = (warp - 2) >> 2;
    const int sub = warp & 3;
    const int r_row = sub * 32 + lane;                // query row within the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(sub * 32) << 16;
    const uint32_t tO = tmem_base + kColO + 64 * g + lane_off;
    uint8_t* stg = smem_raw + Cfg::OFF_STG + (warp - 2) * Cfg::STG;
    uint32_t kbase = 0;                               // score number of the item's first tile
    uint32_t last = 0;                                // the number of this group's previous score tile
    uint32_t bits = 0;                                // per buffer: the phase of this group's next tile there
    bool ok = true;
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    // An item's output is written during the group's next tile, just before that tile's first
    // P U (which overwrites the accumulator) is released: by then the item's last P U has
    // completed, so the group never idles on it.
    bool pend = false;
    float pl = 0.0f;                                  // the pending item's running sum
    float pm = 0.0f;                                  // and its running max (log2 units)
    int pb = 0, ph = 0, pqt = 0;                      // its batch row, head and query tile
    uint32_t plast = 0;                               // the number of its last score tile
    auto write_out = [&]() -> bool {
      const int t = pqt * BQ + r_row;
      float* lse = lse2 != nullptr && t < T ? lse2 + (static_cast<size_t>(pb) * H + ph) * T + t : nullptr;
      pend = false;
      return write_rows<D>(bars, plast, tO, stg, &tm_y, ph * D, pqt * BQ + sub * 32, pb, pl, pm, lse, abort_flag, err);
    };
    const int wrow = sub * 32;                        // first row of this warp within the tile
    for (int r = 0; ok; ++r) {
      Item x;
      if (!next_item(bars, r, x, abort_flag, err, lane)) break;
      const uint32_t knext = kbase + x.total();
      if (g == 1 && !x.two) { kbase = knext; continue; }   // group 1 without a query tile
      const int qt = x.qt0 + g;
      const int t = qt * BQ + r_row;                  // query position
      const int tw = qt * BQ + wrow;                  // the warp's first query
      const int i0 = g == 0 ? x.first0() : 0;
      float mr = -INFINITY;                           // running (lazily raised) reference, log2 units
      float l = 0.0f;                                 // running sum of 2^(s - mr)
      bool ready = false;                             // every row of the warp has a reference
      uint32_t k = kbase + x.number(i0, g);           // the tile's score number, and its buffer
      uint32_t b = k % NSB;
      int kb = x.tile(i0) * BKV;                      // the tile's first key
      bool early = false;                             // the tile's scores were there when the last one was handed over
      for (int i = i0; i < x.n;) {
        const bool first = i == i0;
        if (!__all_sync(0xffffffffu, early) && !mbar_wait_warp(&bars->s_full[g][b], (bits >> b) & 1u, abort_flag, err)) {
          ok = false;
          break;
        }
        bits ^= 1u << b;
        tc_fence_after();
        const uint32_t tS = tmem_base + 128 * b + lane_off;
        // bit n set: this row sees key k0 + n
        auto seen_bits = [&](int k0) -> uint32_t {
          const int hi = t - k0;                      // last key of the row
          const int lo = hi - w.window + 1;           // first key of its window
          const uint32_t to_hi = hi < 0 ? 0u : (hi >= 31 ? ~0u : (2u << hi) - 1u);
          const uint32_t from_lo = lo <= 0 ? ~0u : (lo >= 32 ? 0u : ~0u << lo);
          const int ns = w.sinks - k0;
          const uint32_t sinks = ns <= 0 ? 0u : (ns >= 32 ? ~0u : (1u << ns) - 1u);
          return to_hi & (from_lo | sinks);
        };
        // The tile's keys, CH at a time. A chunk's probabilities are final once its sum is checked (and, rarely,
        // recomputed against a raised reference); they are then stored as bf16 pairs over the buffer's first
        // columns, whose scores have been read. One copy of each loop: the warps' code has to fit the
        // instruction cache.
        int c0 = 0;
        if (ready && i >= x.m && w.sinks <= kFewSinks) {
          // a sink tile before the window with few sinks: its first 16 keys alone
          const float2 nm2 = make_float2(-mr, -mr);
          uint32_t v[16], pk[8];
          tmem_ld_32x32b_x16(tS, v);
          tmem_loaded(v);
          float2 ls = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int q = 0; q < 16; q += 2) {
            const float2 e = fma2_rn(make_float2(__uint_as_float(v[q]), __uint_as_float(v[q + 1])), sc2, nm2);
            const float2 pr = make_float2(q < w.sinks ? ex2_approx(e.x) : 0.0f, q + 1 < w.sinks ? ex2_approx(e.y) : 0.0f);
            ls = add2_rn(ls, pr);
            pk[q / 2] = pack_bf16x2(pr.x, pr.y);
          }
          const float lt = ls.x + ls.y;
          if (!__any_sync(0xffffffffu, !(lt <= kSumLimit))) {
            l += lt;
            c0 = BKV / CH;
            tmem_st_32x32b_x8(tS, pk);
          }
        } else if (ready && kb + BKV - 1 <= tw && (kb > tw + 31 - w.window || kb + BKV <= w.sinks)) {
          // every row sees the whole tile and has its reference: 32 keys at a time, the next 32 scores on their way from
          // tensor memory while these are worked on
          const float2 nm2 = make_float2(-mr, -mr);
          uint32_t va[32], vb[32], pk[CH / 2];
          float2 ls[4];
          auto stream = [&](const uint32_t (&v)[32], int at) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 e = fma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm2);
              const float2 pr = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              ls[(i >> 1) & 3] = add2_rn(ls[(i >> 1) & 3], pr);
              pk[at + i / 2] = pack_bf16x2(pr.x, pr.y);
            }
          };
          tmem_ld_32x32b_x32(tS, va);
          tmem_loaded(va);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld_32x32b_x32(tS + 64 * c + 32, vb);
#pragma unroll
            for (int q = 0; q < 4; ++q) ls[q] = make_float2(0.0f, 0.0f);
            stream(va, 0);
            tmem_loaded(vb);
            if (c == 0) tmem_ld_32x32b_x32(tS + 64, va);
            stream(vb, 16);
            const float2 l2 = add2_rn(add2_rn(ls[0], ls[1]), add2_rn(ls[2], ls[3]));
            const float lt = l2.x + l2.y;
            const bool over = __any_sync(0xffffffffu, !(lt <= kSumLimit));
            if (c == 0) tmem_loaded(va);
            if (over) break;
            l += lt;
            tmem_st_32x32b_x32(tS + 32 * c, pk);
            c0 = c + 1;
          }
        } else if (ready || (first && w.window >= 32)) {
          // the same where a border crosses the tile: 0 for the keys that a row does not see, and 32 keys of which the
          // warp's rows see nothing are left out. In the first tile, the diagonal, all rows of the warp see the key of
          // the first of them: its score is their reference.
          uint32_t va[32], vb[32], pk[CH / 2];
          float2 ls[4];
          auto stream = [&](const uint32_t (&v)[32], int at, int k0, float2 nm2) {
            if (k0 > tw + 31 || (k0 + 31 <= tw - w.window && k0 >= w.sinks)) {
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[at + i] = 0u;
              return;
            }
            const uint32_t seen = seen_bits(k0);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 e = fma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm2);
              const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
              const float2 pr = make_float2((seen >> i) & 1u ? p0 : 0.0f, (seen >> (i + 1)) & 1u ? p1 : 0.0f);
              ls[(i >> 1) & 3] = add2_rn(ls[(i >> 1) & 3], pr);
              pk[at + i / 2] = pack_bf16x2(pr.x, pr.y);
            }
          };
          tmem_ld_32x32b_x32(tS, va);
          if (!ready) {
            uint32_t own[1];
            tmem_ld_32x32b_x1(tS + wrow, own);
            tmem_loaded(own);
            mr = __uint_as_float(own[0]) * scale_log2;
            ready = true;
          }
          const float2 nm2 = make_float2(-mr, -mr);
          tmem_loaded(va);
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            tmem_ld_32x32b_x32(tS + 64 * c + 32, vb);
#pragma unroll
            for (int q = 0; q < 4; ++q) ls[q] = make_float2(0.0f, 0.0f);
            stream(va, 0, kb + CH * c, nm2);
            tmem_loaded(vb);
            if (c == 0) tmem_ld_32x32b_x32(tS + 64, va);
            stream(vb, 16, kb + CH * c + 32, nm2);
            const float2 l2 = add2_rn(add2_rn(ls[0], ls[1]), add2_rn(ls[2], ls[3]));
            const float lt = l2.x + l2.y;
            const bool over = __any_sync(0xffffffffu, !(lt <= kSumLimit));
            if (c == 0) tmem_loaded(va);
            if (over) break;
            l += lt;
            tmem_st_32x32b_x32(tS + 32 * c, pk);
            c0 = c + 1;
          }
        }
#pragma unroll 1
        for (int c = c0; c < BKV / CH; ++c) {
          const int k0 = kb + CH * c;
          uint32_t pk[CH / 2];
          // what the warp's rows tw .. tw + 31 see of the chunk: nothing; not everything (both warp-uniform)
          const bool dead = k0 > tw + 31 || (k0 + CH - 1 <= tw - w.window && k0 >= w.sinks);
          if (dead) {
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) pk[i] = 0u;
          } else {
            float lt;                                 // the row's sum over the chunk
#pragma unroll 1
            for (bool raise = !ready;; raise = true) {
              if (raise) {
                const RowRef rr = raise_reference<D>(bars, tS + CH * c, tS, tO, c * (CH / 32), mr, l, scale_log2,
                                                     seen_bits(k0), seen_bits(k0 + 32), first, last, abort_flag, err);
                mr = rr.mr;
                l = rr.l;
                ok = rr.ok;
                if (!ok) break;
                ready = __all_sync(0xffffffffu, mr != -INFINITY);
              }
              uint32_t v[CH];
              load_chunk(tS + CH * c, v);
              // A score's whole way to a bf16 probability, 2^(s scale - mr), and into the sum, in one run of
              // independent steps, two keys per f32x2 instruction (with the mask as a branch in the middle the
              // exponentials, sums and roundings ran one after the other: 179 against 156 us for 12,001 tokens).
              float2 ls[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) ls[q] = make_float2(0.0f, 0.0f);
              {                                       // 0 for the keys that the row does not see
                const float nm = mr == -INFINITY ? 0.0f : -mr;
                const float2 nm2 = make_float2(nm, nm);
                const uint32_t seen0 = seen_bits(k0), seen1 = seen_bits(k0 + 32);
#pragma unroll
                for (int i = 0; i < CH; i += 2) {
                  const uint32_t seen = i < 32 ? seen0 : seen1;
                  const float2 e = fma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm2);
                  const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
                  const float2 pr = make_float2((seen >> (i & 31)) & 1u ? p0 : 0.0f, (seen >> ((i + 1) & 31)) & 1u ? p1 : 0.0f);
                  ls[(i >> 1) & 3] = add2_rn(ls[(i >> 1) & 3], pr);
                  pk[i / 2] = pack_bf16x2(pr.x, pr.y);
                }
              }
              const float2 l2 = add2_rn(add2_rn(ls[0], ls[1]), add2_rn(ls[2], ls[3]));
              lt = l2.x + l2.y;
              if (raise || !__any_sync(0xffffffffu, !(lt <= kSumLimit))) break;
            }
            if (!ok) break;
            l += lt;
          }
          tmem_st_32x32b_x32(tS + CH / 2 * c, pk);
        }
        // the previous item's output leaves the accumulator before this item's first P U
        if (!ok || (first && pend && !write_out())) { ok = false; break; }
        // the group's next entry: its number, buffer and first key, and whether its scores are there (a wait costs 90
        // cycles even then; the answer to the test comes while the probabilities are stored)
        uint64_t* const full = &bars->p_full[b];
        last = k;
        do {
          const uint32_t step = x.has1(i) ? 2 : 1;
          ++i;
          k += step;
          b += step;
          b = b >= NSB ? b - NSB : b;
          kb = (i == x.m ? x.a * BKV : kb) - BKV;
        } while (g == 1 && i < x.n && !x.has1(i));
        early = i < x.n && mbar_test(&bars->s_full[g][b], (bits >> b) & 1u);
        tmem_st_wait();
        tc_fence_before();                      // our TMEM reads of S and writes of P precede the next MMA
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      if (!ok) break;
      // the item's output is written during the group's next tile (or after the last item)
      pend = true;
      pl = l;
      pm = mr;
      pb = x.b;
      ph = x.h;
      pqt = qt;
      plast = last;
      kbase = knext;
    }
    if (ok && pend) write_out();
    if (lane == 0) bulk_wait_all();              // stores complete before the CTA exits
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tm, const CUtensorMap& tm_y, WinShape w, int* err, float* lse2, cudaStream_t s) {
  using Cfg = AttnCfg<D>;
  static SmemLimit limit;
  int dev = 0, num_sms = 0;
  cudaError_t e = device_sms(&dev, &num_sms);
  if (e == cudaSuccess) e = limit.raise(attn_window_tc_kernel<D>, dev, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  // pairs of query tiles halve the K/U traffic; single tiles where pairs would leave SMs idle
  const long long pairs = static_cast<long long>((w.n_qtiles + 1) / 2) * w.BH;
  w.per_item = pairs >= num_sms ? 2 : 1;
  w.n_groups = (w.n_qtiles + w.per_item - 1) / w.per_item;
  const long long items = static_cast<long long>(w.n_groups) * w.BH;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  w.n_items = static_cast<int>(items);
  const int grid = static_cast<int>(items < num_sms ? items : num_sms);
  const float scale_log2 = kLog2e / sqrtf(static_cast<float>(D));
  return launch_k(attn_window_tc_kernel<D>, dim3(grid), dim3(THREADS), Cfg::SMEM, s, tm, tm_y, w, scale_log2, err, lse2);
}

}  // namespace

cudaError_t launch_attention_window_tc(const CUtensorMap& tm_qkv, const CUtensorMap& tm_y, int B, int T, int H, int Hkv,
                                       int D, int window, int sinks, int* err, float* lse2, cudaStream_t s) {
  WinShape w = {};
  w.T = T;
  w.H = H;
  w.G = H / Hkv;
  w.window = window < T ? window : T;                // beyond T nothing changes; T < 2^30 keeps the arithmetic in range
  w.sinks = sinks < T ? sinks : T;
  w.BH = B * H;
  w.n_qtiles = (T + BQ - 1) / BQ;
  w.sink_tiles = (w.sinks + BKV - 1) / BKV;
  if (D == 64) return launch_d<64>(tm_qkv, tm_y, w, err, lse2, s);
  if (D == 32) return launch_d<32>(tm_qkv, tm_y, w, err, lse2, s);
  return cudaErrorInvalidValue;
}

}  // namespace gptgb
