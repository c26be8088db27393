// Sliding-window attention with sinks on tcgen05 for sm_103a (prompt form).
//
// Query t sees key s if s <= t and (t - s < W or s < S): the last W keys and the sequence's first S ("sinks").
// y = softmax(Q K^T / sqrt(D)) U over the seen keys, per (batch b, head h); H query heads share Hkv key heads.
// Q, K, U are read straight out of the fused projection's rows [B, T, (H + 2 Hkv) D] through a 3-D TMA map (a
// head is a column offset) and the merged heads y [B, T, H D] are stored by TMA.
//
// The work follows the window: a 128-row query tile reads the key tiles from its first row's window start to its
// diagonal, and the tiles that hold sinks, so work and traffic grow with T (W + S), not T^2 / 2. The kernel is
// bound by issuing the softmax's instructions (one exponential and about three more per score), not by the tensor
// core, so a warp leaves out every 64-key half tile of which its 32 rows see nothing (beyond the diagonal, before
// the window, after the sinks) and masks only the half tiles that a border crosses.
//
// Pipeline (one persistent CTA per SM, 352 threads): as in the full causal kernel, a work item is one (b, h) and a
// PAIR of consecutive query tiles that share one stream of 128-key K/U tiles through a four-stage TMA ring; two
// softmax groups of four warps (thread = query row = TMEM lane) own one query tile each and run out of phase.
// Where the pairs would leave SMs without work an item is one query tile. Items are dealt statically, the long
// ones first, forwards and backwards in turn (item r of CTA c: r grid + c, or r grid + grid - 1 - c for odd r):
// all items but a sequence's first few cost the same, and no work counter has to be cleared before the launch.
//
// The score tiles of both groups form ONE sequence: list entry i of the item, group 0's tile then group 1's,
// leaving out what a group does not see. Score number k goes to TMEM buffer k % 3. One warp issues
// S(k + 3) = Q K^T into buffer k % 3 once the P U of number k has completed; another waits for the probabilities
// P(k) (written by the owning group over the first 64 columns of the buffer as bf16 pairs, released in two
// 64-key halves) and issues O_g += P(k) U_j with the A operand in tensor memory.
//
// Softmax: per row one running reference m and sum. The reference starts as the score of key 0 where every row of
// the tile sees it, else as the exact maximum of the first half tile in which the row sees a key; it is raised only
// when a half tile's sum passes 2^16 and the maximum grew by more than 2^8. Sums are fp32; P is rounded to bf16 for
// the second product (the type the tensor core multiplies), which costs at most 2^-8 of sum a |u|.
//
// Tensor memory (512 columns): score buffers at 0, 128, 256; O_g at 384 + 64 g.
// Warps: 0 TMA producer; 1 TMEM allocator and P U issuer; 2-5 softmax group 0; 6-9 group 1; 10 score issuer.
#include "common.cuh"
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
constexpr int NS = 4;                   // K/U ring depth; the MMA warp's look-ahead needs at least 4
constexpr int NSB = 3;                  // score buffers
constexpr uint32_t kColO = 128 * NSB;   // O_g at kColO + 64 g

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

struct __align__(8) AttnBars {
  uint64_t q_empty[2];      // every S of the item that used Q buffer k has been computed
  uint64_t kv_full[NS];     // ring stage holds K_j, U_j (and, for an item's first tile, its query tiles)
  uint64_t kv_empty[NS];
  uint64_t s_full[2][NSB];  // score buffer b holds a new score tile of group g (that group's uses of b, in order)
  uint64_t p_full[NSB][2];  // score buffer b holds that tile's probabilities of keys [64 h, 64 h + 64) (4 warps)
  uint64_t pv_done[NSB];    // the P U that read buffer b has completed (the buffer may take new scores)
  uint64_t o_full[2][3];    // group g's P U number i (its own count) has completed: barrier i % 3
  uint64_t drain[2];        // the issuing warps' own MMAs have completed (exit)
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(AttnBars) <= 512, "barrier block");

// The start-address field is the low 14 bits of a descriptor (address >> 4), and
// every operand here lies below 256 KB, so advancing an operand by `bytes` is a
// plain add of bytes >> 4 to its base descriptor.
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

template <int D>
__device__ __forceinline__ void issue_s(uint32_t tS, uint64_t q_desc, uint64_t k_desc) {
  constexpr uint32_t idesc = idesc_bf16_f32(BQ, BKV, false);
#pragma unroll
  for (int k = 0; k < D / 16; ++k)          // K-major: a K step of 16 bf16 is 32 bytes along the swizzled row
    tc_mma_bf16_warp(tS, desc_add(q_desc, k * 32), desc_add(k_desc, k * 32), idesc, k > 0 ? 1u : 0u);
}

// O += P_h U_h for keys [64 h, 64 h + 64) of a tile: P lies in TMEM over the first 64
// columns of its score buffer (two bf16 per column, row = lane; keys 64 h.. at column 32 h),
// U is MN-major in shared memory (D contiguous per key).
template <int D>
__device__ __forceinline__ void issue_pv_half(uint32_t tO, uint32_t tP, uint64_t u_desc, int h, bool accumulate) {
  using Cfg = AttnCfg<D>;
  constexpr uint32_t idesc = idesc_bf16_f32(BQ, D, true);     // U is MN-major (D contiguous)
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)            // a K step of 16 keys: 8 TMEM columns of P, 16 rows of U
    tc_mma_bf16_ts_warp(tO, tP + 32 * h + 8 * kk, desc_add(u_desc, (64 * h + 16 * kk) * Cfg::ROWB), idesc,
                        (accumulate || kk > 0) ? 1u : 0u);
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

// One item: query tiles qt0 (group 0) and, if `two`, qt0 + 1 (group 1), and the list of key tiles they share:
// entries [0, a) are the sink tiles before the window, entries a.. the tiles from j0 (the window start of qt0's
// first row) to the last diagonal. Group 0 takes entries [0, n0); group 1 takes all but entry a where `skip`
// (its own window starts one tile later and that tile holds no sink).
struct Item {
  int b, h, qt0, a, j0, n0, n;
  bool two, skip;
  __device__ __forceinline__ int tile(int i) const { return i < a ? i : j0 + (i - a); }
  __device__ __forceinline__ bool has1(int i) const { return two && !(skip && i == a); }
  __device__ __forceinline__ int first1() const { return skip && a == 0 ? 1 : 0; }
  // group 1's entries before i
  __device__ __forceinline__ int count1(int i) const { return two ? i - (skip && i > a ? 1 : 0) : 0; }
  // position of (entry i, group g) in the item's score sequence, and the sequence's length
  __device__ __forceinline__ int number(int i, int g) const { return (g ? min(i + 1, n0) : i) + count1(i); }
  __device__ __forceinline__ int total() const { return n0 + count1(n); }
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
  x.j0 = first > 0 ? first / BKV : 0;
  x.a = min(w.sink_tiles, x.j0);
  const int j1 = first + BQ > 0 ? (first + BQ) / BKV : 0;
  x.skip = x.two && j1 > x.j0 && x.j0 >= w.sink_tiles;
  x.n0 = x.a + (x.qt0 - x.j0) + 1;
  x.n = x.n0 + (x.two ? 1 : 0);
  return x;
}

// Walks the score-tile sequence of one CTA for an issuing warp: item r, entry i, group g, with the ring position
// of the item's entry 0.
struct Cursor {
  Item w;
  int r, i, g;
  uint32_t kvb;
  bool valid;
  __device__ __forceinline__ void load(const WinShape& s) {
    const int item = item_of(s, r);
    valid = item >= 0;
    if (valid) w = decode_item(s, item);
  }
  __device__ __forceinline__ void advance(const WinShape& s) {
    if (g == 0 && w.has1(i)) { g = 1; return; }
    if (++i < w.n) { g = (i < w.n0) ? 0 : 1; return; }
    kvb += w.n;
    ++r;
    i = 0;
    g = 0;
    load(s);
  }
  __device__ __forceinline__ uint32_t pos() const { return kvb + i; }
  __device__ __forceinline__ bool first_of_group() const { return g == 0 ? i == 0 : i == w.first1(); }
  // the element is the last MMA reader of its ring position / the item's last score tile
  __device__ __forceinline__ bool last_of_pos() const { return g == 1 || !w.has1(i); }
  __device__ __forceinline__ bool last_of_item() const { return i == w.n - 1 && last_of_pos(); }
};

// 16-byte unit u of row r of a staging box (rows of ROWB bytes) in the TMA swizzle of that width.
template <int ROWB>
__device__ __forceinline__ int swz_unit(int r, int u) {
  return (ROWB == 128) ? (u ^ (r & 7)) : (u ^ ((r >> 1) & 3));
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_empty[i], 1);
      for (int k = 0; k < 3; ++k) mbar_init(&bars->o_full[i][k], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_empty[i], 2);                // K read by the score warp, U by the P U warp
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&bars->s_full[0][i], 1);
      mbar_init(&bars->s_full[1][i], 1);
      mbar_init(&bars->p_full[i][0], 4);
      mbar_init(&bars->p_full[i][1], 4);
      mbar_init(&bars->pv_done[i], 1);
    }
    mbar_init(&bars->drain[0], 1);
    mbar_init(&bars->drain[1], 1);
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
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t issued = 0, last_par = 0;
      uint32_t kv_it = 0;                            // K/U tiles loaded so far (ring position)
      bool ok = true;
      for (int r = 0; ok; ++r) {
        const int item = item_of(w, r);
        if (item < 0) break;
        const Item x = decode_item(w, item);
        const int kh = x.h / w.G;                    // key head
        const int qb = r & 1;                        // Q buffer of this item; its previous user was item r - 2
        if (r >= 2 && !mbar_wait(&bars->q_empty[qb], static_cast<uint32_t>((r >> 1) - 1) & 1u, abort_flag, err)) break;
        for (int i = 0; i < x.n; ++i, ++kv_it) {
          const int s = kv_it % NS;
          const uint32_t use_par = (kv_it / NS) & 1u;
          if (!mbar_wait(&bars->kv_empty[s], use_par ^ 1u, abort_flag, err)) { ok = false; break; }
          // the item's query tiles complete on the barrier of its first K/U tile
          const int nq = (i == 0) ? (x.two ? 2 : 1) : 0;
          const int row = x.tile(i) * BKV;
          mbar_arrive_expect_tx(&bars->kv_full[s], (2 + nq) * Cfg::TILE);
          if (nq > 0) tma_load_3d(sQ + (2 * qb) * Cfg::TILE, &tm, &bars->kv_full[s], x.h * D, x.qt0 * BQ, x.b);
          if (nq > 1) tma_load_3d(sQ + (2 * qb + 1) * Cfg::TILE, &tm, &bars->kv_full[s], x.h * D, (x.qt0 + 1) * BQ, x.b);
          tma_load_3d(sK + s * Cfg::TILE, &tm, &bars->kv_full[s], kcol + kh * D, row, x.b);
          tma_load_3d(sU + s * Cfg::TILE, &tm, &bars->kv_full[s], ucol + kh * D, row, x.b);
          issued |= 1u << s;
          last_par = (last_par & ~(1u << s)) | (use_par << s);
        }
      }
      // never leave with copies in flight into this CTA's shared memory
      for (int s = 0; s < NS; ++s)
        if (issued & (1u << s)) mbar_wait_drain(&bars->kv_full[s], (last_par >> s) & 1u);
    }
  } else if (warp == 1 || warp == 10) {
    // ------------------------------------------------ MMA issuers (whole warp; one elected lane issues)
    // Two warps on different sub-partitions share the issue work, each walking the same
    // sequence of score numbers: warp 1 waits for P(k) and issues O_g += P(k) U_j; warp 10
    // issues S(k) = Q K_j^T into buffer k % 3 once the P U of number k - 3 (which read that
    // buffer) has completed. A ring stage is released after both the last S reading its K and
    // the last P U reading its U; S(k) lies at most three ring positions past the oldest
    // unreleased stage, so four stages never wait on each other.
    {
      const bool pv_warp = warp == 1;
      // base descriptors: Q and K K-major (8-row groups ROWB*8 apart), U MN-major (K-direction
      // 8-row groups ROWB*8 apart)
      const uint64_t dq0 = smem_desc(smem_u32(sQ), 16, 8 * Cfg::ROWB, Cfg::SWZ);
      const uint64_t dk0 = smem_desc(smem_u32(sK), 16, 8 * Cfg::ROWB, Cfg::SWZ);
      const uint64_t du0 = smem_desc(smem_u32(sU), Cfg::TILE, 8 * Cfg::ROWB, Cfg::SWZ);
      Cursor c;
      c.r = 0;
      c.i = 0;
      c.g = 0;
      c.kvb = 0;
      c.load(w);
      uint32_t b = 0;                                // buffer of number k (k % 3)
      uint32_t bits = 0;                             // phase per buffer of the barrier this warp waits on
      if (pv_warp) {
        uint32_t oi0 = 0, oi1 = 0;                   // next o_full barrier per group (P U count % 3)
        while (c.valid) {
          const uint32_t st = c.pos() % NS;
          const uint32_t tOg = tmem_base + kColO + 64 * c.g;
          // keys [0, 64) as soon as the group releases them, then keys [64, 128)
          if (!mbar_wait_warp(&bars->p_full[b][0], (bits >> b) & 1u, abort_flag, err)) break;
          tc_fence_after();
          issue_pv_half<D>(tOg, tmem_base + 128 * b, desc_add(du0, st * Cfg::TILE), 0, !c.first_of_group());
          if (!mbar_wait_warp(&bars->p_full[b][1], (bits >> b) & 1u, abort_flag, err)) break;
          bits ^= 1u << b;
          tc_fence_after();
          issue_pv_half<D>(tOg, tmem_base + 128 * b, desc_add(du0, st * Cfg::TILE), 1, true);
          tc_commit_warp(&bars->pv_done[b]);
          if (c.g) {
            tc_commit_warp(&bars->o_full[1][oi1]);
            oi1 = oi1 == 2 ? 0 : oi1 + 1;
          } else {
            tc_commit_warp(&bars->o_full[0][oi0]);
            oi0 = oi0 == 2 ? 0 : oi0 + 1;
          }
          if (c.last_of_pos()) tc_commit_warp(&bars->kv_empty[st]);   // U_j is consumed
          c.advance(w);
          b = b == NSB - 1 ? 0 : b + 1;
        }
      } else {
        uint32_t n = 0;                              // score number
        uint32_t waited = 0xffffffffu;               // ring position whose K/U (and Q) was last waited for
        while (c.valid) {
          if (n >= NSB) {                            // the P U that read this buffer has completed
            if (!mbar_wait_warp(&bars->pv_done[b], (bits >> b) & 1u, abort_flag, err)) break;
            bits ^= 1u << b;
          }
          const uint32_t pos = c.pos();
          const uint32_t st = pos % NS;
          if (pos != waited) {
            if (!mbar_wait_warp(&bars->kv_full[st], (pos / NS) & 1u, abort_flag, err)) break;
            waited = pos;
          }
          tc_fence_after();
          const uint32_t qb = static_cast<uint32_t>(c.r) & 1u;
          issue_s<D>(tmem_base + 128 * b, desc_add(dq0, (2 * qb + c.g) * Cfg::TILE), desc_add(dk0, st * Cfg::TILE));
          tc_commit_warp(c.g ? &bars->s_full[1][b] : &bars->s_full[0][b]);
          if (c.last_of_pos()) tc_commit_warp(&bars->kv_empty[st]);   // K_j is consumed
          if (c.last_of_item()) tc_commit_warp(&bars->q_empty[qb]);   // every S of the item has read its Q
          c.advance(w);
          b = b == NSB - 1 ? 0 : b + 1;
          ++n;
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
    uint32_t tiles = 0;                               // this group's tiles so far (its P U numbering)
    uint32_t used0 = 0, used1 = 0, used2 = 0;         // this group's score tiles so far in buffers 0, 1, 2
    bool ok = true;
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    // An item's output is written during the group's next tile, just before that tile's first
    // P U (which overwrites the accumulator) is released: by then the item's last P U has
    // completed, so the group never idles on it.
    bool pend = false;
    float pl = 0.0f;                                  // the pending item's running sum
    float pm = 0.0f;                                  // and its running max (log2 units)
    int pb = 0, ph = 0, pqt = 0;                      // its batch row, head and query tile
    uint32_t plast = 0;                               // its last tile (this group's numbering)
    auto write_out = [&]() -> bool {
      if (!mbar_wait_warp(&bars->o_full[g][plast % 3], (plast / 3) & 1u, abort_flag, err)) return false;
      tc_fence_after();
      const float inv = 1.0f / pl;
      uint32_t ov[D];
      if constexpr (D == 64) {
        uint32_t (&o64)[64] = *reinterpret_cast<uint32_t (*)[64]>(ov);
        tmem_ld_32x32b_x64(tO, o64);
      } else {
        uint32_t (&o32)[32] = *reinterpret_cast<uint32_t (*)[32]>(ov);
        tmem_ld_32x32b_x32(tO, o32);
      }
      tmem_ld_wait();
      tc_fence_before();                        // the accumulator may be overwritten after this
      if (lane == 0) bulk_wait_read_all();      // this warp's previous store has read its staging box
      __syncwarp();
      uint8_t* row = stg + lane * Cfg::ROWB;
#pragma unroll
      for (int u = 0; u < Cfg::ROWB / 16; ++u) {
        uint4 v;
        v.x = pack_bf16x2(__uint_as_float(ov[8 * u + 0]) * inv, __uint_as_float(ov[8 * u + 1]) * inv);
        v.y = pack_bf16x2(__uint_as_float(ov[8 * u + 2]) * inv, __uint_as_float(ov[8 * u + 3]) * inv);
        v.z = pack_bf16x2(__uint_as_float(ov[8 * u + 4]) * inv, __uint_as_float(ov[8 * u + 5]) * inv);
        v.w = pack_bf16x2(__uint_as_float(ov[8 * u + 6]) * inv, __uint_as_float(ov[8 * u + 7]) * inv);
        *reinterpret_cast<uint4*>(row + (swz_unit<Cfg::ROWB>(lane, u) << 4)) = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&tm_y, stg, ph * D, pqt * BQ + sub * 32, pb);
        bulk_commit();
      }
      if (lse2 != nullptr) {                      // the row's base-2 log-sum-exp of the scaled scores
        const int t = pqt * BQ + r_row;
        if (t < T) lse2[(static_cast<size_t>(pb) * H + ph) * T + t] = pm + log2f(pl);
      }
      pend = false;
      return true;
    };
    const int wrow = sub * 32;                        // first row of this warp within the tile
    for (int r = 0; ok; ++r) {
      const int item = item_of(w, r);
      if (item < 0) break;
      const Item x = decode_item(w, item);
      const uint32_t knext = kbase + x.total();
      if (g == 1 && !x.two) { kbase = knext; continue; }   // group 1 without a query tile
      const int qt = x.qt0 + g;
      const int t = qt * BQ + r_row;                  // query position
      const int tw = qt * BQ + wrow;                  // the warp's first query
      const int i0 = g == 0 ? 0 : x.first1(), i1 = g == 0 ? x.n0 : x.n;
      float mr = -INFINITY;                           // running (lazily raised) reference, log2 units
      float l = 0.0f;                                 // running sum of 2^(s - mr)
      for (int i = i0; i < i1 && ok; ++i) {
        if (g == 1 && !x.has1(i)) continue;
        const bool first = i == i0;
        // this tile's score number and buffer
        const uint32_t k = kbase + x.number(i, g);
        const uint32_t b = k % NSB;
        const uint32_t use = b == 0 ? used0++ : (b == 1 ? used1++ : used2++);
        if (!mbar_wait_warp(&bars->s_full[g][b], use & 1u, abort_flag, err)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tS = tmem_base + 128 * b + lane_off;
        const int kb = x.tile(i) * BKV;               // first key of the tile
        // bit n set: this row sees key kb_half + n
        auto seen_bits = [&](int kb_half) -> uint64_t {
          const int hi = t - kb_half;                 // last key of the row
          const int lo = hi - w.window + 1;           // first key of its window
          const uint64_t to_hi = hi < 0 ? 0ull : (hi >= 63 ? ~0ull : (2ull << hi) - 1ull);
          const uint64_t from_lo = lo <= 0 ? ~0ull : (lo >= 64 ? 0ull : ~0ull << lo);
          const int ns = w.sinks - kb_half;
          const uint64_t sinks = ns <= 0 ? 0ull : (ns >= 64 ? ~0ull : (1ull << ns) - 1ull);
          return to_hi & (from_lo | sinks);
        };
        // pv = 2^(s*scale - mr) in place of the scores, two keys per f32x2 instruction; 0 for the keys that the
        // row does not see (masked: some row of the warp misses some key of the half); returns the sum
        auto probs = [&](uint32_t (&v)[64], bool masked, uint64_t seen) -> float {
          const float nm = mr == -INFINITY ? 0.0f : -mr;      // no key seen yet: every probability is masked to 0
          const float2 nm2 = make_float2(nm, nm);
          if (masked) {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const float2 e = fma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm2);
              const uint32_t word = i < 32 ? static_cast<uint32_t>(seen) : static_cast<uint32_t>(seen >> 32);
              v[i] = (word >> (i & 31)) & 1u ? __float_as_uint(ex2_approx(e.x)) : 0u;
              v[i + 1] = (word >> ((i + 1) & 31)) & 1u ? __float_as_uint(ex2_approx(e.y)) : 0u;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const float2 e = fma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm2);
              v[i] = __float_as_uint(ex2_approx(e.x));
              v[i + 1] = __float_as_uint(ex2_approx(e.y));
            }
          }
          float2 ls[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) ls[q] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < 64; i += 2)
            ls[(i >> 1) & 3] = add2_rn(ls[(i >> 1) & 3], make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
          const float2 l2 = add2_rn(add2_rn(ls[0], ls[1]), add2_rn(ls[2], ls[3]));
          return l2.x + l2.y;
        };
        // exact maximum of the seen keys of one half, eight independent chains (-inf: none)
        auto half_max = [&](const uint32_t (&v)[64], uint64_t seen) -> float {
          float mx8[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) mx8[q] = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float lo = (static_cast<uint32_t>(seen) >> i) & 1u ? __uint_as_float(v[i]) : -INFINITY;
            const float hi = (static_cast<uint32_t>(seen >> 32) >> i) & 1u ? __uint_as_float(v[32 + i]) : -INFINITY;
            mx8[i & 7] = fmax3(mx8[i & 7], lo, hi);
          }
          return fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        };
        // The two 64-key halves in turn. A half's probabilities are final once its sum is checked
        // (and, rarely, recomputed against a raised max); they are then stored as bf16 pairs over
        // columns [32 hf, 32 hf + 32) of the buffer, whose scores are already in registers.
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t tSh = tS + 64 * hf;
          const int kbh = kb + 64 * hf;
          // what the warp's rows tw .. tw + 31 see of keys kbh .. kbh + 63 (warp-uniform)
          const bool dead = kbh > tw + 31 || (kbh + 63 <= tw - w.window && kbh >= w.sinks);
          uint32_t pk[32];
          if (!dead) {
          const bool masked = kbh + 63 > tw || (kbh <= tw + 31 - w.window && kbh + 64 > w.sinks);
          const uint64_t seen = masked ? seen_bits(kbh) : ~0ull;
          uint32_t sv[64];
          tmem_ld_32x32b_x64(tSh, sv);
          tmem_ld_wait();
          if (first && hf == 0 && kb == 0 && (w.sinks > 0 || tw + 31 < w.window)) {
            mr = __uint_as_float(sv[0]) * scale_log2;         // key 0 is seen by every row of the warp
          } else if (__any_sync(0xffffffffu, mr == -INFINITY)) {
            const float m0 = half_max(sv, seen) * scale_log2;
            if (mr == -INFINITY) mr = m0;
          }
          float lt = probs(sv, masked, seen);
          if (__any_sync(0xffffffffu, !(lt <= kSumLimit))) {
            // rare: this half's exact maximum, a rescale of the running output and sum (and of
            // the first half's stored probabilities) where the max grew by more than 2^8, and
            // the half again against the new reference
            tmem_ld_32x32b_x64(tSh, sv);
            tmem_ld_wait();
            const float m_new = fmaxf(mr, half_max(sv, seen) * scale_log2);
            const bool need = m_new > mr + kRescaleLog2;
            if (__any_sync(0xffffffffu, need)) {
              const float alpha = need ? ex2_approx(mr - m_new) : 1.0f;
              if (need) mr = m_new;
              l *= alpha;
              if (!first) {
                // every earlier P U of the group has completed (its own numbering, barrier i % 3)
                const uint32_t last = tiles - 1;
                if (!mbar_wait_warp(&bars->o_full[g][last % 3], (last / 3) & 1u, abort_flag, err)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t o[32];
                  tmem_ld_32x32b_x32(tO + c * 32, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                  tmem_st_32x32b_x32(tO + c * 32, o);
                }
              }
              if (hf == 1) {                          // the first half's probabilities, already stored
                tmem_st_wait();
                uint32_t q[32];
                tmem_ld_32x32b_x32(tS, q);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float2 f = unpack_bf16x2(q[i]);
                  q[i] = pack_bf16x2(f.x * alpha, f.y * alpha);
                }
                tmem_st_32x32b_x32(tS, q);
              }
              tmem_st_wait();
            }
            tmem_ld_32x32b_x64(tSh, sv);
            tmem_ld_wait();
            lt = probs(sv, masked, seen);
          }
          l += lt;
#pragma unroll
          for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = 0u;
          }
          if (hf == 1) {
            // the previous item's output leaves the accumulator before this item's first P U
            if (first && pend && !write_out()) { ok = false; break; }
            tmem_st_wait();                           // keys [0, 64) are final: hand them to the P U warp
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[b][0]);
          }
          tmem_st_32x32b_x32(tS + 32 * hf, pk);
        }
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();                      // our TMEM reads of S and writes of P precede the next MMA
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[b][1]);
        ++tiles;
      }
      if (!ok) break;
      // the item's output is written during the group's next tile (or after the last item)
      pend = true;
      pl = l;
      pm = mr;
      pb = x.b;
      ph = x.h;
      pqt = qt;
      plast = tiles - 1;
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
  int dev = 0, num_sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_window_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
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
