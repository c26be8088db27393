// Derivative of sliding-window attention with sinks on tcgen05 for sm_103a.
//
// With A recomputed from the forward's row log-sum-exp and Dsum[t] = sum_d dY[t,d] Y[t,d], over the seen pairs
// (s <= t and (t - s < W or s < S)):
//   dA = dY U^T,  dS = A * (dA - Dsum),  dQ = dS K / sqrt(D),  dK = dS^T Q / sqrt(D),  dU = A^T dY,
// where dK and dU of a key head sum over the G query heads that share it.
//
// A work item is one (b, key head), one 128-key tile j and a segment of the query tiles that see it (from j to the
// one whose window ends there; to the sequence's end where the tile holds a sink), head after head of the group, so
// that a group's sum stays in the accumulators. Items are dealt statically, the sink tiles first, forwards and
// backwards in turn, and no work counter has to be cleared.
// Each query tile is taken in two halves g of 64 queries with a tensor-memory buffer each (key = TMEM lane); K_j and
// U_j sit in tensor memory (columns [448, 448 + D)), copied there once per item by the output warps:
//   S^T_g  = K_j Q_{i,g}^T     M=128 keys, N=64 queries, K=D    columns [128 g, 128 g + 64)
//   dP^T_g = U_j dY_{i,g}^T    M=128, N=64, K=D                 columns [128 g + 64, 128 g + 128)
// Four derivative warps per half (one thread per key) turn it into P^T = 2^(S^T log2(e)/sqrt(D) - lse2[q]) and
// dS^T = P^T (dP^T - Dsum[q]), rounded to bf16 for the products below (the type the tensor core multiplies: 2^-8
// of each term) while the tensor core and the other four work on the other half (with one set of four warps
// for both halves a step took 1.8 us, now 1.5: each scheduler had one warp, whose waits nothing covered); a warp writes
// plain zeros for a half of which its 32 keys are not seen. dS^T also goes to shared memory (the MN-major A operand of dQ). Then
//   dU_j += P^T_g dY_{i,g}     A from tensor memory, B = dY rows read MN-major    columns [256, 256 + D)
//   dK_j += dS^T_g Q_{i,g}     A from tensor memory, B = Q rows read MN-major     columns [320, 320 + D)
//   dQ_i  = dS_i K_j           after both halves: A = dS (shared memory), B = K_j  columns [384, 384 + D)
// Four output warps add each dQ_i tile into an fp32 [B][T][H D] buffer with TMA reduce-adds (the order of a query
// tile's few additions varies, below a bf16 step of the result) and, at the end of an item, store dK_j / sqrt(D)
// and dU_j by TMA. Rows of -lse2 and -Dsum are laid out by a first kernel; a last one rounds dQ to bf16 and sums segments.
//
// Bound by shared memory: a step (128 keys x 128 queries) moves about 270 KB through it (operand reads of five products,
// the dS tile written and read, copies in, dQ out), 2,100 of its 2,850 cycles at 128 bytes each; the derivative's chain
// on one half takes about 1,270. A deeper ring of query tiles, or the scores read 16 queries ahead, changed nothing.
// Measured (with the forward, calls back to back): 8,192 tokens, 16 heads on 4, D 64, W 1024: 183 us, 620 TFLOP/s; with
// 12 heads, 8 x 1,000 tokens, W 250: 78 us.
//
// Error of dqkv against 64 bits, relative to its norm: 2.3e-3 to 2.7e-3 on normal inputs, where rounding the result
// alone is 1.7e-3; P and dS rounded to bf16 bring 2.3e-3, the rest is Dsum from the bf16 rows of y.
// Warps (448 threads, one persistent CTA per SM): 0 producer; 1 TMEM allocator and MMA issuer; 2-5 and 6-9 softmax
// derivative of half 0 and 1 (thread = key row); 10-13 output.
#include "attn_window.cuh"
#include "kernels.h"
#include "launch.h"

#include <math.h>

namespace gptgb {

namespace {

constexpr int BT = 128;                 // rows per key or query tile
constexpr int HQ = 64;                  // queries per half tile
constexpr int THREADS = 448;
constexpr int TMEM_COLS = 512;
constexpr int NQ = 3;                   // query-tile ring stages
constexpr int SR = 4;                   // items announced ahead
constexpr int kConsumers = 13;          // warps that read each announced item: MMA, 8 derivative, 4 output
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kColDU = 256, kColDK = 320, kColDQ = 384;   // half g: S^T at 128 g, dP^T at 128 g + 64
constexpr uint32_t kColK = 448;         // K_j (bf16 pairs, D / 2 columns), then U_j: the item's A operands

template <int D>
struct BwdCfg {
  static constexpr int ROWB = D * 2;                              // bytes per row of a Q/K/U/dY tile
  static constexpr uint32_t SWZ = (ROWB == 128) ? SWZ_128B : SWZ_64B;
  static constexpr int TILE = BT * ROWB;
  static constexpr int OFF_K = 0;                                   // [2] item buffers
  static constexpr int OFF_U = 2 * TILE;                            // one: read once, into tensor memory
  static constexpr int OFF_Q = 3 * TILE;                            // [NQ]
  static constexpr int OFF_DY = OFF_Q + NQ * TILE;                  // [NQ]
  static constexpr int OFF_LD = OFF_DY + NQ * TILE;                 // [2][64 pairs] {-lse2 x2, -Dsum x2}
  static constexpr int OFF_DS = (OFF_LD + 2 * BT * 8 + 1023) / 1024 * 1024;
  static constexpr int DS_BUF = 2 * BT * 128;                       // one tile's dS: 2 atoms x 128 keys x 128 B
  static constexpr int OFF_STG = OFF_DS + 2 * DS_BUF;               // 4 output warps x one box of 4 KB
  static constexpr int OFF_BAR = OFF_STG + 4 * 4096;
  static constexpr int SMEM = OFF_BAR + 512;
  static_assert(D == 32 || D == 64, "head width");
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct __align__(16) BwdBars {
  uint64_t kv_full[2], kv_empty[2];     // K_j (buffer r % 2) and U_j of an item
  uint64_t q_full[NQ], q_empty[NQ];     // Q_i, dY_i of a query tile (and its rows' -lse2 and -Dsum: two arrivals)
  uint64_t s_full[2];                   // S^T and dP^T of half g are in tensor memory
  uint64_t p_full[2];                   // the derivative warps wrote half g (4 warps)
  uint64_t dq_full;                     // the current tile's dQ product has completed
  uint64_t dq_free;                     // the output warps read it out of tensor memory (4 warps)
  uint64_t acc_full;                    // the item's dK and dU are complete
  uint64_t acc_free;                    // the output warps read them (4 warps)
  uint64_t kvt_full;                    // the item's K_j and U_j are in tensor memory (4 warps)
  uint64_t kvt_free;                    // the last product reading them has completed
  uint64_t item_full[SR];               // slot r % SR holds the CTA's r-th item (from the producer)
  uint64_t item_empty[SR];              // every other warp has read it
  uint64_t drain;
  __align__(16) int item[SR][8];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(BwdBars) <= 512, "barrier block");


// What a launch computes, and how it is cut. Items: one (b, key head), one key tile j, and a segment of that tile's
// steps. The tiles with sinks see every later query tile and would keep one CTA busy long after the others (and a few
// heads with long windows would leave most CTAs idle), so the tiles of each of the two classes are cut into nseg
// segments; where nseg > 1 a segment's dK and dU go to fp32 slabs that the last kernel sums in order.
struct WinBwdShape {
  int T, H, Hkv, G, window, sinks;   // window >= 1
  int n_qt, sink_tiles, BK;          // BK = B Hkv
  int nseg_s, nseg_w;                // segments per tile with sinks, per other tile
  int n_sink_items, n_items;
};

// Step e0 <= e < e1 is query tile j + e % cnt of query head kh G + e / cnt.
struct Item {
  int b, kh, j, cnt, e0, steps, slot;   // slot: of the fp32 slab, -1: dK and dU are complete
  __device__ __forceinline__ int first_tile() const { return j + e0 % cnt; }
  __device__ __forceinline__ int first_head(int G) const { return kh * G + e0 / cnt; }
};

__host__ __device__ __forceinline__ int tile_count(const WinBwdShape& w, int j) {   // query tiles that see key tile j
  const long long end = j < w.sink_tiles ? w.n_qt : (static_cast<long long>(j) * BT + BT - 1 + w.window - 1) / BT + 1;
  return (end < w.n_qt ? static_cast<int>(end) : w.n_qt) - j;
}
// First step of segment `seg` of nseg.
__device__ __forceinline__ int seg_start(int steps, int seg, int nseg) {
  return static_cast<int>(static_cast<long long>(steps) * seg / nseg);
}

__device__ __forceinline__ Item decode_item(const WinBwdShape& w, int item) {
  Item x;
  const bool sink = item < w.n_sink_items;
  const int nseg = sink ? w.nseg_s : w.nseg_w;
  const int k = sink ? item : item - w.n_sink_items;
  const int q = k / w.BK, bk = k - q * w.BK, seg = q % nseg;
  x.j = q / nseg + (sink ? 0 : w.sink_tiles);
  x.b = bk / w.Hkv;
  x.kh = bk - x.b * w.Hkv;
  x.cnt = tile_count(w, x.j);
  const int steps = w.G * x.cnt;
  x.e0 = seg_start(steps, seg, nseg);
  x.steps = seg_start(steps, seg + 1, nseg) - x.e0;
  x.slot = nseg == 1 ? -1 : item - (w.nseg_s == 1 ? w.n_sink_items : 0);
  return x;
}

// The CTA's items in turn, for its producer: forwards and backwards over the grid, empty segments left out.
struct Items {
  int round = -1;
  __device__ __forceinline__ bool next(const WinBwdShape& w, Item& x) {
    const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    while (true) {
      ++round;
      const long long i = static_cast<long long>(round) * g + ((round & 1) ? g - 1 - c : c);
      if (i >= w.n_items) return false;
      x = decode_item(w, static_cast<int>(i));
      if (x.steps > 0) return true;
    }
  }
};

// What the other warps need of an item. The producer decodes it (a chain of divisions that each warp's first step of
// the item would wait for) and announces it through a ring of SR slots; steps 0 ends the list.
struct Step0 {
  int b, kh, j, end, i, head, steps, slot;   // query tiles [j, end); the first step's tile and head
};
__device__ __forceinline__ bool next_item(BwdBars* bars, int r, Step0& x, volatile int* abort_flag, int* err, int lane) {
  const int slot = r % SR;
  if (!mbar_wait_warp(&bars->item_full[slot], static_cast<uint32_t>(r / SR) & 1u, abort_flag, err)) return false;
  const int4* v = reinterpret_cast<const int4*>(bars->item[slot]);
  const int4 p = v[0], q = v[1];
  x = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
  __syncwarp();
  if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
  return x.steps > 0;
}

// One half tile of the softmax derivative for this thread's key row: reads S^T and dP^T (64 queries
// each) from columns [col, col + 64) and [col + 64, col + 128), writes P^T and dS^T as bf16 pairs
// over [col, col + 32) and [col + 64, col + 96), and dS^T into the row's 128-byte slot `ds_row` of a
// 64-query shared-memory atom, 32 queries at a time. ld: the half's 32 query pairs {-lse2, -lse2, -Dsum,
// -Dsum}. kMasked: keep only the queries ql (counted within the half) whose bit ql of `keep` is set.
template <bool kMasked>
__device__ __forceinline__ void derivative_half(uint32_t col, const float4* __restrict__ ld, float sl2, uint64_t keep,
                                                uint8_t* ds_row, int kr) {
  const float2 sl2v = make_float2(sl2, sl2);
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {                      // 32 queries at a time
    const uint32_t word = c == 0 ? static_cast<uint32_t>(keep) : static_cast<uint32_t>(keep >> 32);
    uint32_t sv[32], dv[32];
    tmem_ld_32x32b_x32(col + 32 * c, sv);
    tmem_ld_32x32b_x32(col + 64 + 32 * c, dv);
    tmem_ld_wait();
    uint32_t pp[16], pd[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float4 L = ld[16 * c + e];
      const float2 x = fma2_rn(make_float2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), sl2v,
                               make_float2(L.x, L.y));
      float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
      if (kMasked) {
        p0 = ((word >> (2 * e)) & 1u) ? p0 : 0.0f;
        p1 = ((word >> (2 * e + 1)) & 1u) ? p1 : 0.0f;
      }
      const float2 d = mul2_rn(make_float2(p0, p1),
                               add2_rn(make_float2(__uint_as_float(dv[2 * e]), __uint_as_float(dv[2 * e + 1])),
                                       make_float2(L.z, L.w)));
      pp[e] = pack_bf16x2(p0, p1);
      pd[e] = pack_bf16x2(d.x, d.y);
    }
    // P^T and dS^T over columns [16 c, 16 c + 16) of their halves (already read)
    tmem_st_32x32b_x16(col + 16 * c, pp);
    tmem_st_32x32b_x16(col + 64 + 16 * c, pd);
#pragma unroll
    for (int u4 = 0; u4 < 4; ++u4) {                 // 16-byte unit u = queries [8 u, 8 u + 8) of the half
      const int u = 4 * c + u4;
      *reinterpret_cast<uint4*>(ds_row + (swz_unit(128, kr, u) << 4)) =
          make_uint4(pd[4 * u4], pd[4 * u4 + 1], pd[4 * u4 + 2], pd[4 * u4 + 3]);
    }
  }
}

// The half tile of a warp whose keys none of its queries sees: P^T and dS^T are zero.
__device__ __forceinline__ void zero_half(uint32_t col, uint8_t* ds_row, int kr) {
  uint32_t z[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) z[k] = 0u;
  tmem_st_32x32b_x32(col, z);
  tmem_st_32x32b_x32(col + 64, z);
#pragma unroll
  for (int u = 0; u < 8; ++u) *reinterpret_cast<uint4*>(ds_row + (swz_unit(128, kr, u) << 4)) = make_uint4(0, 0, 0, 0);
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
attn_window_bwd_tc_kernel(const __grid_constant__ CUtensorMap tm_qkv, const __grid_constant__ CUtensorMap tm_dy,
                   const __grid_constant__ CUtensorMap tm_dkv, const __grid_constant__ CUtensorMap tm_dq,
                   const float* __restrict__ rows, const WinBwdShape w, float sl2,
                   float rsd, float* slabs, int* err) {
  using Cfg = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  BwdBars* bars = reinterpret_cast<BwdBars*>(smem_raw + Cfg::OFF_BAR);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) record_error(err, GPT_DEV_EALIGN);
    return;
  }
  volatile int* abort_flag = &bars->abort_flag;
  const int T = w.T, H = w.H;
  const int kcol = H * D, ucol = (H + w.Hkv) * D;    // first key and value columns of a row

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 4);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&bars->q_full[i], 2);
      mbar_init(&bars->q_empty[i], 1);
    }
    mbar_init(&bars->dq_full, 1);
    mbar_init(&bars->dq_free, 4);
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->acc_free, 4);
    mbar_init(&bars->kvt_full, 4);
    mbar_init(&bars->kvt_free, 1);
    for (int i = 0; i < SR; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], kConsumers);
    }
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_qkv);
    tma_prefetch_desc(&tm_dy);
    tma_prefetch_desc(&tm_dkv);
    tma_prefetch_desc(&tm_dq);
  }
  if (warp == 1) tmem_alloc(&bars->tmem_base, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  pdl_wait();
  pdl_trigger();
  asm volatile("fence.proxy.async.global;" ::: "memory");   // the cleared dQ buffer, before TMA adds into it

  uint8_t* sK = smem_raw + Cfg::OFF_K;
  uint8_t* sU = smem_raw + Cfg::OFF_U;
  uint8_t* sQ = smem_raw + Cfg::OFF_Q;
  uint8_t* sDY = smem_raw + Cfg::OFF_DY;
  float* sLD = reinterpret_cast<float*>(smem_raw + Cfg::OFF_LD);
  uint8_t* sDS = smem_raw + Cfg::OFF_DS;

  if (warp == 0) {
    // ------------------------------------------------ producer (whole warp; lane 0 issues the copies)
    uint32_t qcount = 0;
    bool ok = true;
    uint32_t issued_kv = 0, par_kv = 0, issued_q = 0, par_q = 0;
    Items items;
    Item x;
    for (int r = 0; ok; ++r) {
      const bool have = items.next(w, x);
      const int slot = r % SR;
      if (r >= SR && !mbar_wait_warp(&bars->item_empty[slot], static_cast<uint32_t>(r / SR - 1) & 1u, abort_flag, err)) break;
      if (lane == 0) {
        int4* v = reinterpret_cast<int4*>(bars->item[slot]);
        v[0] = have ? make_int4(x.b, x.kh, x.j, x.j + x.cnt) : make_int4(0, 0, 0, 0);
        v[1] = have ? make_int4(x.first_tile(), x.first_head(w.G), x.steps, x.slot) : make_int4(0, 0, 0, 0);
        mbar_arrive(&bars->item_full[slot]);
      }
      if (!have) break;
      const int kb = r & 1;
      if (r >= 2 && !mbar_wait_warp(&bars->kv_empty[kb], static_cast<uint32_t>((r >> 1) - 1) & 1u, abort_flag, err)) break;
      // the previous item's U has gone to tensor memory
      if (r >= 1 && !mbar_wait_warp(&bars->kvt_full, static_cast<uint32_t>(r - 1) & 1u, abort_flag, err)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->kv_full[kb], 2 * Cfg::TILE);
        tma_load_3d(sK + kb * Cfg::TILE, &tm_qkv, &bars->kv_full[kb], kcol + x.kh * D, x.j * BT, x.b);
        tma_load_3d(sU, &tm_qkv, &bars->kv_full[kb], ucol + x.kh * D, x.j * BT, x.b);
      }
      issued_kv |= 1u << kb;
      par_kv = (par_kv & ~(1u << kb)) | (static_cast<uint32_t>((r >> 1) & 1) << kb);
      int head = x.first_head(w.G), i = x.first_tile();   // query head and tile of the step
      for (int e = 0; e < x.steps; ++e, ++qcount) {
        // Q and dY three steps ahead of the last one done, the rows' values (two slots) two
        const uint32_t qs = qcount % NQ;
        if (qcount >= NQ && !mbar_wait_warp(&bars->q_empty[qs], (qcount / NQ - 1) & 1u, abort_flag, err)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[qs], 2 * Cfg::TILE);
          tma_load_3d(sQ + qs * Cfg::TILE, &tm_qkv, &bars->q_full[qs], head * D, i * BT, x.b);
          tma_load_3d(sDY + qs * Cfg::TILE, &tm_dy, &bars->q_full[qs], head * D, i * BT, x.b);
        }
        issued_q |= 1u << qs;
        par_q = (par_q & ~(1u << qs)) | (((qcount / NQ) & 1u) << qs);
        if (qcount >= 2 && !mbar_wait_warp(&bars->q_empty[(qcount - 2) % NQ], ((qcount - 2) / NQ) & 1u, abort_flag, err)) {
          ok = false;
          if (lane == 0) mbar_arrive(&bars->q_full[qs]);   // the copies' phase completes for the drain below
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[qs], 2 * BT * sizeof(float));
          bulk_load(sLD + (qcount & 1u) * (2 * BT), rows + ((static_cast<size_t>(x.b) * H + head) * w.n_qt + i) * (2 * BT),
                    2 * BT * sizeof(float), &bars->q_full[qs]);
        }
        if (++i == x.j + x.cnt) {
          i = x.j;
          ++head;
        }
      }
    }
    // never leave with copies in flight into this CTA's shared memory
    if (lane == 0) {
      for (int k = 0; k < 2; ++k)
        if (issued_kv & (1u << k)) mbar_wait_drain(&bars->kv_full[k], (par_kv >> k) & 1u);
      for (int k = 0; k < NQ; ++k)
        if (issued_q & (1u << k)) mbar_wait_drain(&bars->q_full[k], (par_q >> k) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (whole warp; one elected lane issues)
    const uint64_t dq0 = smem_desc(smem_u32(sQ), 16, 8 * Cfg::ROWB, Cfg::SWZ);       // K-major (B of S^T)
    const uint64_t dy0 = smem_desc(smem_u32(sDY), 16, 8 * Cfg::ROWB, Cfg::SWZ);      // K-major (B of dP^T)
    const uint64_t qmn0 = smem_desc(smem_u32(sQ), Cfg::TILE, 8 * Cfg::ROWB, Cfg::SWZ);   // MN-major (B of dK)
    const uint64_t dymn0 = smem_desc(smem_u32(sDY), Cfg::TILE, 8 * Cfg::ROWB, Cfg::SWZ); // MN-major (B of dU)
    const uint64_t kmn0 = smem_desc(smem_u32(sK), Cfg::TILE, 8 * Cfg::ROWB, Cfg::SWZ);   // MN-major (B of dQ)
    // dS: MN-major A (queries contiguous): 64-query atoms 16 KB apart, 8-key groups 1 KB apart
    const uint64_t ds0 = smem_desc(smem_u32(sDS), BT * 128, 1024, SWZ_128B);
    constexpr uint32_t id_s = idesc_bf16_f32(BT, HQ, false);
    constexpr uint32_t id_acc = idesc_bf16_f32(BT, D, true);                  // B MN-major
    constexpr uint32_t id_dq = idesc_bf16_f32(BT, D, true) | (1u << 15);      // A and B MN-major
    // S^T and dP^T of half g of the query tile in ring slot qs; A = K_j, U_j from tensor memory (a K step
    // of 16 dimensions: 8 columns)
    auto issue_scores = [&](int g, uint32_t qs) {
      const uint32_t qoff = qs * Cfg::TILE + g * HQ * Cfg::ROWB;
      mma_ts_run<D / 16, 2>(tmem_base + 128 * g, tmem_base + kColK, desc_add(dq0, qoff), id_s, false);
      mma_ts_run<D / 16, 2>(tmem_base + 128 * g + 64, tmem_base + kColK + D / 2, desc_add(dy0, qoff), id_s, false);
      tc_commit_warp(&bars->s_full[g]);
    };
    // dU += P^T_g dY_g and dK += dS^T_g Q_g (a K step of 16 queries: 8 TMEM columns, 16 rows of dY / Q)
    auto issue_acc = [&](int g, uint32_t qs, bool first) {
      const uint32_t qoff = qs * Cfg::TILE + g * HQ * Cfg::ROWB;
      static_assert(HQ / 16 == 4, "K steps of a half");
      mma_ts_run<4, Cfg::ROWB>(tmem_base + kColDU, tmem_base + 128 * g, desc_add(dymn0, qoff), id_acc, !first);
      mma_ts_run<4, Cfg::ROWB>(tmem_base + kColDK, tmem_base + 128 * g + 64, desc_add(qmn0, qoff), id_acc, !first);
    };
    int r = 0;
    Step0 x;
    bool ok = next_item(bars, 0, x, abort_flag, err, lane);
    int steps = ok ? x.steps : 0, e = 0, kb = 0;
    uint32_t qcount = 0, qs = 0, tiles = 0;
    if (ok)
      ok = mbar_wait_warp(&bars->kv_full[0], 0u, abort_flag, err) && mbar_wait_warp(&bars->q_full[0], 0u, abort_flag, err) &&
           mbar_wait_warp(&bars->kvt_full, 0u, abort_flag, err);
    if (ok) {
      tc_fence_after();
      issue_scores(0, qs);
      issue_scores(1, qs);
      if (steps == 1) tc_commit_warp(&bars->kvt_free);   // the item's last reads of K_j, U_j in TMEM
    }
    // A wait costs about 90 cycles even where the phase is complete: each barrier is tested ahead of a run of products,
    // whose issue hides the answer's latency, and waited for only where the answer was no.
    auto settled = [&](bool early, uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, early) || mbar_wait_warp(bar, parity, abort_flag, err);
    };
    bool early_p0 = false;
    while (ok) {
      const bool first = e == 0, last = e == steps - 1;
      if (!settled(early_p0, &bars->p_full[0], tiles & 1u)) break;
      // the previous item's dK and dU have been read out of the accumulators
      if (first && r > 0 && !mbar_wait_warp(&bars->acc_free, static_cast<uint32_t>(r - 1) & 1u, abort_flag, err)) break;
      tc_fence_after();
      const uint32_t qcount2 = qcount + 1, qs2 = qcount2 % NQ;
      const bool early_q = mbar_test(&bars->q_full[qs2], (qcount2 / NQ) & 1u);
      issue_acc(0, qs, first);
      // the next step: the same item's, or the first of the next item
      bool has_next = !last;
      int r2 = r, e2 = e + 1, steps2 = steps, kb2 = kb;
      if (last) {
        has_next = next_item(bars, r + 1, x, abort_flag, err, lane);
        if (has_next) {
          r2 = r + 1;
          e2 = 0;
          steps2 = x.steps;
          kb2 = r2 & 1;
          if (!mbar_wait_warp(&bars->kv_full[kb2], static_cast<uint32_t>(r2 >> 1) & 1u, abort_flag, err)) break;
          if (!mbar_wait_warp(&bars->kvt_full, static_cast<uint32_t>(r2) & 1u, abort_flag, err)) break;
        }
      }
      if (has_next && !settled(early_q, &bars->q_full[qs2], (qcount2 / NQ) & 1u)) break;
      const bool early_p1 = mbar_test(&bars->p_full[1], tiles & 1u);
      if (has_next) {
        tc_fence_after();
        issue_scores(0, qs2);
      }
      if (!settled(early_p1, &bars->p_full[1], tiles & 1u)) break;
      tc_fence_after();
      const bool early_dq = tiles == 0 || mbar_test(&bars->dq_free, (tiles - 1) & 1u);
      issue_acc(1, qs, false);
      tc_commit_warp(&bars->q_empty[qs]);            // Q_i and dY_i are consumed
      if (last) tc_commit_warp(&bars->acc_full);
      // the next scores before dQ: the derivative warps wait for them, nothing waits for dQ
      if (has_next) {
        issue_scores(1, qs2);
        if (e2 == steps2 - 1) tc_commit_warp(&bars->kvt_free);
      }
      if (!settled(early_dq, &bars->dq_free, (tiles - 1) & 1u)) break;
      early_p0 = mbar_test(&bars->p_full[0], (tiles + 1) & 1u);
      tc_fence_after();
      const uint32_t dsoff = (tiles & 1u) * Cfg::DS_BUF;
#pragma unroll
      for (int kk = 0; kk < BT / 64; ++kk)           // a K step of 16 keys: 16 rows of dS and of K_j
        mma_ss_run4<128, Cfg::ROWB>(tmem_base + kColDQ, desc_add(ds0, dsoff + kk * 64 * 128),
                                    desc_add(kmn0, kb * Cfg::TILE + kk * 64 * Cfg::ROWB), id_dq, kk > 0);
      tc_commit_warp(&bars->dq_full);
      if (last) tc_commit_warp(&bars->kv_empty[kb]);   // K_j and U_j are consumed
      if (!has_next) break;
      r = r2;
      e = e2;
      steps = steps2;
      kb = kb2;
      qcount = qcount2;
      qs = qs2;
      ++tiles;
    }
    tc_commit_warp(&bars->drain);
    mbar_wait_drain(&bars->drain, 0);
  } else if (warp < 10) {
    // ------------------------------------------------ softmax derivative (thread = key row; group g: half g)
    const int g = warp < 6 ? 0 : 1;
    const int sub = warp & 3;
    const int kr = sub * 32 + lane;                  // key row within the tile = TMEM lane
    const uint32_t tb = tmem_base + (static_cast<uint32_t>(sub * 32) << 16);
    uint32_t tiles = 0;
    bool ok = true;
    Step0 x;
    for (int r = 0; ok && next_item(bars, r, x, abort_flag, err, lane); ++r) {
      const int s0 = x.j * BT + sub * 32;              // the warp's first key
      // the last query that sees this thread's key, and the same for the warp's first and last key
      const int far = T - 1;
      const int end = s0 + lane < w.sinks ? far : static_cast<int>(min(static_cast<long long>(far), static_cast<long long>(s0) + lane + w.window - 1));
      const int end_lo = s0 + 31 < w.sinks ? far : static_cast<int>(min(static_cast<long long>(far), static_cast<long long>(s0 < w.sinks ? w.sinks : s0) + w.window - 1));
      const int end_hi = s0 < w.sinks ? far : static_cast<int>(min(static_cast<long long>(far), static_cast<long long>(s0) + 31 + w.window - 1));
      int i = x.i;
      for (int e = 0; e < x.steps; ++e, ++tiles) {
        const uint32_t qs = tiles % NQ;
        if (!mbar_wait_warp(&bars->q_full[qs], (tiles / NQ) & 1u, abort_flag, err)) { ok = false; break; }
        const float4* ld = reinterpret_cast<const float4*>(sLD + (tiles & 1u) * (2 * BT)) + 32 * g;
        uint8_t* ds_row = sDS + (tiles & 1u) * Cfg::DS_BUF + g * (BT * 128) + kr * 128;
        if (!mbar_wait_warp(&bars->s_full[g], tiles & 1u, abort_flag, err)) { ok = false; break; }
        tc_fence_after();
        // query q0 + ql is kept for lo <= ql <= hi. The choice of path is the warp's: the TMEM loads in it
        // are warp-wide (.aligned).
        const int q0 = i * BT + g * HQ;
        if (q0 > end_hi || q0 + HQ - 1 < s0) {
          zero_half(tb + 128 * g, ds_row, kr);
        } else if (q0 < s0 + 31 || q0 + HQ - 1 > end_lo) {
          const int hi = end - q0, lo = s0 + lane - q0;
          const uint64_t below_hi = hi < 0 ? 0ull : (hi >= HQ - 1 ? ~0ull : (2ull << hi) - 1ull);
          const uint64_t from_lo = lo >= HQ ? 0ull : (~0ull << (lo > 0 ? lo : 0));
          derivative_half<true>(tb + 128 * g, ld, sl2, below_hi & from_lo, ds_row, kr);
        } else {
          derivative_half<false>(tb + 128 * g, ld, sl2, ~0ull, ds_row, kr);
        }
        tmem_st_wait();
        fence_proxy_async_smem();                    // dS in shared memory is read by the dQ product
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[g]);
        if (++i == x.end) i = x.j;
      }
    }
  } else {
    // ------------------------------------------------ output: dQ reduce-adds and conversion, dK and dU stores
    const int sub = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(sub * 32) << 16;
    uint8_t* stg = smem_raw + Cfg::OFF_STG + (warp - 10) * 4096;
    // K_j and U_j (item buffer kb) into tensor memory as the scores' A operands: this warp's 32 key rows,
    // each row's D values as bf16 pairs
    auto stage_kv = [&](int kb) {
      constexpr int ROWB = Cfg::ROWB;
      const int kr = sub * 32 + lane;
      const uint8_t* krow = sK + kb * Cfg::TILE + kr * ROWB;
      const uint8_t* urow = sU + kr * ROWB;
      uint32_t kw[D / 2], uw[D / 2];
#pragma unroll
      for (int u = 0; u < ROWB / 16; ++u) {
        const uint4 a = *reinterpret_cast<const uint4*>(krow + (swz_unit(ROWB, kr, u) << 4));
        const uint4 c = *reinterpret_cast<const uint4*>(urow + (swz_unit(ROWB, kr, u) << 4));
        kw[4 * u] = a.x; kw[4 * u + 1] = a.y; kw[4 * u + 2] = a.z; kw[4 * u + 3] = a.w;
        uw[4 * u] = c.x; uw[4 * u + 1] = c.y; uw[4 * u + 2] = c.z; uw[4 * u + 3] = c.w;
      }
      if constexpr (D == 64) {
        tmem_st_32x32b_x32(tmem_base + lane_off + kColK, kw);
        tmem_st_32x32b_x32(tmem_base + lane_off + kColK + D / 2, uw);
      } else {
        tmem_st_32x32b_x16(tmem_base + lane_off + kColK, kw);
        tmem_st_32x32b_x16(tmem_base + lane_off + kColK + D / 2, uw);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->kvt_full);
    };
    uint32_t tiles = 0;
    bool ok = true;
    Step0 x, x_next;
    bool have = next_item(bars, 0, x, abort_flag, err, lane);
    if (have) {
      ok = mbar_wait_warp(&bars->kv_full[0], 0u, abort_flag, err);
      if (ok) stage_kv(0);
    }
    for (int r = 0; ok && have; ++r) {
      bool have_next = false;
      int i = x.i, head = x.head;
      for (int e = 0; e < x.steps; ++e, ++tiles) {
        if (e == x.steps - 1) have_next = next_item(bars, r + 1, x_next, abort_flag, err, lane);
        if (e == x.steps - 1 && have_next) {
          // before the item's last dQ: the next item's K_j, U_j, once the item's last scores have read theirs
          if (!mbar_wait_warp(&bars->kvt_free, static_cast<uint32_t>(r) & 1u, abort_flag, err) ||
              !mbar_wait_warp(&bars->kv_full[(r + 1) & 1], static_cast<uint32_t>((r + 1) >> 1) & 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          stage_kv((r + 1) & 1);
        }
        if (e == x.steps - 1) {
          // the item's dK and dU, complete before its last dQ: read first, so that the next item's products may start
          if (!mbar_wait_warp(&bars->acc_full, static_cast<uint32_t>(r) & 1u, abort_flag, err)) { ok = false; break; }
          tc_fence_after();
          constexpr int ROWB = Cfg::ROWB;
          if (x.slot >= 0) {                         // one of several segments: unscaled fp32
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
              float4* dst = reinterpret_cast<float4*>(slabs + ((static_cast<size_t>(x.slot) * 2 + which) * BT + sub * 32 + lane) * D);
#pragma unroll 1
              for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem_base + (which ? kColDU : kColDK) + lane_off + 32 * cc, v);
                tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < 8; ++u)
                  dst[8 * cc + u] = make_float4(__uint_as_float(v[4 * u]), __uint_as_float(v[4 * u + 1]),
                                                __uint_as_float(v[4 * u + 2]), __uint_as_float(v[4 * u + 3]));
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->acc_free);
          } else {
            uint32_t pk[D / 2], pu[D / 2];           // bf16 rows: dK / sqrt(D), dU
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(tmem_base + kColDK + lane_off + 32 * cc, v);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 16; ++u)
                pk[16 * cc + u] = pack_bf16x2(__uint_as_float(v[2 * u]) * rsd, __uint_as_float(v[2 * u + 1]) * rsd);
              tmem_ld_32x32b_x32(tmem_base + kColDU + lane_off + 32 * cc, v);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 16; ++u)
                pu[16 * cc + u] = pack_bf16x2(__uint_as_float(v[2 * u]), __uint_as_float(v[2 * u + 1]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->acc_free);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              if (lane == 0) bulk_wait_read_all();   // the previous copy has read the box
              __syncwarp();
#pragma unroll
              for (int u = 0; u < ROWB / 16; ++u)
                *reinterpret_cast<uint4*>(stg + lane * ROWB + (swz_unit(ROWB, lane, u) << 4)) =
                    which ? make_uint4(pu[4 * u], pu[4 * u + 1], pu[4 * u + 2], pu[4 * u + 3])
                          : make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&tm_dkv, stg, (which ? ucol : kcol) + x.kh * D, x.j * BT + sub * 32, x.b);
                bulk_commit();
              }
            }
          }
        }
        if (!mbar_wait_warp(&bars->dq_full, tiles & 1u, abort_flag, err)) { ok = false; break; }
        tc_fence_after();
        uint32_t v[D];
        if constexpr (D == 64) {
          tmem_ld_32x32b_x64(tmem_base + kColDQ + lane_off, *reinterpret_cast<uint32_t (*)[64]>(v));
        } else {
          tmem_ld_32x32b_x32(tmem_base + kColDQ + lane_off, *reinterpret_cast<uint32_t (*)[32]>(v));
        }
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->dq_free);
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {        // 32 fp32 columns (128 bytes) per box row
          if (lane == 0) bulk_wait_read_all();       // the previous copy has read the box
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(stg + lane * 128 + (swz_unit(128, lane, u) << 4)) =
                make_uint4(v[32 * cc + 4 * u], v[32 * cc + 4 * u + 1], v[32 * cc + 4 * u + 2], v[32 * cc + 4 * u + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_reduce_add_3d(&tm_dq, stg, head * D + 32 * cc, i * BT + sub * 32, x.b);
            bulk_commit();
          }
        }
        if (++i == x.end) {
          i = x.j;
          ++head;
        }
      }
      if (!ok) break;
      x = x_next;
      have = have_next;
    }
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// What the derivative reads of every query row, in its order: per (b, h), tile of 128 rows (the last one filled up with
// zeros) and pair of rows {-lse2, -lse2, -Dsum, -Dsum}, with Dsum[t] = sum_d dY[t,d] Y[t,d], so that a tile's kilobyte is
// one bulk copy, which waits for nothing else (the producer's plain loads of them waited with every step). One warp per
// row, D / 8 lanes per head with 16-byte loads, so each load instruction of the warp reads 512 contiguous bytes of the
// row. It also clears the row of the dQ accumulator (a memset of its own took a launch and as long again). Bound by
// memory at 0.6 of the copy rate (8 x 1,000 tokens, 12 heads: 11 us cold); two or four of a row's loads in flight per
// lane changed the training calls by less than 1 % either way.
template <int D>
__global__ void __launch_bounds__(256)
attn_window_rows_kernel(const __nv_bfloat16* __restrict__ y, const __nv_bfloat16* __restrict__ dy,
                        const float* __restrict__ lse2, float* __restrict__ rows, float* __restrict__ dqacc, int M, int T,
                        int H, int n_qt) {
  pdl_wait();
  pdl_trigger();
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= M) return;
  constexpr int LPH = D / 8;
  const int C = H * D, nv = C / 8;
  const uint4* a4 = reinterpret_cast<const uint4*>(dy + static_cast<size_t>(row) * C);
  const uint4* o4 = reinterpret_cast<const uint4*>(y + static_cast<size_t>(row) * C);
  const int b = static_cast<int>(row / T), t = static_cast<int>(row - static_cast<long long>(b) * T);
  const size_t tp = static_cast<size_t>(n_qt) * BT;  // padded rows
  for (int v0 = 0; v0 < nv; v0 += 32) {            // nv is a multiple of LPH: a head's lanes are all in or all out
    const int v = v0 + lane;
    float acc = 0.0f, ls = 0.0f;
    const size_t bh = static_cast<size_t>(b) * H + v / LPH;
    const bool writer = v < nv && (lane % LPH) == 0;
    if (writer) ls = __ldg(lse2 + bh * T + t);
    if (v < nv) {
      const uint4 a = __ldg(a4 + v), o = __ldg(o4 + v);
      float4* z = reinterpret_cast<float4*>(dqacc + static_cast<size_t>(row) * C) + 2 * v;
      z[0] = z[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = unpack_bf16x2(aw[k]), z2 = unpack_bf16x2(ow[k]);
        acc = fmaf(x.x, z2.x, fmaf(x.y, z2.y, acc));
      }
    }
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (writer) {
      float* dst = rows + (bh * tp + (t & ~1)) * 2 + (t & 1);
      dst[0] = -ls;
      dst[2] = -acc;
      if (t == T - 1) {                              // the last tile's missing rows
        if ((t & 1) == 0) dst[1] = dst[3] = 0.0f;
        for (size_t f = (bh * tp + ((t | 1) + 1)) * 2; f < (bh + 1) * tp * 2; ++f) rows[f] = 0.0f;
      }
    }
  }
}

// The first `nblk` blocks: dqkv[m, c] = bf16(dqacc[m, c] / sqrt(D)) for the first C = H D of a row's columns, four
// consecutive floats per thread and step, so each warp access covers 512 contiguous bytes. Later blocks: dK and dU of
// the key tiles that were cut into segments, their slabs summed in order.
template <int D>
__global__ void __launch_bounds__(256)
attn_window_finish_kernel(const float* __restrict__ dqacc, const float* __restrict__ slabs, __nv_bfloat16* __restrict__ dqkv,
                          int M, const WinBwdShape w, int nblk, float rsd) {
  pdl_wait();
  pdl_trigger();
  const int C = w.H * D, row = C + 2 * w.Hkv * D;
  if (static_cast<int>(blockIdx.x) < nblk) {
    const int c4n = C / 4;
    const long long n = static_cast<long long>(M) * c4n;
    for (long long e = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; e < n;
         e += static_cast<long long>(nblk) * blockDim.x) {
      const int m = static_cast<int>(e / c4n), c = static_cast<int>(e - static_cast<long long>(m) * c4n) * 4;
      const float4 a = __ldg(reinterpret_cast<const float4*>(dqacc) + e);
      *reinterpret_cast<uint2*>(dqkv + static_cast<size_t>(m) * row + c) =
          make_uint2(pack_bf16x2(a.x * rsd, a.y * rsd), pack_bf16x2(a.z * rsd, a.w * rsd));
    }
    return;
  }
  // the tile's first item: the cut tiles are those with sinks (if nseg_s > 1), then the others (if nseg_w > 1)
  constexpr int PARTS = 2 * BT * (D / 4) / 256;      // blocks per tile: four floats of the tile per thread
  int k = (static_cast<int>(blockIdx.x) - nblk) / PARTS;
  const int part = (static_cast<int>(blockIdx.x) - nblk) % PARTS;
  const int sinks = w.nseg_s > 1 ? w.sink_tiles * w.BK : 0;
  const bool sink = k < sinks;
  if (!sink) k -= sinks;
  const int nseg = sink ? w.nseg_s : w.nseg_w;
  const int jj = k / w.BK, bk = k - jj * w.BK, j = jj + (sink ? 0 : w.sink_tiles);
  const int slot0 = (sink ? 0 : (w.nseg_s > 1 ? w.n_sink_items : 0)) + jj * nseg * w.BK + bk;
  const int steps = w.G * tile_count(w, j);
  const int b = bk / w.Hkv, kh = bk - b * w.Hkv;
  const int i = part * 256 + threadIdx.x;
  const int which = i / (BT * (D / 4)), r = i / (D / 4) % BT, c = i % (D / 4);
  if (j * BT + r >= w.T) return;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < nseg; ++s) {
    if (seg_start(steps, s, nseg) == seg_start(steps, s + 1, nseg)) continue;   // an empty segment has no slab
    const float4 v = __ldg(reinterpret_cast<const float4*>(slabs) + static_cast<size_t>(slot0 + s * w.BK) * (2 * BT * (D / 4)) + i);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  const float f = which ? 1.0f : rsd;
  *reinterpret_cast<uint2*>(dqkv + (static_cast<size_t>(b) * w.T + j * BT + r) * row + C + (which * w.Hkv + kh) * D + 4 * c) =
      make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
}

// Cuts the launch into items; the fp32 slabs that it needs.
struct WinBwdPlan {
  WinBwdShape w;
  int slabs, cut_tiles;
};

bool plan_bwd(int B, int T, int H, int Hkv, int window, int sinks, int num_sms, WinBwdPlan* p) {
  WinBwdShape& w = p->w;
  w = {};
  w.T = T;
  w.H = H;
  w.Hkv = Hkv;
  w.G = H / Hkv;
  w.window = window < T ? window : T;
  w.sinks = sinks < T ? sinks : T;
  w.n_qt = (T + BT - 1) / BT;
  w.sink_tiles = (w.sinks + BT - 1) / BT;
  w.BK = B * Hkv;
  const int rest = w.n_qt - w.sink_tiles;
  const long long big_s = w.sink_tiles ? static_cast<long long>(w.G) * w.n_qt : 0;
  const long long big_w = rest ? static_cast<long long>(w.G) * tile_count(w, w.sink_tiles) : 0;
  // a CTA's fair share of the steps; a tile that has more is cut into segments of about half of it, but of 8 steps
  // at least (a segment costs its K and U tiles and, at its end, 64 KB of fp32 sums)
  const long long share = ((big_s * w.sink_tiles + big_w * rest) * w.BK + num_sms - 1) / num_sms;
  const long long len = share / 2 > 8 ? share / 2 : 8;
  const long long ns = big_s > share && big_s > len ? (big_s + len - 1) / len : 1;
  const long long nw = big_w > share && big_w > len ? (big_w + len - 1) / len : 1;
  const long long sink_items = ns * w.sink_tiles * w.BK, items = sink_items + nw * rest * w.BK;
  if (items > 0x7fffffffLL || big_s > 0x7fffffffLL || big_w > 0x7fffffffLL) return false;
  w.nseg_s = static_cast<int>(ns);
  w.nseg_w = static_cast<int>(nw);
  w.n_sink_items = static_cast<int>(sink_items);
  w.n_items = static_cast<int>(items);
  p->slabs = static_cast<int>((ns > 1 ? sink_items : 0) + (nw > 1 ? items - sink_items : 0));
  p->cut_tiles = ((ns > 1 ? w.sink_tiles : 0) + (nw > 1 ? rest : 0)) * w.BK;
  return true;
}

int sm_count() {
  int dev = 0, n = 0;
  return device_sms(&dev, &n) == cudaSuccess ? n : 0;
}

template <int D>
cudaError_t launch_bwd_d(const CUtensorMap& tm_qkv, const CUtensorMap& tm_dy, const CUtensorMap& tm_dkv,
                         const CUtensorMap& tm_dq, const void* y, const void* dy, const float* lse2, float* rows,
                         float* dqacc, float* slabs, void* dqkv, int B, const WinBwdPlan& plan, int num_sms, int* err,
                         cudaStream_t s) {
  using Cfg = BwdCfg<D>;
  const WinBwdShape& w = plan.w;
  static SmemLimit limit;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e == cudaSuccess) e = limit.raise(attn_window_bwd_tc_kernel<D>, dev, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  const int M = B * w.T, C = w.H * D;
  const float rsd = 1.0f / sqrtf(static_cast<float>(D));
  const float sl2 = rsd * kLog2e;
  e = launch_k(attn_window_rows_kernel<D>, dim3(static_cast<unsigned>((M - 1) / 8 + 1)), dim3(256), 0, s,
               static_cast<const __nv_bfloat16*>(y), static_cast<const __nv_bfloat16*>(dy), lse2, rows, dqacc, M, w.T, w.H,
               w.n_qt);
  if (e != cudaSuccess) return e;
  const int grid = w.n_items < num_sms ? w.n_items : num_sms;
  e = launch_k(attn_window_bwd_tc_kernel<D>, dim3(grid), dim3(THREADS), static_cast<size_t>(Cfg::SMEM), s, tm_qkv, tm_dy,
               tm_dkv, tm_dq, static_cast<const float*>(rows), w, sl2, rsd, slabs, err);
  if (e != cudaSuccess) return e;
  const long long n4 = static_cast<long long>(M) * (C / 4);
  const long long cblocks = (n4 + 255) / 256;
  const int nblk = static_cast<int>(cblocks < 8LL * num_sms ? cblocks : 8LL * num_sms);
  return launch_k(attn_window_finish_kernel<D>, dim3(nblk + plan.cut_tiles * (2 * BT * (D / 4) / 256)), dim3(256), 0, s, static_cast<const float*>(dqacc),
                  static_cast<const float*>(slabs), static_cast<__nv_bfloat16*>(dqkv), M, w, nblk, rsd);
}

}  // namespace

size_t attention_window_bwd_row_bytes(int B, int T, int H) {
  return static_cast<size_t>(B) * H * ((T + BT - 1) / BT) * (2 * BT) * sizeof(float);
}

size_t attention_window_bwd_slab_bytes(int B, int T, int H, int Hkv, int D, int window, int sinks) {
  WinBwdPlan p;
  const int num_sms = sm_count();
  if (num_sms <= 0 || !plan_bwd(B, T, H, Hkv, window, sinks, num_sms, &p)) return 0;
  return static_cast<size_t>(p.slabs) * 2 * BT * D * sizeof(float);
}

cudaError_t launch_attention_window_bwd_tc(const CUtensorMap& tm_qkv, const CUtensorMap& tm_dy, const CUtensorMap& tm_dkv,
                                           const CUtensorMap& tm_dq, const void* y, const void* dy, const float* lse2,
                                           float* rows, float* dqacc, float* slabs, void* dqkv, int B, int T, int H,
                                           int Hkv, int D, int window, int sinks, int* err, cudaStream_t s) {
  WinBwdPlan p;
  const int num_sms = sm_count();
  if (num_sms <= 0 || !plan_bwd(B, T, H, Hkv, window, sinks, num_sms, &p)) return cudaErrorInvalidValue;
  if (D == 64)
    return launch_bwd_d<64>(tm_qkv, tm_dy, tm_dkv, tm_dq, y, dy, lse2, rows, dqacc, slabs, dqkv, B, p, num_sms, err, s);
  if (D == 32)
    return launch_bwd_d<32>(tm_qkv, tm_dy, tm_dkv, tm_dq, y, dy, lse2, rows, dqacc, slabs, dqkv, B, p, num_sms, err, s);
  return cudaErrorInvalidValue;
}

}  // namespace gptgb
