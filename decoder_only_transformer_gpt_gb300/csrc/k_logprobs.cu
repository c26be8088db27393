// Log probabilities of given tokens under logits, with entropy and the most probable tokens, and their gradient.
//
// With m the row's largest logit and d = z - m: S = sum e^d, A = sum d e^d, ln p = d - ln S, entropy = ln S - A / S. One pass
// keeps m, S and A per lane against a running maximum (a chunk's maximum first, so S and A are rescaled once a chunk:
// S' = f S, A' = f (A + (m - m') S), f = e^(m - m')). All in fp32, d as a difference, never through a rounded log-sum-exp:
// the gradient gets (m, S), as e^(z - lse) would carry the rounding of lse, 2^-24 |lse| of every probability.
//
// The most probable tokens, behind the sums: every thread has noted the largest logit of each of its chunks. The K-th largest
// of the warps' four largest of those is a floor that K tokens reach, and few others: only the chunks of threads that reach it
// are looked at again (out of L2, where they are not kept in registers), and what reaches it there goes into one pool of keys
// (logit, then lowest index) in shared memory, in any order. A key's place is the number of larger ones, so the result does
// not depend on that order. Where more tokens reach the floor than the pool holds (many equal ones), or there is none (fewer than
// K threads have a logit above -inf), every warp keeps its best 32 in order instead, one a lane, and the lists are joined. (Lists kept up to date while the row went by took 8 to 16
// instructions for every 32 logits, as many as the sums: 4,096 rows of 50,257 with K = 8 took 151 us in fp32 and 124 in bf16;
// lists for every warp behind the sums 135 and 85.)
//
// Bound by memory where rows are many: 4,096 x 50,257 in fp32 121 us with K = 0, 6.8 TB/s, what a copy reaches, and 129 with
// K = 8; in bf16 69 and 82, 6.0 TB/s, the exponentials' units and the sums' instructions close behind. The part after the
// sums reads little and lets the memory rest: that is what K adds. 16 rows with K = 5 4.6 us in a graph, 2.9 with K = 0.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

#include <cooperative_groups.h>
#include <math.h>

namespace gptgb {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kL2E = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = -1e20f;           // stands for differences of -inf in products with 0 (times 2^31 it is finite)
constexpr int kLpWarps = 8;
constexpr int kLpVecs = 4;               // 16-byte vectors a lane and chunk
constexpr int kLpChunk = 32 * kLpVecs;   // vectors a warp and chunk
// Up to this K the floor comes from the warps' four largest logits, else from all (16 rows of 50,257 with K = 20 5.2 and 5.3 us,
// with K = 32 11.5 and 5.5, as the pool then holds too few for what reaches the lower floor).
constexpr int kLpFewTop = 16;
constexpr int kLpPool = 64;              // tokens that are put in order at once
constexpr int kLpGroups = 16;            // maxima that a thread notes: of a chunk each, or of as many as it takes

using Key = unsigned long long;

// Larger logit, larger key; equal logits: lower index, larger key. Never 0. (-0 equals +0.)
__device__ __forceinline__ Key key_of(float v, int index) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<Key>(o) << 32) | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ float value_of(Key k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int index_of(Key k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// The 32 best of two lists in descending order.
__device__ __forceinline__ Key join_lists(Key a, Key b, int lane) {
  const Key r = __shfl_sync(kAll, b, 31 - lane);
  Key x = a > r ? a : r;
#pragma unroll
  for (int k = 16; k; k >>= 1) {
    const Key y = __shfl_xor_sync(kAll, x, k);
    x = ((lane & k) == 0) == (x > y) ? x : y;
  }
  return x;
}

// The same of values.
__device__ __forceinline__ float join_values(float a, float b, int lane) {
  float x = fmaxf(a, __shfl_sync(kAll, b, 31 - lane));
#pragma unroll
  for (int k = 16; k; k >>= 1) {
    const float y = __shfl_xor_sync(kAll, x, k);
    x = (lane & k) == 0 ? fmaxf(x, y) : fminf(x, y);
  }
  return x;
}

// The lanes' values in descending order.
__device__ __forceinline__ float sorted_values(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int k = size >> 1; k; k >>= 1) {
      const float y = __shfl_xor_sync(kAll, v, k);
      const bool down = (lane & size) == 0 || size == 32;   // this run is sorted in descending order
      const bool upper = (lane & k) == 0;
      v = upper == down ? fmaxf(v, y) : fminf(v, y);
    }
  return v;
}

// The largest of the lanes' values, in all of them (a NaN is passed over).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

struct Sums {
  float m, s, a;
};
__device__ __forceinline__ Sums joined_sums(const Sums& x, const Sums& y) {
  const float m = fmaxf(x.m, y.m);
  const float dx = fmaxf(x.m - m, kFar), dy = fmaxf(y.m - m, kFar);
  const float fx = ex2_approx(dx * kL2E), fy = ex2_approx(dy * kL2E);
  return {m, x.s * fx + y.s * fy, fx * (x.a + x.s * dx) + fy * (y.a + y.s * dy)};
}

template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ float2 pair(const uint4& v, int k) {
    const uint32_t* w = &v.x;
    return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ void put(float* p, float x) { *p = x; }
  static constexpr uint32_t kNone = 0xff800000u;     // -inf
  static __device__ __forceinline__ float most(const uint4& v) {
    const float2 a = pair(v, 0), b = pair(v, 1);
    return fmaxf(fmax3(a.x, a.y, b.x), b.y);
  }
  static __device__ __forceinline__ float2 halves(const uint4& v) {   // the largest of each half
    const float2 a = pair(v, 0), b = pair(v, 1);
    return make_float2(fmaxf(a.x, a.y), fmaxf(b.x, b.y));
  }
  static __device__ __forceinline__ float largest(const uint4 (&v)[kLpVecs]) {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kLpVecs; ++k) {
      const float2 a = pair(v[k], 0), b = pair(v[k], 1);
      m = fmax3(m, fmax3(a.x, a.y, b.x), b.y);
    }
    return m;
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ float2 pair(const uint4& v, int k) { return unpack_bf16x2((&v.x)[k]); }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ float most(const uint4& v) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v.x);
    const float2 f = __bfloat1622float2(__hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ float2 halves(const uint4& v) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v.x);
    const float2 a = __bfloat1622float2(__hmax2(w[0], w[1])), b = __bfloat1622float2(__hmax2(w[2], w[3]));
    return make_float2(fmaxf(a.x, a.y), fmaxf(b.x, b.y));
  }
  static __device__ __forceinline__ float largest(const uint4 (&v)[kLpVecs]) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v[0].x);
    __nv_bfloat162 m = w[0];
#pragma unroll
    for (int k = 1; k < 4 * kLpVecs; ++k) m = __hmax2(m, w[k]);   // (a NaN is passed over here and shows in the sums)
    const float2 f = __bfloat1622float2(m);
    return fmaxf(f.x, f.y);
  }
};

struct LpArgs {
  const void* z;
  const int32_t* targets;
  float *logp, *entropy, *stats, *top_logp;
  int32_t* top_ids;
  long long ld, M;
  int V, K, ahead;     // ahead: rows from one that is worked on to one that is not yet
};

// A row, or a stretch of it, as seen by one warp.
template <typename T>
struct Row {
  const T* z;
  int head, nvec;      // values before the first 16-byte boundary, then whole vectors
  __device__ __forceinline__ Row(const void* base, long long ld, int V, long long m) {
    z = static_cast<const T*>(base) + m * ld;
    const int to = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / static_cast<int>(sizeof(T));
    head = min(V, to);
    nvec = (V - head) / Vec<T>::N;
  }
};

// A warp takes a row (WR = 1; eight rows a block), or a block's eight warps do (WR = 8), or those of a cluster of NC blocks: the
// row's chunks go round the warps. FEW: no warp has more than two, which then stay in its registers and are not read again.
// TOP: false where none of the most probable tokens are wanted (K = 0; not of the clusters). It takes fewer registers and no
// shared memory for them: 4,096 x 50,257 121 and 124 us, 256 x 5,000 2.3 and 2.5, 4,096 x 5,000 14.8 and 16.7.
template <typename T, int NC, int WR, bool FEW, bool TOP>
__global__ void __launch_bounds__(kLpWarps * 32, NC > 1 ? 2 : WR == 1 && FEW && TOP ? 3 : 0)
logprobs_kernel(LpArgs a, int* err) {
  using W = Vec<T>;
  constexpr int N = W::N, VALUES = kLpVecs * N;      // values a lane and chunk
  namespace cg = cooperative_groups;
  __shared__ __align__(16) uint4 s_stage[kLpWarps][32][kLpVecs + 1];
  __shared__ float s_max[FEW ? 1 : kLpGroups][kLpWarps * 32];   // the threads' largest logits, by group of chunks
  __shared__ __align__(16) float s_order[kLpWarps][32];   // and over all groups, in order: all, or each warp's four largest
  __shared__ Key s_list[kLpWarps][32], s_lists[NC][32];   // the warps' lists, and the blocks'
  __shared__ Key s_pool[WR == 1 ? kLpWarps : 2][kLpPool], s_best[kLpWarps / WR][32];   // tokens without an order, and in order
  __shared__ int s_count[kLpWarps / WR];             // how many
  __shared__ Sums s_sums[8], s_parts[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = NC == 1 ? 0 : static_cast<int>(blockIdx.x % NC);
  const long long m = WR == 1 ? static_cast<long long>(blockIdx.x) * kLpWarps + warp : blockIdx.x / NC;
  if constexpr (NC > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // every block has started
  pdl_wait();
  pdl_trigger();
  if (WR == 1 && m >= a.M) return;
  const bool lead = WR == 1 || (part == 0 && warp == 0);
  const int team = WR == 1 ? warp : 0;               // of the block's rows
  const Row<T> row(a.z, a.ld, a.V, m);
  const uint4* vecs = reinterpret_cast<const uint4*>(row.z + row.head);
  const int K = TOP ? a.K : 0;
  int target = -1;
  float zt = 0.0f;
  if (lead && lane == 0 && a.targets) {
    target = __ldg(a.targets + m);
    if (static_cast<unsigned>(target) < static_cast<unsigned>(a.V)) {
      zt = W::get(row.z + target);
    } else {
      if (target != -1) record_error(err, GPT_DEV_ETARGET);
      target = -1;
    }
  }
  Sums sum = {kLowest, 0.0f, 0.0f};
  Key best = 0;                                      // this warp's list, one a lane

  auto add = [&](float cm, const uint4 (&v)[kLpVecs]) {
    const float mn = fmaxf(sum.m, cm), dm = fmaxf(sum.m - mn, kFar), f = ex2_approx(dm * kL2E);
    float2 s = make_float2(sum.s * f, 0.0f), e2 = make_float2(f * (sum.a + sum.s * dm), 0.0f);
    const float2 neg = make_float2(-mn, -mn), l2e = make_float2(kL2E, kL2E);
#pragma unroll
    for (int k = 0; k < kLpVecs; ++k)
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float2 d = add2_rn(W::pair(v[k], j), neg), x = mul2_rn(d, l2e);
        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        s = add2_rn(s, e);
        e2 = fma2_rn(e, make_float2(fmaxf(d.x, kFar), fmaxf(d.y, kFar)), e2);
      }
    sum = {mn, s.x + s.y, e2.x + e2.y};
  };
  const int full = row.nvec / kLpChunk;              // chunks without a gap
  const int step = WR == 1 ? 1 : NC * kLpWarps, first = WR == 1 ? 0 : warp * NC + part;
  const int chunks = (row.nvec + kLpChunk - 1) / kLpChunk;
  const int per = ((chunks + step - 1) / step + kLpGroups - 1) / kLpGroups;   // chunks of a group
  float top = -INFINITY, noted = -INFINITY;          // this thread's largest logit, and of the group
  int group = 0, in_group = 0;
  auto use = [&](const uint4 (&v)[kLpVecs]) {
    const float cm = W::largest(v);
    add(cm, v);
    if (K) {
      noted = fmaxf(noted, cm);
      if (++in_group == per) {
        s_max[group++][threadIdx.x] = noted;
        top = fmaxf(top, noted);
        noted = -INFINITY;
        in_group = 0;
      }
    }
  };

  const uint4* at = vecs + static_cast<long long>(first) * kLpChunk + lane;
  auto load = [&](uint4 (&v)[kLpVecs]) {             // the chunk at `at`, which moves on
#pragma unroll
    for (int k = 0; k < kLpVecs; ++k) v[k] = __ldg(at + 32 * k);
    at += static_cast<long long>(step) * kLpChunk;
  };
  auto load_last = [&](int chunk, uint4 (&v)[kLpVecs]) {   // a chunk that the row's last vector may end
#pragma unroll
    for (int k = 0; k < kLpVecs; ++k) {
      const int i = chunk * kLpChunk + k * 32 + lane;
      v[k] = make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
      if (i < row.nvec) v[k] = __ldg(vecs + i);
    }
  };
  uint4 v[kLpVecs], next[kLpVecs];
  float cm0 = -INFINITY, cm1 = -INFINITY;            // FEW: the lane's largest of each chunk
  if constexpr (FEW) {
    if (first < chunks) load_last(first, v);
    if (first + step < chunks) load_last(first + step, next);
    if (first < chunks) add(cm0 = W::largest(v), v);
    if (first + step < chunks) add(cm1 = W::largest(next), next);
    top = fmaxf(cm0, cm1);
  } else {
    if (first < full) load(v);
    for (int c = first; c < full; c += 2 * step) {   // the next chunk on its way while one is used
      const bool two = c + step < full;
      if (two) load(next);
      use(v);
      if (!two) break;
      if (c + 2 * step < full) load(v);
      use(next);
    }
    if (full % step == first && row.nvec > full * kLpChunk) {   // the vectors behind the last whole chunk
      load_last(full, v);
      use(v);
    }
  }
  float ze = -INFINITY;                              // the values before and behind the vectors
  int edge = -1;
  if (lead) {
    const int tail = row.head + row.nvec * N;
    edge = lane < 16 ? (lane < row.head ? lane : -1) : (tail + lane - 16 < a.V ? tail + lane - 16 : -1);
    if (edge >= 0) ze = W::get(row.z + edge);
    const float mn = fmaxf(sum.m, ze), dm = fmaxf(sum.m - mn, kFar), f = ex2_approx(dm * kL2E), d = ze - mn, e = ex2_approx(d * kL2E);
    sum = {mn, sum.s * f + e, f * (sum.a + sum.s * dm) + e * fmaxf(d, kFar)};
  }
  float reached = 0.0f;                              // by K threads' largest logits; -inf: fewer of them are more than that
  if (K) {
    // Blocks take the same time for their rows and so come to this part together, in which nothing is read: the first
    // chunks of a row that comes next are fetched into L2 meanwhile.
    if (NC == 1 && !FEW && lane < 4 && m + a.ahead < a.M) {
      const Row<T> later(a.z, a.ld, a.V, m + a.ahead);
      const int c = first + lane * step;
      const uint4* chunk = reinterpret_cast<const uint4*>(later.z + later.head) + static_cast<long long>(c) * kLpChunk;
      if (c < later.nvec / kLpChunk) prefetch_l2(chunk, kLpChunk * 16);
    }
    if (!FEW && in_group) {
      s_max[group++][threadIdx.x] = noted;
      top = fmaxf(top, noted);
    }
    if ((WR == 1 || warp == 0) && lane == 0) s_count[team] = 0;   // (of every block of a cluster)
    if constexpr (WR == 1) {
      float order = sorted_values(top, lane);
      if constexpr (FEW) {
        if (K > kLpFewTop) {                         // of two numbers a lane, as 32 do not let enough be left out
          float a = cm0, b = cm1;
          if (chunks < 2) {                          // (of few vectors, of which some lanes have none)
            a = b = -INFINITY;
#pragma unroll
            for (int k = 0; k < kLpVecs; ++k) {
              const float2 x = W::halves(v[k]);
              a = fmaxf(a, x.x);
              b = fmaxf(b, x.y);
            }
          }
          order = join_values(sorted_values(a, lane), sorted_values(b, lane), lane);
        }
      }
      reached = __shfl_sync(kAll, order, K - 1);
      __syncwarp();
    } else {
      if (K <= kLpFewTop) {
        float left = top, mine = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float most = warp_max(left);
          if (lane == k) mine = most;
          if (lane == __ffs(__ballot_sync(kAll, left == most)) - 1) left = -INFINITY;
        }
        if (lane < 4) s_order[0][4 * warp + lane] = mine;
        __syncthreads();
        const float x = s_order[0][lane];
        int at = 0;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const float4 y = *reinterpret_cast<const float4*>(&s_order[0][k]);
          at += (y.x > x || (y.x == x && k < lane)) + (y.y > x || (y.y == x && k + 1 < lane)) +
                (y.z > x || (y.z == x && k + 2 < lane)) + (y.w > x || (y.w == x && k + 3 < lane));
        }
        reached = __shfl_sync(kAll, x, __ffs(__ballot_sync(kAll, at == K - 1)) - 1);
      }
      if (K > kLpFewTop || reached == -INFINITY) {   // (too few warps have a chunk, 16 x 2,500 with K = 16 9.4 and 4.5 us; or a mask)
        if (K <= kLpFewTop) __syncthreads();         // the four of every warp are read
        float order = sorted_values(top, lane);
        s_order[warp][lane] = order;
        __syncthreads();
#pragma unroll
        for (int half = kLpWarps / 2; half; half >>= 1) {
          if (warp < half) s_order[warp][lane] = order = join_values(order, s_order[warp + half][lane], lane);
          __syncthreads();
        }
        reached = s_order[0][K - 1];
      }
    }
  }
  // The chunks that may hold a token which passes: passes(a largest logit, the first index of its chunk), use(their 16-byte
  // vectors, one thread's chunk a lane; whether there is one, its largest logit, its number and its thread).
  auto each_chunk = [&](auto&& passes, auto&& use) {
    if constexpr (FEW) {
      if (__any_sync(kAll, cm0 >= reached)) use(v, first < chunks, cm0, first, lane);
      if (__any_sync(kAll, cm1 >= reached)) use(next, first + step < chunks, cm1, first + step, lane);
    } else if (__any_sync(kAll, top >= reached)) {
      // what is read again: as many at once as there are lanes, so that they travel together
      int items = 0, item_chunk = 0, item_lane = 0;
      auto look = [&]() {
#pragma unroll
        for (int k = 0; k < kLpVecs; ++k) {
          const int i = item_chunk * kLpChunk + k * 32 + item_lane;
          v[k] = make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
          if (lane < items && i < row.nvec) v[k] = __ldg(vecs + i);
        }
        use(v, lane < items, W::largest(v), item_chunk, item_lane);
        items = 0;
      };
      for (int g = 0; g < group; ++g) {
        const float most = s_max[g][threadIdx.x];
        if (!__any_sync(kAll, most >= reached)) continue;
        for (int c = first + g * per * step; c < min(chunks, first + (g + 1) * per * step); c += step) {
          unsigned who = __ballot_sync(kAll, passes(most, row.head + (c * kLpChunk + lane) * N));
          while (who) {
            if (lane == items) {
              item_chunk = c;
              item_lane = __ffs(who) - 1;
            }
            who &= who - 1;
            if (++items == 32) look();
          }
        }
      }
      if (items) look();
    }
  };
  // The warp's best tokens, in order, from its chunks.
  auto search = [&]() {
    Key floor_key = (key_of(reached, 0) >> 32) << 32;   // what a token has to pass
    // Puts the lanes' keys that pass into the list, one by one.
    auto insert = [&](Key key) {
      unsigned who = __ballot_sync(kAll, key > floor_key);
#pragma unroll 1
      while (who) {
        const Key k = __shfl_sync(kAll, key, __ffs(who) - 1);
        const int n = __popc(__ballot_sync(kAll, best > k));
        const Key up = __shfl_up_sync(kAll, best, 1);
        best = lane > n ? up : lane == n ? k : best;
        const Key last = __shfl_sync(kAll, best, K - 1);
        if (last > floor_key) floor_key = last;
        who &= who - 1;
        who &= __ballot_sync(kAll, key > floor_key);
      }
    };
    each_chunk([&](float most, int index) { return key_of(most, index) > floor_key; },
               [&](const uint4 (&x)[kLpVecs], bool some, float cm, int chunk, int thread) {
      const Key best_here = some ? key_of(cm, row.head + (chunk * kLpChunk + thread) * N) : 0;
      unsigned who = __ballot_sync(kAll, best_here > floor_key);
      if (__popc(who) > K) {
        // K of them have a value at least as large as the K-th of their largest ones: nothing below it is wanted
        const Key k = (key_of(__shfl_sync(kAll, sorted_values(some ? cm : -INFINITY, lane), K - 1), 0) >> 32) << 32;
        if (k > floor_key) floor_key = k;
        who &= __ballot_sync(kAll, best_here > floor_key);
      }
      if (!who) return;
#pragma unroll
      for (int k = 0; k < kLpVecs; ++k) s_stage[warp][lane][k] = x[k];
      __syncwarp();
      while (who) {
        const int from = __ffs(who) - 1;
        who &= who - 1;
        const int j = lane % VALUES;                 // this lane's value of that chunk's
        const float z = W::get(reinterpret_cast<const T*>(&s_stage[warp][from][0]) + j);
        const int vec = __shfl_sync(kAll, chunk, from) * kLpChunk + (j / N) * 32 + __shfl_sync(kAll, thread, from);
        insert(lane < VALUES && vec < row.nvec ? key_of(z, row.head + vec * N + j % N) : 0);
        who &= __ballot_sync(kAll, best_here > floor_key);
      }
      __syncwarp();                                  // the stage is read before it is filled again
    });
    if (lead) insert(edge >= 0 ? key_of(ze, edge) : 0);
  };
  // Up to kLpPool tokens in any order to one warp: each one's place is the number of larger ones. (Reading them all costs a
  // third of joining eight lists, whose three steps wait for one another.)
  auto ranked = [&](const Key* pool, int n) {
    const Key x = lane < n ? pool[lane] : 0, y = lane + 32 < n ? pool[lane + 32] : 0;
    int at_x = 0, at_y = 0;
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const Key z = pool[k];
      at_x += z > x;
      at_y += z > y;
    }
    s_best[team][lane] = 0;
    __syncwarp();
    if (x && at_x < 32) s_best[team][at_x] = x;
    if (y && at_y < 32) s_best[team][at_y] = y;
    __syncwarp();
    best = s_best[team][lane];
  };
  // Without a floor every token would go to the pool, more than it holds (4,096 x 50,257 in fp32, K = 10, of which a mask leaves 8:
  // 571 us by way of the pool, so 180).
  const bool no_floor = K && reached == -INFINITY && a.V > kLpPool;
  if (K && !no_floor) {
    // Every token that reaches it, in any order: as a rule K of them and a few more.
    const uint32_t room = smem_u32(&s_pool[team][0]);
    auto put = [&](bool hit, int place, float z, int index) {
      asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.shared.b64 [%1], %2;\n\t}" ::"r"(
                       static_cast<int>(hit && static_cast<unsigned>(place) < kLpPool)),
                   "r"(room + 8 * static_cast<uint32_t>(place)), "l"(key_of(z, index))
                   : "memory");
    };
    each_chunk([&](float most, int) { return most >= reached; },
               [&](const uint4 (&x)[kLpVecs], bool some, float cm, int chunk, int thread) {
      unsigned which = 0;                            // this lane's vectors with such a token
      if (some && cm >= reached) {
#pragma unroll
        for (int k = 0; k < kLpVecs; ++k)
          if (chunk * kLpChunk + k * 32 + thread < row.nvec && W::most(x[k]) >= reached) which |= 1u << k;
      }
      // Each lane its own one after the other, but where a warp has the row to itself any lane's: of 200 rows of 500 some have a
      // lane with three, which took 5.7 us instead of 3.5. (A block's warps have fewer to go through: 4,096 x 50,257 in bf16
      // with K = 8 83 us, with any lane's 86.)
      unsigned left = WR == 1 ? __reduce_or_sync(kAll, which) : which;
#pragma unroll 1
      while (left) {
        const int k = __ffs(left) - 1, index = row.head + (chunk * kLpChunk + k * 32 + thread) * N;
        left &= left - 1;
        uint4 y = x[0];
#pragma unroll
        for (int i = 1; i < kLpVecs; ++i)
          if (i == k) y = x[i];
        unsigned hits = 0;
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float2 z = W::pair(y, j);
          if (z.x >= reached) hits |= 1u << (2 * j);
          if (z.y >= reached) hits |= 2u << (2 * j);
        }
        if (WR == 1 && !((which >> k) & 1u)) hits = 0;
        int place = 0;
        if (hits) place = atomicAdd(&s_count[team], __popc(hits));
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const bool hit = (hits >> j) & 1u;
          put(hit, place, j & 1 ? W::pair(y, j / 2).y : W::pair(y, j / 2).x, index + j);
          place += hit;
        }
      }
    });
    if (edge >= 0 && ze >= reached) put(true, atomicAdd(&s_count[team], 1), ze, edge);
    __syncwarp();
  }
  if constexpr (WR == 1) {
    if (K) {
      const int n = no_floor ? kLpPool + 1 : s_count[team];
      if (n <= kLpPool) ranked(s_pool[team], n);
      else search();                                 // (many equal ones, or many large ones in few lanes)
    }
  }
  auto shuffled = [&](const Sums& x, int k) {
    return joined_sums(x, {__shfl_xor_sync(kAll, x.m, k), __shfl_xor_sync(kAll, x.s, k), __shfl_xor_sync(kAll, x.a, k)});
  };
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) sum = shuffled(sum, k);
  if constexpr (WR > 1) {
    // Lists in shared memory to all warps, joined two by two: the larger of each pair of opposite ends is a bitonic sequence of
    // the best 32, sorted in five steps.
    auto join_all = [&](Key (*list)[32], int n) {
#pragma unroll
      for (int half = 4; half; half >>= 1) {
        if (n > half) {
          if (warp < half && warp + half < n) list[warp][lane] = join_lists(list[warp][lane], list[warp + half][lane], lane);
          __syncthreads();
        }
      }
      best = list[0][lane];
    };
    auto join_sums = [&](const Sums* sums, int n) {
      sum = (lane & 7) < n ? sums[lane & 7] : Sums{kLowest, 0.0f, 0.0f};
#pragma unroll
      for (int k = 1; k < 8; k <<= 1) sum = shuffled(sum, k);
    };
    if (lane == 0) s_sums[warp] = sum;
    __syncthreads();
    if (K) {
      const int n = no_floor ? kLpPool + 1 : s_count[0];
      if (n <= kLpPool) {
        if (warp == 0) ranked(s_pool[0], n);
      } else {                                       // (many equal ones, or many large ones in few threads)
        search();
        s_list[warp][lane] = best;
        __syncthreads();
        join_all(s_list, kLpWarps);
      }
    }
    if (warp == 0) join_sums(s_sums, kLpWarps);
    if constexpr (NC > 1) {
      const bool pool = NC * K <= kLpPool;
      auto cluster = cg::this_cluster();
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      if (warp == 0) {
        if (K && !pool) *cluster.map_shared_rank(&s_lists[part][lane], 0) = best;
        if (lane < K && pool) *cluster.map_shared_rank(&s_pool[1][part * K + lane], 0) = best;
        if (lane == 0) *cluster.map_shared_rank(&s_parts[part], 0) = sum;
      }
      cluster.sync();
      if (part) return;
      if (K) {
        if (!pool) join_all(s_lists, NC);
        else if (warp == 0) ranked(s_pool[1], NC * K);
      }
      if (warp == 0) join_sums(s_parts, NC);
    }
    if (warp) return;
  }
  const bool fine = sum.s > 0.0f && sum.s < INFINITY;   // a finite log-sum-exp
  const float ln_s = logf(sum.s), nan = __int_as_float(0x7fffffff);
  if (lane == 0) {
    if (a.logp) a.logp[m] = target < 0 && fine ? 0.0f : fine ? (zt - sum.m) - ln_s : nan;
    if (a.entropy) a.entropy[m] = fine ? ln_s - sum.a / sum.s : nan;
    if (a.stats) *reinterpret_cast<float2*>(a.stats + 2 * m) = fine ? make_float2(sum.m, sum.s) : make_float2(nan, nan);
  }
  if (lane < K) {
    a.top_ids[m * K + lane] = fine ? index_of(best) : -1;
    a.top_logp[m * K + lane] = fine ? (value_of(best) - sum.m) - ln_s : nan;
  }
}

// dz = dlogp (1[j = t] - p) - dentropy p (ln p + entropy), from (m, S): p = e^d / S. Bound by memory: the logits once in,
// once out. A block takes 256 x kGradVecs vectors of a row, two values to an instruction (4,096 x 50,257 in bf16, both calls
// 193 us, one to an instruction 197; eight vectors a thread 192). The last rows come first: they are what the call that made
// (m, S) has left in L2 (the other order took 4 us more; streaming loads or stores 5 to 10).
constexpr int kGradVecs = 4;

struct LpGrad {
  const void* z;
  const int32_t* targets;
  const float *stats, *entropy, *dlogp, *dentropy;
  void* dz;
  long long ld, dld, M;
  int V, segments;     // blocks a row
};

template <typename T>
__global__ void __launch_bounds__(256)
logprobs_grad_kernel(LpGrad a) {
  using W = Vec<T>;
  constexpr int N = W::N;
  pdl_wait();
  pdl_trigger();
  for (long long u = blockIdx.x; u < a.M * a.segments; u += gridDim.x) {
    const long long up = u / a.segments, m = a.M - 1 - up;
    const int seg = static_cast<int>(u - up * a.segments);
    const Row<T> row(a.z, a.ld, a.V, m);
    T* out = static_cast<T*>(a.dz) + m * a.dld;
    const uint4* vecs = reinterpret_cast<const uint4*>(row.z + row.head);
    const long long v0 = static_cast<long long>(seg) * 256 * kGradVecs + threadIdx.x;
    uint4 v[kGradVecs];
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k)
      if (v0 + k * 256 < row.nvec) v[k] = vecs[v0 + k * 256];
    const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * m);
    const float h = a.entropy ? __ldg(a.entropy + m) : 0.0f, ge = a.dentropy ? __ldg(a.dentropy + m) : 0.0f;
    int t = a.targets ? __ldg(a.targets + m) : -1;
    if (static_cast<unsigned>(t) >= static_cast<unsigned>(a.V)) t = -1;
    const float g = t >= 0 && a.dlogp ? __ldg(a.dlogp + m) : 0.0f;
    // dz = e^d (c - ge d) / S with c = -g - ge (entropy - ln S); 1 / S goes into both factors of the row
    const float inv = 1.0f / st.y, c = (-g - ge * (h - logf(st.y))) * inv;
    const float2 off = make_float2(-st.x, -st.x), l2e = make_float2(kL2E, kL2E);
    const float2 slope = make_float2(-ge * inv, -ge * inv), base = make_float2(c, c);
    auto grad = [&](const float2& z) {
      const float2 d = add2_rn(z, off), x = mul2_rn(d, l2e);
      return mul2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)),
                     fma2_rn(make_float2(fmaxf(d.x, kFar), fmaxf(d.y, kFar)), slope, base));
    };
    const bool same = ((reinterpret_cast<uintptr_t>(row.z) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      const long long i = v0 + k * 256;
      if (i >= row.nvec) continue;
      const int index = row.head + static_cast<int>(i) * N;
      float x[N];
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float2 dz = grad(W::pair(v[k], j));
        x[2 * j] = dz.x;
        x[2 * j + 1] = dz.y;
      }
      if (static_cast<unsigned>(t - index) < static_cast<unsigned>(N) && t >= 0) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (t - index == j) x[j] += g;
      }
      if (same) {
        *reinterpret_cast<uint4*>(out + index) = W::pack(x);
      } else {                                       // rows of the gradient that start elsewhere in their 16 bytes
#pragma unroll
        for (int j = 0; j < N; ++j) W::put(out + index + j, x[j]);
      }
    }
    if (seg == 0 && threadIdx.x < 32) {              // the values before and behind the vectors
      const int lane = threadIdx.x, tail = row.head + row.nvec * N;
      const int index = lane < 16 ? (lane < row.head ? lane : -1) : (tail + lane - 16 < a.V ? tail + lane - 16 : -1);
      if (index >= 0) {
        const float z = W::get(row.z + index);
        W::put(out + index, grad(make_float2(z, z)).x + (index == t ? g : 0.0f));
      }
    }
  }
}

template <typename T, int NC, int WR, bool FEW, bool TOP>
cudaError_t launch_rows(const LpArgs& a, int* err, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(WR == 1 ? (a.M + kLpWarps - 1) / kLpWarps : a.M * NC));
  cfg.blockDim = dim3(32 * kLpWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {NC, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = NC > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, NC, WR, FEW, TOP>, a, err);
}

template <typename T, int NC, int WR = kLpWarps>
cudaError_t launch_form(const LpArgs& a, long long chunks, int* err, cudaStream_t s) {
  const bool few = chunks <= 2 * NC * WR;
  if (NC == 1 && !a.K) return few ? launch_rows<T, NC, WR, true, NC != 1>(a, err, s) : launch_rows<T, NC, WR, false, NC != 1>(a, err, s);
  return few ? launch_rows<T, NC, WR, true, true>(a, err, s) : launch_rows<T, NC, WR, false, true>(a, err, s);
}

template <typename T>
cudaError_t launch_logprobs_of(LpArgs a, int* err, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const long long chunks = (static_cast<long long>(a.V) / Vec<T>::N + kLpChunk - 1) / kLpChunk;
  a.ahead = 4 * sms;                                 // (four blocks an SM)
  // A warp a row where its whole row is two chunks, or the rows are short and many and not too many tokens are wanted. Against a
  // block a row (graph replays): 4,096 x 500 with K = 5 7.1 us and 42; 4,096 x 5,000 in fp32 with K = 0 14.6 and 18.6, with K = 5 22.5
  // and 30.7, with K = 16 25.7 and 32.9, but with K = 32, where 32 lanes' largest logits make a low floor, 87 and 35; 4,096 x 10,000
  // in bf16 with K = 5 25 and 45; 1,216 x 1,600 in fp32 6.3 and 8.2, 1,216 x 5,000 11.7 and 10.2, 620 x 5,000 8.2 and 7.1; 1,500 x 8,000
  // in fp32 with K = 0, 16 chunks, 12.5 and 10.9.
  // Clusters of as many blocks as keep all of them at work at once.
  if (chunks <= 2 || (chunks <= 10 && a.M >= 8LL * sms && a.K <= kLpFewTop)) {
    a.ahead *= kLpWarps;
    return launch_form<T, 1, 1>(a, chunks, err, s);
  }
  if (8 * a.M <= 2 * sms && chunks > 4 * kLpWarps) return launch_form<T, 8>(a, chunks, err, s);
  if (4 * a.M <= 2 * sms && chunks > 2 * kLpWarps) return launch_form<T, 4>(a, chunks, err, s);
  if (2 * a.M <= 2 * sms && chunks > kLpWarps) return launch_form<T, 2>(a, chunks, err, s);
  return launch_form<T, 1>(a, chunks, err, s);
}

template <typename T>
cudaError_t launch_grad_of(LpGrad a, cudaStream_t s) {
  a.segments = (a.V / Vec<T>::N + 256 * kGradVecs - 1) / (256 * kGradVecs);
  if (a.segments < 1) a.segments = 1;
  const long long units = a.M * a.segments;
  return launch_k(logprobs_grad_kernel<T>, dim3(static_cast<unsigned>(units < 0x7fffffffLL ? units : 0x7fffffffLL)), dim3(256),
                  0, s, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobRows& x, float* logp, float* entropy, float* stats, int32_t* top_ids,
                            float* top_logp, int K, int* err, cudaStream_t s) {
  LpArgs a = {};
  a.z = x.logits;
  a.targets = x.targets;
  a.logp = logp;
  a.entropy = entropy;
  a.stats = stats;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.ld = x.ld;
  a.M = x.M;
  a.V = x.V;
  a.K = K;
  return x.bf16 ? launch_logprobs_of<__nv_bfloat16>(a, err, s) : launch_logprobs_of<float>(a, err, s);
}

cudaError_t launch_logprobs_bwd(const LogprobRows& x, const float* stats, const float* entropy, const float* dlogp,
                                const float* dentropy, void* dlogits, int64_t dld, cudaStream_t s) {
  LpGrad a = {};
  a.z = x.logits;
  a.targets = x.targets;
  a.stats = stats;
  a.entropy = entropy;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.dz = dlogits;
  a.ld = x.ld;
  a.dld = dld;
  a.M = x.M;
  a.V = x.V;
  return x.bf16 ? launch_grad_of<__nv_bfloat16>(a, s) : launch_grad_of<float>(a, s);
}

}  // namespace gptgb
