// Position rotation of fused rows, alone or on the way into a paged cache of 16-bit or 4-bit rows, and 4-bit rows read back.
//
// Rotation: pair i of the first `rot` values of every query and key head turns by n f_i at position n. Phases are counted
// in turns as 64-bit fractions: turns[i] = f_i / (2 pi) * 2^64 (mod 2^64), so n turns[i] mod 2^64 is the phase of any
// position without rounding (one fp32 product n f_i is off by 2^-25 n f_i: 0.03 rad at position 1,000,000), and 32 bits
// of it go through sincospif. The map is orthogonal: its gradient is the rotation back (sin of the other sign).
//
// A 4-bit row: of its D values the lowest (bf16) and scale = bf16((highest - lowest) / 15), and a code
// min(15, round((x - lowest) / scale)) per value, value 2 j low in byte j. Every step is one rounding in fp32 (1 / scale
// and the products included), so that the same row always gives the same codes. Codes [pages][2][Hkv][page][D / 2] bytes,
// ranges [pages][2][Hkv][page] pairs (scale, lowest).
//
// All three kernels are bound by memory and give a warp one token (or part of one): a lane holds 16 values of a head, two
// 16-byte units that contain each other's pair partners, D / 16 lanes a head. Neighbouring lanes hold neighbouring units, so
// that each load and store covers whole 32-byte sectors (with units 2 i and 2 i + 1 in lane i the L2 moved 1.6 times the bytes:
// 16 x up to 1,024 tokens into 4 bits and back 41 us, now 35.8). A lane computes the sine and cosine of one pair for the whole
// warp, once per token. Eight blocks an SM, with the loads of two steps of heads in flight: 16 x up to 1,024 tokens of 12 heads
// into bf16 pages and rows 27.5 us (155 MB, 5.6 TB/s, 0.84 of a copy's rate); with 6 or 5 blocks 29.0 and 30.5, with 10, whose
// registers spill, 32.8, with one step in flight 29.7. Into 4 bits the instructions count as much (63 % of the issue slots).
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "paged.cuh"

#include <math.h>

namespace gptgb {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kAppendWarps = 4;

struct Row16 {          // 16 values of a head: units u0 and u1
  uint4 a, b;
};

// cs, sn: of pairs 0-3 of unit a and of unit b where they lie side by side, else of the eight pairs that a's values form with b's.
// ta, tb: whether unit a, or b, is turned (apart, only where pairs lie side by side).
__device__ __forceinline__ void turn16(Row16& x, const float (&cs)[8], const float (&sn)[8], bool interleaved, bool ta, bool tb) {
  uint32_t* a = &x.a.x;
  uint32_t* b = &x.b.x;
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 p = unpack_bf16x2(a[k]), q = unpack_bf16x2(b[k]);
      if (ta) a[k] = pack_bf16x2(p.x * cs[k] - p.y * sn[k], p.y * cs[k] + p.x * sn[k]);
      if (tb) b[k] = pack_bf16x2(q.x * cs[4 + k] - q.y * sn[4 + k], q.y * cs[4 + k] + q.x * sn[4 + k]);
    }
  } else if (ta) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 p = unpack_bf16x2(a[k]), q = unpack_bf16x2(b[k]);
      a[k] = pack_bf16x2(p.x * cs[2 * k] - q.x * sn[2 * k], p.y * cs[2 * k + 1] - q.y * sn[2 * k + 1]);
      b[k] = pack_bf16x2(q.x * cs[2 * k] + p.x * sn[2 * k], q.y * cs[2 * k + 1] + p.y * sn[2 * k + 1]);
    }
  }
}

// The codes of a unit's eight values. v * inv + 2^23 leaves the rounded code in the low bits of the sum (ties to even, as
// rintf); the bits above it cancel in the subtraction. (The largest value's code is 15: its quotient is off by the scale's
// rounding, 15 (1 + 2^-8) at most.)
__device__ __forceinline__ uint32_t codes8(const uint4& x, float low, float inv) {
  const uint32_t* a = &x.x;
  const float2 neg = make_float2(-low, -low), by = make_float2(inv, inv);
  const float m = 8388608.0f;
  uint32_t w = 0u - 0xfb000000u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 n = mul2_rn(add2_rn(unpack_bf16x2(a[k]), neg), by);
    // (a packed sum here would be joined with the product, and the product not rounded)
    w += __float_as_uint(__fadd_rn(n.x, m)) * (1u << (8 * k)) + __float_as_uint(__fadd_rn(n.y, m)) * (16u << (8 * k));
  }
  return w;
}

// Scale and lowest value of a row whose values lie in the LANES lanes around this one (bf16 pair), and 1 / scale; a row
// with a value that is not finite, or a range past fp32, is NaN throughout. A scale below the normal numbers counts as 0.
template <int LANES>
__device__ __forceinline__ uint32_t range_of(const Row16& x, float* low, float* inv) {
  const __nv_bfloat162* a = reinterpret_cast<const __nv_bfloat162*>(&x.a.x);
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&x.b.x);
  __nv_bfloat162 mn = __hmin2_nan(a[0], b[0]), mx = __hmax2_nan(a[0], b[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    mn = __hmin2_nan(mn, __hmin2_nan(a[k], b[k]));
    mx = __hmax2_nan(mx, __hmax2_nan(a[k], b[k]));
  }
  // (largest, -lowest) side by side
  __nv_bfloat162 both = __hmax2_nan(__halves2bfloat162(__low2bfloat16(mx), __hneg(__low2bfloat16(mn))),
                                    __halves2bfloat162(__high2bfloat16(mx), __hneg(__high2bfloat16(mn))));
#pragma unroll
  for (int k = 1; k < LANES; k <<= 1) both = __hmax2_nan(both, __shfl_xor_sync(kAll, both, k));
  const float hi = __low2float(both), lo = -__high2float(both);
  const float range = hi - lo;
  float scale = __bfloat162float(__float2bfloat16(__fmul_rn(range, 1.0f / 15.0f)));
  *low = lo;
  *inv = 0.0f;
  if (!(range <= 3.402823466e38f)) return 0x7fff7fffu;
  if (scale < 1.17549435e-38f) scale = 0.0f;
  else *inv = __frcp_rn(scale);
  return pack_bf16x2(scale, lo);
}

struct AppendArgs {
  const uint4* qkv;       // [B, T, (H + 2 Hkv) D] bf16
  uint4* out;             // the same, rotated; qkv itself: in place; nullptr: not wanted
  const int32_t *start, *count, *pos;
  const unsigned long long* turns;   // [rot / 2]; nullptr: no rotation
  uint32_t* ranges;       // 4-bit rows' (scale, lowest)
  long long tokens;       // B T
  int T, H, Hkv, rot, interleaved, inverse;
  int parts;              // warps that share a token
};

// MODE 0: rotation alone; 1: keys and values into c.pool (bf16); 2: into c.pool (codes) and a.ranges.
template <int D, int MODE>
__global__ void __launch_bounds__(kAppendWarps * 32, 8)
append_kernel(PagedCache c, AppendArgs a, int* err) {
  constexpr int U = D / 8, LANES = D / 16, HEADS = 32 / LANES;   // units and lanes of a head, heads side by side
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * kAppendWarps + warp;
  const unsigned tok = w / static_cast<unsigned>(a.parts), part = w - tok * a.parts;
  if (tok >= a.tokens) return;
  const int b = static_cast<int>(tok / static_cast<unsigned>(a.T)), t = static_cast<int>(tok - static_cast<unsigned>(b) * a.T);
  // (on their way together)
  const int count = MODE != 0 && a.count ? __ldg(a.count + b) : a.T;
  const long long first = MODE != 0 && a.start ? __ldg(a.start + b) : 0;
  const long long position = a.pos ? static_cast<long long>(__ldg(a.pos + b)) : first;
  const unsigned long long turn = lane < a.rot / 2 ? __ldg(a.turns + lane) : 0;
  if (t >= count || first < 0) return;               // behind the tokens; no sequence
  // This lane's head (of HEADS side by side) and its two units: i and i + LANES, but of heads that are turned with partners
  // rot / 2 apart, units i and i + rot / 16 in the first rot / 16 lanes, and those behind the first rot values in the others.
  const int i = lane % LANES, hh = lane / LANES, pairs = a.rot / 2, apart = a.rot / 16;
  const bool beyond = i >= apart;
  const int u0 = i, u1 = i + LANES;
  const int t0 = a.interleaved ? i : beyond ? i + apart : i;
  const int t1 = a.interleaved ? u1 : beyond ? i + LANES : i + apart;
  const int c0 = a.interleaved ? 4 * i : 8 * i, c1 = a.interleaved ? 4 * u1 : 8 * i + 4;   // pairs of the first four and the last
  const bool ta = c0 < pairs, tb = c1 < pairs, turns = ta || tb;
  const int NH = a.H + 2 * a.Hkv, heads = a.H + a.Hkv;
  const size_t base = static_cast<size_t>(tok) * NH * U;
  const uint4* src = a.qkv + base;
  uint4* dst = a.out ? a.out + base : nullptr;
  const bool in_place = a.out == a.qkv;
  const long long r = first + t;
  long long row = -1;                                // of the key of head 0 in the pool
  size_t weight = 0;
  if (MODE != 0) {
    if (r >= static_cast<long long>(c.max_pages) << c.page_log2) {
      record_error(err, GPT_DEV_EPAGE);
    } else {
      const int pg = page_of(c, c.table + static_cast<size_t>(b) * c.max_pages, static_cast<int>(r), err);
      const int slot = static_cast<int>(r) & ((1 << c.page_log2) - 1);
      if (pg >= 0) {
        row = static_cast<long long>(row_at(c, pg, 0, 0, slot));
        weight = weight_at(c, pg, 0, slot);
      }
    }
  }
  float cs[8], sn[8];
  if (pairs) {
    float s, co;
    const unsigned long long phase = static_cast<unsigned long long>(position + t) * turn;
    sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &co);   // 2 / 2^32 half turns
    if (a.inverse) s = -s;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int from = ((k < 4 ? c0 : c1) + (k & 3)) & 31;
      cs[k] = __shfl_sync(kAll, co, from);
      sn[k] = __shfl_sync(kAll, s, from);
    }
  }
  // Heads [h0, h1), HEADS side by side in a step of the warp, two steps' loads in flight; those below `heads` are turned.
  auto walk = [&](int h0, int h1, auto&& use) {
    for (h0 += static_cast<int>(part) * HEADS; h0 < h1; h0 += 2 * HEADS * a.parts) {
      Row16 x[2];
      int hd[2];
      const bool two = h0 + HEADS * a.parts < h1;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        hd[k] = h0 + k * HEADS * a.parts + hh;
        if (k && !two) break;
        const int at = min(hd[k], h1 - 1);
        x[k].a = src[static_cast<size_t>(at) * U + (at < heads ? t0 : u0)];
        x[k].b = src[static_cast<size_t>(at) * U + (at < heads ? t1 : u1)];
      }
      use(x[0], hd[0], hd[0] < h1);
      if (two) use(x[1], hd[1], hd[1] < h1);
    }
  };
  auto put = [&](const Row16& x, int hd, int at0, int at1) {
    dst[static_cast<size_t>(hd) * U + at0] = x.a;
    dst[static_cast<size_t>(hd) * U + at1] = x.b;
  };
  if (dst)                                           // without an output the queries are not needed
    walk(0, a.H, [&](Row16& x, int hd, bool ok) {
      turn16(x, cs, sn, a.interleaved, ta, tb);
      if (ok && (turns || !in_place)) put(x, hd, t0, t1);
    });
  walk(a.H, MODE == 0 && in_place ? heads : NH, [&](Row16& x, int hd, bool ok) {
    const bool key = hd < heads;
    const int at0 = key ? t0 : u0, at1 = key ? t1 : u1;
    if (key) turn16(x, cs, sn, a.interleaved, ta, tb);
    if (ok && dst && ((key && turns) || !in_place)) put(x, hd, at0, at1);
    if (MODE == 0) return;
    const int e = hd - a.H;                          // key head, or Hkv + value head
    const bool stored = ok && row >= 0;
    const long long to = row + (static_cast<long long>(e) << c.page_log2);
    if (MODE == 1 && stored) {
      uint4* pool = static_cast<uint4*>(c.pool);
      pool[to * U + at0] = x.a;
      pool[to * U + at1] = x.b;
      if (c.weight && i == 0 && e < a.Hkv) c.weight[weight + (static_cast<size_t>(e) << c.page_log2)] = 0.0f;
    }
    if (MODE == 2) {
      float low, inv;
      const uint32_t range = range_of<LANES>(x, &low, &inv);
      if (stored) {
        uint32_t* codes = static_cast<uint32_t*>(c.pool) + to * U;
        const bool bad = range == 0x7fff7fffu;
        codes[at0] = bad ? 0u : codes8(x.a, low, inv);
        codes[at1] = bad ? 0u : codes8(x.b, low, inv);
        if (i == 0) a.ranges[to] = range;
      }
    }
  });
}

// Rows start[b] + t (t < count[b]) of a 4-bit cache as bf16 rows of Hkv keys, then Hkv values.
template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32)
load4_kernel(PagedCache c, const uint32_t* __restrict__ ranges, const int32_t* __restrict__ start,
             const int32_t* __restrict__ count, uint4* __restrict__ rows, long long tokens, int T, int parts, int* err) {
  constexpr int U = D / 8, LANES = D / 16, HEADS = 32 / LANES;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * kAppendWarps + warp;
  const unsigned tok = w / static_cast<unsigned>(parts), part = w - tok * parts;
  if (tok >= tokens) return;
  const int b = static_cast<int>(tok / static_cast<unsigned>(T)), t = static_cast<int>(tok - static_cast<unsigned>(b) * T);
  if (count && t >= __ldg(count + b)) return;
  const long long first = start ? __ldg(start + b) : 0, r = first + t;
  if (first < 0) return;                             // no sequence
  if (r >= static_cast<long long>(c.max_pages) << c.page_log2) {
    record_error(err, GPT_DEV_EPAGE);
    return;
  }
  const int pg = page_of(c, c.table + static_cast<size_t>(b) * c.max_pages, static_cast<int>(r), err);
  if (pg < 0) return;
  const size_t row = row_at(c, pg, 0, 0, static_cast<int>(r) & ((1 << c.page_log2) - 1));
  const int i = lane % LANES, hh = lane / LANES, NH = 2 * c.Hkv;
  const uint32_t* codes = static_cast<const uint32_t*>(c.pool);
  uint4* dst = rows + static_cast<size_t>(tok) * NH * U;
  for (int h0 = static_cast<int>(part) * HEADS; h0 < NH; h0 += 2 * HEADS * parts) {
    uint32_t x[2][2], range[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const size_t from = row + (static_cast<size_t>(min(h0 + k * HEADS * parts + hh, NH - 1)) << c.page_log2);
      x[k][0] = __ldg(codes + from * U + i);
      x[k][1] = __ldg(codes + from * U + i + LANES);
      range[k] = __ldg(ranges + from);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int hd = h0 + k * HEADS * parts + hh;
      if (hd >= NH) continue;
      const float2 f = unpack_bf16x2(range[k]);      // scale, lowest
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t v[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t two = x[k][j] >> (8 * n);
          v[n] = pack_bf16x2(fmaf(f.x, static_cast<float>(two & 15u), f.y), fmaf(f.x, static_cast<float>((two >> 4) & 15u), f.y));
        }
        dst[static_cast<size_t>(hd) * U + i + j * LANES] = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

// Warps that share a token: one where the tokens alone give every SM eight warps and more, else as many as there are
// groups of heads, so that a step of a few tokens is one group a warp.
int parts_of(long long tokens, int heads, int side_by_side, int sms) {
  const int most = (heads + side_by_side - 1) / side_by_side;
  const long long want = (8LL * sms + tokens - 1) / tokens;
  return want < most ? static_cast<int>(want) : most;
}

template <int MODE>
cudaError_t launch_append(const PagedCache& c, AppendArgs a, int D, int* err, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const int heads = (a.out ? a.H : 0) + 2 * a.Hkv;
  a.parts = parts_of(a.tokens, heads, 512 / D, sms);
  const dim3 grid(static_cast<unsigned>((a.tokens * a.parts + kAppendWarps - 1) / kAppendWarps)), block(32 * kAppendWarps);
  if (D == 64) return launch_k(append_kernel<64, MODE>, grid, block, 0, s, c, a, err);
  return launch_k(append_kernel<32, MODE>, grid, block, 0, s, c, a, err);
}

AppendArgs append_args(const RotaryRows& x, const int32_t* start, const int32_t* count, void* ranges) {
  AppendArgs a = {};
  a.qkv = static_cast<const uint4*>(x.qkv);
  a.out = static_cast<uint4*>(x.out);
  a.start = start;
  a.count = count;
  a.pos = x.pos;
  a.turns = reinterpret_cast<const unsigned long long*>(x.turns);
  a.ranges = static_cast<uint32_t*>(ranges);
  a.tokens = static_cast<long long>(x.B) * x.T;
  a.T = x.T;
  a.H = x.H;
  a.Hkv = x.Hkv;
  a.rot = x.turns ? x.rot : 0;
  a.interleaved = x.interleaved;
  a.inverse = x.inverse;
  return a;
}

}  // namespace

cudaError_t launch_rotary(const RotaryRows& x, cudaStream_t s) {
  return launch_append<0>(PagedCache{}, append_args(x, nullptr, nullptr, nullptr), x.D, nullptr, s);
}

cudaError_t launch_paged_append(const PagedCache& c, const RotaryRows& x, const int32_t* start, const int32_t* count,
                                int* err, cudaStream_t s) {
  return launch_append<1>(c, append_args(x, start, count, nullptr), x.D, err, s);
}

cudaError_t launch_paged_append4(const PagedCache& c, void* ranges, const RotaryRows& x, const int32_t* start,
                                 const int32_t* count, int* err, cudaStream_t s) {
  return launch_append<2>(c, append_args(x, start, count, ranges), x.D, err, s);
}

cudaError_t launch_paged_load4(const PagedCache& c, const void* ranges, const int32_t* start, const int32_t* count,
                               void* rows, int B, int T, int D, int* err, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const long long tokens = static_cast<long long>(B) * T;
  const int parts = parts_of(tokens, 2 * c.Hkv, 512 / D, sms);
  const dim3 grid(static_cast<unsigned>((tokens * parts + kAppendWarps - 1) / kAppendWarps)), block(32 * kAppendWarps);
  const uint32_t* r = static_cast<const uint32_t*>(ranges);
  uint4* out = static_cast<uint4*>(rows);
  if (D == 64) return launch_k(load4_kernel<64>, grid, block, 0, s, c, r, start, count, out, tokens, T, parts, err);
  return launch_k(load4_kernel<32>, grid, block, 0, s, c, r, start, count, out, tokens, T, parts, err);
}

}  // namespace gptgb
