// Keys and values into a paged cache held in 4 bits, queries and keys normed and
// rotated on the way, and the cache's values back in 16 bits.
//
// Mathematics.  Norm and rotation are those of attn_rope.cu.  A row of D elements
// of the input type (of a key: what norm and rotation leave, rounded to it) is cut into
// groups of G = min(D, 64).  With a group's minimum m and maximum M,
//     s = the smallest number of the input type with 15 s >= M - m,
//     c_d = round((x_d - m) / s), ties to even, 0 where s is 0;
// the cache stands for s c_d + m, at most s / 2 from x_d.  (Where 15 s + m would pass the
// type's largest number, s is the next one below.)  A group with an element that is
// not finite, or whose spread passes FP32, gets the scale NaN and reads as NaN.
//
// Precision.  A code jumps where (x - m) / s passes a half, and a key's rounding to
// the input type jumps, too, so an error of 2^-24 would now and then be one of a whole step
// and the same prompt give other codes on another way.  Keys are therefore computed as
// unevaluated sums of two FP32 numbers (Dekker's and Knuth's error-free products and
// sums), off by about 2^-46, and rounded once; the quotient is rounded correctly (one
// Newton step on the reciprocal's product, after Markstein).  Queries are computed in
// FP32 and rounded once, as in attn_rope.cu.
//
// Memory bounds it for prompts: q is read and written once, k and v are read once and leave
// 9/32 of their bytes.  D/16 threads hold a row, as in attn_rope.cu, and a row's sums,
// minima and maxima take log2(D/16) shuffles each.  Blocks of q, of k and of v are apart,
// so that no warp does two kinds of work, and take turns, so that the arithmetic of k runs
// beside the traffic of q.
//
// Measured (GB300; BF16, 32 + 2 x 8 heads of 128, norm and rotation): 16 x 1000 tokens 69.4 us, of
// which q is 22 and k's two-part arithmetic 10 (51 us at the measured copy bandwidth; the
// issue slots bound it: some 230 instructions for a warp's four rows of v, 620 for k, 148 for q); 16000
// tokens of 32 + 2 x 8 heads of 64 and of 32 39.5 and 26.5 us (26.2 and 13.2 at the copy bandwidth); 999
// tokens of 16 + 2 x 4 heads of 64 4.3 us; 8 tokens 2.8 us, the launch and the chain slot -> page.
// Unpacking the 16000 tokens' keys takes 8.2 us (6.2 at the copy bandwidth).
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "launchers.h"
#include "cache_ptx.cuh"
#include "rope_device.cuh"

namespace etattn {

namespace {

constexpr int kAppendThreads = 128;  // (16000 tokens: 68.4 us; 256: 71.3, 64: 72.7)

// hi + lo, |lo| at most half a step of hi.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Two two_product(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
// hi + lo for |hi| well above |lo|
__device__ __forceinline__ Two renormed(float hi, float lo) {
  const float s = __fadd_rn(hi, lo);
  return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ Two operator+(const Two& a, const Two& b) {
  const Two s = two_sum(a.hi, b.hi);
  return renormed(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
// 1 / sqrt(x): with y near it and e = 1 - x y^2, y (1 + e/2 + 3 e^2 / 8).
__device__ __forceinline__ Two two_rsqrt(const Two& x) {
  const float y = rsqrtf(x.hi);
  const Two s = two_product(y, y);
  const float e = __fmaf_rn(-x.lo, s.hi, __fmaf_rn(-x.hi, s.lo, __fmaf_rn(-x.hi, s.hi, 1.f)));
  return renormed(y, __fmul_rn(y, __fmul_rn(e, __fmaf_rn(e, 0.375f, 0.5f))));
}
// The same on pairs of numbers (paired FP32 arithmetic has no subtraction).
constexpr uint64_t kMinusOnes = 0xbf800000bf800000ull;
__device__ __forceinline__ uint64_t sub_pair(uint64_t a, uint64_t b) { return fma_pair(b, kMinusOnes, a); }
__device__ __forceinline__ void two_sum_pair(uint64_t a, uint64_t b, uint64_t& hi, uint64_t& lo) {
  hi = add_pair(a, b);
  const uint64_t bb = sub_pair(hi, a);
  lo = add_pair(sub_pair(a, sub_pair(hi, bb)), sub_pair(b, bb));
}
// The sum rounded to odd, so that rounding it on to 16 bits is rounding once.
__device__ __forceinline__ float to_odd(float hi, float lo) {
  const uint32_t b = __float_as_uint(hi);
  if (lo == 0.f || (b & 1u)) return hi;
  return __uint_as_float(((b ^ __float_as_uint(lo)) >> 31) ? b - 1u : b | 1u);
}

// The smaller of two pairs of 16-bit values, keeping a NaN; and a pair with its signs
// turned.  A group's minimum and maximum travel as the pair (min, -max).
template <bool BF16>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (min, -max) of the eight values in four words.
template <bool BF16>
__device__ __forceinline__ uint32_t extremes(const uint32_t* w) {
  constexpr uint32_t kSigns = 0x80008000u;
  const uint32_t lo = min_pair<BF16>(min_pair<BF16>(w[0], w[1]), min_pair<BF16>(w[2], w[3]));
  const uint32_t hi = min_pair<BF16>(min_pair<BF16>(w[0] ^ kSigns, w[1] ^ kSigns), min_pair<BF16>(w[2] ^ kSigns, w[3] ^ kSigns));
  return min_pair<BF16>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
}

template <bool BF16>
__device__ __forceinline__ float from16(uint32_t b) {
  float x, unused;
  if (BF16) unpack_bf16x2(b, x, unused);
  else unpack_f16x2(b, x, unused);
  return x;
}

// A group's scale and minimum, as the cache holds them, and what its codes need.
struct Quant {
  uint32_t word;                    // scale in the low half, minimum in the high one
  float min, scale, inverse, lift;  // scale and inverse of lift times the group; lift 0: all codes are 0
};
// From (min, -max).
template <bool BF16>
__device__ __forceinline__ Quant quant_of(uint32_t extreme) {
  float mn, mx;
  if (BF16) unpack_bf16x2(extreme, mn, mx);
  else unpack_f16x2(extreme, mn, mx);
  // The spread, and whether it is above its rounding to FP32 (in FP16 it is exact, in BF16 a
  // small minimum beside a large maximum may fall below it).
  const float span = __fsub_rn(-mx, mn);
  const bool above = BF16 && two_sum(-mx, -mn).lo > 0.f;
  // The product is off by a few 2^-24, so its rounding by a step of the 16-bit type at
  // most; 15 s is exact in FP32 and tells.
  auto covers = [&](uint32_t scale) { return 15.f * from16<BF16>(scale) > span || (15.f * from16<BF16>(scale) == span && !above); };
  uint32_t b = (BF16 ? pack_bf16x2(span * (1.f / 15.f), 0.f) : pack_f16x2(span * (1.f / 15.f), 0.f)) & 0xffffu;
  if (!covers(b)) ++b;
  else if (b > 0 && covers(b - 1)) --b;
  // Code 15 must not stand for more than the type holds (the difference is exact where it decides).
  if (mn > (BF16 ? 0x1.fep127f : 65504.f) - 15.f * from16<BF16>(b)) --b;
  Quant z;
  z.word = __byte_perm(b, extreme, 0x5410);
  z.min = mn;
  z.scale = from16<BF16>(b);
  // Scales of BF16 may be denormals of FP32: lifted, their reciprocal and the
  // remainders are normal.
  z.lift = BF16 && z.scale < 0x1p-64f ? 0x1p80f : 1.f;
  if (BF16) z.scale *= z.lift;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(z.inverse) : "f"(z.scale));
  if (z.scale == 0.f) z.inverse = z.lift = 0.f;
  if (!(span < INFINITY)) z = Quant{0x7fff7fffu, 0.f, 1.f, 0.f, 0.f};  // NaN
  return z;
}
// The codes of the eight values in four words, the first in the lowest bits.  x - m is
// rounded to FP32, and so is the quotient, correctly: by an approximate reciprocal and
// the remainder (a quotient by 8 or 11 bits is never as near to the middle of two FP32
// numbers as that is off).
template <bool BF16>
__device__ __forceinline__ uint32_t codes8(const uint32_t* x, const Quant& z) {
  const uint64_t min2 = packed_pair(z.min, z.min), inverse2 = packed_pair(z.inverse, z.inverse), minus2 = packed_pair(-z.scale, -z.scale);
  uint64_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    if (BF16) unpack_bf16x2(x[i], a, b);
    else unpack_f16x2(x[i], a, b);
    t[i] = sub_pair(packed_pair(a, b), min2);
  }
  if (BF16 && z.lift > 1.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = mul_pair(t[i], packed_pair(z.lift, z.lift));
  }
  uint32_t two[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q = mul_pair(t[i], inverse2);
    // 1.5 * 2^23 rounds to whole numbers, ties to even, in the lowest bits.
    constexpr uint64_t kRound = 0x4b4000004b400000ull;
    const float2 n = parts_of(add_pair(fma_pair(fma_pair(q, minus2, t[i]), inverse2, q), kRound));
    two[i] = __float_as_uint(n.x) + (__float_as_uint(n.y) << 4);  // its lowest byte
  }
  const uint32_t w = __byte_perm(__byte_perm(two[0], two[1], 0x0040), __byte_perm(two[2], two[3], 0x0040), 0x5410);
  return z.lift == 0.f ? 0u : w;  // (a NaN makes any code)
}

// A row of 16-bit values, the chunks' four words each, into its block.
// APART: the chunks are one of either group.
template <int D, bool BF16, bool APART>
__device__ __forceinline__ void store_row(uint8_t* block, int slot, int page_keys, const uint32_t (&y)[8], const Chunks& ch,
                                          int lane, bool on) {
  constexpr int G = D < 64 ? D : 64, H = D / G, LANES = D / 16;
  constexpr uint32_t kNone = BF16 ? 0x7f807f80u : 0x7c007c00u;  // infinities
  const int ga = H == 1 || APART ? 0 : ch.first / G, gb = H == 1 ? 0 : APART ? 1 : ch.second / G;
  const uint32_t a = extremes<BF16>(y), b = extremes<BF16>(y + 4);
  Quant za, zb;  // of the two chunks
  uint32_t word;  // of group `lane`, in the lanes below H
  if constexpr (H == 1) {
    uint32_t e = min_pair<BF16>(a, b);
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) e = min_pair<BF16>(e, __shfl_xor_sync(0xffffffffu, e, off));
    za = zb = quant_of<BF16>(e);
    word = za.word;
  } else {
    // The lower lanes come to hold group 0 and the upper ones group 1: each makes one
    // quantiser and gets the other.
    const int mine = lane / (LANES / 2);
    const uint32_t e0 = APART ? a : min_pair<BF16>(ga == 0 ? a : kNone, gb == 0 ? b : kNone);
    const uint32_t e1 = APART ? b : min_pair<BF16>(ga == 1 ? a : kNone, gb == 1 ? b : kNone);
    uint32_t e = min_pair<BF16>(mine ? e1 : e0, __shfl_xor_sync(0xffffffffu, mine ? e0 : e1, LANES / 2));
#pragma unroll
    for (int off = LANES / 4; off > 0; off >>= 1) e = min_pair<BF16>(e, __shfl_xor_sync(0xffffffffu, e, off));
    const Quant z = quant_of<BF16>(e);
    Quant other;
    other.word = __shfl_xor_sync(0xffffffffu, z.word, LANES / 2);
    other.inverse = __shfl_xor_sync(0xffffffffu, z.inverse, LANES / 2);
    other.lift = __shfl_xor_sync(0xffffffffu, z.lift, LANES / 2);
    if (BF16) unpack_bf16x2(other.word, other.scale, other.min);
    else unpack_f16x2(other.word, other.scale, other.min);
    if (BF16) other.scale *= other.lift;
    za = ga == mine ? z : other;
    zb = gb == mine ? z : other;
    word = lane == 1 ? other.word : z.word;
  }
  const uint32_t ca = codes8<BF16>(y, za), cb = codes8<BF16>(y + 4, zb);
  if (!on) return;
  const uint32_t part = (uint32_t)page_keys * (G / 2 + 4);
  uint8_t* codes = block + slot * (G / 2);
  *reinterpret_cast<uint32_t*>(codes + ga * part + (ch.first & (G - 1)) / 2) = ca;
  *reinterpret_cast<uint32_t*>(codes + gb * part + (ch.second & (G - 1)) / 2) = cb;
  if (lane < H)
    *reinterpret_cast<uint32_t*>(block + lane * part + (uint32_t)page_keys * (G / 2) + slot * 4) = word;
}

// A key's row: norm and rotation in two-part arithmetic, rounded to the input type.
// w, c and s: the weights, cosines and signed sines of the thread's elements, in pairs.
template <int D, bool BF16, bool INTER, bool FULL>
__device__ __forceinline__ void key_row(const uint64_t (&w)[8], const uint64_t (&c)[8], const uint64_t (&s)[8],
                                        const Chunks& ch, bool norm, float eps, uint32_t (&u)[8]) {
  uint64_t x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float a, b;
    if (BF16) unpack_bf16x2(u[j], a, b);
    else unpack_f16x2(u[j], a, b);
    x[j] = packed_pair(a, b);
  }
  Two r{1.f, 0.f};
  if (norm) {
    Two ss;
    bool zero = false;  // an infinite element: 1 / sqrt is 0
#pragma unroll 1
    for (bool again = false;; again = true) {
      uint64_t hi = mul_pair(x[0], x[0]), lo = 0;  // (exact within FP32's range)
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        uint64_t e;
        two_sum_pair(hi, mul_pair(x[j], x[j]), hi, e);
        lo = add_pair(lo, e);
      }
      const float2 h = parts_of(hi), l = parts_of(lo);
      ss = Two{h.x, l.x} + Two{h.y, l.y};
#pragma unroll
      for (int off = D / 32; off > 0; off >>= 1)
        ss = ss + Two{__shfl_xor_sync(0xffffffffu, ss.hi, off), __shfl_xor_sync(0xffffffffu, ss.lo, off)};
      // Squares of BF16 numbers may leave FP32's range.  Rows of such are scaled by a power of two,
      // eps by its square, so that the larger of both is near 1 (the norm takes it away again).
      // (16000 tokens 68.9 us without the test, 69.3 with it.)
      const bool far = !(ss.hi < 0x1p100f) || (ss.hi < 0x1p-60f && eps < 0x1p-60f);
      if (again || !__any_sync(0xffffffffu, far)) break;
      float big = 0.f;
      int nan = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = parts_of(x[j]);
        big = fmaxf(big, fmaxf(fabsf(v.x), fabsf(v.y)));
        nan |= v.x != v.x || v.y != v.y;
      }
#pragma unroll
      for (int off = D / 32; off > 0; off >>= 1) {
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
        nan |= __shfl_xor_sync(0xffffffffu, nan, off);
      }
      const int e = max((int)(__float_as_uint(big) >> 23) - 126, ((int)(__float_as_uint(eps) >> 23) - 127) / 2);
      const float by = far ? __uint_as_float((uint32_t)(127 - max(-126, min(126, e))) << 23) : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = mul_pair(x[j], packed_pair(by, by));
      eps = eps * by * by;
      zero = big == INFINITY && nan == 0;
    }
    r = two_rsqrt(Two{ss.hi * (1.f / D), ss.lo * (1.f / D)} + Two{eps, 0.f});
    if (zero) r = Two{0.f, 0.f};
  }
  const uint64_t rh = packed_pair(r.hi, r.hi), rl = packed_pair(r.lo, r.lo), minus_rh = packed_pair(-r.hi, -r.hi);
  float hi[16], lo[16];
  // How near a rounding comes to a tie: the distance of the bits that it cuts off to it.
  constexpr uint32_t kCut = BF16 ? 0xffffu : 0x1fffu, kTie = BF16 ? 0x8000u : 0x1000u;
  uint32_t near = kCut;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // t + e = n w cos + (partner n w) sin, times r.
    uint64_t t = mul_pair(x[j], w[j]), e = 0;  // (exact, as the squares)
    const bool turn = FULL || (j < 4 ? ch.turn_first : ch.turn_second);
    if (turn) {
      uint64_t xo = INTER ? x[j] : x[j ^ 4], wo = INTER ? w[j] : w[j ^ 4];
      uint64_t b = mul_pair(xo, wo);
      if (INTER) b = packed_pair(parts_of(b).y, parts_of(b).x);
      const uint64_t p = mul_pair(t, c[j]), q = mul_pair(b, s[j]);
      const uint64_t pe = fma_pair(t, c[j], mul_pair(p, kMinusOnes)), qe = fma_pair(b, s[j], mul_pair(q, kMinusOnes));
      two_sum_pair(p, q, t, e);
      e = add_pair(e, add_pair(pe, qe));
    }
    if (norm) {
      const uint64_t y = mul_pair(t, rh);
      const uint64_t ye = mul_pair(fma_pair(t, minus_rh, y), kMinusOnes);
      e = fma_pair(t, rl, fma_pair(e, rh, ye));
      t = y;
    }
    const uint64_t sum = add_pair(t, e);
    const float2 h = parts_of(sum), l = parts_of(sub_pair(e, sub_pair(sum, t)));
    // (What neither norm nor rotation touches passes through as it is, -0 among it.)
    const bool as_is = !norm && !turn;
    hi[2 * j] = as_is ? parts_of(t).x : h.x, hi[2 * j + 1] = as_is ? parts_of(t).y : h.y;
    lo[2 * j] = l.x, lo[2 * j + 1] = l.y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      near = min(near, (__float_as_uint(hi[2 * j + i]) ^ kTie) & kCut);
      if (!BF16 && fabsf(hi[2 * j + i]) < 0x1p-14f) near = 0u;  // (there it cuts off more)
    }
  }
  // The lower part decides a tie alone, which is rare.
  if (near == 0u) {
#pragma unroll
    for (int j = 0; j < 16; ++j) hi[j] = to_odd(hi[j], lo[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = BF16 ? pack_bf16x2(hi[2 * j], hi[2 * j + 1]) : pack_f16x2(hi[2 * j], hi[2 * j + 1]);
}

// A group of D/16 threads takes consecutive heads of one token, as in attn_rope.cu: HQ of
// q or HP of k or v.
template <int D, bool BF16, int HQ, int HP, bool INTER, bool FULL>
__global__ void __launch_bounds__(kAppendThreads, 6) append_q4_kernel(const __grid_constant__ AppendQ4Params p) {
  constexpr int LANES = D / 16, GROUPS = kAppendThreads / LANES;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES;
  const Chunks ch = chunks_of(D, lane, FULL ? D : p.rope_dim, INTER);
  // The block's kind of rows: those of k and v are spread among those of q, so that
  // their arithmetic runs beside q's traffic.
  const int before = min(p.others, (int)(blockIdx.x * p.others_step >> 32));  // blocks of k and v before this one
  const bool is_q = min(p.others, (int)((blockIdx.x + 1) * p.others_step >> 32)) == before;
  const int kind = is_q ? 0 : 1 + (before & 1);
  const int block = is_q ? (int)blockIdx.x - before : before >> 1;
  const int heads = kind == 0 ? p.Hq : p.Hkv, step = kind == 0 ? HQ : HP, per_token = (heads + step - 1) / step;
  const int64_t item = (int64_t)block * GROUPS + threadIdx.x / LANES;
  const bool live = item < (int64_t)p.total_tokens * per_token;
  const uint64_t groups = kind == 0 ? p.q_groups : p.kv_groups;
  const int t = !live ? 0 : groups == 0 ? (int)item : (int)__umul64hi((uint64_t)item, groups);
  const int h0 = live ? (int)(item - (int64_t)t * per_token) * step : 0;
  const int64_t st = kind == 0 ? p.q_st : kind == 1 ? p.k_st : p.v_st;
  const int64_t sh = kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh;
  const uint16_t* in = static_cast<const uint16_t*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) + t * st + h0 * sh;

  constexpr bool STAGED = HP > 1;
  extern __shared__ uint4 cells[];
  uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
  auto fetch = [&](int i) {
    if (live && h0 + i < heads) {
      if constexpr (STAGED) {
        copy_async(cells + (2 * i) * kAppendThreads + threadIdx.x, in + i * sh + ch.first);
        copy_async(cells + (2 * i + 1) * kAppendThreads + threadIdx.x, in + i * sh + ch.second);
      } else {
        ra = *reinterpret_cast<const uint4*>(in + ch.first);
        rb = *reinterpret_cast<const uint4*>(in + ch.second);
      }
    }
    if constexpr (STAGED) copy_commit();
  };
  if (kind == 0) {
#pragma unroll
    for (int i = 0; i < HQ; ++i) fetch(i);
  } else {
#pragma unroll
    for (int i = 0; i < HP; ++i) fetch(i);
  }

  // The token's place; without one, nothing of it is written.
  const int page_keys = 1 << p.page_shift;
  const int64_t place = live ? p.slots[t] : -1;
  int64_t pos = 0;
  bool ok = place >= 0;
  if (ok) {
    ok = (place >> p.page_shift) < p.num_pages;
    if (p.rope_dim > 0) {
      pos = p.positions[t];
      ok = ok && pos >= 0 && pos < p.max_position;
    }
    if (!ok && lane == 0) atomicCAS(p.status, 0, (int)kDevBadIndex);
  }
  const int64_t page = ok ? place >> p.page_shift : 0;
  const int slot = ok ? (int)(place & (page_keys - 1)) : 0;

  const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  float w[16], c8[8], s8[8];
  if (kind != 2) {
    load_weight<BF16>(weight, ch, w);
    load_angles(c8, s8, p.cos, p.sin, pos, FULL ? D : p.rope_dim, ch, ok);
  }
  if (kind == 0) {
    uint16_t* out = static_cast<uint16_t*>(p.q_out) + t * p.qo_st + h0 * p.qo_sh;
    float P[16], Q[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      P[j] = w[j] * c8[pair_of<INTER>(j)];
      Q[j] = (is_first<INTER>(j) ? -1.f : 1.f) * w[partner<INTER>(j)] * s8[pair_of<INTER>(j)];
    }
#pragma unroll
    for (int i = 0; i < HQ; ++i) {
      float x[16], y[16];
      if constexpr (STAGED) {
        copy_wait_for(HQ - 1 - i);
        ra = cells[(2 * i) * kAppendThreads + threadIdx.x];
        rb = cells[(2 * i + 1) * kAppendThreads + threadIdx.x];
      }
      unpack16<BF16>(ra, rb, x);
      const float ss = row_sum<LANES>(dot16(x, x));
      turn16<INTER, FULL>(x, P, Q, ch, y);
      if (weight != nullptr) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int j = 0; j < 16; j += 2) fma2_keep(y[j], y[j + 1], y[j], y[j + 1], r, r, -0.f, -0.f);
      }
      if (ok && h0 + i < heads) store16<BF16>(out + i * p.qo_sh, ch, y);
    }
  } else {
    uint8_t* out = kind == 1 ? p.k_pages + page * p.kp_sp : p.v_pages + page * p.vp_sp;
    const int64_t oh = kind == 1 ? p.kp_sh : p.vp_sh;
    uint64_t w2[8], c2[8], s2[8];
    if (kind == 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int a = 2 * j, b = 2 * j + 1;
        w2[j] = packed_pair(w[a], w[b]);
        c2[j] = packed_pair(c8[pair_of<INTER>(a)], c8[pair_of<INTER>(b)]);
        const float sa = s8[pair_of<INTER>(a)], sb = s8[pair_of<INTER>(b)];
        s2[j] = packed_pair(is_first<INTER>(a) ? -sa : sa, is_first<INTER>(b) ? -sb : sb);
      }
    }
    if constexpr (STAGED) copy_wait<0>();
    auto row = [&](int i, auto KEY) {
      if constexpr (STAGED) {
        ra = cells[(2 * i) * kAppendThreads + threadIdx.x];
        rb = cells[(2 * i + 1) * kAppendThreads + threadIdx.x];
      }
      uint32_t y[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
      if constexpr (decltype(KEY)::value) key_row<D, BF16, INTER, FULL>(w2, c2, s2, ch, weight != nullptr, p.eps, y);
      store_row<D, BF16, FULL || INTER>(out + (h0 + i) * oh, slot, page_keys, y, ch, lane, ok && h0 + i < heads);
    };
    if (kind == 1) {
#pragma unroll 1
      for (int i = 0; i < HP; ++i) row(i, std::true_type{});
    } else {  // (two at a time: 2 % faster for 16000 tokens than one)
#pragma unroll 2
      for (int i = 0; i < HP; ++i) row(i, std::false_type{});
    }
  }
}

// A thread takes eight elements of four neighbouring rows, all on their way at once;
// neighbours take neighbouring elements.
constexpr int kUnpackRows = 4;
template <int D, bool BF16>
__global__ void __launch_bounds__(256) unpack_q4_kernel(const __grid_constant__ UnpackQ4Params p) {
  constexpr int G = D < 64 ? D : 64, PER = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int d = (int)(item % PER) * 8;
  int64_t row = item / PER;
  const int page_keys = 1 << p.page_shift, slot = (int)(row & (page_keys / kUnpackRows - 1)) * kUnpackRows;
  row >>= p.page_shift - 2;
  const int64_t page = div_pos(row, p.Hkv);
  const int head = (int)(row - page * p.Hkv);
  if (page >= p.num_pages) return;
  const uint8_t* part = p.pages + page * p.p_sp + head * p.p_sh + (int64_t)(d / G) * page_keys * (G / 2 + 4);
  const uint8_t* codes = part + (int64_t)slot * (G / 2) + (d & (G - 1)) / 2;
  uint32_t w[kUnpackRows];
#pragma unroll
  for (int i = 0; i < kUnpackRows; ++i) w[i] = *reinterpret_cast<const uint32_t*>(codes + i * (G / 2));
  const uint4 sm = *reinterpret_cast<const uint4*>(part + (int64_t)page_keys * (G / 2) + (int64_t)slot * 4);
  const uint32_t words[4] = {sm.x, sm.y, sm.z, sm.w};
  uint16_t* out = static_cast<uint16_t*>(p.out) + page * p.o_sp + head * p.o_sh + slot * p.o_st + d;
#pragma unroll
  for (int j = 0; j < kUnpackRows; ++j) {
    float s, m, x[8];
    if (BF16) unpack_bf16x2(words[j], s, m);
    else unpack_f16x2(words[j], s, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn((float)((w[j] >> 4 * i) & 15u), s, m);
    *reinterpret_cast<uint4*>(out + j * p.o_st) = pack8<BF16>(x);
  }
}
static_assert(kUnpackRows == 4, "the scales and minima of four rows are one load");

template <int D, bool BF16, int HQ, int HP, bool INTER, bool FULL>
cudaError_t launch_append(const AppendQ4Params& p, unsigned blocks, cudaStream_t s) {
  auto kern = append_q4_kernel<D, BF16, HQ, HP, INTER, FULL>;
  static_assert(HQ >= HP, "");
  constexpr int SMEM = HP > 1 ? HQ * 2 * kAppendThreads * 16 : 0;
  if (SMEM > 48 * 1024) {
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = opt_in(kern, SMEM, configured);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(blocks), kAppendThreads, SMEM, s, p);
}

// Blocks with hq heads of q and hp of k or v a group; *kv of them for k, as many for v.
template <int D>
int64_t append_blocks(const AppendQ4Params& p, int hq, int hp, int64_t* kv) {
  constexpr int GROUPS = kAppendThreads / (D / 16);
  *kv = ((int64_t)p.total_tokens * ((p.Hkv + hp - 1) / hp) + GROUPS - 1) / GROUPS;
  return ((int64_t)p.total_tokens * ((p.Hq + hq - 1) / hq) + GROUPS - 1) / GROUPS + 2 * *kv;
}

template <int D, bool BF16, int HQ, int HP>
cudaError_t append(const AppendQ4Params& p0, cudaStream_t s) {
  AppendQ4Params p = p0;
  int64_t kv;
  const int64_t blocks = append_blocks<D>(p, HQ, HP, &kv);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // k and v's blocks come in the first 6/7 of the launch: theirs take longer, and at the
  // end the GPU would wait for a few of them (16000 tokens: 73.6 us spread over all of it,
  // 71.3, 69.1, 68.4 and 69.5 over 95, 90, 86 and 80 %; all of it and 86 % with 8, 16, 40 and 64 heads
  // of q 54.4 and 50.9, 60.8 and 56.7, 81.7 and 76.4, 105 and 99.3, with 32 of each at 8000 tokens 98.0 and 94.4,
  // without q no difference, with heads of 64 42.6 and 39.5, of 32 27.9 and 26.4).  The product with all
  // blocks is no less than their number.
  p.others = (int)(2 * kv);
  const uint64_t even = (((uint64_t)p.others << 32) + blocks - 1) / blocks;
  p.others_step = std::min(even + even / 6, uint64_t{1} << 32);
  // Rounded up: with an item (below 2^37) a quotient whose fraction stays below 1.
  auto one_over = [](int heads, int each) {
    const uint64_t groups = (heads + each - 1) / each;
    return groups <= 1 ? 0 : ~uint64_t{0} / groups + 1;
  };
  p.q_groups = one_over(p.Hq, HQ);
  p.kv_groups = one_over(p.Hkv, HP);
  const bool full = p.rope_dim == D;
  if (p.interleaved)
    return full ? launch_append<D, BF16, HQ, HP, true, true>(p, (unsigned)blocks, s)
                : launch_append<D, BF16, HQ, HP, true, false>(p, (unsigned)blocks, s);
  return full ? launch_append<D, BF16, HQ, HP, false, true>(p, (unsigned)blocks, s)
              : launch_append<D, BF16, HQ, HP, false, false>(p, (unsigned)blocks, s);
}

// One head a group for small calls, else four (eight of q), which read a token's place, angles
// and weights for all of them.  Measured, us of either (BF16, 32 + 2 x 8 heads): of 128, 3.2 and 6.8 at 64
// tokens, 7.2 and 10.7 at 800, 19.0 and 19.2 at 2400 (7200 blocks of one head), 36 and 28 at
// 4800, 115 and 69 at 16000; of 64, 4.8 and 8.5 at 800, 18.9 and 18.8 at 4800 (7200), 58 and 39 at
// 16000.  At 16000 tokens of the former two, four and eight heads of k and v beside eight of q
// take 74.7, 68.4 and 73.8 us, four of all 70.1.
constexpr int kOneHeadBlocks = 7296;  // 48 on each of a GB300's 152 SMs
template <int D, bool BF16>
cudaError_t append_any(const AppendQ4Params& p, cudaStream_t s) {
  int64_t kv;
  return append_blocks<D>(p, 1, 1, &kv) <= kOneHeadBlocks ? append<D, BF16, 1, 1>(p, s) : append<D, BF16, 8, 4>(p, s);
}

template <int D, bool BF16>
cudaError_t unpack(const UnpackQ4Params& p, cudaStream_t s) {
  const int64_t items = ((int64_t)p.num_pages * p.Hkv << p.page_shift) / kUnpackRows * (D / 8), blocks = (items + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(unpack_q4_kernel<D, BF16>, dim3((unsigned)blocks), 256, 0, s, p);
}

}  // namespace

cudaError_t launch_append_q4(int D, bool bf16, const AppendQ4Params& p, cudaStream_t s) {
  switch (D) {
    case 32: return bf16 ? append_any<32, true>(p, s) : append_any<32, false>(p, s);
    case 64: return bf16 ? append_any<64, true>(p, s) : append_any<64, false>(p, s);
    default: return bf16 ? append_any<128, true>(p, s) : append_any<128, false>(p, s);
  }
}

cudaError_t launch_unpack_q4(int D, bool bf16, const UnpackQ4Params& p, cudaStream_t s) {
  switch (D) {
    case 32: return bf16 ? unpack<32, true>(p, s) : unpack<32, false>(p, s);
    case 64: return bf16 ? unpack<64, true>(p, s) : unpack<64, false>(p, s);
    default: return bf16 ? unpack<128, true>(p, s) : unpack<128, false>(p, s);
  }
}

}  // namespace etattn
