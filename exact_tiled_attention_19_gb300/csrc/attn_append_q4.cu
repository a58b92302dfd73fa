// Keys and values into a paged cache held in 4 bits, queries and keys normed and
// rotated on the way, and the cache's values back in 16 bits.
//
// Mathematics.  Norm and rotation are those of attn_rope.cu.  A row of D elements
// of the input type (of a key: what norm and rotation leave, rounded to it) is cut into
// groups of G = min(D, 64).  With a group's minimum m and maximum M,
//     s = the smallest number of the input type with 15 s >= M - m,
//     c_d = round((x_d - m) / s), ties to even, 0 where s is 0;
// the cache stands for s c_d + m, at most s / 2 from x_d.  A group with an element that is
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
// so that no warp does two kinds of work.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "launchers.h"
#include "cache_ptx.cuh"
#include "rope_device.cuh"

namespace etattn {

namespace {

constexpr int kAppendThreads = 256;

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
__device__ __forceinline__ Two operator*(const Two& a, const Two& b) {
  const Two p = two_product(a.hi, b.hi);
  return renormed(p.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, p.lo)));
}
// 1 / sqrt(x): with y near it and e = 1 - x y^2, y (1 + e/2 + 3 e^2 / 8).
__device__ __forceinline__ Two two_rsqrt(const Two& x) {
  const float y = rsqrtf(x.hi);
  const Two s = two_product(y, y);
  const float e = __fmaf_rn(-x.lo, s.hi, __fmaf_rn(-x.hi, s.lo, __fmaf_rn(-x.hi, s.hi, 1.f)));
  return renormed(y, __fmul_rn(y, __fmul_rn(e, __fmaf_rn(e, 0.375f, 0.5f))));
}
// The sum rounded to odd, so that rounding it on to 16 bits is rounding once.
__device__ __forceinline__ float to_odd(const Two& x) {
  const uint32_t b = __float_as_uint(x.hi);
  if (x.lo == 0.f || (b & 1u)) return x.hi;
  return __uint_as_float(((b ^ __float_as_uint(x.lo)) >> 31) ? b - 1u : b | 1u);
}

// min and max that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t bits16(float x) { return (BF16 ? pack_bf16x2(x, 0.f) : pack_f16x2(x, 0.f)) & 0xffffu; }
template <bool BF16>
__device__ __forceinline__ float from16(uint32_t b) {
  float x, unused;
  if (BF16) unpack_bf16x2(b, x, unused);
  else unpack_f16x2(b, x, unused);
  return x;
}

// A group's scale and minimum, as the cache holds them, and what its codes need.
struct Quant {
  uint32_t word;            // scale in the low half, minimum in the high one
  float min, scale, inverse, lift;  // scale and inverse of lift times the group; lift 0: all codes are 0
};
template <bool BF16>
__device__ __forceinline__ Quant quant_of(float mn, float mx) {
  Quant z{0x7fff7fffu, 0.f, 1.f, 0.f, 0.f};  // NaN, codes 0
  const float span = mx - mn;
  if (!(span < INFINITY)) return z;
  uint32_t b = bits16<BF16>(__fdiv_rn(span, 15.f));
  if (15.f * from16<BF16>(b) < span) ++b;  // (15 s is exact in FP32)
  z.word = b | bits16<BF16>(mn) << 16;
  z.min = mn;
  const float s = from16<BF16>(b);
  if (s > 0.f) {
    z.lift = s < 0x1p-64f ? 0x1p80f : 1.f;  // keeps the reciprocal and the remainders normal
    z.scale = s * z.lift;
    z.inverse = __frcp_rn(z.scale);
  }
  return z;
}
// The codes of eight values, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float* x, const Quant& z) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float t = __fsub_rn(x[i], z.min) * z.lift;
    const float q0 = __fmul_rn(t, z.inverse);
    const float q = __fmaf_rn(__fmaf_rn(-q0, z.scale, t), z.inverse, q0);
    w = (w << 4) | (__float_as_uint(__fadd_rn(q, 12582912.f)) & 15u);  // 1.5 * 2^23: rounds to whole numbers
  }
  return z.lift == 0.f ? 0u : w;  // (a NaN makes any code)
}

// A row of 16-bit values into its block.
template <int D, bool BF16>
__device__ __forceinline__ void store_row(uint8_t* block, int slot, int page_keys, const float (&y)[16], const Chunks& ch,
                                          int lane, bool on) {
  constexpr int G = D < 64 ? D : 64, H = D / G, LANES = D / 16;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const bool a = H == 1 || ch.first / G == h, b = H == 1 || ch.second / G == h;
    float mn = INFINITY, mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (a) mn = min_nan(mn, y[j]), mx = max_nan(mx, y[j]);
      if (b) mn = min_nan(mn, y[8 + j]), mx = max_nan(mx, y[8 + j]);
    }
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) {
      mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, off));
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    }
    const Quant z = quant_of<BF16>(mn, mx);
    if (on) {
      uint8_t* part = block + (int64_t)h * page_keys * (G / 2 + 4);
      uint8_t* codes = part + (int64_t)slot * (G / 2);
      if (a) *reinterpret_cast<uint32_t*>(codes + (ch.first & (G - 1)) / 2) = codes8(y, z);
      if (b) *reinterpret_cast<uint32_t*>(codes + (ch.second & (G - 1)) / 2) = codes8(y + 8, z);
      if (lane == 0) *reinterpret_cast<uint32_t*>(part + (int64_t)page_keys * (G / 2) + (int64_t)slot * 4) = z.word;
    }
  }
}

// A key's row: norm and rotation in two-part arithmetic, rounded to the input type.
template <int D, bool BF16, bool INTER, bool FULL>
__device__ __forceinline__ void key_row(const float (&x)[16], const float (&w)[16], const float (&c)[8], const float (&s)[8],
                                        const Chunks& ch, bool norm, float eps, float (&y)[16]) {
  Two r{1.f, 0.f};
  if (norm) {
    Two ss{0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) {  // (squares of 16-bit numbers are exact)
      const Two t = two_sum(ss.hi, __fmul_rn(x[j], x[j]));
      ss = Two{t.hi, __fadd_rn(ss.lo, t.lo)};
    }
#pragma unroll
    for (int off = D / 32; off > 0; off >>= 1)
      ss = ss + Two{__shfl_xor_sync(0xffffffffu, ss.hi, off), __shfl_xor_sync(0xffffffffu, ss.lo, off)};
    r = two_rsqrt(Two{ss.hi * (1.f / D), ss.lo * (1.f / D)} + Two{eps, 0.f});
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int o = partner<INTER>(j);
    const bool turn = FULL || (j < 8 ? ch.turn_first : ch.turn_second);
    Two t{__fmul_rn(x[j], w[j]), 0.f};  // (exact, as the squares)
    if (turn) {
      const float angle = is_first<INTER>(j) ? -s[pair_of<INTER>(j)] : s[pair_of<INTER>(j)];
      t = two_product(t.hi, c[pair_of<INTER>(j)]) + two_product(__fmul_rn(x[o], w[o]), angle);
    }
    // What neither norm nor rotation touches passes through as it is.
    y[j] = norm ? to_odd(t * r) : to_odd(t);
  }
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const uint32_t u = BF16 ? pack_bf16x2(y[j], y[j + 1]) : pack_f16x2(y[j], y[j + 1]);
    if (BF16) unpack_bf16x2(u, y[j], y[j + 1]);
    else unpack_f16x2(u, y[j], y[j + 1]);
  }
}

// A group of D/16 threads takes HP consecutive heads of one token, as in attn_rope.cu.
template <int D, bool BF16, int HP, bool INTER, bool FULL>
__global__ void __launch_bounds__(kAppendThreads, 2) append_q4_kernel(const __grid_constant__ AppendQ4Params p) {
  constexpr int LANES = D / 16, GROUPS = kAppendThreads / LANES;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES;
  const Chunks ch = chunks_of(D, lane, FULL ? D : p.rope_dim, INTER);
  // The block's kind of rows.
  const int kind = (int)blockIdx.x < p.q_blocks ? 0 : (int)blockIdx.x < p.q_blocks + p.kv_blocks ? 1 : 2;
  const int block = (int)blockIdx.x - (kind == 0 ? 0 : kind == 1 ? p.q_blocks : p.q_blocks + p.kv_blocks);
  const int heads = kind == 0 ? p.Hq : p.Hkv, per_token = (heads + HP - 1) / HP;
  const int64_t item = (int64_t)block * GROUPS + threadIdx.x / LANES;
  const bool live = item < (int64_t)p.total_tokens * per_token;
  const int t = live ? (int)div_pos(item, per_token) : 0;
  const int h0 = live ? (int)(item - (int64_t)t * per_token) * HP : 0;
  const int64_t st = kind == 0 ? p.q_st : kind == 1 ? p.k_st : p.v_st;
  const int64_t sh = kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh;
  const uint16_t* in = static_cast<const uint16_t*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) + t * st + h0 * sh;

  constexpr bool STAGED = HP > 1;
  extern __shared__ uint4 cells[];
  uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
#pragma unroll
  for (int i = 0; i < HP; ++i) {
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
    if (!ok) atomicCAS(p.status, 0, (int)kDevBadIndex);
  }
  const int64_t page = ok ? place >> p.page_shift : 0;
  const int slot = ok ? (int)(place & (page_keys - 1)) : 0;

  const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  float w[16], c8[8], s8[8];
  if (kind != 2) {
    load_weight<BF16>(weight, ch, w);
    load_angles(c8, s8, p.cos, p.sin, pos, FULL ? D : p.rope_dim, ch, ok);
  }
  auto row = [&](int i, float(&x)[16]) {
    if constexpr (STAGED) {
      copy_wait_for(HP - 1 - i);
      ra = cells[(2 * i) * kAppendThreads + threadIdx.x];
      rb = cells[(2 * i + 1) * kAppendThreads + threadIdx.x];
    }
    unpack16<BF16>(ra, rb, x);
  };

  if (kind == 0) {
    uint16_t* out = static_cast<uint16_t*>(p.q_out) + t * p.qo_st + h0 * p.qo_sh;
    float P[16], Q[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      P[j] = w[j] * c8[pair_of<INTER>(j)];
      Q[j] = (is_first<INTER>(j) ? -1.f : 1.f) * w[partner<INTER>(j)] * s8[pair_of<INTER>(j)];
    }
#pragma unroll
    for (int i = 0; i < HP; ++i) {
      float x[16], y[16];
      row(i, x);
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
#pragma unroll 1
    for (int i = 0; i < HP; ++i) {
      float x[16], y[16];
      row(i, x);
      if (kind == 1) {
        key_row<D, BF16, INTER, FULL>(x, w, c8, s8, ch, weight != nullptr, p.eps, y);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = x[j];
      }
      store_row<D, BF16>(out + (h0 + i) * oh, slot, page_keys, y, ch, lane, ok && h0 + i < heads);
    }
  }
}

// A thread takes eight elements of a row, neighbours neighbouring ones.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) unpack_q4_kernel(const __grid_constant__ UnpackQ4Params p) {
  constexpr int G = D < 64 ? D : 64, PER = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int d = (int)(item % PER) * 8;
  int64_t row = item / PER;
  const int page_keys = 1 << p.page_shift, slot = (int)(row & (page_keys - 1));
  row >>= p.page_shift;
  const int64_t page = div_pos(row, p.Hkv);
  const int head = (int)(row - page * p.Hkv);
  if (page >= p.num_pages) return;
  const uint8_t* part = p.pages + page * p.p_sp + head * p.p_sh + (int64_t)(d / G) * page_keys * (G / 2 + 4);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(part + (int64_t)slot * (G / 2) + (d & (G - 1)) / 2);
  const uint32_t sm = *reinterpret_cast<const uint32_t*>(part + (int64_t)page_keys * (G / 2) + (int64_t)slot * 4);
  float s, m, x[8];
  if (BF16) unpack_bf16x2(sm, s, m);
  else unpack_f16x2(sm, s, m);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn((float)((w >> 4 * i) & 15u), s, m);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + page * p.o_sp + head * p.o_sh + slot * p.o_st + d) = pack8<BF16>(x);
}

template <int D, bool BF16, int HP, bool INTER, bool FULL>
cudaError_t launch_append(const AppendQ4Params& p, unsigned blocks, cudaStream_t s) {
  auto kern = append_q4_kernel<D, BF16, HP, INTER, FULL>;
  constexpr int SMEM = HP > 1 ? HP * 2 * kAppendThreads * 16 : 0;
  if (SMEM > 48 * 1024) {
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = opt_in(kern, SMEM, configured);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(blocks), kAppendThreads, SMEM, s, p);
}

template <int D>
int64_t append_blocks(const AppendQ4Params& p, int hp, int64_t* q, int64_t* kv) {
  constexpr int GROUPS = kAppendThreads / (D / 16);
  *q = ((int64_t)p.total_tokens * ((p.Hq + hp - 1) / hp) + GROUPS - 1) / GROUPS;
  *kv = ((int64_t)p.total_tokens * ((p.Hkv + hp - 1) / hp) + GROUPS - 1) / GROUPS;
  return *q + 2 * *kv;
}

template <int D, bool BF16, int HP>
cudaError_t append(const AppendQ4Params& p0, cudaStream_t s) {
  AppendQ4Params p = p0;
  int64_t q, kv;
  const int64_t blocks = append_blocks<D>(p, HP, &q, &kv);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  p.q_blocks = (int)q;
  p.kv_blocks = (int)kv;
  const bool full = p.rope_dim == D;
  if (p.interleaved)
    return full ? launch_append<D, BF16, HP, true, true>(p, (unsigned)blocks, s)
                : launch_append<D, BF16, HP, true, false>(p, (unsigned)blocks, s);
  return full ? launch_append<D, BF16, HP, false, true>(p, (unsigned)blocks, s)
              : launch_append<D, BF16, HP, false, false>(p, (unsigned)blocks, s);
}

// One head a group while its blocks all run at once, else eight.
constexpr int kOneHeadBlocks = 304;
template <int D, bool BF16>
cudaError_t append_any(const AppendQ4Params& p, cudaStream_t s) {
  int64_t q, kv;
  return append_blocks<D>(p, 1, &q, &kv) <= kOneHeadBlocks ? append<D, BF16, 1>(p, s) : append<D, BF16, 8>(p, s);
}

template <int D, bool BF16>
cudaError_t unpack(const UnpackQ4Params& p, cudaStream_t s) {
  const int64_t items = ((int64_t)p.num_pages * p.Hkv << p.page_shift) * (D / 8), blocks = (items + 255) / 256;
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
