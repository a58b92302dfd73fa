// What the kernels that norm and rotate rows have in common.  D/16 threads hold a
// row of D elements, two 16-byte chunks each, with both elements of every pair in
// one thread.
#pragma once

#include <cstdint>

#include "cache_ptx.cuh"

namespace etattn {

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) unpack_bf16x2(w[i], f[2 * i], f[2 * i + 1]);
    else unpack_f16x2(w[i], f[2 * i], f[2 * i + 1]);
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = BF16 ? pack_bf16x2(f[2 * i], f[2 * i + 1]) : pack_f16x2(f[2 * i], f[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's own 16-byte cells of shared memory, filled by asynchronous copies
// that it alone waits for.
__device__ __forceinline__ void copy_async(uint4* cell, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(cell)), "l"(src) : "memory");
}
// The same for what neighbouring groups read too: through L1.
__device__ __forceinline__ void copy_async_shared(uint4* cell, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(cell)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
// copy_wait for a count that becomes a constant when its loop is unrolled.
__device__ __forceinline__ void copy_wait_for(int pending) {
  switch (pending) {
    case 0: copy_wait<0>(); break;
    case 1: copy_wait<1>(); break;
    case 2: copy_wait<2>(); break;
    case 3: copy_wait<3>(); break;
    case 4: copy_wait<4>(); break;
    case 5: copy_wait<5>(); break;
    case 6: copy_wait<6>(); break;
    default: copy_wait<7>(); break;
  }
}

// The sum over the LANES threads that hold a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// A thread's two chunks of a row: element offsets, whether they are rotated
// and where the angles of the thread's pairs 0-3 and 4-7 start in a table row.
// Neighbouring lanes hold neighbouring chunks, so that a warp's access covers
// whole sectors.  Pairs of halves: (first + j, second + j), the elements past
// rope_dim in two runs of their own; side by side: a chunk's own neighbours.
struct Chunks {
  int first, second;
  bool turn_first, turn_second;
  int angle_first, angle_second;
};
__device__ __forceinline__ Chunks chunks_of(int D, int lane, int rope_dim, bool interleaved) {
  if (interleaved) {
    const int a = 8 * lane, b = D / 2 + 8 * lane;
    return {a, b, a < rope_dim, b < rope_dim, a / 2, b / 2};
  }
  const int n = rope_dim / 16;
  if (lane < n) return {8 * lane, rope_dim / 2 + 8 * lane, true, true, 8 * lane, 8 * lane + 4};
  const int a = rope_dim + 8 * (lane - n);
  return {a, a + (D - rope_dim) / 2, false, false, 0, 0};
}

// cos and sin of the thread's eight pairs (1 and 0 where nothing rotates).
__device__ __forceinline__ void load_angles(float (&c)[8], float (&s)[8], const float* cos, const float* sin,
                                            int64_t pos, int rope_dim, const Chunks& ch, bool on) {
  const float* pc = cos + pos * (rope_dim / 2);
  const float* ps = sin + pos * (rope_dim / 2);
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on && (j == 0 ? ch.turn_first : ch.turn_second)) {
      const int at = j == 0 ? ch.angle_first : ch.angle_second;
      c4 = *reinterpret_cast<const float4*>(pc + at);
      s4 = *reinterpret_cast<const float4*>(ps + at);
    }
    c[j] = c4.x, c[j + 1] = c4.y, c[j + 2] = c4.z, c[j + 3] = c4.w;
    s[j] = s4.x, s[j + 1] = s4.y, s[j + 2] = s4.z, s[j + 3] = s4.w;
  }
}

// Index of element i's partner among the thread's 16 (chunk first: 0-7,
// second: 8-15) and of their pair.
template <bool INTER>
__device__ __forceinline__ constexpr int partner(int i) { return INTER ? (i ^ 1) : (i ^ 8); }
template <bool INTER>
__device__ __forceinline__ constexpr int pair_of(int i) { return INTER ? (i >> 1) : (i & 7); }
template <bool INTER>
__device__ __forceinline__ constexpr bool is_first(int i) { return INTER ? (i & 1) == 0 : i < 8; }

template <bool BF16>
__device__ __forceinline__ void load_weight(const void* w, const Chunks& ch, float (&f)[16]) {
  if (w != nullptr) {
    float lo[8], hi[8];
    unpack8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + ch.first), lo);
    unpack8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + ch.second), hi);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = lo[j], f[8 + j] = hi[j];
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = 1.f;
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&x)[16]) {
  float lo[8], hi[8];
  unpack8<BF16>(a, lo);
  unpack8<BF16>(b, hi);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = lo[j], x[8 + j] = hi[j];
}
template <bool BF16>
__device__ __forceinline__ void store16(uint16_t* row, const Chunks& ch, const float (&y)[16]) {
  float lo[8], hi[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) lo[j] = y[j], hi[j] = y[8 + j];
  *reinterpret_cast<uint4*>(row + ch.first) = pack8<BF16>(lo);
  *reinterpret_cast<uint4*>(row + ch.second) = pack8<BF16>(hi);
}
// sum of a[j] * b[j]
__device__ __forceinline__ float dot16(const float (&a)[16], const float (&b)[16]) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int j = 0; j < 16; j += 2) fma2_keep(s0, s1, a[j], a[j + 1], b[j], b[j + 1], s0, s1);
  return s0 + s1;
}
// y = x P + x_partner Q, and x P alone for an element that does not rotate: its
// "partner" and that one's weight may be infinite, and 0 times infinity is not
// 0.  Adding -0 to x P changes no value, so P = 1 passes x through as it is.
template <bool INTER, bool FULL>
__device__ __forceinline__ void turn16(const float (&x)[16], const float (&P)[16], const float (&Q)[16],
                                       const Chunks& ch, float (&y)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const bool turn = FULL || (j < 8 ? ch.turn_first : ch.turn_second);
    float t0, t1, u0, u1;
    fma2_keep(t0, t1, x[j], x[j + 1], P[j], P[j + 1], -0.f, -0.f);
    fma2_keep(u0, u1, x[partner<INTER>(j)], x[partner<INTER>(j + 1)], Q[j], Q[j + 1], t0, t1);
    y[j] = turn ? u0 : t0;
    y[j + 1] = turn ? u1 : t1;
  }
}

}  // namespace etattn
