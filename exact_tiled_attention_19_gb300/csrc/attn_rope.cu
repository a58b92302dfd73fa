// Queries and keys before attention: the RMS norm of every head and the
// rotation by position in one pass, its gradients, and the append to a paged
// key-value cache with both applied on the way.
//
// Mathematics.  A row x is one head of one token, D elements, with weight w:
//     r = (mean_d x_d^2 + eps)^(-1/2),   n_d = x_d r w_d      (no w: n = x)
// and the first R elements are rotated in pairs (a, b) by the angle of the
// token's position and of the pair:
//     y_a = n_a cos - n_b sin,   y_b = n_b cos + n_a sin,
// pairs (i, i + R/2) or, interleaved, (2i, 2i + 1).  With g the rotation of
// the upstream gradient by the negative angle,
//     dw_d = sum over rows of g_d x_d r,
//     dx_d = r (g_d w_d - x_d r^2 mean_e(g_e w_e x_e)).
//
// Everything is computed in FP32 from the 16-bit inputs and rounded once, to
// the type of the output.  Each row is read and written once, so memory
// bounds these kernels.  D/8 threads hold a row, 16 bytes each.
#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "launchers.h"
#include "sm103_ptx.cuh"

namespace etattn {

namespace {

constexpr int kThreads = 256;

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

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// The thread's share of a token's angles: chunk c holds elements 8c .. 8c+7.
// Paired with the other half, element j has cos[j], sin[j] of its own; side by
// side, pair j of the chunk (elements 2j, 2j + 1) has cos[j], sin[j], j < 4.
struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ void load_angles(Angles& a, const float* cos, const float* sin, int64_t pos, int rope_dim,
                                            bool interleaved, int chunk) {
  const int half = rope_dim / 2;
  if (8 * chunk >= rope_dim) return;
  const int first = interleaved ? 4 * chunk : (8 * chunk < half ? 8 * chunk : 8 * chunk - half);
  const float* pc = cos + pos * half + first;
  const float* ps = sin + pos * half + first;
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    if (j == 4 && interleaved) break;
    const float4 c4 = *reinterpret_cast<const float4*>(pc + j), s4 = *reinterpret_cast<const float4*>(ps + j);
    a.c[j] = c4.x, a.c[j + 1] = c4.y, a.c[j + 2] = c4.z, a.c[j + 3] = c4.w;
    a.s[j] = s4.x, a.s[j + 1] = s4.y, a.s[j + 2] = s4.z, a.s[j + 3] = s4.w;
  }
}

// Rotates the thread's eight elements by sign * angle.  Every thread of the
// warp takes part (the other half of a row is in its other threads).
__device__ __forceinline__ void rotate(float (&n)[8], const Angles& a, int rope_dim, bool interleaved, int chunk,
                                       float sign) {
  if (rope_dim == 0) return;
  if (interleaved) {
    if (8 * chunk >= rope_dim) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float c = a.c[j], s = sign * a.s[j], x = n[2 * j], y = n[2 * j + 1];
      n[2 * j] = x * c - y * s;
      n[2 * j + 1] = y * c + x * s;
    }
    return;
  }
  const int half_chunks = rope_dim / 16;
  const bool first = chunk < half_chunks, second = !first && chunk < 2 * half_chunks;
  const int lane = threadIdx.x & 31;
  const int other = first ? lane + half_chunks : second ? lane - half_chunks : lane;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float o = __shfl_sync(0xffffffffu, n[j], other);
    // first half: x cos - y sin; second: y cos + x sin
    if (first) n[j] = n[j] * a.c[j] - o * (sign * a.s[j]);
    else if (second) n[j] = n[j] * a.c[j] + o * (sign * a.s[j]);
  }
}

template <bool BF16>
__device__ __forceinline__ void load_weight(const void* w, int chunk, float (&f)[8]) {
  if (w != nullptr) {
    unpack8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + 8 * chunk), f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.f;
  }
}

// Where a token stands: its position, and in the paged form its page and slot.
struct Place {
  bool ok;        // the token has a valid place
  int64_t pos;
  int64_t k_off, v_off;  // element offsets of (page, slot) in k_pages and v_pages
};

__device__ __forceinline__ Place place_of(const RopeParams& p, int t) {
  Place r{false, 0, 0, 0};
  if (!p.paged) {
    r.pos = p.positions != nullptr ? p.positions[t] : 0;
    r.ok = p.rope_dim == 0 || (r.pos >= 0 && r.pos < p.max_position);
    if (!r.ok) atomicCAS(p.status, 0, (int)kDevBadIndex);
    return r;
  }
  // The sequence of token t: equal shares, or the last s with cu[s] <= t.
  int s, first, n;
  if (p.cu_seqlens == nullptr) {
    n = p.tokens_per_seq;
    s = t / n;
    first = s * n;
  } else {
    int lo = 0, hi = p.num_seqs;  // cu[lo] <= t < cu[hi], once cu is checked
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_seqlens[mid] <= t) lo = mid;
      else hi = mid;
    }
    s = lo;
    first = p.cu_seqlens[s];
    const int end = p.cu_seqlens[s + 1];
    if (t >= end && s + 1 == p.num_seqs) return r;  // a row behind the last sequence
    n = end - first;
    if (first > t || t >= end || first < 0 || end > p.total_tokens) {
      atomicCAS(p.status, 0, (int)kDevBadSeqlens);
      return r;
    }
  }
  const int64_t pos = (int64_t)p.seqlens_k[s] - n + (t - first);
  if (pos < 0) return r;  // the token has no place in the cache
  const int64_t col = pos >> p.page_shift;
  if (col >= p.max_pages) {
    atomicCAS(p.status, 0, (int)kDevBadSeqlens);
    return r;
  }
  if (p.rope_dim > 0 && pos >= p.max_position) {
    atomicCAS(p.status, 0, (int)kDevBadIndex);
    return r;
  }
  const int page = p.block_table[(int64_t)s * p.table_stride + col];
  if (page < 0 || page >= p.num_pages) {
    atomicCAS(p.status, 0, (int)kDevBadIndex);
    return r;
  }
  const int64_t slot = pos & ((1 << p.page_shift) - 1);
  r.ok = true;
  r.pos = pos;
  r.k_off = page * p.kp_sp + slot * p.kp_st;
  r.v_off = page * p.vp_sp + slot * p.vp_st;
  return r;
}

// Group of D/8 threads: HP consecutive heads of one token, so that the
// position, its angles and the weights are read once for all of them.  The
// heads of a token are numbered q, then k, then (paged) v; a group's heads are
// all of one kind.
template <int D, bool BF16, int HP>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeParams p) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  const int chunk = threadIdx.x % LANES;
  const int cq = (p.Hq + HP - 1) / HP, ck = (p.Hk + HP - 1) / HP, per_token = cq + (p.paged ? 2 : 1) * ck;
  const int64_t item = (int64_t)blockIdx.x * GROUPS + threadIdx.x / LANES;
  const bool live = item < (int64_t)p.total_tokens * per_token;
  const int t = live ? (int)(item / per_token) : 0;
  int c = live ? (int)(item - (int64_t)t * per_token) : 0;
  const int kind = c < cq ? 0 : c < cq + ck ? 1 : 2;
  c -= kind == 0 ? 0 : kind == 1 ? cq : cq + ck;
  const int h0 = c * HP, heads = kind == 0 ? p.Hq : p.Hk;
  const void* src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  const int64_t st = kind == 0 ? p.q_st : kind == 1 ? p.k_st : p.v_st;
  const int64_t sh = kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh;
  const uint16_t* in = static_cast<const uint16_t*>(src) + t * st + 8 * chunk;

  uint4 raw[HP];
#pragma unroll
  for (int i = 0; i < HP; ++i)
    raw[i] = live && h0 + i < heads ? *reinterpret_cast<const uint4*>(in + (h0 + i) * sh) : make_uint4(0, 0, 0, 0);

  Place at{false, 0, 0, 0};
  if (live) at = place_of(p, t);
  const bool ok = live && at.ok;
  uint16_t* out;
  int64_t oh;
  if (kind == 0) {
    out = static_cast<uint16_t*>(p.q_out) + t * p.qo_st;
    oh = p.qo_sh;
  } else if (kind == 1) {
    out = static_cast<uint16_t*>(p.k_out) + (p.paged ? at.k_off : t * p.kp_st);
    oh = p.kp_sh;
  } else {
    out = static_cast<uint16_t*>(p.v_out) + at.v_off;
    oh = p.vp_sh;
  }
  out += 8 * chunk;

  const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  float w[8];
  load_weight<BF16>(weight, chunk, w);
  Angles ang;
  const int rope_dim = kind == 2 ? 0 : p.rope_dim;
  if (ok && rope_dim > 0) load_angles(ang, p.cos, p.sin, at.pos, rope_dim, p.interleaved, chunk);

#pragma unroll
  for (int i = 0; i < HP; ++i) {
    float x[8];
    unpack8<BF16>(raw[i], x);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    ss = row_sum<LANES>(ss);
    const float r = weight != nullptr ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    // A warp holds groups of different kinds: all of them shuffle.
    rotate(x, ang, p.rope_dim, p.interleaved, rope_dim > 0 ? chunk : 1 << 20, 1.f);
    if (ok && h0 + i < heads)
      *reinterpret_cast<uint4*>(out + (h0 + i) * oh) = kind == 2 ? raw[i] : pack8<BF16>(x);
  }
}

// Gradients.  Each group strides over (token, HP heads) items and keeps the
// weight gradients of its rows in registers; a block leaves one partial sum
// per weight element, and rope_bwd_weights_kernel adds them in a fixed order.
template <int D, bool BF16, int HP>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(RopeBwdParams p) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  const int chunk = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const int cq = (p.Hq + HP - 1) / HP, ck = (p.Hk + HP - 1) / HP, per_token = cq + ck;
  const int64_t items = (int64_t)p.total_tokens * per_token, stride = (int64_t)gridDim.x * GROUPS;
  float accq[8], acck[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) accq[j] = acck[j] = 0.f;

  // Every warp makes the same number of rounds in all its groups (shuffles).
  const int64_t first = (int64_t)blockIdx.x * GROUPS + grp;
  const int64_t rounds = (items - (int64_t)blockIdx.x * GROUPS + stride - 1) / stride;
  for (int64_t round = 0; round < rounds; ++round) {
    const int64_t item = first + round * stride;
    const bool live = item < items;
    const int t = live ? (int)(item / per_token) : 0;
    const int c = live ? (int)(item - (int64_t)t * per_token) : 0;
    const bool is_q = c < cq;
    const int h0 = (is_q ? c : c - cq) * HP, heads = is_q ? p.Hq : p.Hk;
    const int64_t xh = is_q ? p.q_sh : p.k_sh, gh = is_q ? p.dqo_sh : p.dko_sh, oh = is_q ? p.dq_sh : p.dk_sh;
    const uint16_t* in = static_cast<const uint16_t*>(is_q ? p.q : p.k) + t * (is_q ? p.q_st : p.k_st) + 8 * chunk;
    const uint16_t* up =
        static_cast<const uint16_t*>(is_q ? p.dq_out : p.dk_out) + t * (is_q ? p.dqo_st : p.dko_st) + 8 * chunk;
    uint16_t* out = static_cast<uint16_t*>(is_q ? p.dq : p.dk) + t * (is_q ? p.dq_st : p.dk_st) + 8 * chunk;

    uint4 rx[HP], rg[HP];
#pragma unroll
    for (int i = 0; i < HP; ++i) {
      const bool on = live && h0 + i < heads;
      rx[i] = on ? *reinterpret_cast<const uint4*>(in + (h0 + i) * xh) : make_uint4(0, 0, 0, 0);
      rg[i] = on ? *reinterpret_cast<const uint4*>(up + (h0 + i) * gh) : make_uint4(0, 0, 0, 0);
    }
    int64_t pos = 0;
    bool ok = live;
    if (live && p.rope_dim > 0) {
      pos = p.positions[t];
      ok = pos >= 0 && pos < p.max_position;
      if (!ok) atomicCAS(p.status, 0, (int)kDevBadIndex);
    }
    Angles ang;
    if (ok && p.rope_dim > 0) load_angles(ang, p.cos, p.sin, pos, p.rope_dim, p.interleaved, chunk);
    const void* weight = is_q ? p.q_weight : p.k_weight;
    float w[8], dw[8];
    load_weight<BF16>(weight, chunk, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = 0.f;

#pragma unroll
    for (int i = 0; i < HP; ++i) {
      float x[8], g[8];
      unpack8<BF16>(rx[i], x);
      unpack8<BF16>(rg[i], g);
      rotate(g, ang, p.rope_dim, p.interleaved, chunk, -1.f);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(x[j], x[j], ss);
        dot = fmaf(g[j] * w[j], x[j], dot);
      }
      ss = row_sum<LANES>(ss);
      dot = row_sum<LANES>(dot);
      if (weight != nullptr) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const float m = r * r * (dot * (1.f / D));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (ok) dw[j] = fmaf(g[j] * x[j], r, dw[j]);
          g[j] = r * (g[j] * w[j] - x[j] * m);
        }
      }
      if (ok && h0 + i < heads) *reinterpret_cast<uint4*>(out + (h0 + i) * oh) = pack8<BF16>(g);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      accq[j] += is_q ? dw[j] : 0.f;
      acck[j] += is_q ? 0.f : dw[j];
    }
  }

  if (p.dq_weight == nullptr && p.dk_weight == nullptr) return;
  __shared__ float sums[GROUPS][2 * D];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sums[grp][8 * chunk + j] = accq[j];
    sums[grp][D + 8 * chunk + j] = acck[j];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) v += sums[g][e];
    p.partials[(int64_t)blockIdx.x * 2 * D + e] = v;
  }
}

// dw[e] = sum over the blocks' partials, 32 elements a block: 8 strided sums
// in parallel, joined in order, so the result does not depend on timing.
__global__ void __launch_bounds__(256) rope_bwd_weights_kernel(const float* partials, int blocks, int D, float* dqw,
                                                               float* dkw) {
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  float v = 0.f;
  for (int b = part; b < blocks; b += 8) v += partials[(int64_t)b * 2 * D + e];
  __shared__ float s[8][32];
  s[part][lane] = v;
  __syncthreads();
  if (part != 0) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += s[i][lane];
  if (e < D) {
    if (dqw != nullptr) dqw[e] = v;
  } else if (dkw != nullptr) {
    dkw[e - D] = v;
  }
}

template <int D, bool BF16, int HP>
cudaError_t fwd(const RopeParams& p, cudaStream_t s) {
  constexpr int GROUPS = kThreads / (D / 8);
  const int64_t cq = (p.Hq + HP - 1) / HP, ck = (p.Hk + HP - 1) / HP;
  const int64_t blocks = ((cq + (p.paged ? 2 : 1) * ck) * p.total_tokens + GROUPS - 1) / GROUPS;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  rope_kernel<D, BF16, HP><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t bwd(const RopeBwdParams& p, cudaStream_t s) {
  if (p.blocks > 0) rope_bwd_kernel<D, BF16, kRopeBwdHeads><<<(unsigned)p.blocks, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (p.dq_weight == nullptr && p.dk_weight == nullptr)) return e;
  rope_bwd_weights_kernel<<<2 * D / 32, 256, 0, s>>>(p.partials, p.blocks, D, p.dq_weight, p.dk_weight);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int D, bool bf16, const RopeParams& p, cudaStream_t s) {
  switch (D) {
    case 32: return bf16 ? fwd<32, true, 1>(p, s) : fwd<32, false, 1>(p, s);
    case 64: return bf16 ? fwd<64, true, 1>(p, s) : fwd<64, false, 1>(p, s);
    default: return bf16 ? fwd<128, true, 1>(p, s) : fwd<128, false, 1>(p, s);
  }
}

cudaError_t launch_rope_bwd(int D, bool bf16, const RopeBwdParams& p, cudaStream_t s) {
  switch (D) {
    case 32: return bf16 ? bwd<32, true>(p, s) : bwd<32, false>(p, s);
    case 64: return bf16 ? bwd<64, true>(p, s) : bwd<64, false>(p, s);
    default: return bf16 ? bwd<128, true>(p, s) : bwd<128, false>(p, s);
  }
}

}  // namespace etattn
