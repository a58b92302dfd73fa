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
// bounds these kernels once the instructions per element are few.  D/16
// threads hold a row, two 16-byte chunks each, chosen so that both elements of
// every pair are in one thread: pair rotation needs no exchange, and a row's
// two sums take log2(D/16) shuffles.  All heads of a group of threads share
// the token and so the coefficients: with P = w cos and Q = -/+ w sin of the
// partner folded together, an output is r (x P + x_partner Q), in paired FP32
// arithmetic.
//
// Measured (GB300, 16384 tokens, 32 + 8 heads of 128, BF16, CUDA graph; the
// plain copy reaches 6.80 TB/s): norm and rotation 54.2 us, 6.35 TB/s (51.4
// without the rotation, whose angles each group reads again); gradients 80 us,
// 6.39 TB/s; 16000 tokens into a cache 64.1 us, 6.26 TB/s; 8 tokens 2.3 us.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "launchers.h"
#include "cache_ptx.cuh"

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
    if (!r.ok) atomicCAS(p.status, 0, kDevBadIndex);
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
  const int keys = p.seqlens_k[s];
  const int64_t pos = (int64_t)keys - n + (t - first);
  if (keys >= 0 && pos < 0) return r;  // the token has no place in the cache
  const int64_t col = pos >> p.page_shift;
  if (keys < 0 || col >= p.max_pages) {
    atomicCAS(p.status, 0, (int)kDevBadSeqlens);
    return r;
  }
  if (p.rope_dim > 0 && pos >= p.max_position) {
    atomicCAS(p.status, 0, kDevBadIndex);
    return r;
  }
  const int page = p.block_table[(int64_t)s * p.table_stride + col];
  if (page < 0 || page >= p.num_pages) {
    atomicCAS(p.status, 0, kDevBadIndex);
    return r;
  }
  const int64_t slot = pos & ((1 << p.page_shift) - 1);
  r.ok = true;
  r.pos = pos;
  r.k_off = page * p.kp_sp + slot * p.kp_st;
  r.v_off = page * p.vp_sp + slot * p.vp_st;
  return r;
}

// Offsets that do not fit need not meet a token (one that decreases ends a
// sequence before it begins), so the grid's threads look at all of them: while
// a block's rows are on their way where a group takes one head (under 0.1 us at
// 8 to 256 tokens; at the end 0.1 to 0.3 us), at the end, out of line, where it
// takes several (no time at 16000 tokens; in line anywhere, the loop over the
// rows was compiled into one that took 2 % longer without offsets and 4 % with).
// 64 tokens in a batch of 20000 sequences: 5.2 us, 17 when one block looks.
__device__ __forceinline__ void check_offsets(const int* cu, int num_seqs, int total, int* status) {
  // (64 bits: 2^24 blocks, which 2^30 tokens of one head make, are 2^32 threads.)
  for (int64_t s = (int64_t)blockIdx.x * kThreads + threadIdx.x; s < num_seqs; s += (int64_t)gridDim.x * kThreads) {
    const int begin = cu[s], end = cu[s + 1];
    if (begin < 0 || end < begin || end > total) atomicCAS(status, 0, (int)kDevBadSeqlens);
  }
}
__device__ __noinline__ void check_offsets_apart(const int* cu, int num_seqs, int total, int* status) {
  check_offsets(cu, num_seqs, total, status);
}

// A group of D/16 threads takes HP consecutive heads of one token, so that the
// position, its angles and the weights are read once for all of them.  The
// heads of a token are numbered q, then k, then (paged) v; a group's heads are
// all of one kind.  FULL: the whole head is rotated.
template <int D, bool BF16, int HP, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, HP > 1 ? 3 : 4) rope_kernel(const __grid_constant__ RopeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int LANES = D / 16, GROUPS = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const Chunks ch = chunks_of(D, lane, FULL ? D : p.rope_dim, INTER);
  const int cq = (p.Hq + HP - 1) / HP, ck = (p.Hk + HP - 1) / HP, per_token = cq + (p.paged ? 2 : 1) * ck;
  const int64_t item = (int64_t)blockIdx.x * GROUPS + threadIdx.x / LANES;
  const bool live = item < (int64_t)p.total_tokens * per_token;
  const int t = live ? (int)div_pos(item, per_token) : 0;
  int c = live ? (int)(item - (int64_t)t * per_token) : 0;
  const int kind = c < cq ? 0 : c < cq + ck ? 1 : 2;
  c -= kind == 0 ? 0 : kind == 1 ? cq : cq + ck;
  const int h0 = c * HP, heads = kind == 0 ? p.Hq : p.Hk;
  const void* src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  const int64_t st = kind == 0 ? p.q_st : kind == 1 ? p.k_st : p.v_st;
  const int64_t sh = kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh;
  const uint16_t* in = static_cast<const uint16_t*>(src) + t * st + h0 * sh;

  // One row a group (few rows: latency counts) waits in registers; several are
  // all on their way at once into the thread's cells, [row][half][thread].
  constexpr bool STAGED = HP > 1;
  extern __shared__ uint4 cells[];
  uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    if (live && h0 + i < heads) {
      if constexpr (STAGED) {
        copy_async(cells + (2 * i) * kThreads + threadIdx.x, in + i * sh + ch.first);
        copy_async(cells + (2 * i + 1) * kThreads + threadIdx.x, in + i * sh + ch.second);
      } else {
        ra = *reinterpret_cast<const uint4*>(in + ch.first);
        rb = *reinterpret_cast<const uint4*>(in + ch.second);
      }
    }
    if constexpr (STAGED) copy_commit();
  }

  if (!STAGED && p.cu_seqlens != nullptr)
    check_offsets(p.cu_seqlens, p.num_seqs, p.total_tokens, p.status);
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
  out += h0 * oh;

  const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  float P[16], Q[16];
  {
    float w[16], c8[8], s8[8];
    load_weight<BF16>(weight, ch, w);
    load_angles(c8, s8, p.cos, p.sin, ok ? at.pos : 0, FULL ? D : p.rope_dim, ch, ok && kind != 2);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      P[j] = w[j] * c8[pair_of<INTER>(j)];
      Q[j] = (is_first<INTER>(j) ? -1.f : 1.f) * w[partner<INTER>(j)] * s8[pair_of<INTER>(j)];
    }
  }

#pragma unroll
  for (int i = 0; i < HP; ++i) {
    if constexpr (STAGED) {
      copy_wait_for(HP - 1 - i);
      ra = cells[(2 * i) * kThreads + threadIdx.x];
      rb = cells[(2 * i + 1) * kThreads + threadIdx.x];
    }
    float x[16], y[16];
    unpack16<BF16>(ra, rb, x);
    const float ss = row_sum<LANES>(dot16(x, x));
    turn16<INTER, FULL>(x, P, Q, ch, y);
    if (weight != nullptr) {
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int j = 0; j < 16; j += 2) fma2_keep(y[j], y[j + 1], y[j], y[j + 1], r, r, -0.f, -0.f);
    }
    if (ok && h0 + i < heads) {
      if (kind == 2) {
        *reinterpret_cast<uint4*>(out + i * oh + ch.first) = ra;
        *reinterpret_cast<uint4*>(out + i * oh + ch.second) = rb;
      } else {
        store16<BF16>(out + i * oh, ch, y);
      }
    }
  }
  if (STAGED && p.cu_seqlens != nullptr && (int64_t)blockIdx.x * kThreads < p.num_seqs)
    check_offsets_apart(p.cu_seqlens, p.num_seqs, p.total_tokens, p.status);
}

// Gradients.  The first q_blocks blocks take q's rows and the others k's.  Each
// group strides over (token, HP heads) items and keeps the weight gradient of
// its rows in registers; a block leaves one partial sum per weight element,
// and rope_bwd_weights_kernel adds them in a fixed order.
template <int D, bool BF16, int HP, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, 2) rope_bwd_kernel(const __grid_constant__ RopeBwdParams p) {
  constexpr int LANES = D / 16, GROUPS = kThreads / LANES;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const Chunks ch = chunks_of(D, lane, FULL ? D : p.rope_dim, INTER);
  const bool is_q = (int)blockIdx.x < p.q_blocks;
  const int block = is_q ? blockIdx.x : blockIdx.x - p.q_blocks;
  const int blocks = is_q ? p.q_blocks : p.blocks - p.q_blocks;
  const int heads = is_q ? p.Hq : p.Hk;
  const int64_t xh = is_q ? p.q_sh : p.k_sh, gh = is_q ? p.dqo_sh : p.dko_sh, oh = is_q ? p.dq_sh : p.dk_sh;
  const int64_t xt = is_q ? p.q_st : p.k_st, gt = is_q ? p.dqo_st : p.dko_st, ot = is_q ? p.dq_st : p.dk_st;
  const uint16_t* x0 = static_cast<const uint16_t*>(is_q ? p.q : p.k);
  const uint16_t* g0 = static_cast<const uint16_t*>(is_q ? p.dq_out : p.dk_out);
  uint16_t* d0 = static_cast<uint16_t*>(is_q ? p.dq : p.dk);
  const void* weight = is_q ? p.q_weight : p.k_weight;
  float w[16], acc[16];
  load_weight<BF16>(weight, ch, w);
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;

  // Items are (token, HP heads), the group's own `stride` apart; a step of the
  // walk is step_t tokens and step_h heads, with a carry.
  const int per_token = (heads + HP - 1) / HP, stride = blocks * GROUPS;
  const int step_t = stride / per_token, step_h = (stride - step_t * per_token) * HP, all_h = per_token * HP;
  struct Item {
    int t, h;  // token (p.total_tokens or more: past the end) and first head
  };
  auto next = [&](Item x) {
    x.t += step_t;
    x.h += step_h;
    if (x.h >= all_h) x.h -= all_h, ++x.t;
    return x;
  };
  // While row i of an item is worked on, the item's later rows and the next
  // item's earlier ones are on their way into the thread's cells ([row][x, x,
  // dy, dy][thread]), and so are the next item's angles ([set][cos, cos, sin,
  // sin][thread]); positions are read an item ahead of that.
  extern __shared__ uint4 cells[];
  uint4* const row_cells = cells + threadIdx.x;
  uint4* const angle_cells = cells + HP * 4 * kThreads + threadIdx.x;
  const bool turn_first = p.rope_dim > 0 && ch.turn_first, turn_second = p.rope_dim > 0 && ch.turn_second;
  auto position = [&](Item x) { return x.t < p.total_tokens && p.rope_dim > 0 ? p.positions[x.t] : -1; };
  auto fetch_row = [&](Item x, int i) {
    if (x.t < p.total_tokens && x.h + i < heads) {
      const uint16_t* in = x0 + x.t * xt + (x.h + i) * xh;
      const uint16_t* up = g0 + x.t * gt + (x.h + i) * gh;
      copy_async(row_cells + (4 * i) * kThreads, in + ch.first);
      copy_async(row_cells + (4 * i + 1) * kThreads, in + ch.second);
      copy_async(row_cells + (4 * i + 2) * kThreads, up + ch.first);
      copy_async(row_cells + (4 * i + 3) * kThreads, up + ch.second);
    }
  };
  auto fetch_angles = [&](int pos, int set) {
    if (pos < 0 || pos >= p.max_position) return;
    const int64_t row = (int64_t)pos * (p.rope_dim / 2);
    uint4* dst = angle_cells + set * 4 * kThreads;
    if (turn_first) {
      copy_async_shared(dst, p.cos + row + ch.angle_first);
      copy_async_shared(dst + 2 * kThreads, p.sin + row + ch.angle_first);
    }
    if (turn_second) {
      copy_async_shared(dst + kThreads, p.cos + row + ch.angle_second);
      copy_async_shared(dst + 3 * kThreads, p.sin + row + ch.angle_second);
    }
  };
  const int start = block * GROUPS + grp;
  Item item{start / per_token, (start % per_token) * HP};
  Item after = next(item), second = next(after);
  int pos = position(item), pos_next = position(after), set = 0;
  fetch_angles(pos, 0);
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    fetch_row(item, i);
    copy_commit();
  }
  // A warp's groups walk on until the last of them is past the end (they
  // shuffle together).
  for (; __any_sync(0xffffffffu, item.t < p.total_tokens); set ^= 1, item = after, after = second, second = next(second)) {
    const bool live = item.t < p.total_tokens;
    uint16_t* out = d0 + (live ? item.t * ot + item.h * oh : 0);
    const int h0 = item.h;
    const bool ok = live && (p.rope_dim == 0 || (pos >= 0 && pos < p.max_position));
    if (live && !ok) atomicCAS(p.status, 0, kDevBadIndex);
    fetch_angles(pos_next, set ^ 1);  // part of the next group that is committed
    pos = pos_next;
    pos_next = position(second);
    float c8[8], s8[8];

#pragma unroll
    for (int i = 0; i < HP; ++i) {
      copy_wait<HP - 1>();
      const bool on = ok && h0 + i < heads;
      if (i == 0) {
        const float* c4 = reinterpret_cast<const float*>(angle_cells + set * 4 * kThreads);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = (j >> 2) * kThreads * 4 + (j & 3);
          const bool turn = j < 4 ? turn_first : turn_second;
          c8[j] = turn ? c4[at] : 1.f;
          s8[j] = turn ? c4[2 * kThreads * 4 + at] : 0.f;
        }
      }
      float x[16], g[16];
      unpack16<BF16>(row_cells[(4 * i) * kThreads], row_cells[(4 * i + 1) * kThreads], x);
      {
        float dy[16], P[16], Q[16];
        unpack16<BF16>(row_cells[(4 * i + 2) * kThreads], row_cells[(4 * i + 3) * kThreads], dy);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          P[j] = c8[pair_of<INTER>(j)];
          Q[j] = is_first<INTER>(j) ? s8[pair_of<INTER>(j)] : -s8[pair_of<INTER>(j)];
        }
        turn16<INTER, FULL>(dy, P, Q, ch, g);
      }
      if (weight != nullptr) {
        float gw[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) fma2_keep(gw[j], gw[j + 1], g[j], g[j + 1], w[j], w[j + 1], 0.f, 0.f);
        const float ss = row_sum<LANES>(dot16(x, x));
        const float dot = row_sum<LANES>(dot16(gw, x));
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const float m = -r * (dot * (1.f / D)) * r;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float n0, n1;  // the normed row
          fma2_keep(n0, n1, x[j], x[j + 1], r, r, 0.f, 0.f);
          if (on) fma2_keep(acc[j], acc[j + 1], g[j], g[j + 1], n0, n1, acc[j], acc[j + 1]);
          fma2_keep(n0, n1, x[j], x[j + 1], m, m, gw[j], gw[j + 1]);
          fma2_keep(g[j], g[j + 1], n0, n1, r, r, 0.f, 0.f);
        }
      }
      if (on) store16<BF16>(out + i * oh, ch, g);
      fetch_row(after, i);  // x and dy of this row are in registers
      copy_commit();
    }
  }

  if (weight == nullptr) return;
  // The block's sum, over its groups in order, through the cells (which no
  // copy is on its way to any more).
  float* sums = reinterpret_cast<float*>(cells);  // [GROUPS][D]
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sums[grp * D + ch.first + j] = acc[j];
    sums[grp * D + ch.second + j] = acc[8 + j];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kThreads) {
    float v = 0.f;
#pragma unroll 8
    for (int g = 0; g < GROUPS; ++g) v += sums[g * D + e];
    p.partials[(int64_t)blockIdx.x * D + e] = v;
  }
}

// dw[e] = sum over the partials of q's blocks (blockIdx.y = 0) or k's, 32
// elements a block: 32 strided sums in parallel, joined in order, so the
// result does not depend on timing.
__global__ void __launch_bounds__(1024) rope_bwd_weights_kernel(const float* partials, int q_blocks, int blocks, int D,
                                                                float* dqw, float* dkw) {
  pdl_wait();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  float* dst = blockIdx.y == 0 ? dqw : dkw;
  if (dst == nullptr) return;
  const int end = blockIdx.y == 0 ? q_blocks : blocks;
  float v = 0.f;
#pragma unroll 8
  for (int b = (blockIdx.y == 0 ? 0 : q_blocks) + part; b < end; b += 32) v += partials[(int64_t)b * D + e];
  __shared__ float s[32][33];
  s[lane][part] = v;
  __syncthreads();
  v = row_sum<32>(s[part][lane]);  // warp `part` adds up element `part`
  if (lane == 0) dst[blockIdx.x * 32 + part] = v;
}

// The dynamic shared-memory opt-in is per device; set once per device.
template <typename P>
cudaError_t opt_in(void (*kern)(P), int smem, std::atomic<unsigned long long>& configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) configured.fetch_or(bit);
  }
  return e;
}

template <int D, bool BF16, int HP, bool INTER, bool FULL>
cudaError_t launch_fwd(const RopeParams& p, unsigned blocks, cudaStream_t s) {
  auto kern = rope_kernel<D, BF16, HP, INTER, FULL>;
  constexpr int SMEM = HP > 1 ? HP * 2 * kThreads * 16 : 0;
  if (SMEM > 48 * 1024) {
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = opt_in(kern, SMEM, configured);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(blocks), kThreads, SMEM, s, p);
}

// Blocks of `hp` heads a group over all items.
template <int D>
int64_t fwd_blocks(const RopeParams& p, int hp) {
  constexpr int GROUPS = kThreads / (D / 16);
  const int64_t cq = (p.Hq + hp - 1) / hp, ck = (p.Hk + hp - 1) / hp;
  return ((cq + (p.paged ? 2 : 1) * ck) * p.total_tokens + GROUPS - 1) / GROUPS;
}

template <int D, bool BF16, int HP>
cudaError_t fwd(const RopeParams& p, cudaStream_t s) {
  const int64_t blocks = fwd_blocks<D>(p, HP);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const bool full = p.rope_dim == D;
  if (p.interleaved)
    return full ? launch_fwd<D, BF16, HP, true, true>(p, (unsigned)blocks, s)
                : launch_fwd<D, BF16, HP, true, false>(p, (unsigned)blocks, s);
  return full ? launch_fwd<D, BF16, HP, false, true>(p, (unsigned)blocks, s)
              : launch_fwd<D, BF16, HP, false, false>(p, (unsigned)blocks, s);
}

// One head a group while its blocks all run at once (four on each of a GB300's
// 152 SMs), else four, and eight (which read the angles and weights half as
// often) when more moves than the 126 MB L2 holds.  Measured with 32 + 8 heads
// of 128, us with 1 / 4 / 8 heads a group: 3.1 / 4.0 / 5.1 at 128 tokens, 4.8 /
// 4.5 / 5.1 at 512, 6.7 / 5.6 / 6.3 at 1024, 19 / 12.3 / 12.4 at 4096 (84 MB),
// 46 / 33.6 / 31.3 at 8192 and 87 / 59 / 55 at 16384; heads of 64: 4.8 / 4.8 /
// 5.5 at 1024, 20 / 13.0 / 13.5 at 8192 (84 MB), 46 / 33.9 / 32.1 at 16384.
constexpr int kOneHeadBlocks = 608;
constexpr int64_t kL2Bytes = 126 << 20;
template <int D, bool BF16>
cudaError_t fwd_any(const RopeParams& p, cudaStream_t s) {
  if (fwd_blocks<D>(p, 1) <= kOneHeadBlocks) return fwd<D, BF16, 1>(p, s);
  const int64_t heads = (int64_t)p.Hq + (p.paged ? 2 : 1) * p.Hk;
  return 4 * D * heads * p.total_tokens > kL2Bytes ? fwd<D, BF16, 8>(p, s) : fwd<D, BF16, 4>(p, s);
}

template <int D, bool BF16, bool INTER, bool FULL>
cudaError_t launch_bwd(const RopeBwdParams& p, cudaStream_t s) {
  auto kern = rope_bwd_kernel<D, BF16, kRopeBwdHeads, INTER, FULL>;
  constexpr int SMEM = (kRopeBwdHeads + 2) * 4 * kThreads * 16;
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = opt_in(kern, SMEM, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.blocks), kThreads, SMEM, s, p);
}

template <int D, bool BF16>
cudaError_t bwd(const RopeBwdParams& p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.blocks > 0) {
    const bool full = p.rope_dim == D;
    if (p.interleaved) e = full ? launch_bwd<D, BF16, true, true>(p, s) : launch_bwd<D, BF16, true, false>(p, s);
    else e = full ? launch_bwd<D, BF16, false, true>(p, s) : launch_bwd<D, BF16, false, false>(p, s);
  }
  if (e != cudaSuccess || (p.dq_weight == nullptr && p.dk_weight == nullptr)) return e;
  return launch_pdl(rope_bwd_weights_kernel, dim3(D / 32, 2), 1024, 0, s, (const float*)p.partials, p.q_blocks, p.blocks,
                    D, p.dq_weight, p.dk_weight);
}

}  // namespace

cudaError_t launch_rope(int D, bool bf16, const RopeParams& p, cudaStream_t s) {
  switch (D) {
    case 32: return bf16 ? fwd_any<32, true>(p, s) : fwd_any<32, false>(p, s);
    case 64: return bf16 ? fwd_any<64, true>(p, s) : fwd_any<64, false>(p, s);
    default: return bf16 ? fwd_any<128, true>(p, s) : fwd_any<128, false>(p, s);
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
