// Attention of a few new query rows per sequence over a paged key-value
// cache (a decode step), exact and in one pass over the cache.
//
// Mathematics.  Row i of a sequence reads the keys E(i) of the eligibility
// rule in etattn.h and keeps the streaming state (m, l, acc) of its base-2
// logits, rescaled whenever m grows; partial states of disjoint key sets
// merge by M = max m_s, l = sum l_s 2^(m_s - M), acc likewise.
//
// What bounds it: every key and value is read once and meets few query rows
// (the query heads of its KV head times the new tokens), far below the tensor
// core's ridge point, so the HBM does.  The kernel therefore keeps as many
// bytes in flight as shared memory holds and keeps the CTAs equally long:
//  * The key tiles of all (sequence, KV head, row tile) units are laid on one
//    line, in units order, and cut into `shares` equal pieces, one per CTA,
//    whatever the sequences' lengths.  A unit cut by a boundary leaves
//    partial states in the workspace and paged_join_kernel joins them.
//  * One producer warp looks up the pages of a tile and issues one TMA box
//    per page and 64 columns (the lanes work on different pages), STAGES
//    tiles ahead.
//  * Four consumer warps take a quarter of a tile's keys each, with a private
//    state, so that they never wait for one another inside a unit; the four
//    states merge through shared memory at its end.  The products run on
//    m16n8k16 MMAs: 16 or 32 rows per unit would leave 7/8 or 3/4 of a
//    128-row tcgen05 tile empty, and the products are no bound here.
//
// Masked keys: only tiles at the edge of some row's range are masked.  There
// a score of a key outside the row's range becomes -inf whatever the key
// holds, and the product with V runs once per token of the tile with the
// values outside that token's range replaced by 0, so that nothing stored
// outside a row's range (a NaN in a page's unused slots, say) reaches it.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "launchers.h"
#include "sm103_ptx.cuh"

namespace etattn {

template <int D_, int MT_>
struct PagedCfg {
  static constexpr int D = D_, MT = MT_;
  static constexpr int TK = D == 128 ? 64 : 128;      // keys per tile
  static constexpr int WK = TK / 4;                   // keys per consumer warp
  static constexpr int COLS = D > 64 ? 64 : D;        // columns of one TMA box
  static constexpr int HALVES = D / COLS;
  static constexpr int ROW_BYTES = COLS * 2;          // 128, or 64 for D = 32
  static constexpr int SUB_BYTES = TK * ROW_BYTES;    // one box column of a tile
  static constexpr int TILE_BYTES = HALVES * SUB_BYTES;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K and V
  static constexpr int STAGES = D == 32 ? 6 : 3;
  // Columns merged at a time: the four warps' rows fill 16 KB (MT = 16), or
  // 8 KB (MT = 32, which also holds Q), so that two CTAs fit on an SM.
  static constexpr int MERGE_COLS = MT == 16 ? (D < 64 ? D : 64) : 16;
  static constexpr int MERGE_BYTES = 4 * MT * MERGE_COLS * 4;
  static constexpr int Q_BYTES = MT == 16 ? 0 : MT * D * 2;
  static constexpr int OFF_MERGE = STAGES * STAGE_BYTES;
  static constexpr int OFF_Q = OFF_MERGE + MERGE_BYTES;
  static constexpr int OFF_STATE = OFF_Q + Q_BYTES;   // m and l: 2 x 4 warps x MT
  static constexpr int OFF_SCAN = OFF_STATE + 2 * 4 * MT * 4;
  static constexpr int OFF_BARS = OFF_SCAN + 64;
  static constexpr int SMEM_BYTES = OFF_BARS + 2 * STAGES * 8;
  static constexpr int CONSUMERS = 128, THREADS = 160;
};

// Everything of one sequence that the roles need.
struct PagedSeq {
  int n;        // new tokens (0: nothing to do)
  int t0;       // its first row of q
  int Lk;       // keys
  int tile0;    // first key tile any row reads
  int tiles;    // key tiles of a unit (at least 1: an empty unit still writes its rows)
  int nrt;      // row tiles
  int units;    // Hkv * nrt
};

template <class C>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int s) {
  PagedSeq q;
  q.n = p.tokens_per_seq;
  q.t0 = s * q.n;
  bool ok = true;
  if (p.cu_seqlens_q != nullptr) {
    q.t0 = p.cu_seqlens_q[s];
    const int end = p.cu_seqlens_q[s + 1];
    ok = q.t0 >= 0 && end >= q.t0 && end <= p.total_q && end - q.t0 <= p.max_seqlen_q;
    q.n = end - q.t0;
  }
  q.Lk = p.seqlens_k[s];
  ok = ok && q.Lk >= 0 && q.Lk <= p.max_keys;
  if (!ok) {
    atomicCAS(p.status, 0, (int)kDevBadSeqlens);
    q.n = 0;
  }
  // Keys that some row reads: row i stands at key position i + Lk - n.
  const int c0 = q.Lk - q.n;
  const int lo = max(0, c0 - p.win_left);
  const int hi = (int)min((int64_t)q.Lk - 1, (int64_t)q.Lk - 1 + p.win_right);
  q.tile0 = lo / C::TK;
  q.tiles = hi >= lo ? hi / C::TK - q.tile0 + 1 : 1;
  q.nrt = (q.n * p.group + C::MT - 1) / C::MT;
  q.units = p.Hkv * q.nrt;
  return q;
}

// A position on the line of tiles.
struct PagedWalk {
  PagedSeq q;
  int s, unit, tile;
};

template <class C>
__device__ __forceinline__ void paged_next_unit(const PagedParams& p, PagedWalk& w) {
  w.tile = 0;
  if (++w.unit < w.q.units) return;
  w.unit = 0;
  do {
    ++w.s;
    if (w.s >= p.num_seqs) {
      w.q.units = 0;
      return;
    }
    w.q = paged_seq<C>(p, w.s);
  } while (w.q.units == 0);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Byte offset of 16-byte column `c16` of row `row` in a tile as TMA writes it
// (128-byte swizzle: bits 4-6 take bits 7-9; 64-byte: bits 4-5 take bits 7-8).
template <class C>
__device__ __forceinline__ uint32_t tile_off(int row, int c16) {
  if constexpr (C::ROW_BYTES == 128) {
    return (uint32_t)((c16 >> 3) * C::SUB_BYTES + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
  } else {
    return (uint32_t)(row * 64 + ((c16 ^ ((row >> 1) & 3)) << 4));
  }
}

// Splits the line: where CTA `c` of `shares` starts, and its length.
__device__ __forceinline__ int64_t share_start(int64_t total, int shares, int c) {
  const int64_t each = total / shares, rest = total - each * shares;
  return c * each + min((int64_t)c, rest);
}
// The CTA that owns tile x.
__device__ __forceinline__ int share_of(int64_t total, int shares, int64_t x) {
  const int64_t each = total / shares, rest = total - each * shares;
  const int64_t big = rest * (each + 1);
  return (int)(x < big ? x / (each + 1) : rest + (x - big) / each);
}

template <int D, int MT, bool BF16>
__global__ void __launch_bounds__(160, 2) attn_paged_kernel(const __grid_constant__ CUtensorMap kmap,
                                                            const __grid_constant__ CUtensorMap vmap,
                                                            const __grid_constant__ PagedParams p) {
  using C = PagedCfg<D, MT>;
  constexpr int NM = MT / 16;  // 16-row MMA tiles
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty = full + C::STAGES;
  volatile int64_t* scan = reinterpret_cast<volatile int64_t*>(smem + C::OFF_SCAN);

  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 4);
    }
    fence_mbar_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  pdl_wait();

  // ------------------------------------------------ this CTA's piece of the line
  // Thread i sums up the tiles of its run of sequences; the thread whose run
  // holds the piece's first tile finds the place inside it.
  const int per = (p.num_seqs + C::THREADS - 1) / C::THREADS;
  const int s_begin = min(p.num_seqs, tid * per), s_end = min(p.num_seqs, s_begin + per);
  int64_t mine = 0;
  for (int s = s_begin; s < s_end; ++s) {
    const PagedSeq q = paged_seq<C>(p, s);
    mine += (int64_t)q.units * q.tiles;
  }
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < 5; ++w) {
    const int64_t v = scan[w];
    if (w < warp) before += v;
    total += v;
  }
  __syncthreads();
  const int share = blockIdx.x;
  const int64_t begin = share_start(total, p.shares, share), end = share_start(total, p.shares, share + 1);
  PagedShare* desc = p.desc + share;
  if (begin >= end) {
    if (tid == 0 && p.shares > 1) desc->parts = 0;
    return;
  }
  if (begin >= before && begin < before + mine) {
    int64_t at = before;
    for (int s = s_begin;; ++s) {
      const PagedSeq q = paged_seq<C>(p, s);
      const int64_t len = (int64_t)q.units * q.tiles;
      if (begin < at + len) {
        scan[0] = s;
        scan[1] = (begin - at) / q.tiles;
        scan[2] = (begin - at) % q.tiles;
        break;
      }
      at += len;
    }
  }
  __syncthreads();
  PagedWalk w;
  w.s = (int)scan[0];
  w.unit = (int)scan[1];
  w.tile = (int)scan[2];
  w.q = paged_seq<C>(p, w.s);
  const int count = (int)(end - begin);  // tiles of this CTA

  // The join of a unit that began in an earlier CTA is shared by the CTAs
  // that continue it: each leaves itself the unit and its CTAs.
  if (tid == 0 && p.shares > 1) {
    if (w.tile > 0) {
      const int64_t u0 = begin - w.tile;
      desc->t0 = w.q.t0;
      desc->n = w.q.n;
      desc->head0 = (w.unit / w.q.nrt) * p.group;
      desc->row0 = (w.unit % w.q.nrt) * MT;
      desc->first = share_of(total, p.shares, u0);
      desc->parts = share_of(total, p.shares, u0 + w.q.tiles - 1) - desc->first + 1;
    } else {
      desc->parts = 0;
    }
  }

  if (warp == 4) {
    // ---------------------------------------------- producer
    const int page_keys = 1 << p.page_shift;
    const int box_keys = min(page_keys, C::TK);
    const int boxes = C::TK / box_keys;  // pages of a tile (1 when a page holds whole tiles)
    const uint32_t box_bytes = (uint32_t)box_keys * C::ROW_BYTES;
    const uint64_t policy = l2_policy_evict_first();
    uint32_t phase = 1;
    int stage = 0;
    for (int i = 0; i < count; ++i) {
      const int head = w.unit / w.q.nrt;
      const int key0 = (w.q.tile0 + w.tile) * C::TK;
      // Keys that some row of the sequence reads; a box past them is not loaded.
      const int lo = max(0, w.q.Lk - w.q.n - p.win_left);
      const int hi = (int)min((int64_t)w.q.Lk - 1, (int64_t)w.q.Lk - 1 + p.win_right);
      if (!mbar_wait(empty + stage, phase, p.status)) return;
      uint8_t* base = smem + stage * C::STAGE_BYTES;
      uint32_t loads = 0;
      for (int b0 = 0; b0 < boxes; b0 += 32) {
        const int b = b0 + lane, k0 = key0 + b * box_keys;
        const bool on = b < boxes && k0 <= hi && k0 + box_keys > lo;
        loads += __popc(__ballot_sync(0xffffffffu, on));
      }
      if (lane == 0) mbar_arrive_expect_tx(full + stage, loads * 2 * C::HALVES * box_bytes);
      __syncwarp();
      for (int b = lane; b < boxes; b += 32) {
        const int k0 = key0 + b * box_keys;
        if (!(k0 <= hi && k0 + box_keys > lo)) continue;
        int page = p.block_table[(int64_t)w.s * p.table_stride + (k0 >> p.page_shift)];
        if (page < 0 || page >= p.num_pages) {
          atomicCAS(p.status, 0, (int)kDevBadIndex);
          page = p.num_pages;  // past the map: the box is filled with zeros
        }
        const int slot = k0 & (page_keys - 1);
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h) {
          uint8_t* dst = base + h * C::SUB_BYTES + b * box_bytes;
          tma_load_4d_hint(dst, &kmap, full + stage, h * C::COLS, (p.hn_swapped & 1) ? head : slot,
                           (p.hn_swapped & 1) ? slot : head, page, policy);
          tma_load_4d_hint(dst + C::TILE_BYTES, &vmap, full + stage, h * C::COLS, (p.hn_swapped & 2) ? head : slot,
                           (p.hn_swapped & 2) ? slot : head, page, policy);
        }
      }
      __syncwarp();
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
      if (++w.tile == w.q.tiles) paged_next_unit<C>(p, w);
    }
    return;
  }

  // ------------------------------------------------ consumers
  const int g = lane >> 2, t4 = lane & 3;
  float* st_m = reinterpret_cast<float*>(smem + C::OFF_STATE);
  float* st_l = st_m + 4 * MT;
  float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
  uint32_t phase = 0;
  int stage = 0, left = count;
  bool alive = true;
  while (left > 0) {
    const int head0 = (w.unit / w.q.nrt) * p.group, row0 = (w.unit % w.q.nrt) * MT;
    const int rows = min(MT, w.q.n * p.group - row0);
    const int delta = w.q.Lk - w.q.n;
    // The tokens of this row tile and the rows' key ranges (rows g, g + 8, ...).
    const int tok_first = row0 / p.group, tok_last = (row0 + rows - 1) / p.group;
    int tok[2 * NM], row_lo[2 * NM], row_hi[2 * NM];
#pragma unroll
    for (int j = 0; j < 2 * NM; ++j) {
      const int r = g + 8 * j;
      tok[j] = min((row0 + r) / p.group, tok_last);
      const int c = tok[j] + delta;
      row_lo[j] = max(0, c - p.win_left);
      row_hi[j] = (int)min((int64_t)w.q.Lk - 1, (int64_t)c + p.win_right);
    }
    // Keys in [in_lo, in_hi] are read by every row of the tile.
    const int in_lo = max(0, tok_last + delta - p.win_left);
    const int in_hi = (int)min((int64_t)w.q.Lk - 1, (int64_t)tok_first + delta + p.win_right);

    // Q: fragments in registers (MT = 16), or rows in shared memory.
    auto q_row = [&](int r) {
      const int rr = row0 + r, i = rr / p.group;
      return static_cast<const uint16_t*>(p.q) + (int64_t)(w.q.t0 + i) * p.q_st +
             (int64_t)(head0 + rr - i * p.group) * p.q_sh;
    };
    uint32_t qf[NM == 1 ? D / 16 : 1][4];
    if constexpr (NM == 1) {
      const uint16_t* r0 = g < rows ? q_row(g) : nullptr;
      const uint16_t* r1 = g + 8 < rows ? q_row(g + 8) : nullptr;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int d = ks * 16 + 2 * t4;
        qf[ks][0] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + d) : 0u;
        qf[ks][1] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + d) : 0u;
        qf[ks][2] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + d + 8) : 0u;
        qf[ks][3] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + d + 8) : 0u;
      }
    } else {
      // 16-byte column c of row r at r * 2D + ((c ^ (r & 7 of the row's columns)) * 16).
      constexpr int CH = D / 8, SWZ = CH < 8 ? CH - 1 : 7;
      for (int x = tid; x < MT * CH; x += C::CONSUMERS) {
        const int r = x / CH, c = x % CH;
        const uint4 v = r < rows ? *reinterpret_cast<const uint4*>(q_row(r) + 8 * c) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + r * 2 * D + ((c ^ (r & SWZ)) << 4)) = v;
      }
      named_barrier(1, C::CONSUMERS);
    }

    float m[2 * NM], l[2 * NM], o[NM][D / 8][4];
#pragma unroll
    for (int j = 0; j < 2 * NM; ++j) m[j] = -INFINITY, l[j] = 0.f;
#pragma unroll
    for (int a = 0; a < NM; ++a)
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[a][n][i] = 0.f;

    const bool from_start = w.tile == 0;
    const int here = min(left, w.q.tiles - w.tile);
    const bool to_end = w.tile + here == w.q.tiles;
    for (int x = 0; x < here; ++x) {
      const int key0 = (w.q.tile0 + w.tile + x) * C::TK + warp * C::WK;
      if (alive) alive = mbar_wait(full + stage, phase, p.status);
      if (alive) {
        const uint32_t kbase = smem_u32(smem + stage * C::STAGE_BYTES), vbase = kbase + C::TILE_BYTES;
        constexpr int KB = C::WK / 16;
        // S = Q K^T for the warp's keys.
        float sc[NM][2 * KB][4];
#pragma unroll
        for (int a = 0; a < NM; ++a)
#pragma unroll
          for (int n = 0; n < 2 * KB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[a][n][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t qa[NM][4];
          if constexpr (NM == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) qa[0][i] = qf[ks][i];
          } else {
            constexpr int CH = D / 8, SWZ = CH < 8 ? CH - 1 : 7;
#pragma unroll
            for (int a = 0; a < NM; ++a) {
              const int r = a * 16 + (lane & 15), c = ks * 2 + (lane >> 4);
              ldsm4(qa[a], smem_u32(smem + C::OFF_Q) + r * 2 * D + ((c ^ (r & SWZ)) << 4));
            }
          }
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            uint32_t b[4];
            // matrices: keys 0-7 / d 0-7, keys 0-7 / d 8-15, keys 8-15 / d 0-7, keys 8-15 / d 8-15
            const int row = warp * C::WK + kb * 16 + ((lane >> 4) << 3) + (lane & 7);
            ldsm4(b, kbase + tile_off<C>(row, ks * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int a = 0; a < NM; ++a) {
              mma16816<BF16>(sc[a][2 * kb], qa[a], b[0], b[1]);
              mma16816<BF16>(sc[a][2 * kb + 1], qa[a], b[2], b[3]);
            }
          }
        }
        const bool edge = key0 < in_lo || key0 + C::WK - 1 > in_hi;
        float mx[2 * NM];
#pragma unroll
        for (int j = 0; j < 2 * NM; ++j) mx[j] = -INFINITY;
#pragma unroll
        for (int a = 0; a < NM; ++a)
#pragma unroll
          for (int n = 0; n < 2 * KB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 2 * a + (i >> 1);
              float s = sc[a][n][i] * p.scale_log2;
              if (edge) {
                const int key = key0 + n * 8 + 2 * t4 + (i & 1);
                if (key < row_lo[j] || key > row_hi[j]) s = -INFINITY;
              }
              sc[a][n][i] = s;
              mx[j] = fmaxf(mx[j], s);
            }
        bool grew = false;
#pragma unroll
        for (int j = 0; j < 2 * NM; ++j) {
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 1));
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 2));
          grew = grew || mx[j] > m[j];
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int j = 0; j < 2 * NM; ++j) {
            const float mn = fmaxf(m[j], mx[j]);
            const float f = mn == -INFINITY ? 1.f : ex2_approx(m[j] - mn);
            m[j] = mn;
            l[j] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[j >> 1][n][2 * (j & 1)] *= f;
              o[j >> 1][n][2 * (j & 1) + 1] *= f;
            }
          }
        }
        // P = 2^(S - m), rounded to the input type for the product with V (a
        // relative half step per weight); l sums the unrounded values.
        uint32_t pf[NM][KB][4];
#pragma unroll
        for (int a = 0; a < NM; ++a)
#pragma unroll
          for (int n = 0; n < 2 * KB; ++n) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 2 * a + (i >> 1);
              e[i] = ex2_approx(sc[a][n][i] - (m[j] == -INFINITY ? 0.f : m[j]));
              l[j] += e[i];
            }
            pf[a][n >> 1][(n & 1) * 2] = BF16 ? pack_bf16x2(e[0], e[1]) : pack_f16x2(e[0], e[1]);
            pf[a][n >> 1][(n & 1) * 2 + 1] = BF16 ? pack_bf16x2(e[2], e[3]) : pack_f16x2(e[2], e[3]);
          }
        // O += P V.
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          // matrices (transposed): keys 0-7 / d 0-7, keys 8-15 / d 0-7, keys 0-7 / d 8-15, keys 8-15 / d 8-15
          const int row = warp * C::WK + kb * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
          if (!edge) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t b[4];
              ldsm4_trans(b, vbase + tile_off<C>(row, 2 * n + (lane >> 4)));
#pragma unroll
              for (int a = 0; a < NM; ++a) {
                mma16816<BF16>(o[a][2 * n], pf[a][kb], b[0], b[1]);
                mma16816<BF16>(o[a][2 * n + 1], pf[a][kb], b[2], b[3]);
              }
            }
          } else {
            // One pass per token: its range alone survives in V, and only its
            // rows take the product.
            const int key = key0 + kb * 16 + 2 * t4;
            for (int tk = tok_first; tk <= tok_last; ++tk) {
              const int lo = max(0, tk + delta - p.win_left);
              const int hi = (int)min((int64_t)w.q.Lk - 1, (int64_t)tk + delta + p.win_right);
              auto keep = [&](int k) { return k >= lo && k <= hi; };
              const uint32_t m0 = (keep(key) ? 0xffffu : 0u) | (keep(key + 1) ? 0xffff0000u : 0u);
              const uint32_t m1 = (keep(key + 8) ? 0xffffu : 0u) | (keep(key + 9) ? 0xffff0000u : 0u);
              if (__all_sync(0xffffffffu, (m0 | m1) == 0u)) continue;
#pragma unroll
              for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                ldsm4_trans(b, vbase + tile_off<C>(row, 2 * n + (lane >> 4)));
#pragma unroll
                for (int a = 0; a < NM; ++a)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816<BF16>(d, pf[a][kb], b[2 * h] & m0, b[2 * h + 1] & m1);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                      if (tok[2 * a + (i >> 1)] == tk) o[a][2 * n + h][i] += d[i];
                  }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + stage);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    left -= here;

    // Merge the four warps' states.
#pragma unroll
    for (int j = 0; j < 2 * NM; ++j) {
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
      if (t4 == 0) {
        st_m[warp * MT + g + 8 * j] = m[j];
        st_l[warp * MT + g + 8 * j] = l[j];
      }
    }
    named_barrier(1, C::CONSUMERS);
    float inv[2 * NM];
#pragma unroll
    for (int j = 0; j < 2 * NM; ++j) {
      const int r = g + 8 * j;
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) mm = fmaxf(mm, st_m[x * MT + r]);
      const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int x = 0; x < 4; ++x) ll += st_l[x * MT + r] * ex2_approx(st_m[x * MT + r] - ref);
      inv[j] = ll == 0.f ? 0.f : ex2_approx(m[j] - ref) / ll;  // no key: 0; a NaN sum stays one
    }
    const bool whole = from_start && to_end;
    // Where this piece of the unit goes: the output, or the workspace (slot 0
    // for a unit that began earlier, slot 1 for one that begins here).
    const int64_t part_row = ((int64_t)share * 2 + (from_start ? 1 : 0)) * MT;
    if (tid < rows) {
      const int r = tid;
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) mm = fmaxf(mm, st_m[x * MT + r]);
      const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int x = 0; x < 4; ++x) ll += st_l[x * MT + r] * ex2_approx(st_m[x * MT + r] - ref);
      const float lse = ll == 0.f ? -INFINITY : ref * 0.6931471805599453f + logf(ll);
      if (whole) {
        if (p.lse != nullptr) {
          const int rr = row0 + r, i = rr / p.group;
          p.lse[(int64_t)(head0 + rr - i * p.group) * p.total_q + w.q.t0 + i] = lse;
        }
      } else {
        p.part_lse[part_row + r] = lse;
      }
    }
    constexpr int MC = C::MERGE_COLS;
    auto swz = [](int r) { return MC >= 32 ? (r & 3) << 3 : ((r >> 1) & 1) << 3; };
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += MC) {
#pragma unroll
      for (int a = 0; a < NM; ++a)
#pragma unroll
        for (int n = 0; n < MC / 8; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = a * 16 + g + 8 * h;
            const float f = inv[2 * a + h];
            float2 v = make_float2(o[a][c0 / 8 + n][2 * h], o[a][c0 / 8 + n][2 * h + 1]);
            v.x *= f;
            v.y *= f;
            *reinterpret_cast<float2*>(merge + (warp * MT + r) * MC + ((n * 8) ^ swz(r)) + 2 * t4) = v;
          }
      named_barrier(1, C::CONSUMERS);
      for (int x = tid; x < rows * (MC / 8); x += C::CONSUMERS) {
        const int r = x / (MC / 8), c = (x % (MC / 8)) * 8;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float4* src = reinterpret_cast<const float4*>(merge + (y * MT + r) * MC + (c ^ swz(r)));
          const float4 u0 = src[0], u1 = src[1];
          v[0] += u0.x, v[1] += u0.y, v[2] += u0.z, v[3] += u0.w;
          v[4] += u1.x, v[5] += u1.y, v[6] += u1.z, v[7] += u1.w;
        }
        if (whole) {
          const int rr = row0 + r, i = rr / p.group;
          uint32_t u[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            u[k] = BF16 ? pack_bf16x2(v[2 * k], v[2 * k + 1]) : pack_f16x2(v[2 * k], v[2 * k + 1]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (int64_t)(w.q.t0 + i) * p.o_st +
                                    (int64_t)(head0 + rr - i * p.group) * p.o_sh + c0 + c) =
              make_uint4(u[0], u[1], u[2], u[3]);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (part_row + r) * D + c0 + c);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
      named_barrier(1, C::CONSUMERS);
    }
    w.tile += here;
    if (left > 0) paged_next_unit<C>(p, w);
  }
}

}  // namespace etattn
