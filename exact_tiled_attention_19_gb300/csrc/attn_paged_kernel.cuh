// Attention of a few new query rows per sequence over a paged key-value
// cache (a decode step), exact and in one pass over the cache.
//
// Mathematics.  Row i of a sequence reads the keys E(i) of the eligibility
// rule in etattn.h and keeps the streaming state (m, l, acc) of its base-2
// logits, rescaled whenever m grows; partial states of disjoint key sets
// merge by M = max m_s, l = sum l_s 2^(m_s - M), acc likewise.
//
// What bounds it: every key and value is read once for each row tile of up to
// 32 query rows (the query heads of its KV head times the new tokens: one tile
// in a decode step), far below the tensor core's ridge point, so the HBM does.  The kernel therefore keeps as many
// bytes in flight as shared memory holds and keeps the CTAs equally long:
//  * The key tiles of all (sequence, KV head, row tile) units are laid on one
//    line, in units order, and cut into `shares` equal pieces, one per CTA,
//    whatever the sequences' lengths.  A unit cut by a boundary leaves
//    partial states in the workspace and paged_join_kernel joins them.
//    Entering a unit costs about a tile's time beside its tiles, so a unit is
//    kUnitCost tiles longer on the line than it is.
//  * One producer warp walks the line: it looks up the pages of a tile one
//    tile ahead and issues one TMA box for K and one for V per page (the lanes
//    work on different pages), STAGES tiles ahead; a unit's Q rows and its
//    description go through a slot of their own, so that the consumers find
//    the next unit ready.
//  * Four consumer warps take a quarter of a tile's keys each, with a private
//    state, so that they never wait for one another inside a unit; the four
//    states merge through shared memory at its end.  The products run on
//    m16n8k16 MMAs: 16 rows would leave 7/8 of a 128-row tcgen05 tile empty,
//    and the products are no bound here.  Units of up to 32 rows have a second
//    group of four warps for rows 16 .. 31, on the same tiles.
//
// Masked keys: only tiles at the edge of some row's range are masked.  There
// a score of a key outside the row's range becomes -inf whatever the key
// holds, and the values that no row of the group reads are replaced by 0.  A
// value that some of them read and others do not meets weights of 0 in the
// latter; where such a value is not finite, the product runs once per token
// instead, with the values outside that token's range replaced by 0.  So
// nothing stored outside a row's range (a NaN in a page's unused slots, say)
// reaches it.
//
// Precision: scores, maxima, sums, accumulators and partial rows are FP32.  P
// meets V in two parts of the input type, P = hi + lo, so that a weight is off
// by 2^-16 of itself (BF16) and not by 2^-9: with P in one part the outputs
// were off from 64 bits by up to 12 % more than a rounding of the exact ones.
// The second product costs 0 to 2 % where the cache bounds (8 x 32768 keys 164.3
// us against 163.2, 64 ragged sequences 80.7 against 81.0), 9 to 15 % for units
// of 32 rows (202 against 185, heads of 64 134 against 116), 5 % for units of
// two tiles (220 against 209).
//
// Measured (GB300, D = 128, 32 query and 8 KV heads, BF16, one new token, CUDA
// graph, over several boxes): 8 sequences of 32768 keys 162 to 166 us, 6.5 to
// 6.6 TB/s of the 6.80 that a plain copy reaches; one of 524288 keys 320 to 326
// us, 6.6 to 6.7 TB/s; 64 of 1 .. 16384 keys 79 to 81 us, 5.9 to 6.05 TB/s (the
// units of short sequences cost their entry); one of 1000 keys 9 us (two
// launches, three dependent loads, the join).  32 rows (8 new tokens) over 8 x
// 32768 keys: 202 us, 64 rows 388.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "launchers.h"
#include "cache_ptx.cuh"

namespace etattn {

template <int D_, int MT_>
struct PagedCfg {
  static constexpr int D = D_, MT = MT_;
  static constexpr int GROUPS = MT / 16;              // of four consumer warps, 16 rows each
  static constexpr int TK = 8192 / D;                 // keys per tile: 16 KB each of K and V
  static constexpr int WK = TK / 4;                   // keys per consumer warp
  static constexpr int COLS = D > 64 ? 64 : D;        // columns of a box row
  static constexpr int HALVES = D / COLS;
  static constexpr int ROW_BYTES = COLS * 2;          // 128, or 64 for D = 32
  static constexpr int TILE_BYTES = TK * D * 2;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K and V
  // As many stages as let two CTAs of 16 rows (113 KB each), or one of 32,
  // share an SM.
  static constexpr int STAGES = 3 * GROUPS;
  static constexpr int MERGE_BYTES = 4 * 16 * 32 * 4; // a group's: four warps' 16 rows, 32 columns
  static constexpr int Q_PITCH = 2 * D + 16;          // padded: no bank conflicts
  static constexpr int OFF_MERGE = STAGES * STAGE_BYTES;
  static constexpr int OFF_Q = OFF_MERGE + GROUPS * MERGE_BYTES;
  static constexpr int OFF_STATE = OFF_Q + MT * Q_PITCH;  // a group's m and l: 2 x 4 warps x 16
  static constexpr int OFF_UNIT = OFF_STATE + GROUPS * 2 * 4 * 16 * 4;
  static constexpr int OFF_BARS = OFF_UNIT + 48;
  static constexpr int SMEM_BYTES = OFF_BARS + 2 * (STAGES + 1) * 8;
  static_assert(GROUPS == 1 ? SMEM_BYTES <= 115712 : SMEM_BYTES <= 232448, "two CTAs per SM, or one");
  static constexpr int CONSUMER_WARPS = 4 * GROUPS, THREADS = 32 * (CONSUMER_WARPS + 1);
};

// Tiles that entering a unit costs.  8 KV heads of 128, us with 1 / 2 / 3 / 4: 64
// ragged sequences of up to 16384 keys 86.6 / 79.6 / 79.4 / 79.9, 512 of up to
// 2048 keys 121 / 103 / 108 / 115.
constexpr int kUnitCost = 2;

// What FP16 weights, and the accumulators with them, are multiplied by.
constexpr float kF16Weight = 32768.f;

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

// A stretch of one unit's tiles, as the producer hands it to the consumers.
struct PagedUnit {
  int t0, n, Lk;         // the sequence
  int head0, row0;       // first query head, first row of the row tile
  int tile, tiles;       // first tile (of the sequence) and how many; 0 tiles: no more units
  int from_start, to_end;
  int pad[3];
};
static_assert(sizeof(PagedUnit) == 48, "");

// The sequences s_base .. s_base + 31, one per lane.
template <class C>
struct PagedWindow {
  PagedSeq mine;
  int base;
  __device__ __forceinline__ void load(const PagedParams& p, int s0, int lane) {
    base = s0;
    mine.n = mine.t0 = mine.Lk = mine.tile0 = mine.nrt = mine.units = 0;
    mine.tiles = 1;
    if (s0 + lane < p.num_seqs) mine = paged_seq<C>(p, s0 + lane);
  }
  __device__ __forceinline__ PagedSeq at(int s) const {
    const int src = s - base;
    PagedSeq q;
    q.n = __shfl_sync(0xffffffffu, mine.n, src);
    q.t0 = __shfl_sync(0xffffffffu, mine.t0, src);
    q.Lk = __shfl_sync(0xffffffffu, mine.Lk, src);
    q.tile0 = __shfl_sync(0xffffffffu, mine.tile0, src);
    q.tiles = __shfl_sync(0xffffffffu, mine.tiles, src);
    q.nrt = __shfl_sync(0xffffffffu, mine.nrt, src);
    q.units = __shfl_sync(0xffffffffu, mine.units, src);
    return q;
  }
};

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

// x, y >= 0 as hi + lo, each a pair of 16-bit values: hi by cutting bits off (no
// rounding to wait for), lo the rest, rounded.  hi is cut from a little less
// than x, so that lo is not 0 unless x is (or is 2^-28 of the largest weight in
// FP16): an infinite value must not meet 0.  Together they are off by 2^-16 of x
// (BF16: a rest of at most 2^-7 x, rounded by 2^-9 of it) or 2^-21 (FP16: cut
// from one step less, a rest of at most 2^-9 x, rounded by 2^-12 of it).
template <bool BF16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  constexpr uint32_t kKept = BF16 ? 0xffff0000u : 0xffffe000u;
  const uint32_t a = __viaddmax_s32(__float_as_int(x), BF16 ? -1 : -0x2000, 0);
  const uint32_t b = __viaddmax_s32(__float_as_int(y), BF16 ? -1 : -0x2000, 0);
  const float ha = __uint_as_float(a & kKept), hb = __uint_as_float(b & kKept);
  hi = BF16 ? __byte_perm(a, b, 0x7632) : pack_f16x2(ha, hb);
  lo = BF16 ? pack_bf16x2(x - ha, y - hb) : pack_f16x2(x - ha, y - hb);
}

// The halves of a register that hold keys k and k + 1 within [lo, hi], as a mask.
__device__ __forceinline__ uint32_t half_mask(int k, int lo, int hi) {
  return (k >= lo && k <= hi ? 0xffffu : 0u) | (k + 1 >= lo && k + 1 <= hi ? 0xffff0000u : 0u);
}

// Bits 15 and 31: whether the low and the high half are infinite or NaN (their
// exponent carries over when it is all ones).
template <bool BF16>
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
  return ((w & (BF16 ? 0x7f807f80u : 0x7c007c00u)) + (BF16 ? 0x00800080u : 0x04000400u)) & 0x80008000u;
}

// One arrival of the warp (by the lane that `arrives`) on `bar`, giving back shared memory that it has read.
// A read is issued before the arrival but need not have been served by then:
// nothing makes the arrival wait for a register that is still on its way, and a
// refill then overtakes the last reads (it did, where bank conflicts held them
// up).  So the arrival's address takes in `seen`, a value made of a register of
// every read (a read delivers its registers together), and with `zero` (a 0
// that the compiler does not know) leaves it where it is.
__device__ __forceinline__ void release_after(uint64_t* bar, uint32_t seen, uint32_t zero, bool arrives) {
  const uint32_t off = seen & zero;
  __syncwarp();
  if (arrives) mbar_arrive(reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(bar) + off));
  __syncwarp();
}

// Byte offset of 16-byte column `c16` in row `row` of a tile, beside where the
// row starts: TMA's 128-byte swizzle (bits 4-6 take bits 7-9), or its 64-byte
// one (bits 4-5 take bits 7-8).  `half` is the distance of columns 64 .. 127.
template <class C>
__device__ __forceinline__ uint32_t col_off(int row, int c16, uint32_t half) {
  if constexpr (C::ROW_BYTES == 128) {
    return (c16 >= 8 ? half : 0u) + (uint32_t)(((c16 & 7) ^ (row & 7)) << 4);
  } else {
    return (uint32_t)((c16 ^ ((row >> 1) & 3)) << 4);
  }
}

// The line cut into shares: the first `rest` of them one longer than `each`.
struct PagedCut {
  int64_t each, rest;
  __device__ __forceinline__ PagedCut(int64_t total, int shares) {
    each = div_pos(total, shares);
    rest = total - each * shares;
  }
  __device__ __forceinline__ int64_t start(int c) const { return c * each + min((int64_t)c, rest); }
  __device__ __forceinline__ int holder(int64_t x) const {
    const int64_t big = rest * (each + 1);
    return (int)(x < big ? div_pos(x, each + 1) : rest + div_pos(x - big, each));
  }
};

// What the producer warp knows of the ring: the stage to fill next, the parity
// to wait for on its `empty`, and on Q's.
struct PagedRing {
  int stage = 0;
  uint32_t phase = 1, uphase = 1;
};

// A wait that the whole warp takes the same way.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status)) != 0;
}

// The producer warp's walk along its piece of the line.  False: a wait ran out.
template <class C>
__device__ __forceinline__ bool paged_walk(const CUtensorMap& kmap, const CUtensorMap& vmap, const PagedParams& p,
                                           uint8_t* smem, int lane, PagedRing& ring) {
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty = full + C::STAGES;
  uint64_t* ufull = empty + C::STAGES;
  uint64_t* uempty = ufull + 1;
  PagedUnit* handed = reinterpret_cast<PagedUnit*>(smem + C::OFF_UNIT);

  // Nothing to join, until the end says otherwise: whatever the workspace held
  // must not be taken for a unit if a wait of this CTA runs out.
  const int share = blockIdx.x;
  PagedShare* desc = p.desc + share;
  if (lane == 0 && p.shares > 1) desc->parts = 0;

  // This CTA's piece of the line: lane i sums up its run of sequences; the
  // lane whose run holds the piece's start finds the sequence.  (With up to 32
  // sequences a run is the lane's sequence of the window.)
  PagedWindow<C> win;
  win.load(p, 0, lane);
  const bool one_each = p.num_seqs <= 32;
  const int per = (p.num_seqs + 31) / 32;
  const int s_begin = min(p.num_seqs, lane * per), s_end = min(p.num_seqs, s_begin + per);
  auto length = [](const PagedSeq& q) { return (int64_t)q.units * (q.tiles + kUnitCost); };
  int64_t mine = 0;
  if (one_each) mine = length(win.mine);
  else
    for (int s = s_begin; s < s_end; ++s) mine += length(paged_seq<C>(p, s));
  int64_t incl = mine;
  if (__all_sync(0xffffffffu, mine < (1 << 26))) {  // every sum fits in 32 bits
    int sum = (int)mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    incl = sum;
  } else {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
  }
  const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
  const PagedCut cut(total, p.shares);
  const int64_t begin = cut.start(share), end = cut.start(share + 1);
  if (begin >= end) return true;
  int s = lane;
  int64_t at = incl - mine;
  const bool holds = begin >= at && begin < incl;
  if (holds && !one_each)
    for (s = s_begin;; ++s) {
      const int64_t len = length(paged_seq<C>(p, s));
      if (begin < at + len) break;
      at += len;
    }
  const int holder = __ffs(__ballot_sync(0xffffffffu, holds)) - 1;
  s = __shfl_sync(0xffffffffu, s, holder);
  at = __shfl_sync(0xffffffffu, at, holder);
  if (!one_each) win.load(p, s, lane);
  PagedSeq q = win.at(s);
  int unit = (int)div_pos(begin - at, q.tiles + kUnitCost);
  int64_t u0 = at + (int64_t)unit * (q.tiles + kUnitCost);  // where the unit lies on the line
  int tile = max(0, (int)(begin - u0) - kUnitCost);

  PagedShare mark{};  // for the join, written at the end
  int64_t mark_u0 = 0;
  int mark_tiles = 0;
  if (tile > 0) {
    mark.t0 = q.t0;
    mark.n = q.n;
    mark.head0 = (unit / q.nrt) * p.group;
    mark.row0 = (unit % q.nrt) * C::MT;
    mark_u0 = u0 + kUnitCost;
    mark_tiles = q.tiles;
  }

  const int page_keys = 1 << p.page_shift;
  const int box_keys = min(page_keys, C::TK);
  const int boxes = C::TK / box_keys;  // pages of a tile (1 when a page holds whole tiles); at most 32
  const uint32_t box_bytes = (uint32_t)box_keys * 2 * C::D;
  const uint64_t policy = l2_policy_evict_first();

  // Unit by unit; `stop` is the end of this share's tiles in the unit.
  while (true) {
    const int stop = (int)max((int64_t)0, min((int64_t)q.tiles, end - u0 - kUnitCost));
    if (tile < stop) {
      const int head = unit / q.nrt;
      const int row0 = (unit - head * q.nrt) * C::MT, rows = min(C::MT, q.n * p.group - row0);
      // Keys that some row of the sequence reads; a box beside them is not loaded.
      const int lo = max(0, q.Lk - q.n - p.win_left);
      const int hi = (int)min((int64_t)q.Lk - 1, (int64_t)q.Lk - 1 + p.win_right);
      const int* table = p.block_table + (int64_t)s * p.table_stride;
      auto wants = [&](int k0) { return lane < boxes && k0 <= hi && k0 + box_keys > lo; };
      auto look_up = [&](int t) {
        const int k0 = (q.tile0 + t) * C::TK + lane * box_keys;
        return wants(k0) ? table[k0 >> p.page_shift] : 0;
      };
      int page = look_up(tile);

      if (!warp_wait(uempty, ring.uphase, p.status)) return false;
      ring.uphase ^= 1;
      if (lane == 0) {
        *handed = PagedUnit{q.t0, q.n, q.Lk, head * p.group, row0, q.tile0 + tile, stop - tile, tile == 0,
                            stop == q.tiles, {0, 0, 0}};
        mbar_arrive_expect_tx(ufull, (uint32_t)rows * 2 * C::D);
      }
      __syncwarp();
      if (lane < rows) {
        const int rr = row0 + lane, i = rr / p.group;
        bulk_load(smem + C::OFF_Q + lane * C::Q_PITCH,
                  static_cast<const uint16_t*>(p.q) + (int64_t)(q.t0 + i) * p.q_st +
                      (int64_t)(head * p.group + rr - i * p.group) * p.q_sh,
                  2 * C::D, ufull);
      }

      for (; tile < stop; ++tile) {
        const int k0 = (q.tile0 + tile) * C::TK + lane * box_keys;
        const bool on = wants(k0);
        int pg = page;
        if (tile + 1 < stop) page = look_up(tile + 1);
        const uint32_t loads = __popc(__ballot_sync(0xffffffffu, on));
        if (!warp_wait(empty + ring.stage, ring.phase, p.status)) return false;
        uint8_t* base = smem + ring.stage * C::STAGE_BYTES;
        if (lane == 0) mbar_arrive_expect_tx(full + ring.stage, loads * 2 * box_bytes);
        __syncwarp();
        if (on) {
          if (pg < 0 || pg >= p.num_pages) {
            atomicCAS(p.status, 0, kDevBadIndex);
            pg = p.num_pages;  // past the map: the box is filled with zeros
          }
          const int slot = k0 & (page_keys - 1);
          uint8_t* dst = base + lane * box_bytes;
          tma_load_5d_hint(dst, &kmap, full + ring.stage, 0, slot, 0, head, pg, policy);
          tma_load_5d_hint(dst + C::TILE_BYTES, &vmap, full + ring.stage, 0, slot, 0, head, pg, policy);
        }
        __syncwarp();
        if (++ring.stage == C::STAGES) {
          ring.stage = 0;
          ring.phase ^= 1;
        }
      }
    }
    // The next unit of the line.
    u0 += q.tiles + kUnitCost;
    if (u0 >= end) break;
    tile = 0;
    if (++unit == q.units) {
      unit = 0;
      do {  // u0 < end <= total: some later sequence has units
        if (++s == win.base + 32) win.load(p, s, lane);
        q = win.at(s);
      } while (q.units == 0);
    }
  }
  // The join of a unit that began in an earlier share is shared by those that
  // continue it: each leaves itself the unit and its shares.
  if (lane == 0 && mark_tiles > 0) {
    mark.first = cut.holder(mark_u0);
    mark.parts = cut.holder(mark_u0 + mark_tiles - 1) - mark.first + 1;
    *desc = mark;
  }
  return true;
}

// The producer warp: the walk, the end of the line, and its copies seen home.
template <class C>
__device__ __forceinline__ void paged_producer(const CUtensorMap& kmap, const CUtensorMap& vmap, const PagedParams& p,
                                               uint8_t* smem, int lane) {
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* ufull = full + 2 * C::STAGES;
  uint64_t* uempty = ufull + 1;
  PagedRing ring;
  const bool ended = paged_walk<C>(kmap, vmap, p, smem, lane, ring) && warp_wait(uempty, ring.uphase, p.status);
  if (ended && lane == 0) {
    reinterpret_cast<PagedUnit*>(smem + C::OFF_UNIT)->tiles = 0;
    mbar_arrive(ufull);
  }
  // Wait (bounded) until the last load into every stage has landed, and Q's, so
  // that no copy writes shared memory after the CTA has ended.  After a normal
  // run they have, or do soon, and Q's slot was free, after which ufull went on;
  // where a wait ran out some may not.
#pragma unroll 1
  for (int i = 0; i < C::STAGES; ++i)
    mbar_wait(full + i, i < ring.stage ? ring.phase ^ 1 : ring.phase, nullptr, 2 * kWaitLimitNs);
  if (!ended) mbar_wait(ufull, ring.uphase, nullptr, 2 * kWaitLimitNs);
}

// Barriers among a group's four warps.  For the only group the id is a
// constant: in a register it made entering and leaving a unit 0.5 us longer
// (15 % at 16000 units of two tiles); a branch between two constants made the
// two-group kernel's loop 7 % slower.
template <class C>
__device__ __forceinline__ void group_barrier(int grp) {
  named_barrier(C::GROUPS == 1 ? 1 : 1 + grp, 128);
}
template <class C>
__device__ __forceinline__ bool group_any(int grp, bool x) {
  return named_barrier_or(C::GROUPS == 1 ? 1 : 1 + grp, 128, x);
}

// Adds up a group's four warps' scaled rows, MC columns at a time through its
// 8 KB of shared memory, and writes them: the output, or the unit's partial
// rows.  Rows from ROWS on are nobody's.
template <class C, bool BF16, int MC, int ROWS>
__device__ __forceinline__ void paged_merge(const PagedParams& p, const PagedUnit& w, int grp, int rows, float* merge,
                                            const float (&o)[C::D / 8][4], const float (&inv)[2], bool whole,
                                            int64_t part_row) {
  static_assert(4 * ROWS * MC * 4 <= C::MERGE_BYTES, "");
  const int tid = C::GROUPS == 1 ? threadIdx.x : threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3, row0 = w.row0 + 16 * grp;
  auto swz = [](int r) { return (r & 3) << 3; };  // keeps a warp's eight rows out of one another's banks
#pragma unroll
  for (int c0 = 0; c0 < C::D; c0 += MC) {
#pragma unroll
    for (int n = 0; n < MC / 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = g + 8 * h;
        if (ROWS < 16 && r >= ROWS) continue;
        *reinterpret_cast<float2*>(merge + (warp * ROWS + r) * MC + ((n * 8) ^ swz(r)) + 2 * t4) =
            make_float2(o[c0 / 8 + n][2 * h] * inv[h], o[c0 / 8 + n][2 * h + 1] * inv[h]);
      }
    group_barrier<C>(grp);
    for (int x = tid; x < rows * (MC / 8); x += 128) {
      const int r = x / (MC / 8), c = (x % (MC / 8)) * 8;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float4* src = reinterpret_cast<const float4*>(merge + (y * ROWS + r) * MC + (c ^ swz(r)));
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
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (int64_t)(w.t0 + i) * p.o_st +
                                  (int64_t)(w.head0 + rr - i * p.group) * p.o_sh + c0 + c) =
            make_uint4(u[0], u[1], u[2], u[3]);
      } else {
        float4* dst = reinterpret_cast<float4*>(p.part_o + (part_row + r) * C::D + c0 + c);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    // The next columns, or the next unit's (whose state the warps write first,
    // and meet, before they come here again).
    if (c0 + MC < C::D) group_barrier<C>(grp);
  }
}

template <int D, int MT, bool BF16>
__global__ void __launch_bounds__(PagedCfg<D, MT>::THREADS, MT == 16 ? 2 : 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ PagedParams p) {
  using C = PagedCfg<D, MT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty = full + C::STAGES;
  uint64_t* ufull = empty + C::STAGES;
  uint64_t* uempty = ufull + 1;

  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, C::CONSUMER_WARPS);
    }
    mbar_init(ufull, 1);
    mbar_init(uempty, C::CONSUMER_WARPS);
    fence_mbar_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  __syncthreads();
  pdl_wait();
  if (warp == C::CONSUMER_WARPS) {
    paged_producer<C>(kmap, vmap, p, smem, lane);
    return;
  }

  // ------------------------------------------------ consumers
  // The warp's 16 rows, and its quarter of a tile's keys.
  const int grp = C::GROUPS == 1 ? 0 : warp >> 2, quarter = C::GROUPS == 1 ? warp : warp & 3;
  const int g = lane >> 2, t4 = lane & 3;
  float* st_m = reinterpret_cast<float*>(smem + C::OFF_STATE) + grp * 128;
  float* st_l = st_m + 64;
  float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE + grp * C::MERGE_BYTES);
  const int share = blockIdx.x;
  // A tile is laid out box by box, [box][half][key][64 columns].  ldmatrix
  // takes an address per lane: for K (two 8-key blocks of two 8-column blocks
  // each) and, transposed, V the lane's key within 16 keys and its column.
  constexpr int KB = C::WK / 16;
  const int box_keys = min(1 << p.page_shift, C::TK);
  const uint32_t half = (uint32_t)box_keys * C::ROW_BYTES;
  const int krow = ((lane >> 4) << 3) + (lane & 7), kcol = (lane >> 3) & 1;
  const int vrow = (((lane >> 3) & 1) << 3) + (lane & 7), vcol = lane >> 4;
  uint32_t kstart[KB], vstart[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    auto start = [&](int row) {
      return (uint32_t)(row + (C::HALVES - 1) * (row & ~(box_keys - 1))) * C::ROW_BYTES;
    };
    kstart[kb] = start(quarter * C::WK + kb * 16 + krow);
    vstart[kb] = start(quarter * C::WK + kb * 16 + vrow);
  }

  uint32_t phase = 0, uphase = 0;
  int stage = 0;
  bool alive = true;
  while (true) {
    // A wait that ran out in one warp ends its group, here, where none of them
    // waits in a barrier for another.
    alive = alive && mbar_wait(ufull, uphase, p.status);
    uphase ^= 1;
    if (group_any<C>(grp, !alive)) return;
    __syncwarp();
    const PagedUnit w = *reinterpret_cast<const PagedUnit*>(smem + C::OFF_UNIT);
    if (w.tiles == 0) return;
    const int row0 = w.row0 + 16 * grp;
    const int rows = min(16, w.n * p.group - row0);  // none (or fewer) for the second group of a short unit
    const bool upper = rows > 8;                     // rows 8 .. 15 are somebody's
    const int delta = w.Lk - w.n;
    // The tokens of the group's rows and the key ranges of rows g and g + 8.
    const int tok_first = row0 / p.group, tok_last = (row0 + max(rows, 1) - 1) / p.group;
    int tok[2], row_lo[2], row_hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tok[h] = min((row0 + g + 8 * h) / p.group, tok_last);
      const int c = tok[h] + delta;
      row_lo[h] = max(0, c - p.win_left);
      row_hi[h] = (int)min((int64_t)w.Lk - 1, (int64_t)c + p.win_right);
    }
    // Keys in [in_lo, in_hi] are read by every row of the group.
    const int in_lo = max(0, tok_last + delta - p.win_left);
    const int in_hi = (int)min((int64_t)w.Lk - 1, (int64_t)tok_first + delta + p.win_right);

    // Q's fragments; rows past the last hold anything, and nothing of them is
    // written.
    uint32_t qf[D / 16][4];
    uint32_t qseen = (uint32_t)(w.t0 | w.n | w.Lk | w.head0 | w.row0 | w.tile | w.tiles | w.from_start | w.to_end);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      ldsm4(qf[ks], smem_u32(smem + C::OFF_Q) + (16 * grp + (lane & 15)) * C::Q_PITCH + (ks * 2 + (lane >> 4)) * 16);
      qseen |= qf[ks][0];
    }
    release_after(uempty, qseen, p.zero, lane == 0);

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

    for (int x = 0; x < w.tiles; ++x) {
      const int key0 = (w.tile + x) * C::TK + quarter * C::WK;
      alive = alive && mbar_wait(full + stage, phase, p.status);
      alive = __all_sync(0xffffffffu, alive);  // and the lanes, which leave the wait one by one, are together
      uint32_t seen = 0;  // everything read of V (what is read of K goes into the maxima)
      if (alive && rows > 0) {
        const uint32_t kbase = smem_u32(smem + stage * C::STAGE_BYTES), vbase = kbase + C::TILE_BYTES;
        // S = Q K^T for the warp's keys.
        float sc[2 * KB][4];
#pragma unroll
        for (int n = 0; n < 2 * KB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            uint32_t b[4];
            // matrices: keys 0-7 / d 0-7, keys 0-7 / d 8-15, keys 8-15 / d 0-7, keys 8-15 / d 8-15
            ldsm4(b, kbase + kstart[kb] + col_off<C>(krow, ks * 2 + kcol, half));
            mma16816<BF16>(sc[2 * kb], qf[ks], b[0], b[1]);
            mma16816<BF16>(sc[2 * kb + 1], qf[ks], b[2], b[3]);
          }
        const bool edge = key0 < in_lo || key0 + C::WK - 1 > in_hi;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2 * KB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = i >> 1;
            float s = sc[n][i] * p.scale_log2;
            if (edge) {
              const int key = key0 + n * 8 + 2 * t4 + (i & 1);
              if (key < row_lo[h] || key > row_hi[h]) s = -INFINITY;
            }
            sc[n][i] = s;
            mx[h] = fmaxf(mx[h], s);
          }
        bool grew = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          grew = grew || ((h == 0 || upper) && mx[h] > m[h]);
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[h], mx[h]);
            const float f = mn == -INFINITY ? 1.f : ex2_approx(m[h] - mn);
            m[h] = mn;
            l[h] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * h] *= f;
              o[n][2 * h + 1] *= f;
            }
          }
        }
        // P = 2^(S - m) in two parts of the input type for the products with V;
        // l sums the same values.  FP16 holds P times 2^15, so that weights
        // keep their bits down to 2^-29 of the largest and count down to 2^-40:
        // in a long cache very many small ones add up.  (A reference 15 below
        // the maximum instead would round either itself or the largest weight.)
        uint32_t pf[KB][4], pl[KB][4];
#pragma unroll
        for (int n = 0; n < 2 * KB; ++n) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = i >> 1;
            e[i] = ex2_approx(sc[n][i] - (m[h] == -INFINITY ? 0.f : m[h]));
            l[h] += e[i];
          }
          if (!BF16) {
            fma2(e[0], e[1], e[0], e[1], kF16Weight, kF16Weight, 0.f, 0.f);
            fma2(e[2], e[3], e[2], e[3], kF16Weight, kF16Weight, 0.f, 0.f);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int x = (n & 1) * 2 + i;
            split_pair<BF16>(e[2 * i], e[2 * i + 1], pf[n >> 1][x], pl[n >> 1][x]);
          }
        }
        // O += P V.
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          // matrices (transposed): keys 0-7 / d 0-7, keys 8-15 / d 0-7, keys 0-7 / d 8-15, keys 8-15 / d 8-15
          auto load = [&](uint32_t(&b)[4], int n) {
            ldsm4_trans(b, vbase + vstart[kb] + col_off<C>(vrow, 2 * n + vcol, half));
            seen |= b[0];
          };
          auto products = [&](int n, const uint32_t(&b)[4]) {
            mma16816<BF16>(o[2 * n], pf[kb], b[0], b[1]);
            mma16816<BF16>(o[2 * n + 1], pf[kb], b[2], b[3]);
            mma16816<BF16>(o[2 * n], pl[kb], b[0], b[1]);
            mma16816<BF16>(o[2 * n + 1], pl[kb], b[2], b[3]);
          };
          if (!edge) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t b[4];
              load(b, n);
              products(n, b);
            }
            continue;
          }
          // V outside the range of all rows is taken as 0.  A key that some rows
          // read and others do not has weight 0 in the latter, which is enough
          // if its V is finite.  If not: one pass per token, in which its range
          // alone survives in V and its rows alone take the products.
          const int key = key0 + kb * 16 + 2 * t4;
          bool apart = false;
          if (tok_first != tok_last) {
            const int lo = max(0, tok_first + delta - p.win_left);
            const int hi = (int)min((int64_t)w.Lk - 1, (int64_t)tok_last + delta + p.win_right);
            const uint32_t m0 = half_mask(key, lo, hi), m1 = half_mask(key + 8, lo, hi);
            uint32_t bad = 0;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t b[4];
              load(b, n);
              bad |= non_finite<BF16>(b[0] & m0) | non_finite<BF16>(b[1] & m1) | non_finite<BF16>(b[2] & m0) |
                     non_finite<BF16>(b[3] & m1);
            }
            apart = __any_sync(0xffffffffu, bad != 0u);
          }
          if (!apart) {
            const int lo = max(0, tok_first + delta - p.win_left);
            const int hi = (int)min((int64_t)w.Lk - 1, (int64_t)tok_last + delta + p.win_right);
            const uint32_t m0 = half_mask(key, lo, hi), m1 = half_mask(key + 8, lo, hi);
            if (__any_sync(0xffffffffu, (m0 | m1) != 0u)) {
#pragma unroll
              for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                load(b, n);
                b[0] &= m0, b[1] &= m1, b[2] &= m0, b[3] &= m1;
                products(n, b);
              }
            }
          } else {
            for (int tk = tok_first; tk <= tok_last; ++tk) {
              const int lo = max(0, tk + delta - p.win_left);
              const int hi = (int)min((int64_t)w.Lk - 1, (int64_t)tk + delta + p.win_right);
              const uint32_t m0 = half_mask(key, lo, hi), m1 = half_mask(key + 8, lo, hi);
#pragma unroll
              for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                load(b, n);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float d[4] = {o[2 * n + h][0], o[2 * n + h][1], o[2 * n + h][2], o[2 * n + h][3]};
                  mma16816<BF16>(d, pf[kb], b[2 * h] & m0, b[2 * h + 1] & m1);
                  mma16816<BF16>(d, pl[kb], b[2 * h] & m0, b[2 * h + 1] & m1);
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (tok[i >> 1] == tk) o[2 * n + h][i] = d[i];
                }
              }
            }
          }
        }
      }
      // (Without having waited the warp gives nothing back: the stage's load may be on its way.)
      release_after(empty + stage, seen, p.zero, lane == 0 && alive);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (rows <= 0) continue;  // (the whole group)

    // Merge the four warps' states.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (t4 == 0) {
        st_m[quarter * 16 + g + 8 * h] = m[h];
        st_l[quarter * 16 + g + 8 * h] = l[h];
      }
    }
    group_barrier<C>(grp);
    // Row r's largest maximum (0 for none) and its sum.
    auto state_of = [&](int r, float& ref, float& sum) {
      float mm = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) mm = fmaxf(mm, st_m[x * 16 + r]);
      ref = mm == -INFINITY ? 0.f : mm;
      sum = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) sum += st_l[x * 16 + r] * ex2_approx(st_m[x * 16 + r] - ref);
    };
    float inv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float ref, sum;
      state_of(g + 8 * h, ref, sum);
      inv[h] = sum == 0.f ? 0.f : ex2_approx(m[h] - ref) / sum;  // no key: 0; a NaN sum stays one
      if (!BF16) inv[h] *= 1.f / kF16Weight;
    }
    const bool whole = w.from_start && w.to_end;
    // Where this piece of the unit goes: the output, or the workspace (slot 0
    // for a unit that began earlier, slot 1 for one that begins here).
    const int64_t part_row = ((int64_t)share * 2 + (w.from_start ? 1 : 0)) * MT + 16 * grp;
    const int r = C::GROUPS == 1 ? tid : tid & 127;
    if (r < rows) {
      float ref, sum;
      state_of(r, ref, sum);
      const float lse = sum == 0.f ? -INFINITY : ref * 0.6931471805599453f + logf(sum);
      if (!whole) {
        p.part_lse[part_row + r] = lse;
      } else if (p.lse != nullptr) {
        const int rr = row0 + r, i = rr / p.group;
        p.lse[(int64_t)(w.head0 + rr - i * p.group) * p.total_q + w.t0 + i] = lse;
      }
    }
    __syncwarp();
    // All columns at once for up to four rows, half of 128 for eight, 32 for more.
    if (rows <= 4) paged_merge<C, BF16, D, 4>(p, w, grp, rows, merge, o, inv, whole, part_row);
    else if (rows <= 8) paged_merge<C, BF16, (D < 64 ? D : 64), 8>(p, w, grp, rows, merge, o, inv, whole, part_row);
    else paged_merge<C, BF16, 32, 16>(p, w, grp, rows, merge, o, inv, whole, part_row);
  }
}

}  // namespace etattn
