// Attention of a few new query rows per sequence over a paged key-value cache
// held in 4 bits, exact over the values that the cache stands for and in one
// pass over it.  Work line, producer and joined partial states are those of
// attn_paged_kernel.cuh; the consumers compute on the codes.
//
// Mathematics.  Element d of key j, in group h of G = min(D, 64) elements, is
//     k_jd = s_jh c_jd + m_jh,   c_jd in 0 .. 15,
// with scale s and minimum m in the type of q, and values likewise.  So
//     <q_i, k_j>      = sum_h ( s_jh <q_ih, c_jh> + m_jh sum_d q_id ),
//     sum_j P_ij v_jd = sum_j (P_ij s_jh) c_jd + sum_j P_ij m_jh,
// products of small whole numbers on the tensor core, with a scale and a minimum
// per key and group applied to their FP32 results (keys) or to the weights in FP32
// (values).  The cache's codes are never turned into 16-bit numbers in memory.
//
// Codes as operands.  The bits of a code in the low bits of a half make the
// denormal c 2^-24, which the tensor core multiplies exactly; one position higher
// (bits 4 to 7) they make c 2^-20.  So a word of eight codes becomes four operand
// registers by four ANDs and one shift, with no conversion and no offset to take
// away: the minimum goes into a term of its own.  The order of the elements within
// a product does not matter as long as q has the same one; q's elements that meet
// codes at the higher position are divided by 16, as are the outputs at them.
//   Both products have the codes as their left operand (m16n8k16), so that 8 rows
// fill the right one: S^T = K Q^T with 16 keys, O^T = V^T P^T with 16 elements.  A lane has
// the scores of one key in the former, and of one row in P^T: an 8 x 8 transpose of the
// weights, already scaled and rounded, lies between.  A register of V^T holds two keys
// of one element: transposed loads bring 16 bits of two keys together.
//
// Precision.  q's rows are scaled by powers of two so that their largest element
// is within 2^14 .. 2^15, and held as FP16: exact for both input types (elements below
// 2^-29 of the largest lose bits).  Scores, maxima, sums, minima terms and accumulators are
// FP32.  Weights times scales, P s, are multiplied by a power of two per row and group, which
// takes the largest P s that the row has seen in the warp to 2^5.5 or more (2^4.5 right after
// larger scores), and rounded to FP16: in two parts of together 2^-21 for FP16 outputs, in one
// for BF16 ones, whose 2^-11 is an eighth of the output's own rounding (two there take 62.5 us
// where one takes 55.6 for 8 x 32768 keys, 128 and 98 with 16 rows; with one, outputs are up to 1.02 times
// as far from 64 bits as those of FP32 weights).  A P s below 2^-19 of the row's largest loses bits, by
// 2^-28 of that at most.  The tensor core cuts off what falls below an
// accumulator's last bit, always downwards, and codes are never negative, so a
// running sum would drift.  A tile's products with V therefore start anew and are added to
// the running sums in FP32; and they start from -8 times the sum of the tile's weights, so
// that what accumulates is sum (P s)(c - 8), of both signs and small, while the minima's
// term takes m + 8 s instead of m.  One sequence of 524288 keys: outputs in BF16 were 1.6 times
// as far from 64 bits as a rounding of the exact ones with one running sum; in FP16 2.9 times
// with tiles that start from 0, 1.15 times now.
//   A row's weights are taken against a reference m that is set again only when a score
// passes it by 2^6 (kSlack), and the power of two when a P s may pass what FP16 holds.  Both go by
// the row's own scores, and by the scales of keys that it reads times their weights, so that no
// other row and nothing outside the row's range changes a bit of its result, and a key of a large
// scale that counts for nothing in a row takes nothing from its others.  (One power of two for all
// rows of a warp, by the scales alone, lost the rows' other keys where one had values 2^30 times as
// large; it took 54.7 us for 8 x 32768 keys where a row's own takes 55.6, 16 rows 93.6 and 97.8.)
//
// Up to 4 rows (PAIRED; a decode step of four query heads a KV head), 128 elements.
// The right operands' columns 4 .. 7 are the same rows again, for the second group of
// elements: a lane applies the scales of one group, not of both.  Q's operands are 0
// in the other group's columns, so that one accumulator takes the products of both groups
// side by side, and the two parts of a score are in neighbouring lanes; the weights'
// likewise.  (8 x 32768 keys took 57.2 us instead of 62.7 with the kernel for 8 rows, 512 sequences
// up to 2048 keys 77 instead of 92.)  Heads of 64 or 32 have one group: there the second columns are the
// same rows for a warp's second half of keys (a second side, with a state of its own, as if
// another warp had them), and every scale, exponential and transpose serves twice as many
// keys (8 x 32768 keys, heads of 64, 34.8 to 32.0 us; of 32 27.3 to 24.8; 512 sequences 59.8 to 56.7 and 54.2
// to 50.7).
//
// What bounds it.  A key and a value of D = 128 are 144 bytes, 3.6 times fewer than in 16
// bits, and 16 of them cost a warp as many instructions as 16 bits would: the loads alone
// take 50 us of the 55 for 8 x 32768 keys (44.6 at the copy bandwidth), the instructions of the
// consumers half of all issue slots (2.0 of 4 a cycle), of which the integer units
// take 51 %; the tensor pipe is busy 27 %.  (Heads of 64 and 32: 1.8 and 2.0, 46 %, 22 and 15 %;
// 16 rows 1.7, 33 %, 30 %: no unit is full, fixed latencies and waits for tiles lie in between.)  So everything here saves instructions per key: no
// conversions, scales on pairs, maxima looked at only when they matter.  And code: short sequences run
// it through once a unit, so what a key that not all rows read may need (`values`, odd) is apart (512
// short sequences of 16 rows 203 us with it in every edge tile, 181 without).
//   mma.sync and not tcgen05: a tile of 128 query rows would be 15/16 empty, and the codes would
// have to be written to shared memory as numbers first.  Three CTAs of four consumer warps an
// SM: two took 64.5 us where three took 62.7; four (96 registers a thread, two stages) take 56.3
// where three take 54.7.
//
// Measured (GB300; BF16, 32 query and 8 KV heads of 128, one new token, unless said; device
// time; % of the measured copy bandwidth): 8 x 32768 keys 55.5 us (80 %), in FP16 62.0; 1 x 524288
// 107.5 us (83 %); 64 sequences of 1 to 16384 keys 35.4 us (56 %); 16 rows (4 tokens) 8 x 32768 97.7
// us; heads of 64 32.0, of 32 24.6.  The
// cache in 16 bits takes 164, 325 and 80 us for the first, the second and the 64 sequences.
#pragma once

#include <cstdint>
#include <type_traits>

#include "attn_paged_kernel.cuh"

namespace etattn {

template <int D_, int MT_>
struct PagedQ4Cfg {
  static constexpr int D = D_, MT = MT_;
  // What a unit costs next to a tile (of twice the keys for the smaller heads).  1, 2 and 3 took (before a
  // row had a power of two of its own), us for 64 ragged sequences and for 512 short ones: 4 rows of 128 38.0, 34.7, 36.0 and 69.0, 66.5, 72.8; 8
  // rows 45.4, 39.8, 41.2 and 87.4, 79.6, 85.8; 16 rows 87.2, 71.1, 65.3 and 198, 178, 170; heads of 64
  // 28.4, 29.8, 31.5 and 59.7, 65.0, 70.9, 16 rows of them 42.5, 42.2, 45.2 and 102, 99.2, 106; of 32
  // 23.2, 24.4, - and 47.0, 51.1, -, 16 rows 34.9, 34.0, - and 78.7, 76.6, -.
  static constexpr int UNIT_COST = (D == 128 ? 2 : 1) + (MT == 16 ? 1 : 0);
  static constexpr int GROUPS = 1;                    // of four consumer warps
  static constexpr int G = D < 64 ? D : 64, H = D / G;
  static constexpr int TK = paged_q4_tile_keys(D);    // keys per tile
  static constexpr int WK = TK / 4, NT = WK / 8;      // per consumer warp, and in blocks of 8
  static constexpr int SPREAD = 32;                   // keys of the largest box whose blocks different warps take
  static constexpr int PANEL = G / 2 + 4;             // bytes of a key's group: codes, scale and minimum
  static constexpr int ROW_BYTES = H * PANEL;
  static_assert(ROW_BYTES == q4_slot_bytes(D), "");
  static constexpr int TILE_BYTES = TK * ROW_BYTES;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K and V: 18 KB, or 10 KB for D = 32
  static constexpr bool PAIRED = MT == 4;
  static constexpr int SIDES = PAIRED && H == 1 ? 2 : 1;  // runs of keys with a state of their own in a warp
  static_assert(MT == 8 || MT == 16 || PAIRED, "");
  // Three CTAs of up to 8 rows share an SM, or two of 16; one more of heads of 32, whose stages are
  // smaller (three or four, us: 64 ragged sequences 24.7 and 23.3, 512 short ones 50.9 and 47.1; 16
  // rows, two or three, 39.2 and 34.4, 82.4 and 78.7).  With four of heads of 64 two stages are left
  // (8 x 32768 keys 32.0 and 33.7), and three of 16 rows of them spill (FP16 58.8 and 60.5).
  static constexpr int CTAS = paged_q4_ctas(MT, D);
  static constexpr int BUDGET = CTAS == 4 ? 57344 : CTAS == 3 ? 76800 : 115712;
  static constexpr int COLS = PAIRED ? D : G;            // elements that are merged at a time
  static constexpr int MERGE_BYTES = 4 * MT * SIDES * COLS * 4;  // four warps' rows
  static constexpr int WIDE = MT * COLS > 4 * 128 ? 8 : 4, CHUNKS = COLS / WIDE;  // elements that a thread writes of them
  static_assert(MT * CHUNKS <= 128, "");
  static constexpr int Q_PITCH = 2 * D + 16;            // padded: no bank conflicts
  static constexpr int STATE_BYTES = (2 + H) * 4 * 16 * 4;  // m, l and minima's terms: 4 warps x 16 each
  static constexpr int FIXED = MERGE_BYTES + MT * Q_PITCH + STATE_BYTES + 48;
  static constexpr int FIT = (BUDGET - FIXED - 192) / STAGE_BYTES;
  static constexpr int STAGES = FIT < 11 ? FIT : 11;
  static constexpr int OFF_MERGE = STAGES * STAGE_BYTES;
  static constexpr int OFF_Q = OFF_MERGE + MERGE_BYTES;
  static constexpr int OFF_STATE = OFF_Q + MT * Q_PITCH;
  static constexpr int OFF_UNIT = OFF_STATE + STATE_BYTES;
  static constexpr int OFF_BARS = OFF_UNIT + 48;
  static constexpr int SMEM_BYTES = OFF_BARS + 2 * (STAGES + 1) * 8;
  static_assert(STAGES >= 3 && SMEM_BYTES <= BUDGET, "");
  static constexpr int CONSUMER_WARPS = 4, THREADS = 32 * (CONSUMER_WARPS + 1);
};

// A box: a block of the cache (one page and head: for every group the codes of its
// slots, then their scales and minima) in one copy, or, where a page holds more than
// a tile, the tile's slots of every part.
template <class C>
struct PagedQ4Boxes {
  const PagedQ4Params& p;
  uint64_t policy;
  uint32_t bytes;  // of a box of K, or of V
  __device__ __forceinline__ explicit PagedQ4Boxes(const PagedQ4Params& p_)
      : p(p_), policy(l2_policy_evict_first()), bytes((uint32_t)min(1 << p_.page_shift, C::TK) * C::ROW_BYTES) {}
  // Large boxes one after the other; small ones so that those of a warp, NT in a
  // row, lie SPREAD keys apart, with those of the other warps between them.
  __device__ __forceinline__ void load(uint8_t* stage, int box, int slot, int head, int page, uint64_t* bar) const {
    const uint8_t* src[2] = {p.k_pages + page * p.kp_sp + head * p.kp_sh, p.v_pages + page * p.vp_sp + head * p.vp_sh};
    uint8_t* dst = stage + ((1 << p.page_shift) <= C::SPREAD
                                ? (box % C::NT) * (C::SPREAD * C::ROW_BYTES) + (box / C::NT) * bytes
                                : box * bytes);
#pragma unroll
    for (int i = 0; i < 2; ++i, dst += C::TILE_BYTES) {
      if ((1 << p.page_shift) <= C::TK) {
        bulk_load_hint(dst, src[i], bytes, bar, policy);
      } else {
        const int64_t page_keys = 1 << p.page_shift;
#pragma unroll
        for (int h = 0; h < C::H; ++h) {
          const uint8_t* from = src[i] + h * page_keys * C::PANEL;
          uint8_t* to = dst + h * C::TK * C::PANEL;
          bulk_load_hint(to, from + slot * (C::G / 2), C::TK * (C::G / 2), bar, policy);
          bulk_load_hint(to + C::TK * (C::G / 2), from + page_keys * (C::G / 2) + slot * 4, C::TK * 4, bar, policy);
        }
      }
    }
  }
  // (Recorded; the rows of that sequence mean nothing.)
  __device__ __forceinline__ int bad_page(const PagedParams&) const { return 0; }
};

// d = A B
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// d = A B + c
__device__ __forceinline__ void mma16816_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                              const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// x, y as hi + lo, two pairs of halves: hi by cutting bits off, lo the rest, rounded.
__device__ __forceinline__ void split_halves(float x, float y, uint32_t& hi, uint32_t& lo) {
  const float hx = __uint_as_float(__float_as_uint(x) & 0xffffe000u), hy = __uint_as_float(__float_as_uint(y) & 0xffffe000u);
  hi = pack_f16x2(hx, hy);
  lo = pack_f16x2(x - hx, y - hy);
}

// A scale (low half) and a minimum.
template <bool BF16>
__device__ __forceinline__ void scale_and_min(uint32_t w, float& s, float& m) {
  if (BF16) unpack_bf16x2(w, s, m);
  else unpack_f16x2(w, s, m);
}

// Four (or two) 8 x 8 matrices of 16-bit values, transposed; eight lanes each give their
// rows.  (Volatile, so that it stays behind the wait, but free of the other loads.)
__device__ __forceinline__ void codes_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void codes_trans(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}

// The 8 x 8 matrix of halves that the warp holds, a row of four registers each, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

constexpr uint32_t kLowCodes = 0x000f000fu, kHighCodes = 0x00f000f0u;

// Adds up the four warps' rows, COLS elements at a time, normalises and writes them: the
// output, or the unit's partial rows.  A lane holds elements 4 g .. and 32 + 4 g .. of
// two rows (and of those 8 further down) of every group, or of its own; a thread writes
// WIDE elements of row `tid / CHUNKS`, of whose sum `inv` is the inverse.
template <class C, bool BF16>
__device__ __forceinline__ void paged_q4_merge(const PagedParams& p, const PagedUnit& w, int rows, float* merge,
                                               const float (&o)[C::PAIRED ? 1 : C::H][(C::MT + 7) / 8][2][C::G / 8],
                                               float inv, bool whole, int64_t part_row) {
  constexpr int G = C::G, RUN = G / 8, COLS = C::COLS, WIDE = C::WIDE;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int row = tid / C::CHUNKS, c = (tid % C::CHUNKS) * WIDE;
  // Where a row's four elements x4 lie: eight lanes that store together hit eight
  // different quarters of the banks.
  auto place = [](int r, int x4) {
    if (C::PAIRED && C::H == 2) return (x4 ^ (r & 2) ^ ((x4 >> 2) & 4)) * 4;
    return (x4 ^ (r & 6)) * 4;
  };
#pragma unroll
  for (int h = 0; h < C::D / COLS; ++h) {
#pragma unroll
    for (int hr = 0; hr < (C::MT + 7) / 8; ++hr)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        constexpr bool APART = C::PAIRED && C::H == 2;  // (its lanes have a group each; of two sides rows 4 .. are the second's)
        const int r = APART ? 2 * (t4 & 1) + j : 8 * hr + 2 * t4 + j, at = (APART ? (t4 >> 1) * G : 0) + g * 4;
        float* dst = merge + (warp * C::MT * C::SIDES + r) * COLS;
        const float(&v)[RUN] = o[h][hr][j];
#pragma unroll
        for (int i = 0; i < RUN; i += 4)
          *reinterpret_cast<float4*>(dst + place(r, at / 4 + 2 * i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    group_barrier<C>(0);
    if (row < rows) {
      float v[WIDE];
#pragma unroll
      for (int i = 0; i < WIDE; ++i) v[i] = 0.f;
#pragma unroll
      for (int y = 0; y < 4 * C::SIDES; ++y) {
        const float* src = merge + (y * C::MT + row) * COLS;
#pragma unroll
        for (int i = 0; i < WIDE; i += 4) {
          const float4 u = *reinterpret_cast<const float4*>(src + place(y % C::SIDES * C::MT + row, (c + i) / 4));
          v[i] += u.x, v[i + 1] += u.y, v[i + 2] += u.z, v[i + 3] += u.w;
        }
      }
#pragma unroll
      for (int i = 0; i < WIDE; ++i) v[i] *= inv;
      if (whole) {
        const int rr = w.row0 + row, i = rr / p.group;
        uint32_t u[WIDE / 2];
#pragma unroll
        for (int k = 0; k < WIDE / 2; ++k)
          u[k] = BF16 ? pack_bf16x2(v[2 * k], v[2 * k + 1]) : pack_f16x2(v[2 * k], v[2 * k + 1]);
        uint16_t* dst = static_cast<uint16_t*>(p.o) + (int64_t)(w.t0 + i) * p.o_st +
                        (int64_t)(w.head0 + rr - i * p.group) * p.o_sh + h * COLS + c;
        if constexpr (WIDE == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
        else *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
      } else {
        float* dst = p.part_o + (part_row + row) * C::D + h * COLS + c;
#pragma unroll
        for (int i = 0; i < WIDE; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
    // The next elements, or the next unit's (whose state the warps write first, and
    // meet, before they come here again).
    if (h + 1 < C::D / COLS) group_barrier<C>(0);
  }
}

template <int D, int MT, bool BF16, bool SPREAD>
__global__ void __launch_bounds__(PagedQ4Cfg<D, MT>::THREADS, PagedQ4Cfg<D, MT>::CTAS)
    attn_paged_q4_kernel(const __grid_constant__ PagedQ4Params p) {
  using C = PagedQ4Cfg<D, MT>;
  constexpr int G = C::G, H = C::H, NT = C::NT, RH = (MT + 7) / 8;
  constexpr bool PAIRED = C::PAIRED;
  constexpr int SIDES = C::SIDES, NB = NT / SIDES;  // blocks of 8 keys of a side
  constexpr int PARTS = PAIRED ? 2 : H;        // of the codes that have operands of Q of their own: groups, or sides
  constexpr int HL = PAIRED ? 1 : H;           // groups whose scales a lane applies
  constexpr int KW = G / 32, ON = G / 16;      // words of a key's group that a lane reads; blocks of 16 elements
  constexpr bool TWO = !BF16;                  // weights in two parts
  // Rows' key ranges are kept where there are registers for them, or made again at the edges (4
  // rows 55.7 and 56.0 us, 8 rows 63.2 and 61.5, 16 rows 100.3 and 97.9).
  constexpr bool RANGES = PAIRED;
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
  }
  __syncthreads();
  pdl_wait();
  if (warp == C::CONSUMER_WARPS) {
    paged_producer<C>(PagedQ4Boxes<C>(p), p, smem, lane);
    return;
  }

  // ------------------------------------------------ consumers
  const int quarter = warp, g = lane >> 2, t4 = lane & 3;
  // The first of the lane's rows (of the first 8), its group or side where it has one, and
  // the row of its state.
  const int row_at = PAIRED ? 2 * (t4 & 1) : 2 * t4, mine = PAIRED ? t4 >> 1 : 0;
  const int mine_group = H == 2 ? mine : 0, state_at = SIDES == 2 ? 2 * t4 : row_at;
  float* st_m = reinterpret_cast<float*>(smem + C::OFF_STATE);
  float* st_l = st_m + 64;
  float* st_low = st_l + 64;
  float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
  // Q's operands, which the warp reads again for every tile (the registers are needed
  // for the values): where the rows are merged, which happens after the last tile.
  uint4* q_ops = reinterpret_cast<uint4*>(merge) + quarter * (PARTS * KW * RH * 32) + lane;
  static_assert(4 * PARTS * KW * RH * 32 * 16 <= C::MERGE_BYTES, "");
  const int share = blockIdx.x;
  // Blocks of 8 keys lie in one box each.  The warp takes NT of them: neighbours in a
  // large box, or the same place of NT boxes (SPREAD), which lie a constant step apart
  // either way.  Its first one, key `key_at` of the tile, starts `first` bytes (its
  // scales `first_scale` bytes) into the tile; groups are `panel` apart.
  constexpr uint32_t kCodeStep = SPREAD ? C::SPREAD * C::ROW_BYTES : 8 * (G / 2);
  constexpr uint32_t kScaleStep = SPREAD ? C::SPREAD * C::ROW_BYTES : 8 * 4;
  const int box_keys = min(1 << p.page_shift, C::TK);
  const uint32_t panel = (uint32_t)box_keys * C::PANEL;
  const int key_step = SPREAD ? box_keys : 8;
  // Where the second part of the codes and scales lies: the other group, or the other side.
  const uint32_t code_part = H == 2 ? panel : NB * kCodeStep, scale_part = H == 2 ? panel : NB * kScaleStep;
  const int key_lane = g + (SIDES == 2 ? mine * NB * key_step : 0);
  int key_at, box_at, in_box;  // the latter two: where the box starts, and the block's first key in it
  if (SPREAD) {
    const int per_box = box_keys >> 3, row = quarter / per_box;  // blocks of a box; the warp's row of NT boxes
    in_box = (quarter - row * per_box) * 8;
    key_at = row * NT * box_keys + in_box;
    box_at = row * box_keys * C::ROW_BYTES;
  } else {
    key_at = quarter * C::WK;
    in_box = key_at & (box_keys - 1);
    box_at = (key_at - in_box) * C::ROW_BYTES;
  }
  const uint32_t first = box_at + in_box * (G / 2), first_scale = box_at + box_keys * (G / 2) + in_box * 4;
  // The lane's part of a block: elements G/4 t4 .. of key g, with its scales.  Of values it
  // gets elements 4 g .. (and 32 + 4 g ..) of keys 2 t4 and 2 t4 + 1 by transposed loads
  // of 8 keys' 16 bytes, of which it gives one address: of two blocks, G / 32 loads each.
  const uint32_t k_at = first + g * (G / 2) + t4 * (G / 8), s_at = first_scale + g * 4 + mine * scale_part;
  const uint32_t v_at = C::TILE_BYTES + first + (lane & 7) * (G / 2) +
                        (G == 64 ? (lane >> 4) * 16 + ((lane >> 3) & 1) * kCodeStep : ((lane >> 3) & 1) * kCodeStep);

  uint32_t phase = 0, uphase = 0;
  int stage = 0;
  bool alive = true;
  while (true) {
    // A wait that ran out in one warp ends them all, here, where none of them waits
    // in a barrier for another.
    alive = alive && mbar_wait(ufull, uphase, p.status);
    uphase ^= 1;
    if (group_any<C>(0, !alive)) return;
    __syncwarp();
    const PagedUnit w = *reinterpret_cast<const PagedUnit*>(smem + C::OFF_UNIT);
    if (w.tiles == 0) return;
    const int row0 = w.row0, rows = min(MT, w.n * p.group - row0);
    const int delta = w.Lk - w.n, Lk = w.Lk;
    // The tokens of the rows and the key ranges of the lane's.
    // (x beyond a token's first row is at least 1/2 / 2^16 of a token from the next one,
    // the FP32 product less than 2^-18 of 16 off.)
    const int tok_first = row0 / p.group;
    const float in_token = (float)(row0 - tok_first * p.group) + 0.5f;
    auto tok_of = [&](int x) { return tok_first + (int)((in_token + (float)x) * p.one_over_group); };
    const int tok_last = tok_of(rows - 1);
    int row_lo[RANGES ? RH : 1][2], row_hi[RANGES ? RH : 1][2];
    auto ranges = [&](int r) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = min(tok_of(row_at + i + 8 * r), tok_last) + delta;
        row_lo[RANGES ? r : 0][i] = max(0, c - p.win_left);
        row_hi[RANGES ? r : 0][i] = (int)min((int64_t)Lk - 1, (int64_t)c + p.win_right);
      }
    };
#pragma unroll
    for (int r = 0; RANGES && r < RH; ++r) ranges(r);
    // Keys in [in_lo, in_hi] are read by every row.
    const int in_lo = max(0, tok_last + delta - p.win_left);
    const int in_hi = (int)min((int64_t)w.Lk - 1, (int64_t)tok_first + delta + p.win_right);

    // Q's operands: rows scaled by 2^up; their groups' sums (in units of 2^-24), and
    // what brings a score back.  Rows past the last hold anything, and nothing of
    // them is written.
    uint64_t qsum[RH][HL], back[RH];  // of the lane's rows: columns 2 t4 and 2 t4 + 1
    auto of_rows = [&](float x) { return packed_pair(__shfl_sync(0xffffffffu, x, 8 * t4), __shfl_sync(0xffffffffu, x, 8 * t4 + 4)); };
    uint32_t qseen = (uint32_t)(w.t0 | w.n | w.Lk | w.head0 | w.row0 | w.tile | w.tiles | w.from_start | w.to_end);
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      float x[H][KW][8];
      float big = 0.f;
      const uint8_t* src = smem + C::OFF_Q + (PAIRED ? g & 3 : g + 8 * r) * C::Q_PITCH + t4 * (G / 2);
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int y = 0; y < KW; ++y) {
          const uint4 u = *reinterpret_cast<const uint4*>(src + h * 2 * G + y * 16);
          qseen |= u.x | u.y | u.z | u.w;
          const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            scale_and_min<BF16>(v[i], x[h][y][2 * i], x[h][y][2 * i + 1]);
            big = fmaxf(big, fmaxf(fabsf(x[h][y][2 * i]), fabsf(x[h][y][2 * i + 1])));
          }
        }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // (big = 1.x 2^e: 2^(14 - e), within what FP32 holds.)
      const int e = max(-90, min(110, (int)(__float_as_uint(big) >> 23) - 127));
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      const float down = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 + e + 10) << 23), 0x1p-126f);
      back[r] = of_rows(down);
      float total[HL];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float sum = 0.f;
#pragma unroll
        for (int y = 0; y < KW; ++y) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[h][y][i] *= up;
            sum += x[h][y][i];
          }
          const uint4 v = make_uint4(pack_f16x2(x[h][y][0], x[h][y][4]), pack_f16x2(x[h][y][1] * 0.0625f, x[h][y][5] * 0.0625f),
                                     pack_f16x2(x[h][y][2], x[h][y][6]), pack_f16x2(x[h][y][3] * 0.0625f, x[h][y][7] * 0.0625f));
#pragma unroll
          for (int part = h; part < PARTS; part += H)  // (0 in the columns of the other group, or side)
            q_ops[((part * KW + y) * RH + r) * 32] = !PAIRED || (g >> 2) == part ? v : make_uint4(0, 0, 0, 0);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (HL == H || (g >> 2) == h) total[HL == H ? h : 0] = sum * 0x1p-24f;
      }
#pragma unroll
      for (int h = 0; h < HL; ++h) qsum[r][h] = of_rows(total[h]);
    }
    release_after(uempty, qseen, p.zero, lane == 0);
    __syncwarp();

    // m: a reference for the row's weights, its largest score when it was last set.  Later
    // ones may pass it by kSlack (in powers of two) before it is set again, which spares
    // most tiles the maximum over their keys; weights are 2^kSlack at most.
    constexpr float kSlack = 6.f;
    float m[RH][2];
    uint64_t l[RH], low[RH][HL], o[RH][HL][ON][2];
#pragma unroll
    for (int r = 0; r < RH; ++r) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[r][i] = row_at + i + 8 * r < rows ? -INFINITY : INFINITY;  // (a row that is nobody's never grows)
      l[r] = 0;
#pragma unroll
      for (int h = 0; h < HL; ++h) {
        low[r][h] = 0;
#pragma unroll
        for (int n = 0; n < ON; ++n) o[r][h][n][0] = o[r][h][n][1] = 0;
      }
    }
    // What P s is multiplied by before it becomes FP16: a new one takes the row's largest so far to
    // 2^5.5 .. 2^7.5, and it is set again when a P s may pass 2^15.5.  `lifts`: two rows' as BF16
    // numbers, the first's in the low half.
    constexpr float kPre = BF16 ? 0x1p-8f : 1.f;  // of scales beforehand, so that P s stays within FP32
    constexpr int kExpShift = BF16 ? 7 : 10, kExpMax = BF16 ? 255 : 31;
    // P = 2^x, a scale's exponent E and that of the power of two: x + E + lift - kBias is the product's.
    constexpr int kBias = BF16 ? 127 + 127 + 8 : 15 + 127, kLiftTo = 6, kLiftPast = 14, kLiftMost = 247;
    constexpr int kMagic = 0x4b000000;  // 2^23 as a number: whole numbers beside it are its lowest bits
    uint32_t lifts[RH][HL];
    int top[HL];  // the largest exponent of a scale that passes nothing in the lane's rows whatever its weight
#pragma unroll
    for (int h = 0; h < HL; ++h) {
      top[h] = -1;
#pragma unroll
      for (int r = 0; r < RH; ++r) lifts[r][h] = (uint32_t)kLiftMost << 23 | kLiftMost << 7;
    }
    auto lift_of = [&](int h, int r, int i) { return __uint_as_float(i == 0 ? lifts[r][h] << 16 : lifts[r][h] & 0xffff0000u); };
    auto power = [](int biased) { return biased <= 0 ? 0.f : __uint_as_float((uint32_t)biased << 23); };
    auto number = [](int x) { return __uint_as_float((uint32_t)(kMagic + x)); };

    for (int x = 0; x < w.tiles; ++x) {
      const int tile0 = (w.tile + x) * C::TK, key0 = tile0 + key_at;
      alive = alive && mbar_wait(full + stage, phase, p.status);
      alive = __all_sync(0xffffffffu, alive);  // and the lanes, which leave the wait one by one, are together
      uint32_t seen = 0;  // of products that everything read of V has gone into (what is read of K goes into the maxima)
      if (alive) {
        const uint8_t* tile = smem + stage * C::STAGE_BYTES;
        const bool edge = tile0 < in_lo || tile0 + C::TK - 1 > in_hi;
        // Scores of the warp's keys, in units of 1 / back, 16 keys at a time: of key g of
        // two blocks.
        uint64_t sc[NB][RH];
        // The products of one part's codes with q; `first`: from 0.
        auto dots = [&](int h, int kb, const uint4(&q)[KW][RH], float(&part)[RH][4], bool first) {
          uint32_t c[2][KW];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint8_t* at = tile + k_at + (2 * kb + u) * kCodeStep + h * code_part;
            if constexpr (KW == 2) {
              const uint2 x = *reinterpret_cast<const uint2*>(at);
              c[u][0] = x.x, c[u][KW - 1] = x.y;
            } else {
              c[u][0] = *reinterpret_cast<const uint32_t*>(at);
            }
          }
#pragma unroll
          for (int y = 0; y < KW; ++y)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t c0 = j == 0 ? c[0][y] : c[0][y] >> 8, c1 = j == 0 ? c[1][y] : c[1][y] >> 8;
              const uint32_t a[4] = {c0 & kLowCodes, c1 & kLowCodes, c0 & kHighCodes, c1 & kHighCodes};
#pragma unroll
              for (int r = 0; r < RH; ++r) {
                const uint4 b = q[y][r];
                if (first && y == 0 && j == 0) mma16816_first(part[r], a, b.x, b.y);
                else mma16816<false>(part[r], a, j == 0 ? b.x : b.z, j == 0 ? b.y : b.w);
              }
            }
        };
        // Their scales and minima; `h`: of the lane's groups.
        auto scaled = [&](int h, int kb, const float(&part)[RH][4]) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float s, mn;
            scale_and_min<BF16>(*reinterpret_cast<const uint32_t*>(tile + s_at + (2 * kb + u) * kScaleStep + h * scale_part), s, mn);
            const uint64_t s2 = packed_pair(s, s), mn2 = packed_pair(mn, mn);
#pragma unroll
            for (int r = 0; r < RH; ++r) {
              uint64_t& x = sc[2 * kb + u][r];
              x = h == 0 ? mul_pair(mn2, qsum[r][h]) : fma_pair(mn2, qsum[r][h], x);
              x = fma_pair(s2, packed_pair(part[r][2 * u], part[r][2 * u + 1]), x);
            }
          }
        };
        auto q_of = [&](int h, uint4(&q)[KW][RH]) {
#pragma unroll
          for (int y = 0; y < KW; ++y)
#pragma unroll
            for (int r = 0; r < RH; ++r) q[y][r] = q_ops[((h * KW + y) * RH + r) * 32];
        };
        if constexpr (PAIRED) {
          uint4 q[PARTS][KW][RH];
#pragma unroll
          for (int h = 0; h < PARTS; ++h) q_of(h, q[h]);
#pragma unroll
          for (int kb = 0; kb < NB / 2; ++kb) {
            float part[RH][4];
#pragma unroll
            for (int h = 0; h < PARTS; ++h) dots(h, kb, q[h], part, h == 0);
            scaled(0, kb, part);
          }
#pragma unroll
          for (int n = 0; H == 2 && n < NB; ++n) {  // the other group's part
            const float2 x = parts_of(sc[n][0]);
            sc[n][0] = add_pair(sc[n][0], packed_pair(__shfl_xor_sync(0xffffffffu, x.x, 2), __shfl_xor_sync(0xffffffffu, x.y, 2)));
          }
        } else {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            uint4 q[KW][RH];
            q_of(h, q);
#pragma unroll
            for (int kb = 0; kb < NB / 2; ++kb) {
              float part[RH][4];
              dots(h, kb, q, part, true);
              scaled(h, kb, part);
            }
          }
        }
        // Whether what code 8 of a key that not all rows read stands for is not finite: a weight of 0
        // would not take it away.  (What lies in slots of nobody's may be anything.)
        bool odd = false;
        if (edge) {
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            const int key = key0 + n * key_step + key_lane;
#pragma unroll
            for (int h = 0; h < HL; ++h) {
              float s, mn;
              scale_and_min<BF16>(*reinterpret_cast<const uint32_t*>(tile + C::TILE_BYTES + s_at + n * kScaleStep + h * scale_part), s, mn);
              odd = odd || (!(fabsf(fmaf(s, 8.f, mn)) < INFINITY) && (key < in_lo || key > in_hi));
            }
          }
          odd = __any_sync(0xffffffffu, odd);
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            if constexpr (!RANGES) ranges(r);
            const int(&lo)[2] = row_lo[RANGES ? r : 0], (&hi)[2] = row_hi[RANGES ? r : 0];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              const int key = key0 + n * key_step + key_lane;
              float2 x = parts_of(sc[n][r]);
              if (key < lo[0] || key > hi[0]) x.x = -INFINITY;
              if (key < lo[1] || key > hi[1]) x.y = -INFINITY;
              sc[n][r] = packed_pair(x.x, x.y);
            }
          }
        }
        // Whether some score passes the reference that weights are taken against by more
        // than 2^kSlack allows, or a scale is so large that with such a weight P s might pass what
        // FP16 holds (scales' bits order like the numbers, none of which is negative; the minima
        // beside them are cut off).
        float mx[RH][2];
        bool grew = false;
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          mx[r][0] = mx[r][1] = -INFINITY;
#pragma unroll
          for (int n = 0; n < NB; n += 2) {
            const float2 x = parts_of(sc[n][r]), y = parts_of(sc[n + 1][r]);
            mx[r][0] = max3(mx[r][0], x.x, y.x);
            mx[r][1] = max3(mx[r][1], x.y, y.y);
          }
          const float2 f = parts_of(back[r]);  // (NaN while there was no key: not larger)
          grew = grew || fmaf(mx[r][0], f.x, -m[r][0]) > kSlack || fmaf(mx[r][1], f.y, -m[r][1]) > kSlack;
        }
        uint32_t sm[NB][HL];  // the values' scales and minima
        int most[HL];
        bool large = false;
#pragma unroll
        for (int h = 0; h < HL; ++h) {
          uint32_t bits = 0u;
#pragma unroll
          for (int n = 0; n < NB; n += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
              sm[n + u][h] = *reinterpret_cast<const uint32_t*>(tile + C::TILE_BYTES + s_at + (n + u) * kScaleStep + h * scale_part);
            bits = __vimax3_u16x2(bits, sm[n][h], sm[n + 1][h]);
          }
          most[h] = (int)((bits & 0xffffu) >> kExpShift);
          large = large || most[h] > top[h];
        }
        if (__any_sync(0xffffffffu, grew || large)) {
          // With the weights that the lane has: its largest score of every row, its largest scale.
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            float past = -INFINITY;
#pragma unroll
            for (int r = 0; r < RH; ++r)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                past = fmaxf(past, fmaf(mx[r][i], i == 0 ? parts_of(back[r]).x : parts_of(back[r]).y, -m[r][i]) +
                                       number(__float_as_uint(lift_of(h, r, i)) >> 23));
            grew = grew || __float_as_int(past) + most[h] >= kMagic + kLiftPast + kBias;
          }
          if (__any_sync(0xffffffffu, grew)) {
            // Row by row, by its own scores and the scales of keys that it reads alone: what
            // brought the warp here may be another's.
            uint64_t exps[NB][HL];  // the scales' exponents (0 for NaN: such a row is NaN whatever its lift)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int h = 0; h < HL; ++h) {
                const int ex = (int)((sm[n][h] & 0xffffu) >> kExpShift);
                const float e = number(ex < kExpMax ? ex : 0);
                exps[n][h] = packed_pair(e, e);
              }
#pragma unroll
            for (int h = 0; h < HL; ++h) top[h] = kExpMax;
            // The largest exponent of P s of either row, in a half each.
            auto far_of = [&](int h, int r) {
              float2 far = make_float2(0x1p23f, 0x1p23f);
              const uint64_t ref = packed_pair(m[r][0] == -INFINITY ? 0.f : -m[r][0], m[r][1] == -INFINITY ? 0.f : -m[r][1]);
#pragma unroll
              for (int n = 0; n < NB; n += 2) {
                const float2 e = parts_of(add_pair(fma_pair(sc[n][r], back[r], ref), exps[n][h]));
                const float2 d = parts_of(add_pair(fma_pair(sc[n + 1][r], back[r], ref), exps[n + 1][h]));
                far = make_float2(max3(far.x, e.x, d.x), max3(far.y, e.y, d.y));
              }
              uint32_t both = __byte_perm(__float_as_uint(far.x), __float_as_uint(far.y), 0x5410);
#pragma unroll
              for (int by = 4; by < 32; by <<= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, by));
              return both;
            };
            auto set_lifts = [&](int h, int r, const int(&now)[2]) {
              lifts[r][h] = (uint32_t)now[0] << 7 | (uint32_t)now[1] << 23;
#pragma unroll
              for (int i = 0; i < 2; ++i)  // (not for a row that is nobody's)
                if (m[r][i] != INFINITY) top[h] = min(top[h], kLiftPast - (int)kSlack + kBias - now[i]);
            };
            if (x == 0) {  // nothing to scale yet
#pragma unroll
              for (int r = 0; r < RH; ++r) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float mn = mx[r][i];
#pragma unroll
                  for (int by = 4; by < 32; by <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, by));
                  m[r][i] = fmaxf(m[r][i], mn * (i == 0 ? parts_of(back[r]).x : parts_of(back[r]).y));
                }
#pragma unroll
                for (int h = 0; h < HL; ++h) {
                  const uint32_t far = far_of(h, r);
                  set_lifts(h, r, {min(kLiftMost, kLiftTo + kBias - (int)(far & 0xffffu)), min(kLiftMost, kLiftTo + kBias - (int)(far >> 16))});
                }
              }
            } else {
#pragma unroll
              for (int r = 0; r < RH; ++r) {
                float part[2];  // 2^(m - its new value) is part, 0.5 .. 1, times 2^-up
                int up[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float mn = mx[r][i];
#pragma unroll
                  for (int by = 4; by < 32; by <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, by));
                  const float f = i == 0 ? parts_of(back[r]).x : parts_of(back[r]).y;
                  const bool set = fmaf(mn, f, -m[r][i]) > kSlack;
                  mn *= f;
                  up[i] = set ? (int)fminf(mn - m[r][i], 1000.f) : 0;
                  part[i] = set ? ex2_approx(m[r][i] - mn + (float)up[i]) : 1.f;
                  if (set) m[r][i] = mn;
                }
                const uint64_t f2 = packed_pair(part[0] * power(127 - up[0]), part[1] * power(127 - up[1]));
                l[r] = mul_pair(l[r], f2);
#pragma unroll
                for (int h = 0; h < HL; ++h) {
                  low[r][h] = mul_pair(low[r][h], f2);
                  const uint32_t far = far_of(h, r);
                  float by[2];
                  int now[2];
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const int was = (int)(__float_as_uint(lift_of(h, r, i)) >> 23), e = (int)(i == 0 ? far & 0xffffu : far >> 16);
                    // The largest P s so far fell by `up` powers of two, so that there is room above it.
                    now[i] = min(was + up[i], kLiftMost);
                    if (now[i] + e > kLiftPast + kBias) now[i] = kLiftTo + kBias - e;
                    by[i] = part[i] * power(127 - up[i] + now[i] - was);
                  }
                  set_lifts(h, r, now);
                  const uint64_t o2 = packed_pair(by[0], by[1]);
#pragma unroll
                  for (int n = 0; n < ON; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) o[r][h][n][i] = mul_pair(o[r][h][n][i], o2);
                }
              }
            }
          }
        }
        // P = 2^(S - m).
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          const uint64_t ref = packed_pair(m[r][0] == -INFINITY ? 0.f : -m[r][0], m[r][1] == -INFINITY ? 0.f : -m[r][1]);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            const float2 e = parts_of(fma_pair(sc[n][r], back[r], ref));
            sc[n][r] = packed_pair(ex2_approx(e.x), ex2_approx(e.y));
            l[r] = add_pair(l[r], sc[n][r]);
          }
        }
        // O^T += codes^T (P s)^T, and P m, group by group.  ODD: a key that the row does
        // not read may have any scale and minimum.
        auto values = [&](auto ODD) {
          float part[RH][ON][4], base[RH][4];
          // Codes of one group and 16 keys with the weights; `first`: from `base`.
          auto products = [&](int h, int kb, const uint32_t(&hi)[RH][2], const uint32_t(&lo)[RH][2], bool first) {
            // Four elements of two keys, a key's in a half, of either block.
            auto block = [&](int n, uint32_t b0, uint32_t b1) {
              const uint32_t v[4] = {b0 & kLowCodes, b0 & kHighCodes, b1 & kLowCodes, b1 & kHighCodes};
#pragma unroll
              for (int r = 0; r < RH; ++r) {
                if (first) mma16816_from(part[r][n], v, hi[r][0], hi[r][1], base[r]);
                else mma16816<false>(part[r][n], v, hi[r][0], hi[r][1]);
                if (TWO) mma16816<false>(part[r][n], v, lo[r][0], lo[r][1]);
              }
            };
            const uint32_t from = smem_u32(tile) + v_at + 2 * kb * kCodeStep + h * code_part;
            constexpr int X = RH == 1 ? ON : 2;
#pragma unroll
            for (int n0 = 0; n0 < ON; n0 += X) {
              uint32_t x[X];
              codes_trans(x, from + 8 * n0);
#pragma unroll
              for (int n = 0; n < X; n += 2) {
                block(n0 + n, x[n], x[n + 1]);
                block(n0 + n + 1, x[n] >> 8, x[n + 1] >> 8);
              }
            }
          };
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            uint32_t hi[NB / 2][RH][2], lo[NB / 2][RH][2];
            uint64_t lift[RH];
#pragma unroll
            for (int r = 0; r < RH; ++r) lift[r] = packed_pair(lift_of(h, r, 0), lift_of(h, r, 1));
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              float s, mn;
              scale_and_min<BF16>(sm[n][h], s, mn);
              mn = fmaf(s, 8.f, mn);  // what code 8 stands for
              s *= kPre;
              const uint64_t s2 = packed_pair(s, s), mn2 = packed_pair(mn, mn);
#pragma unroll
              for (int r = 0; r < RH; ++r) {
                // (In this order: a scale alone may be too large for the row's lift, where its weight is small.)
                float2 ws = parts_of(mul_pair(mul_pair(sc[n][r], s2), lift[r]));
                if constexpr (decltype(ODD)::value) {
                  const float2 e = parts_of(sc[n][r]), was = parts_of(low[r][h]);
                  float2 now = parts_of(fma_pair(sc[n][r], mn2, low[r][h]));
                  if (e.x == 0.f) ws.x = 0.f, now.x = was.x;
                  if (e.y == 0.f) ws.y = 0.f, now.y = was.y;
                  low[r][h] = packed_pair(now.x, now.y);
                } else {
                  low[r][h] = fma_pair(sc[n][r], mn2, low[r][h]);
                }
                uint32_t &a = hi[n / 2][r][n % 2], &b = lo[n / 2][r][n % 2];
                if (TWO) split_halves(ws.x, ws.y, a, b), b = transposed(b);
                else a = pack_f16x2(ws.x, ws.y);
                a = transposed(a);
              }
            }
            // The sums start from -8 times the weights, which is the same for all elements.
            constexpr uint32_t kMinusEights[4] = {0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u};
#pragma unroll
            for (int kb = 0; kb < NB / 2; ++kb)
#pragma unroll
              for (int r = 0; r < RH; ++r) {
                if (kb == 0) mma16816_first(base[r], kMinusEights, hi[0][r][0], hi[0][r][1]);
                else mma16816<false>(base[r], kMinusEights, hi[kb][r][0], hi[kb][r][1]);
                if (TWO) mma16816<false>(base[r], kMinusEights, lo[kb][r][0], lo[kb][r][1]);
              }
            if constexpr (PAIRED) {
#pragma unroll
              for (int x = 0; x < PARTS; ++x) {
                const uint32_t own = (g >> 2) == x ? ~0u : 0u;  // the columns of this group, or side
#pragma unroll
                for (int kb = 0; kb < NB / 2; ++kb) {
                  const uint32_t a[RH][2] = {{hi[kb][0][0] & own, hi[kb][0][1] & own}};
                  const uint32_t b[RH][2] = {{TWO ? lo[kb][0][0] & own : 0u, TWO ? lo[kb][0][1] & own : 0u}};
                  products(x, kb, a, b, x == 0 && kb == 0);
                }
              }
            } else {
#pragma unroll
              for (int kb = 0; kb < NB / 2; ++kb) products(h, kb, hi[kb], lo[kb], kb == 0);
            }
#pragma unroll
            for (int r = 0; r < RH; ++r)
#pragma unroll
              for (int n = 0; n < ON; ++n) {
                o[r][h][n][0] = add_pair(o[r][h][n][0], packed_pair(part[r][n][0], part[r][n][1]));
                o[r][h][n][1] = add_pair(o[r][h][n][1], packed_pair(part[r][n][2], part[r][n][3]));
              }
            seen |= __float_as_uint(part[0][0][0]) | __float_as_uint(part[0][ON - 1][0]);
          }
        };
        if (odd) values(std::true_type{});
        else values(std::false_type{});
      }
      // (Without having waited the warp gives nothing back: the stage's load may be on its way.)
      release_after(empty + stage, seen, p.zero, lane == 0 && alive);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }

    // Merge the four warps' states.
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      // (of the keys of all lanes that have the row)
      auto put_total = [&](uint64_t x, float* to) {
        float2 f = parts_of(x);
#pragma unroll
        for (int by = 4; by < 32; by <<= 1) {
          f.x += __shfl_xor_sync(0xffffffffu, f.x, by);
          f.y += __shfl_xor_sync(0xffffffffu, f.y, by);
        }
        if (g == 0) to[0] = f.x, to[1] = f.y;
      };
      // (Two lanes have a row where it is there for both groups, and write the same.)
      const int at = quarter * 16 + 8 * r + state_at;
      if (g == 0) st_m[at] = m[r][0], st_m[at + 1] = m[r][1];
      put_total(l[r], st_l + at);
#pragma unroll
      for (int h = 0; h < HL; ++h) put_total(low[r][h], st_low + (h + mine_group) * 64 + at);
    }
    group_barrier<C>(0);
    // The warp's rows against the largest maximum of the four (0 for none): powers of
    // two taken back (apart, as together they may pass FP32), minima added.
    float full_o[HL][RH][2][2 * ON];
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      float2 most = make_float2(-INFINITY, -INFINITY);
#pragma unroll
      for (int x = 0; x < 4 * SIDES; ++x) {
        const float2 y = *reinterpret_cast<const float2*>(st_m + x / SIDES * 16 + x % SIDES * MT + 8 * r + row_at);
        most = make_float2(fmaxf(most.x, y.x), fmaxf(most.y, y.y));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float ref = j == 0 ? most.x : most.y, f = ex2_approx(m[r][j] - (ref == -INFINITY ? 0.f : ref));
        const float even = 0x1p24f / kPre * f, odd = 0x1p20f / kPre * f;
#pragma unroll
        for (int h = 0; h < HL; ++h) {
          const float unit = __uint_as_float((254u << 23) - __float_as_uint(lift_of(h, r, j)));  // 1 / its power of two
          const float add = st_low[(h + mine_group) * 64 + quarter * 16 + 8 * r + state_at + j] * f;
#pragma unroll
          for (int n = 0; n < ON; ++n) {
            const float2 x = parts_of(o[r][h][n][0]), y = parts_of(o[r][h][n][1]);
            full_o[h][r][j][2 * n] = fmaf((j == 0 ? x.x : x.y) * even, unit, add);
            full_o[h][r][j][2 * n + 1] = fmaf((j == 0 ? y.x : y.y) * odd, unit, add);
          }
        }
      }
    }
    const bool whole = w.from_start && w.to_end;
    // Where this piece of the unit goes: the output, or the workspace (slot 0
    // for a unit that began earlier, slot 1 for one that begins here).
    const int64_t part_row = ((int64_t)share * 2 + (w.from_start ? 1 : 0)) * MT;
    // The sum of the row that the thread writes a part of.
    float inv = 0.f;
    if (tid < rows * C::CHUNKS) {
      const int r = tid / C::CHUNKS;
      float ref = -INFINITY, sum = 0.f;
#pragma unroll
      for (int x = 0; x < 4 * SIDES; ++x) ref = fmaxf(ref, st_m[x / SIDES * 16 + x % SIDES * MT + r]);
      if (ref == -INFINITY) ref = 0.f;
#pragma unroll
      for (int x = 0; x < 4 * SIDES; ++x) {
        const int at = x / SIDES * 16 + x % SIDES * MT + r;
        sum += st_l[at] * ex2_approx(st_m[at] - ref);
      }
      inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: 0; a NaN sum stays one
      if (tid % C::CHUNKS == 0) {
        const float lse = sum == 0.f ? -INFINITY : ref * 0.6931471805599453f + logf(sum);
        if (!whole) {
          p.part_lse[part_row + r] = lse;
        } else if (p.lse != nullptr) {
          const int rr = row0 + r, i = rr / p.group;
          p.lse[(int64_t)(w.head0 + rr - i * p.group) * p.total_q + w.t0 + i] = lse;
        }
      }
    }
    __syncwarp();
    paged_q4_merge<C, BF16>(p, w, rows, merge, full_o, inv, whole, part_row);
  }
}

}  // namespace etattn
