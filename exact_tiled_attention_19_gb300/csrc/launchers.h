// Internal declarations of the per-variant kernel launchers (one per head dim
// and element type), implemented in attn_fwd_inst.cu.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace etattn {

struct FwdParams;

#define ETATTN_DECLARE_LAUNCHER(name)                                                                     \
  cudaError_t name(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const FwdParams& p, \
                   dim3 grid, int nsub, bool general, bool ksplit, bool split, cudaStream_t stream);

ETATTN_DECLARE_LAUNCHER(launch_fwd_d32_0)
ETATTN_DECLARE_LAUNCHER(launch_fwd_d32_1)
ETATTN_DECLARE_LAUNCHER(launch_fwd_d64_0)
ETATTN_DECLARE_LAUNCHER(launch_fwd_d64_1)
ETATTN_DECLARE_LAUNCHER(launch_fwd_d128_0)
ETATTN_DECLARE_LAUNCHER(launch_fwd_d128_1)

#undef ETATTN_DECLARE_LAUNCHER

// Merge of split-KV partial states (attn_combine.cu).  Row r is the lse
// index of an output row; its slice-s state is part_o[(s * rows + r) * D ..]
// and part_lse[s * rows + r].
struct CombineParams {
  const float* part_o;
  const float* part_lse;
  int64_t rows;                  // rows per slice (the size of lse)
  int num_splits;
  void* o;                       // output in the input type
  float* lse;                    // or nullptr
  int64_t o_sb, o_sh, o_sn;      // element strides of o (batch, head, token)
  int Hq, Nq;                    // batched layout: row = (b * Hq + h) * Nq + t
  int packed;                    // packed layout: row = h * total + t
  int64_t total;                 // packed: query tokens
};

cudaError_t launch_combine(int D, bool bf16, const CombineParams& c, cudaStream_t stream);

// Backward pass (attn_bwd_aux.cu, attn_bwd_inst.cu).
struct BwdParams;

// Before the backward kernel: one row per (batch, query head, query) of
// [B * Hq][Nq_pad].
struct BwdPreParams {
  const void* o;                 // forward output, input type
  const void* dout;              // upstream gradient, input type
  const float* lse;              // [B, Hq, Nq] contiguous
  int64_t o_sb, o_sh, o_sn;      // element strides (batch, head, token); d-stride 1
  int64_t do_sb, do_sh, do_sn;
  int64_t rows;                  // B * Hq * Nq_pad
  int Hq, Nq, Nq_pad;
  float scale;
  float* nsd;                    // out: [B * Hq][Nq_pad], -scale * <dO, O>
  float* nlse2;                  // out: [B * Hq][Nq_pad], -lse * log2(e)
  float* dq_acc;                 // out: [B, Hq, Nq, D] zeroed
};

// After: FP32 dQ to the input type.
struct BwdConvertParams {
  const float* dq_acc;           // [B, Hq, Nq, D]
  void* dq;
  int64_t dq_sb, dq_sh, dq_sn;
  int64_t rows;                  // B * Hq * Nq
  int Hq, Nq;
};

cudaError_t launch_bwd_pre(int D, bool bf16, const BwdPreParams& c, cudaStream_t stream);
cudaError_t launch_bwd_convert(int D, bool bf16, const BwdConvertParams& c, cudaStream_t stream);

#define ETATTN_DECLARE_BWD_LAUNCHER(name)                                                                  \
  cudaError_t name(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dout, \
                   const CUtensorMap& dq_acc, const BwdParams& p, dim3 grid, cudaStream_t stream);

ETATTN_DECLARE_BWD_LAUNCHER(launch_bwd_d32_0)
ETATTN_DECLARE_BWD_LAUNCHER(launch_bwd_d32_1)
ETATTN_DECLARE_BWD_LAUNCHER(launch_bwd_d64_0)
ETATTN_DECLARE_BWD_LAUNCHER(launch_bwd_d64_1)
ETATTN_DECLARE_BWD_LAUNCHER(launch_bwd_d128_0)
ETATTN_DECLARE_BWD_LAUNCHER(launch_bwd_d128_1)

#undef ETATTN_DECLARE_BWD_LAUNCHER

// Programmatic stream serialisation (as for the forward kernel): the grid may
// be scheduled while its predecessor on the stream ends; griddepcontrol.wait
// in the kernel keeps its memory accesses behind the predecessor's completion.
template <typename... A>
cudaError_t launch_pdl(void (*kern)(A...), dim3 grid, int threads, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
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

// Query/key norm and rotation, plain or into a paged cache (attn_rope.cu).
// Strides in elements: token, head (pages: page, head, token); d-stride 1.
struct RopeParams {
  const void *q, *k, *v;           // [T, Hq, D], [T, Hk, D]; v: paged form only
  const void *q_weight, *k_weight; // [D] in the input type, or nullptr: no norm
  const float *cos, *sin;          // [max_position, rope_dim / 2]
  const int* positions;            // [T]: plain form
  void *q_out, *k_out, *v_out;     // [T, H, D]; paged: k_out, v_out are the pages
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh;
  int64_t kp_sp, kp_sh, kp_st, vp_sp, vp_sh, vp_st;  // plain form: kp_st, kp_sh of k_out
  int total_tokens, Hq, Hk;
  int rope_dim, interleaved, max_position;
  float eps;
  int paged;
  const int *block_table, *seqlens_k, *cu_seqlens;   // cu_seqlens nullptr: tokens_per_seq each
  int64_t table_stride;
  int num_seqs, tokens_per_seq, max_pages, num_pages, page_shift;
  int* status;
};

// Its gradients.
struct RopeBwdParams {
  const void *q, *k, *dq_out, *dk_out;
  const void *q_weight, *k_weight;
  const float *cos, *sin;
  const int* positions;
  void *dq, *dk;
  float *dq_weight, *dk_weight;    // [D] or nullptr
  float* partials;                 // [blocks][D]
  int64_t q_st, q_sh, k_st, k_sh, dqo_st, dqo_sh, dko_st, dko_sh, dq_st, dq_sh, dk_st, dk_sh;
  int total_tokens, Hq, Hk;
  int rope_dim, interleaved, max_position;
  float eps;
  int q_blocks, blocks;            // blocks for q's rows, and all
  int* status;
};

constexpr int kRopeBwdHeads = 2;   // heads a group of threads takes at a time

cudaError_t launch_rope(int D, bool bf16, const RopeParams& p, cudaStream_t stream);
cudaError_t launch_rope_bwd(int D, bool bf16, const RopeBwdParams& p, cudaStream_t stream);

// Norm, rotation and the append to a cache held in 4 bits (attn_append_q4.cu).
struct AppendQ4Params {
  const void *q, *k, *v;           // [T, Hq, D], [T, Hkv, D]
  const void *q_weight, *k_weight; // [D] in the input type, or nullptr: no norm
  const float *cos, *sin;          // [max_position, rope_dim / 2]
  const int* positions;            // [T], or nullptr when rope_dim is 0
  const int64_t* slots;            // [T]: page * page_size + slot; negative: no place
  void* q_out;                     // [T, Hq, D]
  uint8_t *k_pages, *v_pages;      // blocks of one page and head, byte strides
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh;
  int64_t kp_sp, kp_sh, vp_sp, vp_sh;
  int total_tokens, Hq, Hkv;
  int rope_dim, interleaved, max_position;
  float eps;
  int num_pages, page_shift;
  int others;                      // blocks of the launch that are of k or v, as many each
  uint64_t others_step;            // how many of them come with every block, times 2^32
  uint64_t q_groups, kv_groups;    // one over a token's groups of heads, times 2^64 (0: one group)
  int* status;
};
cudaError_t launch_append_q4(int D, bool bf16, const AppendQ4Params& p, cudaStream_t stream);

// The way back: 16-bit values of a cache's blocks.
struct UnpackQ4Params {
  const uint8_t* pages;
  void* out;                       // [num_pages, Hkv, page_size, D]
  int64_t p_sp, p_sh;              // bytes
  int64_t o_sp, o_sh, o_st;        // elements
  int num_pages, Hkv, page_shift;
};
cudaError_t launch_unpack_q4(int D, bool bf16, const UnpackQ4Params& p, cudaStream_t stream);

// Pages handed out for a step's tokens and taken back (attn_tables.cu).
constexpr int kTablesNoScratch = 4096;  // sequences whose sums are in shared memory
struct TablesParams {
  const int *amount, *seqlens;     // [S]: new tokens, or keys that stay; keys before
  int* table;                      // [S, max_pages] (truncate only reads it)
  int* free_pages;                 // [capacity] (extend only reads it)
  const int* free_count;
  int *seqlens_out, *free_count_out;
  int *cu_seqlens, *positions;     // extend: [S + 1], [total_tokens]
  int64_t* slots;                  // extend: [total_tokens]
  int* first;                      // scratch [S + 1] past kTablesNoScratch sequences: pages before each
  int64_t table_stride;
  int num_seqs, max_pages, capacity, total_tokens, page_shift;
  int extend;
  int fill;                        // whether the first launch fills in the pages and tokens, too
  int* status;
};
cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream);

// Attention over a paged cache (attn_paged_inst.cu).
// What a CTA whose piece begins inside a unit leaves for the join.
struct PagedShare {
  int t0, n, head0, row0;          // the unit: first q row, new tokens, first query head, first row of the tile
  int first, parts;                // the shares it spans (parts = 0: nothing to join)
  int pad[2];
};

struct PagedParams {
  const void* q;                   // [total_q, Hq, D]
  void* o;
  float* lse;                      // [Hq, total_q] or nullptr
  int64_t q_st, q_sh, o_st, o_sh;
  const int *block_table, *seqlens_k, *cu_seqlens_q;  // cu_seqlens_q nullptr: tokens_per_seq each
  int64_t table_stride;
  int num_seqs, tokens_per_seq, max_seqlen_q, total_q;
  int Hkv, group;
  int max_keys;                    // block-table width * page size, at most 2^30
  int num_pages, page_shift;
  int win_left, win_right;
  float scale_log2;
  int row_tile, shares;
  PagedShare* desc;                // [shares]
  float *part_lse, *part_o;        // [shares][2][row_tile], [shares][2][row_tile][D]
  uint32_t zero;                   // 0 (the kernel's release_after)
  int* status;
};

#define ETATTN_DECLARE_PAGED_LAUNCHER(name) \
  cudaError_t name(const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, cudaStream_t stream);

ETATTN_DECLARE_PAGED_LAUNCHER(launch_paged_d32_0)
ETATTN_DECLARE_PAGED_LAUNCHER(launch_paged_d32_1)
ETATTN_DECLARE_PAGED_LAUNCHER(launch_paged_d64_0)
ETATTN_DECLARE_PAGED_LAUNCHER(launch_paged_d64_1)
ETATTN_DECLARE_PAGED_LAUNCHER(launch_paged_d128_0)
ETATTN_DECLARE_PAGED_LAUNCHER(launch_paged_d128_1)

#undef ETATTN_DECLARE_PAGED_LAUNCHER

// The same over a cache held in 4 bits (attn_paged_q4_inst.cu): blocks of one
// page and head, with byte strides.
// What the host's plan and checks have in common with the kernels: bytes of a slot in a
// block (the codes and every group's scale and minimum), keys of a tile, and CTAs an SM for
// units of `rows` rows (4, 8 or 16).
constexpr int q4_slot_bytes(int D) { return D / 2 + 4 * (D < 64 ? 1 : D / 64); }
constexpr int paged_q4_tile_keys(int D) { return D == 128 ? 128 : 256; }
constexpr int paged_q4_ctas(int rows, int D) { return (rows == 16 ? 2 : 3) + (D == 32 ? 1 : 0); }
struct PagedQ4Params : PagedParams {
  const uint8_t *k_pages, *v_pages;
  int64_t kp_sp, kp_sh, vp_sp, vp_sh;
  float one_over_group;
};

#define ETATTN_DECLARE_PAGED_Q4_LAUNCHER(name) cudaError_t name(const PagedQ4Params& p, cudaStream_t stream);

ETATTN_DECLARE_PAGED_Q4_LAUNCHER(launch_paged_q4_d32_0)
ETATTN_DECLARE_PAGED_Q4_LAUNCHER(launch_paged_q4_d32_1)
ETATTN_DECLARE_PAGED_Q4_LAUNCHER(launch_paged_q4_d64_0)
ETATTN_DECLARE_PAGED_Q4_LAUNCHER(launch_paged_q4_d64_1)
ETATTN_DECLARE_PAGED_Q4_LAUNCHER(launch_paged_q4_d128_0)
ETATTN_DECLARE_PAGED_Q4_LAUNCHER(launch_paged_q4_d128_1)

#undef ETATTN_DECLARE_PAGED_Q4_LAUNCHER

}  // namespace etattn
