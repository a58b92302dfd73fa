// Block tables, slots and positions from the sequences' lengths, on the device:
// pages handed out for a step's new tokens, and taken back.
//
// With p keys a page, a sequence of L keys that gets n new ones takes
//     ceil((L + n) / p) - ceil(L / p)
// pages; page number i of all (sequence by sequence, column by column) comes from
// the top of a stack, free[count - 1 - i].  A sequence of which K keys stay gives
// back ceil(L / p) - ceil(K / p) pages, page i of all to free[count + i].
//
// Two prefix sums over the sequences and then independent tokens and pages: a few
// bytes each, so launches and chains of dependent loads bound it.  One launch of one
// cluster does the whole step.  Each CTA sums up its run of sequences; the CTAs
// exchange the sums, after which every one of them knows whether the step fits, before
// anything is written; then each writes its sequences' offsets, and after a second
// barrier all threads take the tokens and pages, which find their sequence by
// bisection.  One CTA is enough for small steps (no exchange); a step of many tokens
// has them filled in by a second launch as wide as the GPU.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "launchers.h"
#include "cache_ptx.cuh"

namespace etattn {

namespace {

constexpr int kTableThreads = 1024, kCtas = 8;

// Tokens and pages, in 64 bits: lengths are checked one by one, their sums by these.
struct Sums {
  int64_t tokens, pages;
  __device__ __forceinline__ Sums& operator+=(const Sums& o) {
    tokens += o.tokens;
    pages += o.pages;
    return *this;
  }
};

// What one sequence adds.  False: its lengths do not fit.
__device__ __forceinline__ bool sequence_sums(const TablesParams& p, int s, Sums& x) {
  const int64_t page = int64_t(1) << p.page_shift, L = p.seqlens[s], n = p.amount[s];
  const int64_t after = p.extend ? L + n : n;
  x = Sums{0, 0};
  if (L < 0 || n < 0 || (p.extend ? after : L) > p.max_pages * page || (p.extend ? after > (1 << 30) : n > L)) return false;
  const int64_t held = (L + page - 1) >> p.page_shift, wanted = (after + page - 1) >> p.page_shift;
  x.tokens = p.extend ? n : 0;
  x.pages = p.extend ? wanted - held : held - wanted;
  return true;
}

__device__ __forceinline__ Sums shuffled_up(const Sums& x, int by) {
  return Sums{__shfl_up_sync(0xffffffffu, x.tokens, by), __shfl_up_sync(0xffffffffu, x.pages, by)};
}

// The sums before this thread's, and of the whole block.
__device__ __forceinline__ Sums block_scan(Sums x, Sums& all, Sums (&warps)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums incl = x;
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const Sums o = shuffled_up(incl, by);
    if (lane >= by) incl += o;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  Sums w = warps[lane], wi = w;
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const Sums o = shuffled_up(wi, by);
    if (lane >= by) wi += o;
  }
  all = Sums{__shfl_sync(0xffffffffu, wi.tokens, 31), __shfl_sync(0xffffffffu, wi.pages, 31)};
  const Sums before = Sums{__shfl_sync(0xffffffffu, wi.tokens - w.tokens, warp), __shfl_sync(0xffffffffu, wi.pages - w.pages, warp)};
  return Sums{before.tokens + incl.tokens - x.tokens, before.pages + incl.pages - x.pages};
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster, with what they wrote.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// `src` of this CTA as CTA `rank` has it.
__device__ __forceinline__ int64_t remote_load(const int64_t* src, uint32_t rank) {
  uint32_t a;
  int64_t x;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(src)), "r"(rank));
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(x) : "r"(a) : "memory");
  return x;
}

// The last s with first[s] <= x, first[0] = 0.
__device__ __forceinline__ int holder_of(const int* first, int num_seqs, int x) {
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Item i: the i-th token's place, and the i-th page.  Only what the scan wrote is
// read, and table entries and free pages that this step does not write.
__device__ __forceinline__ void fill_token(const TablesParams& p, int t, int tokens, int top) {
  if (t >= tokens) {  // behind the last sequence
    p.positions[t] = 0;
    p.slots[t] = -1;
    return;
  }
  const int page = 1 << p.page_shift;
  const int s = holder_of(p.cu_seqlens, p.num_seqs, t);
  const int begin = p.cu_seqlens[s], n = p.cu_seqlens[s + 1] - begin;
  const int L = p.seqlens_out[s] - n, pos = L + t - begin;
  const int held = (int)(((int64_t)L + page - 1) >> p.page_shift), col = pos >> p.page_shift;
  const int number = col < held ? p.table[(int64_t)s * p.table_stride + col] : p.free_pages[top - 1 - (p.first[s] + col - held)];
  p.positions[t] = pos;
  p.slots[t] = ((int64_t)number << p.page_shift) + (pos & (page - 1));
}
__device__ __forceinline__ void fill_page(const TablesParams& p, int i, int base) {
  const int64_t page = 1 << p.page_shift;
  const int s = holder_of(p.first, p.num_seqs, i);
  if (p.extend) {
    const int64_t L = p.seqlens_out[s] - (p.cu_seqlens[s + 1] - p.cu_seqlens[s]);
    const int64_t col = ((L + page - 1) >> p.page_shift) + i - p.first[s];
    p.table[s * p.table_stride + col] = p.free_pages[base - 1 - i];
  } else {
    const int64_t col = ((p.seqlens_out[s] + page - 1) >> p.page_shift) + i - p.first[s];
    p.free_pages[base + i] = p.table[s * p.table_stride + col];
  }
}
__device__ __forceinline__ void fill_step(const TablesParams& p, int64_t at, int64_t stride) {
  const int pages = p.first[p.num_seqs], after = *p.free_count_out;
  const int base = p.extend ? after + pages : after - pages;  // the stack's height before the step
  if (p.extend) {
    const int tokens = p.cu_seqlens[p.num_seqs];
    for (int64_t t = at; t < p.total_tokens; t += stride) fill_token(p, (int)t, tokens, base);
  }
  for (int64_t i = at; i < pages; i += stride) fill_page(p, (int)i, base);
}

__global__ void __launch_bounds__(kTableThreads) tables_kernel(const __grid_constant__ TablesParams p) {
  __shared__ Sums warps[32];
  __shared__ int64_t own[3];  // the CTA's tokens, pages and whether a sequence does not fit
  pdl_launch_dependents();
  pdl_wait();
  const int rank = (int)cluster_rank(), ctas = (int)cluster_size(), tid = threadIdx.x;
  // This CTA's run of sequences, 1024 at a time.
  const int per = (p.num_seqs + ctas - 1) / ctas;
  const int s0 = min(p.num_seqs, rank * per), s1 = min(p.num_seqs, s0 + per);
  const int count = *p.free_count;
  Sums mine{0, 0}, one;
  bool bad = false;
  for (int s = s0 + tid; s < s1; s += kTableThreads) {
    bad = !sequence_sums(p, s, one) || bad;
    mine += one;
  }
  Sums all;
  const Sums before = block_scan(mine, all, warps);  // of the only round, where there is one
  bad = __syncthreads_or(bad) != 0;
  Sums offset{0, 0};
  if (ctas > 1) {
    if (tid == 0) own[0] = all.tokens, own[1] = all.pages, own[2] = bad;
    cluster_sync();
    all = Sums{0, 0};
    for (int r = 0; r < ctas; ++r) {
      const Sums x{remote_load(&own[0], r), remote_load(&own[1], r)};
      if (r < rank) offset += x;
      all += x;
      bad = bad || remote_load(&own[2], r) != 0;
    }
  }
  // Every CTA comes to the same verdict.
  bad = bad || count < 0 || count > p.capacity || all.tokens > p.total_tokens;
  const bool none = !bad && (p.extend ? all.pages > count : all.pages > p.capacity - count);
  const bool refused = bad || none;
  if (refused && rank == 0 && tid == 0) atomicCAS(p.status, 0, none ? (int)kDevNoPages : (int)kDevBadSeqlens);

  Sums at = offset;
  for (int s = s0 + tid; s - tid < s1; s += kTableThreads) {
    Sums x{0, 0}, block;
    const bool on = s < s1;
    if (on && !refused) sequence_sums(p, s, x);
    Sums here;
    if (s1 - s0 <= kTableThreads) {
      here = Sums{at.tokens + before.tokens, at.pages + before.pages};
      block = Sums{0, 0};
    } else {
      here = block_scan(x, block, warps);
      here += at;
    }
    at += block;
    if (on) {
      const int after = refused ? p.seqlens[s] : p.extend ? p.seqlens[s] + p.amount[s] : p.amount[s];
      p.seqlens_out[s] = after;
      p.first[s] = refused ? 0 : (int)here.pages;
      if (p.extend) p.cu_seqlens[s] = refused ? 0 : (int)here.tokens;
    }
  }
  if (rank == 0 && tid == 0) {
    const int pages = refused ? 0 : (int)all.pages;
    p.first[p.num_seqs] = pages;
    if (p.extend) p.cu_seqlens[p.num_seqs] = refused ? 0 : (int)all.tokens;
  }
  // (All CTAs have read the count before the first barrier; a single one reads it above.)
  __syncthreads();
  if (rank == 0 && tid == 0) {
    const int pages = refused ? 0 : (int)all.pages;
    *p.free_count_out = p.extend ? count - pages : count + pages;
  }
  // (What a CTA has in shared memory is read by the others up to here.)
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  if (p.fill) fill_step(p, (int64_t)rank * kTableThreads + tid, (int64_t)ctas * kTableThreads);
}

__global__ void __launch_bounds__(256) tables_fill_kernel(const __grid_constant__ TablesParams p) {
  pdl_launch_dependents();
  pdl_wait();
  fill_step(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

}  // namespace

// One CTA for steps that it can look at in a round or few, else a cluster of eight; a
// second launch, twice the GPU's width, where there are more tokens than that.
constexpr int kOneCtaItems = 2048, kClusterTokens = 32768;

cudaError_t launch_tables(const TablesParams& p0, cudaStream_t stream) {
  TablesParams p = p0;
  const int64_t items = p.extend ? p.total_tokens : std::min<int64_t>((int64_t)p.num_seqs * p.max_pages, p.capacity);
  const int ctas = p.num_seqs <= kTableThreads && items <= kOneCtaItems ? 1 : kCtas;
  p.fill = !p.extend || p.total_tokens <= kClusterTokens;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTableThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tables_kernel, p);
  if (e != cudaSuccess || p.fill) return e;
  const int64_t blocks = std::min<int64_t>((p.total_tokens + 255) / 256, 304 * 4);
  return launch_pdl(tables_fill_kernel, dim3((unsigned)blocks), 256, 0, stream, p);
}

}  // namespace etattn
