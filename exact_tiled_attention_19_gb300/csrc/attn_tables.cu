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
// bytes each, so launches and chains of dependent loads bound it.
//  * Up to 4096 sequences, every CTA sums all of them up, a thread one or four, and has the
//    sums in shared memory, where tokens and pages find their sequence by bisection: no
//    CTA waits for another, and one launch of as many CTAs as the tokens want does
//    everything.  Where lengths and count are updated in place, none may be written before all
//    CTAs have read them: a cluster of eight with a barrier then, or for many tokens a
//    launch of one CTA and a wide one after it.
//  * More sequences are divided among a cluster of eight, which exchanges its sums, after
//    which every CTA knows whether the step fits, before anything is written; the
//    offsets go through memory.  (Eight, as a cluster is the widest group that may wait for its
//    own in a launch; a wider sum would be three launches and a scratch that outlives them, for
//    batches that are rare: 20000 sequences take 18.5 us, 14.9 to truncate.)  A step of many tokens has them filled in by a second
//    launch as wide as the GPU.
//
// Measured (GB300, device time): 8 sequences, one token each, 3.6 us; 1000 sequences with prompts,
// 7.0 us in one launch (11.8 by the cluster, whose barriers and exchange cost about 3 us);
// 4000 sequences truncated 6.4 us (10.0 by the cluster); 20000 sequences, one token each, 18.5 us.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "launchers.h"
#include "cache_ptx.cuh"

namespace etattn {

namespace {

constexpr int kTableThreads = 1024, kCtas = 8;
static_assert(kTablesNoScratch == 4 * kTableThreads, "");

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

// Where the sums of a step are: tokens and pages before each sequence, and the keys
// that each has then.
struct Step {
  const int *cu, *first, *after;
  int tokens, pages, base;  // of the step; the stack's height before it
};

// Token t's place.  Only the step's sums are read, and table entries and free pages
// that this step does not write.
__device__ __forceinline__ void fill_token(const TablesParams& p, const Step& x, int t) {
  if (t >= x.tokens) {  // behind the last sequence
    p.positions[t] = 0;
    p.slots[t] = -1;
    return;
  }
  const int page = 1 << p.page_shift;
  const int s = holder_of(x.cu, p.num_seqs, t);
  const int begin = x.cu[s], L = x.after[s] - (x.cu[s + 1] - begin), pos = L + t - begin;
  const int held = (int)(((int64_t)L + page - 1) >> p.page_shift), col = pos >> p.page_shift;
  const int number = col < held ? p.table[(int64_t)s * p.table_stride + col] : p.free_pages[x.base - 1 - (x.first[s] + col - held)];
  p.positions[t] = pos;
  p.slots[t] = ((int64_t)number << p.page_shift) + (pos & (page - 1));
}
// Page i of the step.
__device__ __forceinline__ void fill_page(const TablesParams& p, const Step& x, int i) {
  const int64_t page = 1 << p.page_shift;
  const int s = holder_of(x.first, p.num_seqs, i);
  const int64_t kept = p.extend ? x.after[s] - (x.cu[s + 1] - x.cu[s]) : x.after[s];
  const int64_t at = s * p.table_stride + ((kept + page - 1) >> p.page_shift) + i - x.first[s];
  if (p.extend) p.table[at] = p.free_pages[x.base - 1 - i];
  else p.free_pages[x.base + i] = p.table[at];
}
__device__ __forceinline__ void fill_step(const TablesParams& p, const Step& x, int64_t at, int64_t stride) {
  if (p.extend)
    for (int64_t t = at; t < p.total_tokens; t += stride) fill_token(p, x, (int)t);
  for (int64_t i = at; i < x.pages; i += stride) fill_page(p, x, (int)i);
}
// The step that an earlier launch, or an earlier part of this one, left in memory.
__device__ __forceinline__ Step step_in_memory(const TablesParams& p) {
  Step x{p.cu_seqlens, p.first, p.seqlens_out, 0, p.first[p.num_seqs], 0};
  x.tokens = p.extend ? p.cu_seqlens[p.num_seqs] : 0;
  x.base = p.extend ? *p.free_count_out + x.pages : *p.free_count_out - x.pages;
  return x;
}

// Whether a step fits; if not, it is recorded once.
__device__ __forceinline__ bool step_refused(const TablesParams& p, const Sums& all, bool bad, int count, bool record) {
  bad = bad || count < 0 || count > p.capacity || all.tokens > p.total_tokens;
  const bool none = !bad && (p.extend ? all.pages > count : all.pages > p.capacity - count);
  if ((bad || none) && record) atomicCAS(p.status, 0, none ? (int)kDevNoPages : (int)kDevBadSeqlens);
  return bad || none;
}

// Up to 1024 PER sequences, PER of a thread.  again: the lengths and the count have been
// updated by an earlier launch, and this one takes the step from what it wrote.
template <int PER>
__global__ void __launch_bounds__(kTableThreads) tables_small_kernel(const __grid_constant__ TablesParams p, int again) {
  __shared__ Sums warps[32];
  extern __shared__ int sums[];  // [3][1024 PER + 1]
  constexpr int kMost = kTableThreads * PER;
  int *s_cu = sums, *s_first = sums + kMost + 1, *s_after = sums + 2 * (kMost + 1);
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, s0 = tid * PER;
  const bool writes = blockIdx.x == 0 && !again;
  int count = again ? *p.free_count_out : *p.free_count;
  Sums each[PER], mine{0, 0}, all;
  bool bad = false;
  int before[PER], after[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = s0 + i;
    before[i] = after[i] = 0;
    each[i] = Sums{0, 0};
    if (s >= p.num_seqs) continue;
    if (again) {  // (of an extension alone: a truncation is one launch)
      const int n = p.cu_seqlens[s + 1] - p.cu_seqlens[s];
      const int64_t page = int64_t(1) << p.page_shift, L = p.seqlens_out[s] - n;
      after[i] = p.seqlens_out[s];
      each[i] = Sums{n, ((L + n + page - 1) >> p.page_shift) - ((L + page - 1) >> p.page_shift)};
    } else {
      bad = !sequence_sums(p, s, each[i]) || bad;
      before[i] = p.seqlens[s];
      after[i] = p.extend ? before[i] + p.amount[s] : p.amount[s];
    }
    mine += each[i];
  }
  Sums here = block_scan(mine, all, warps);
  bad = __syncthreads_or(bad) != 0;
  bool refused = false;
  if (again) count += (int)all.pages;  // (what it was before)
  else refused = step_refused(p, all, bad, count, writes && tid == 0);
  if (refused) all = Sums{0, 0};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (s0 + i < p.num_seqs) {
      s_cu[s0 + i] = refused ? 0 : (int)here.tokens;
      s_first[s0 + i] = refused ? 0 : (int)here.pages;
      s_after[s0 + i] = refused ? before[i] : after[i];
    }
    here += each[i];
  }
  if (tid == 0) s_cu[p.num_seqs] = (int)all.tokens, s_first[p.num_seqs] = (int)all.pages;
  // Everybody has read what is updated in place: in this CTA, and in the cluster.
  if (cluster_size() > 1) cluster_sync();
  else __syncthreads();
  if (writes) {
    for (int s = tid; s < p.num_seqs; s += kTableThreads) p.seqlens_out[s] = s_after[s];
    if (p.extend)
      for (int s = tid; s <= p.num_seqs; s += kTableThreads) p.cu_seqlens[s] = s_cu[s];
    if (tid == 0) *p.free_count_out = p.extend ? count - (int)all.pages : count + (int)all.pages;
  }
  if (!p.fill) return;
  const Step step{s_cu, s_first, s_after, (int)all.tokens, (int)all.pages, count};
  fill_step(p, step, (int64_t)blockIdx.x * kTableThreads + tid, (int64_t)gridDim.x * kTableThreads);
}

// More sequences: one cluster.
__global__ void __launch_bounds__(kTableThreads) tables_kernel(const __grid_constant__ TablesParams p) {
  __shared__ Sums warps[32];
  __shared__ int64_t own[3];  // the CTA's tokens, pages and whether a sequence does not fit
  pdl_launch_dependents();
  pdl_wait();
  const int rank = (int)cluster_rank(), tid = threadIdx.x;
  constexpr int ctas = kCtas;
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
  if (tid == 0) own[0] = all.tokens, own[1] = all.pages, own[2] = bad;
  cluster_sync();
  all = Sums{0, 0};
  for (int r = 0; r < ctas; ++r) {
    const Sums x{remote_load(&own[0], r), remote_load(&own[1], r)};
    if (r < rank) offset += x;
    all += x;
    bad = bad || remote_load(&own[2], r) != 0;
  }
  // Every CTA comes to the same verdict.
  const bool refused = step_refused(p, all, bad, count, rank == 0 && tid == 0);

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
  if (rank == 0 && tid == 0) {  // (all CTAs have read the count before the first barrier)
    const int pages = refused ? 0 : (int)all.pages;
    *p.free_count_out = p.extend ? count - pages : count + pages;
  }
  cluster_sync();  // (what a CTA has in shared memory is read by the others up to here)
  if (p.fill) fill_step(p, step_in_memory(p), (int64_t)rank * kTableThreads + tid, (int64_t)ctas * kTableThreads);
}

__global__ void __launch_bounds__(256) tables_fill_kernel(const __grid_constant__ TablesParams p) {
  pdl_launch_dependents();
  pdl_wait();
  fill_step(p, step_in_memory(p), (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

}  // namespace

// Tokens and pages that one CTA takes; tokens that a cluster does before a wide launch of
// their own is faster: where the sums are in shared memory (in place; 4000 sequences with
// 16000 tokens and their truncation 15.9 us by the cluster, 18.5 by two launches), and where they are
// in memory, which eight CTAs bisect more slowly (5000 tokens 12.5 and 13.4, 16000 14.3 and 13.2,
// 32000 18.6 and 12.8).
constexpr int kOneCtaItems = 2048, kClusterTokens = 32768, kClusterTokensInMemory = 8192, kWideCtas = 304;

cudaError_t launch_tables(const TablesParams& p0, cudaStream_t stream) {
  TablesParams p = p0;
  p.fill = 1;
  // (Of a truncation the pages are known to their bound alone.)
  const int64_t items = p.extend ? p.total_tokens : std::min<int64_t>((int64_t)p.num_seqs * p.max_pages, p.capacity);
  auto launch = [&](auto kern, int smem, int ctas, int cluster, auto... more) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.dynamicSmemBytes = smem;
    cfg.blockDim = dim3(kTableThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, more...);
  };
  if (p.num_seqs <= kTablesNoScratch) {
    const bool one_each = p.num_seqs <= kTableThreads;
    const int smem = 3 * ((one_each ? 1 : 4) * kTableThreads + 1) * 4;
    if (!one_each) {
      static std::atomic<unsigned long long> configured{0};
      int dev = 0;
      cudaError_t e = cudaGetDevice(&dev);
      if (e != cudaSuccess) return e;
      const unsigned long long bit = 1ull << (dev & 63);
      if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(tables_small_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
      }
    }
    auto small = [&](int ctas, int cluster, int again) {
      return launch(one_each ? tables_small_kernel<1> : tables_small_kernel<4>, smem, ctas, cluster, again);
    };
    if (items <= kOneCtaItems) return small(1, 1, 0);
    const bool in_place = p.seqlens == p.seqlens_out || p.free_count == p.free_count_out;
    const int wide = (int)std::min<int64_t>((items + kTableThreads - 1) / kTableThreads, kWideCtas);
    if (!in_place) return small(wide, 1, 0);
    if (!p.extend || items <= kClusterTokens) return small(kCtas, kCtas, 0);
    p.fill = 0;
    const cudaError_t e = small(1, 1, 0);
    if (e != cudaSuccess) return e;
    p.fill = 1;
    return small(wide, 1, 1);
  }
  p.fill = !p.extend || p.total_tokens <= kClusterTokensInMemory;
  const cudaError_t e = launch(tables_kernel, 0, kCtas, kCtas);
  if (e != cudaSuccess || p.fill) return e;
  const int64_t blocks = std::min<int64_t>((p.total_tokens + 255) / 256, 4 * kWideCtas);
  return launch_pdl(tables_fill_kernel, dim3((unsigned)blocks), 256, 0, stream, p);
}

}  // namespace etattn
