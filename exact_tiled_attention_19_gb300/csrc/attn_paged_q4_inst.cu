// The instantiations of attention over a 4-bit paged cache for one (head dim,
// element type) and its launcher, compiled once per variant with
// -DETATTN_INST_D=<32|64|128> -DETATTN_INST_BF16=<0|1> (like attn_paged_inst.cu).
#include <atomic>
#include <cuda_runtime.h>

#include "attn_paged_join.cuh"
#include "attn_paged_q4_kernel.cuh"
#include "launchers.h"

#ifndef ETATTN_INST_D
#error "ETATTN_INST_D must be defined"
#endif
#ifndef ETATTN_INST_BF16
#error "ETATTN_INST_BF16 must be defined"
#endif

#define ETATTN_PCAT2(a, b, c) a##b##_##c
#define ETATTN_PCAT(a, b, c) ETATTN_PCAT2(a, b, c)
#define ETATTN_PAGED_Q4_LAUNCHER ETATTN_PCAT(launch_paged_q4_d, ETATTN_INST_D, ETATTN_INST_BF16)

namespace etattn {

namespace {

template <int MT, bool SPREAD>
cudaError_t launch_one(const PagedQ4Params& p, cudaStream_t stream) {
  using C = PagedQ4Cfg<ETATTN_INST_D, MT>;
  auto kern = attn_paged_q4_kernel<ETATTN_INST_D, MT, ETATTN_INST_BF16 != 0, SPREAD>;
  // The dynamic shared-memory opt-in is per device; set it once per device.
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  e = launch_pdl(kern, dim3(p.shares), C::THREADS, C::SMEM_BYTES, stream, p);
  if (e != cudaSuccess || p.shares == 1) return e;
  return launch_pdl(paged_join_kernel<ETATTN_INST_D, ETATTN_INST_BF16 != 0>, dim3(p.shares), 256, 0, stream,
                    static_cast<const PagedParams&>(p));
}

template <int MT>
cudaError_t launch_rows(const PagedQ4Params& p, cudaStream_t stream) {
  return (1 << p.page_shift) <= PagedQ4Cfg<ETATTN_INST_D, MT>::SPREAD ? launch_one<MT, true>(p, stream)
                                                                      : launch_one<MT, false>(p, stream);
}

}  // namespace

cudaError_t ETATTN_PAGED_Q4_LAUNCHER(const PagedQ4Params& p, cudaStream_t stream) {
  if (p.row_tile == 4) return launch_rows<4>(p, stream);
  return p.row_tile == 8 ? launch_rows<8>(p, stream) : launch_rows<16>(p, stream);
}

}  // namespace etattn
