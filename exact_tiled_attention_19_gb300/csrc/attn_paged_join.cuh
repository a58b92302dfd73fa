// The second launch of attention over a paged cache.
#pragma once

#include <cstdint>

#include "launchers.h"
#include "cache_ptx.cuh"

namespace etattn {

// Joins the partial states of every unit that a share boundary cut: with
// normalised partial rows O_s and their lse_s, M = max lse_s and
// w_s = exp(lse_s - M):  O = sum w_s O_s / sum w_s,  lse = M + ln sum w_s.
// Block c belongs to share c.  A unit over the shares first .. first + parts
// - 1 has parts - 1 boundaries; the blocks of the shares after the first take
// every (parts - 1)-th row of it, so that a unit cut into many parts is joined
// by many blocks.  A block with several rows gives each to a warp; one with a
// single row (many parts) gives its warps every eighth part of it and adds
// their sums in shared memory.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p) {
  pdl_wait();
  const PagedShare u = p.desc[blockIdx.x];
  if (u.parts == 0) return;
  constexpr int PER = D / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = min(p.row_tile, u.n * p.group - u.row0);
  const int r0 = (int)blockIdx.x - u.first - 1, step = u.parts - 1;  // rows r0, r0 + step, ...
  const bool by_warp = r0 + step < rows;
  auto slot = [&](int part) { return ((int64_t)(u.first + part) * 2 + (part == 0 ? 1 : 0)) * p.row_tile; };
  __shared__ float s_acc[8][D], s_max[8], s_sum[8];
  for (int r = by_warp ? r0 + warp * step : r0; r < rows; r += by_warp ? 8 * step : rows) {
    // A running state over the warp's parts, four at a time: their loads go
    // out together.
    float mx = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    const int hop = by_warp ? 1 : 8;
    for (int s = by_warp ? 0 : warp; s < u.parts; s += 4 * hop) {
      float lse[4], v[4][PER];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool on = s + k * hop < u.parts;
        const int64_t at = slot(on ? s + k * hop : 0) + r;
        lse[k] = on ? p.part_lse[at] : -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[k][i] = on ? p.part_o[at * D + lane * PER + i] : 0.f;
      }
      float top = mx;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = fmaxf(top, lse[k]);
      const float ref = top == -INFINITY ? 0.f : top;  // no key yet, or only NaN sums
      const float f = expf(mx - ref);                  // 0 while there was none
      sum *= f;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] *= f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w = expf(lse[k] - ref);
        sum += w;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += w * v[k][i];  // (a part without a key is a row of zeros)
      }
      mx = top;
    }
    if (!by_warp) {
#pragma unroll
      for (int i = 0; i < PER; ++i) s_acc[warp][lane * PER + i] = acc[i];
      if (lane == 0) s_max[warp] = mx, s_sum[warp] = sum;
      __syncthreads();
      if (warp != 0) return;
#pragma unroll
      for (int x = 0; x < 8; ++x) mx = fmaxf(mx, s_max[x]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        // A warp that saw only NaN sums has s_max -inf and a NaN s_sum.
        const float w = s_max[x] == -INFINITY ? (s_sum[x] == 0.f ? 0.f : 1.f) : expf(s_max[x] - ref);
        sum += w * s_sum[x];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += w * s_acc[x][lane * PER + i];
      }
    }
    if (mx == -INFINITY) mx = 0.f;
    const int rr = u.row0 + r, i = rr / p.group;
    const int head = u.head0 + rr - i * p.group;
    // A row without a key is 0; a NaN sum stays one.
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* dst = static_cast<uint16_t*>(p.o) + (int64_t)(u.t0 + i) * p.o_st + (int64_t)head * p.o_sh + lane * PER;
    if constexpr (PER == 1) {
      dst[0] = (uint16_t)(BF16 ? pack_bf16x2(acc[0] * inv, 0.f) : pack_f16x2(acc[0] * inv, 0.f));
    } else {
#pragma unroll
      for (int j = 0; j < PER; j += 2)
        *reinterpret_cast<uint32_t*>(dst + j) =
            BF16 ? pack_bf16x2(acc[j] * inv, acc[j + 1] * inv) : pack_f16x2(acc[j] * inv, acc[j + 1] * inv);
    }
    if (p.lse != nullptr && lane == 0)
      p.lse[(int64_t)head * p.total_q + u.t0 + i] = sum == 0.f ? -INFINITY : mx + logf(sum);
  }
}

}  // namespace etattn
