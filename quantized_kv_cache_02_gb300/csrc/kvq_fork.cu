// The copies of kvq_fork: whole sequences of a cache, in place and all at once.
//
// Bound: HBM.  Every live column of a source is read once and written to each
// of its copies, so one source sampled n times costs 1 + n passes over its
// bytes and not 2 n.  What must not move is not moved: a paged cache's blocks are
// shared (a flushed page is never written again), so only its block-table row, range
// maxima and window are copied; dead rows of a window's ring stay as they are.
//
// Sources may be overwritten by the same call (a beam search's survivors change
// places).  No thread depends on another: it holds the same columns of every
// sequence, and the host orders the steps so that each sequence is read before it is
// written; of a cycle one sequence's columns wait in registers.

#include <algorithm>

#include "kvq_internal.h"

namespace kvq {
namespace {

struct alignas(16) Quad {
  uint32_t w[4];
};

template <typename V, int N>
__device__ __forceinline__ void copy_columns(const ForkParams<N>& p, const ForkRegion& r, int unit, int64_t col0) {
  V v[kForkDepth], held[kForkDepth];
  bool held_live[kForkDepth] = {};
  auto place = [&](int seq) {
    if (r.by_layout) return r.base + p.layout[seq].page_base + unit * p.layout[seq].unit_stride;
    return r.base + seq * r.seq_stride + unit * r.unit_stride;
  };
  for (int at = p.component[blockIdx.y]; at < p.component[blockIdx.y + 1]; ++at) {
    const ForkStep& s = p.step[at];
    bool live[kForkDepth];
    const int64_t bytes = r.live_tokens ? s.ctr.quantized / r.live_tokens * r.live_bytes : r.live_bytes;
    const uint8_t* src = s.held ? nullptr : place(s.src);
#pragma unroll
    for (int e = 0; e < kForkDepth; ++e) {
      const int64_t off = (col0 + e * kForkThreads) * (int64_t)sizeof(V);
      if (s.held) {
        live[e] = held_live[e];
        v[e] = held[e];
        continue;
      }
      if (r.ring) {
        // a row of the ring holds a token of the window
        const int64_t row = off / r.ring;
        const int from = s.ctr.quantized % p.rcap;
        const int after = (int)row >= from ? (int)row - from : (int)row - from + p.rcap;
        live[e] = row < p.rcap && after < s.ctr.total - s.ctr.quantized;
      } else {
        live[e] = off < bytes;
      }
      if (live[e]) v[e] = *reinterpret_cast<const V*>(src + off);
    }
    if (s.count == 0) {
#pragma unroll
      for (int e = 0; e < kForkDepth; ++e) {
        held[e] = v[e];
        held_live[e] = live[e];
      }
    }
    for (int d = 0; d < s.count; ++d) {
      uint8_t* dst = place(p.dst[s.first + d]);
#pragma unroll
      for (int e = 0; e < kForkDepth; ++e)
        if (live[e]) *reinterpret_cast<V*>(dst + (col0 + e * kForkThreads) * (int64_t)sizeof(V)) = v[e];
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ ForkParams<N> p) {
  int n = 0;
  while (n + 1 < p.n_regions && p.region[n + 1].first_block <= blockIdx.x) ++n;
  const ForkRegion& r = p.region[n];
  const int64_t per_unit = (r.cols + kForkCols - 1) / kForkCols;
  const int64_t at = blockIdx.x - r.first_block;
  const int unit = (int)(at / per_unit);
  const int64_t col0 = (at - unit * per_unit) * kForkCols + threadIdx.x;
  pdl_wait();
  pdl_release();
  if (r.grain == 16) copy_columns<Quad, N>(p, r, unit, col0);
  else copy_columns<uint32_t, N>(p, r, unit, col0);
}

}  // namespace

cudaError_t launch_fork(const ForkParams<kMaxForkSteps>& p, int steps, int copies, int64_t blocks, int components,
                        cudaStream_t s) {
  const dim3 grid((unsigned)blocks, (unsigned)components), block(kForkThreads);
  if (steps > kFewForkSteps || copies > kFewForkSteps) return launch_pdl(fork_kernel<kMaxForkSteps>, grid, block, 0, s, p);
  ForkParams<kFewForkSteps> few;
  few.n_regions = p.n_regions;
  few.rcap = p.rcap;
  few.layout = p.layout;
  std::copy(p.region, p.region + p.n_regions, few.region);
  std::copy(p.component, p.component + components + 1, few.component);
  std::copy(p.step, p.step + steps, few.step);
  std::copy(p.dst, p.dst + copies, few.dst);
  return launch_pdl(fork_kernel<kFewForkSteps>, grid, block, 0, s, few);
}

}  // namespace kvq
