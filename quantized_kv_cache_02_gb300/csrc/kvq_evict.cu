// Eviction of a prompt's light tokens (kvq_evict): per (sequence, KV head)
// unit choose the kept tokens, then gather their Key and Value rows into the
// layout that kvq_append takes.
//
// Choice: the first ``first`` and the last ``recent`` tokens stay; of the ones
// between, the ``left`` heaviest, equal weights by lowest token.  A radix
// select over the weights' order-preserving bits finds the left-th largest
// value in four 8-bit passes; one ordered pass then writes the kept tokens.
// Gather: 16 bytes a thread, K and V of a kept row together.

#include "kvq_prompt.h"

namespace kvq {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kGatherThreads = 256;

// Weights in increasing order as unsigned words: -0 equals 0, NaN is lowest.
__device__ __forceinline__ uint32_t order_bits(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sum[kSelThreads / 32];
  __shared__ uint32_t sh_prefix, sh_left;
  const int h = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const EvictSeq sq = p.seq[blockIdx.y];
  int32_t* out = p.index + sq.out_row + (int64_t)h * sq.keep;
  pdl_wait();
  pdl_release();
  if (sq.keep >= sq.len) {  // nothing is evicted
    for (int i = t; i < sq.len; i += kSelThreads) out[i] = i;
    return;
  }
  const float* w = p.weights + (int64_t)h * p.n_tokens + sq.start;
  const int lo = p.first, hi = sq.len - p.recent;  // the tokens that compete
  const uint32_t left = (uint32_t)(sq.keep - p.first - p.recent);
  uint32_t prefix = 0;  // the top bits of the left-th largest, and how many of its equals stay
  if (t == 0) sh_left = left;
  for (int shift = 24; shift >= 0 && left > 0; shift -= 8) {
    if (t < 256) hist[t] = 0;
    __syncthreads();
    for (int i = lo + t; i < hi; i += kSelThreads) {
      const uint32_t x = order_bits(w[i]);
      if (shift == 24 || (x >> (shift + 8)) == prefix) atomicAdd(&hist[(x >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255 - 8 l .. 248 - 8 l; find where the count from the top passes the rank
      uint32_t c[8], mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mine += c[j] = hist[255 - 8 * lane - j];
      uint32_t incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      const uint32_t rank = sh_left;
      uint32_t before = incl - mine;
      __syncwarp();
      if (before < rank && rank <= incl) {
        int j = 0;
        while (before + c[j] < rank) before += c[j++];
        sh_prefix = prefix << 8 | (uint32_t)(255 - 8 * lane - j);
        sh_left = rank - before;
      }
    }
    __syncthreads();
    prefix = sh_prefix;
  }
  __syncthreads();
  // tokens above the value stay, and the first ``ties`` equal ones
  const uint32_t ties = left > 0 ? sh_left : 0u;
  uint32_t n_out = 0, n_tie = 0;
  for (int i0 = 0; i0 < sq.len; i0 += kSelThreads) {
    const int i = i0 + t;
    bool stay = false, tie = false;
    if (i < sq.len) {
      stay = i < lo || i >= hi;
      if (!stay && left > 0) {
        const uint32_t x = order_bits(w[i]);
        stay = x > prefix;
        tie = x == prefix;
      }
    }
    const uint32_t bs = __ballot_sync(0xffffffffu, stay), bt = __ballot_sync(0xffffffffu, tie);
    const uint32_t below = (1u << lane) - 1u;
    __syncthreads();
    if (lane == 0) warp_sum[warp] = (uint32_t)__popc(bs) << 16 | (uint32_t)__popc(bt);
    __syncthreads();
    // both counts of a step fit 16 bits: one scan over the warps' pairs
    const uint32_t pair = warp_sum[lane];
    uint32_t incl = pair;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    const uint32_t excl = __shfl_sync(0xffffffffu, incl - pair, warp);
    const uint32_t total = __shfl_sync(0xffffffffu, incl, 31);
    const uint32_t tie_rank = n_tie + (excl & 0xffffu) + (uint32_t)__popc(bt & below);
    const uint32_t ties_before = min(tie_rank, ties);
    const uint32_t pos = n_out + (excl >> 16) + (uint32_t)__popc(bs & below) + ties_before;
    if (stay || (tie && tie_rank < ties)) out[pos] = i;
    n_out += total >> 16;
    n_tie += total & 0xffffu;
  }
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const __grid_constant__ EvictParams p) {
  const int h = blockIdx.y;
  const EvictSeq sq = p.seq[blockIdx.z];
  const int per = p.row_bytes / 16;
  const int64_t base = sq.out_row + (int64_t)h * sq.keep;
  const int64_t n = (int64_t)sq.keep * per;
  pdl_wait();
  pdl_release();
  for (int64_t i = (int64_t)blockIdx.x * kGatherThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kGatherThreads) {
    const int r = (int)(i / per), c = (int)(i - (int64_t)r * per) * 16;
    const int64_t tok = (int64_t)sq.start + p.index[base + r];
    const uint4 a = *reinterpret_cast<const uint4*>(p.k + tok * p.k_ts + (int64_t)h * p.k_hs + c);
    const uint4 b = *reinterpret_cast<const uint4*>(p.v + tok * p.v_ts + (int64_t)h * p.v_hs + c);
    *reinterpret_cast<uint4*>(p.k_out + (base + r) * p.row_bytes + c) = a;
    *reinterpret_cast<uint4*>(p.v_out + (base + r) * p.row_bytes + c) = b;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int32_t max_len, int32_t max_keep, cudaStream_t s) {
  (void)max_len;
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(p.Hkv, p.n_seqs), dim3(kSelThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  const int64_t chunks = (int64_t)max_keep * (p.row_bytes / 16);
  const unsigned bx = (unsigned)((chunks + 4 * kGatherThreads - 1) / (4 * kGatherThreads));
  return launch_pdl(evict_gather_kernel, dim3(bx, p.Hkv, p.n_seqs), dim3(kGatherThreads), 0, s, p);
}

}  // namespace kvq
