// Eviction of a prompt's light tokens (kvq_evict): per (sequence, KV head)
// unit choose the kept tokens, then gather their Key and Value rows into the
// layout that kvq_append takes.
//
// Choice.  The first ``first`` and the last ``recent`` tokens stay; of the ones
// between, the ``left`` heaviest, equal weights by lowest token.  A cluster of up
// to 16 CTAs takes a unit, a run of its tokens each, kept in shared memory as
// order-preserving words.  A radix select finds the left-th largest word in
// passes of 11, 11 and 10 bits (each CTA counts its run, all read every CTA's
// counts through distributed shared memory: one cluster barrier a pass); one
// ordered pass then writes the kept tokens.  Every weight is read once.
//
// Gather.  A thread has four 16-byte pieces of K and of V in flight.  Bound by
// HBM: 16 bytes a kept piece read and written.  Small choices gather in the
// choosing CTA and save the second launch.

#include <algorithm>

#include "kvq_prompt.h"

namespace kvq {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;
constexpr int kCached = 48 * 1024;   // words of a run that shared memory holds; a longer one is read again a pass
constexpr int kGatherThreads = 256, kPieces = 4 * kGatherThreads;

// Weights in increasing order as unsigned words: -0 equals 0, NaN is lowest.
__device__ __forceinline__ uint32_t order_bits(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct SelShared {
  uint32_t hist[3][kBins];
  uint32_t warp_sum[kSelWarps];
  uint32_t above[kSelWarps], equal[kSelWarps];  // kept and tied words of each warp's stretch
  uint32_t totals[2];                           // of the CTA
  uint32_t digit, rank;
};

__device__ __forceinline__ void cluster_barrier(int size) {
  __syncwarp();
  if (size > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
}
// A word of another rank's shared memory.
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, int rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Sum over the threads before this one (and, in *all, over all).
__device__ __forceinline__ uint32_t scan_before(uint32_t x, SelShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sh.warp_sum[warp] = incl;
  __syncthreads();
  uint32_t w = sh.warp_sum[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  const uint32_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return incl - x + (warp > 0 ? before : 0u);
}

// Copy kept rows [r0, r0 + rows) of a unit.
__device__ __forceinline__ void gather_rows(const EvictParams& p, const EvictSeq& sq, int h, int64_t r0, int rows,
                                            int per, int t, int threads) {
  const int64_t base = sq.out_row + (int64_t)h * sq.keep + r0;
  const int n = rows * per;
  for (int i0 = t; i0 < n; i0 += 4 * threads) {
    uint4 a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e * threads;
      if (i < n) {
        const int r = i / per, c = (i - r * per) * 16;
        const int64_t tok = (int64_t)sq.start + p.index[base + r];
        a[e] = __ldcs(reinterpret_cast<const uint4*>(p.k + tok * p.k_ts + (int64_t)h * p.k_hs + c));
        b[e] = __ldcs(reinterpret_cast<const uint4*>(p.v + tok * p.v_ts + (int64_t)h * p.v_hs + c));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e * threads;
      if (i < n) {
        const int r = i / per, c = (i - r * per) * 16;
        *reinterpret_cast<uint4*>(p.k_out + (base + r) * p.row_bytes + c) = a[e];
        *reinterpret_cast<uint4*>(p.v_out + (base + r) * p.row_bytes + c) = b[e];
      }
    }
  }
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint8_t sel_smem[];
  SelShared& sh = *reinterpret_cast<SelShared*>(sel_smem);
  uint32_t* run = reinterpret_cast<uint32_t*>(sel_smem + sizeof(SelShared));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int size = gridDim.x, rank = blockIdx.x, h = blockIdx.y;  // a cluster is one unit
  const EvictSeq sq = p.seq[blockIdx.z];
  int32_t* out = p.index + sq.out_row + (int64_t)h * sq.keep;
  for (int i = t; i < 3 * kBins; i += kSelThreads) sh.hist[0][i] = 0;
  pdl_wait();
  pdl_release();
  if (sq.keep >= sq.len) {  // nothing is evicted
    for (int i = rank * kSelThreads + t; i < sq.len; i += size * kSelThreads) out[i] = i;
  } else {
    const int lo = p.first, hi = sq.len - p.recent;  // the tokens that compete
    const uint32_t left = (uint32_t)(sq.keep - p.first - p.recent);
    for (int i = rank * kSelThreads + t; i < lo; i += size * kSelThreads) out[i] = i;
    for (int i = rank * kSelThreads + t; i < p.recent; i += size * kSelThreads) out[lo + left + i] = hi + i;
    if (left > 0) {
      // this CTA's run of them
      const int share = (hi - lo + size - 1) / size, r0 = min(hi, lo + rank * share), n = min(hi, r0 + share) - r0;
      const float* w = p.weights + (int64_t)h * p.n_tokens + sq.start + r0;
      const bool cached = share <= kCached;
      auto word = [&](int i) { return cached ? run[i] : order_bits(w[i]); };
      __syncthreads();
      uint32_t prefix = 0, need = left;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        uint32_t* hist = sh.hist[pass];
        const int whole = (n + kSelThreads - 1) / kSelThreads * kSelThreads;
#pragma unroll 4
        for (int i = t; i < whole; i += kSelThreads) {
          bool in = i < n;
          uint32_t x = 0;
          if (in) {
            if (pass == 0) {
              x = order_bits(__ldcs(w + i));
              if (cached) run[i] = x;
            } else {
              x = word(i);
              in = x >> (pass == 1 ? 21 : 10) == prefix;
            }
          }
          const uint32_t d = (x >> shift) & mask;
          // equal weights (a prompt's many zeros) would queue up at one counter
          int same;
          __match_all_sync(0xffffffffu, in ? d : ~0u, &same);
          if (same) {
            if (lane == 0 && in) atomicAdd(&hist[d], 32u);
          } else if (in) {
            atomicAdd(&hist[d], 1u);
          }
        }
        cluster_barrier(size);
        // bins from the top, two a thread, over the cluster
        uint32_t c0 = 0, c1 = 0;
        const int b0 = kBins - 1 - 2 * t;
        if (size > 1) {
#pragma unroll 4
          for (int r = 0; r < size; ++r) {
            c0 += peer_word(hist + b0, r);
            c1 += peer_word(hist + b0 - 1, r);
          }
        } else {
          c0 = hist[b0];
          c1 = hist[b0 - 1];
        }
        const uint32_t before = scan_before(c0 + c1, sh);
        if (before < need && need <= before + c0 + c1) {
          const bool second = need > before + c0;
          sh.digit = (uint32_t)(second ? b0 - 1 : b0);
          sh.rank = need - before - (second ? c0 : 0u);
        }
        __syncthreads();
        prefix = pass == 2 ? prefix << 10 | sh.digit : prefix << 11 | sh.digit;
        need = sh.rank;
        __syncthreads();
      }
      // Words above the left-th largest stay, and the first ``need`` equal to it.
      // Each warp counts a stretch of the run, then writes it in order.
      const int stretch = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31, s0 = min(n, warp * stretch),
                s1 = min(n, s0 + stretch);
      uint32_t above = 0, equal = 0;
      for (int i0 = s0; i0 < s1; i0 += 32) {
        const uint32_t x = i0 + lane < s1 ? word(i0 + lane) : 0u;
        above += __popc(__ballot_sync(0xffffffffu, i0 + lane < s1 && x > prefix));
        equal += __popc(__ballot_sync(0xffffffffu, i0 + lane < s1 && x == prefix));
      }
      if (lane == 0) {
        sh.above[warp] = above;
        sh.equal[warp] = equal;
      }
      __syncthreads();
      uint32_t wa = sh.above[lane], we = sh.equal[lane];  // running sums over the warps
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t ya = __shfl_up_sync(0xffffffffu, wa, d), ye = __shfl_up_sync(0xffffffffu, we, d);
        if (lane >= d) {
          wa += ya;
          we += ye;
        }
      }
      if (t == 31) {
        sh.totals[0] = wa;
        sh.totals[1] = we;
      }
      uint32_t n_above = __shfl_sync(0xffffffffu, wa, warp) - above, n_equal = __shfl_sync(0xffffffffu, we, warp) - equal;
      cluster_barrier(size);
      if (size > 1) {
        for (int r = 0; r < rank; ++r) {
          n_above += peer_word(&sh.totals[0], r);
          n_equal += peer_word(&sh.totals[1], r);
        }
      }
      const uint32_t below = (1u << lane) - 1u;
      for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t x = i < s1 ? word(i) : 0u;
        const bool up = i < s1 && x > prefix, tie = i < s1 && x == prefix;
        const uint32_t ba = __ballot_sync(0xffffffffu, up), be = __ballot_sync(0xffffffffu, tie);
        const uint32_t ties = n_equal + __popc(be & below);
        if (up || (tie && ties < need))
          out[lo + n_above + __popc(ba & below) + min(ties, need)] = r0 + i;
        n_above += __popc(ba);
        n_equal += __popc(be);
      }
      if (size > 1) cluster_barrier(size);  // no rank ends while another reads its counts
    }
  }
  if (p.gather_here) {
    __syncthreads();
    gather_rows(p, sq, h, 0, sq.keep, p.row_bytes / 16, t, kSelThreads);
  }
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const __grid_constant__ EvictParams p) {
  const EvictSeq sq = p.seq[blockIdx.z];
  const int per = p.row_bytes / 16, rows = kPieces / per;
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  pdl_wait();
  pdl_release();
  if (r0 < sq.keep)
    gather_rows(p, sq, blockIdx.y, r0, (int)min((int64_t)rows, sq.keep - r0), per, threadIdx.x, kGatherThreads);
}

}  // namespace

cudaError_t launch_evict(EvictParams& p, int32_t max_len, int32_t max_keep, cudaStream_t s, int* launches) {
  // one CTA for a few thousand tokens, else runs of about 4096 over a cluster
  int size = 1;
  while (size < kMaxCluster && max_len > 8192 * size) size *= 2;
  const int share = (max_len + size - 1) / size;
  const size_t smem = sizeof(SelShared) + (size_t)std::min(share, kCached) * sizeof(uint32_t);
  // up to 64 KB of rows a unit the choosing CTA copies them itself
  p.gather_here = size == 1 && (int64_t)max_keep * p.row_bytes <= 32 * 1024;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(sizeof(SelShared) + kCached * sizeof(uint32_t)));
  if (e == cudaSuccess && size > 8)
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)size, (unsigned)p.Hkv, (unsigned)p.n_seqs);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = size > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
  *launches = 1;
  if (e != cudaSuccess || p.gather_here) return e;
  const int rows = kPieces / (p.row_bytes / 16);
  *launches = 2;
  return launch_pdl(evict_gather_kernel, dim3((unsigned)((max_keep + rows - 1) / rows), p.Hkv, p.n_seqs),
                    dim3(kGatherThreads), 0, s, p);
}

}  // namespace kvq
