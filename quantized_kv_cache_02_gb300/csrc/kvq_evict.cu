// Eviction of a prompt's light tokens (kvq_evict): per (sequence, KV head)
// unit choose the kept tokens, then gather their Key and Value rows into the
// layout that kvq_append takes.
//
// Choice.  The first ``first`` and the last ``recent`` tokens stay; of the ones
// between, the ``left`` heaviest, equal weights by lowest token.  A cluster of up
// to 16 CTAs takes a unit, a run of its tokens each, kept in shared memory as
// order-preserving words.  A radix select finds the left-th largest word eight
// bits at a time (each CTA counts its run, all add up every CTA's 256 counts
// through distributed shared memory: one cluster barrier a pass); one ordered
// pass then writes the kept tokens.  Every weight is read once.
// Eight units of 432,000 tokens take 27 us as clusters of 12, which run at
// once; of 16 (in two waves, or two CTAs an SM) 56 and 41 us, and passes of 11
// bits, whose 2048 counters are read from every peer, 163 us.
//
// Gather.  The unit's CTAs then copy its rows, an equal share each, with four
// 16-byte pieces of K and of V in flight a thread.  Bound by HBM: 16 bytes a kept
// piece read and written.  A second kernel for the copies has every SM for few
// units but starts later and costs the host a launch: eight ragged prompts (67 MB
// in all) 22.8 us against 19.6 us, one of 432,000 tokens (132 MB) 47.7 us against
// 48.5 us.

#include <algorithm>
#include <atomic>

#include "kvq_prompt.h"

namespace kvq {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kCached = 55 * 1024;   // words of a run that shared memory holds; a longer one is read again a pass

// Weights in increasing order as unsigned words: -0 equals 0, NaN is lowest.
__device__ __forceinline__ uint32_t order_bits(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct SelShared {
  uint32_t hist[4][256];                        // the CTA's counts, a pass each
  uint32_t sums[256];                           // the cluster's
  uint32_t above[kSelWarps], equal[kSelWarps];  // running sums of each warp's kept and tied words
  uint32_t totals[2];                           // of the CTA
  uint32_t digit, rank;
};
constexpr int kSelSmemMax = (int)(sizeof(SelShared) + kCached * sizeof(uint32_t));
static_assert(kSelSmemMax <= 227 * 1024, "a run has to fit shared memory");

template <bool CLUSTER>
__device__ __forceinline__ void unit_barrier() {
  __syncwarp();
  if (CLUSTER)
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

// Four words of another rank's shared memory.
__device__ __forceinline__ uint4 peer_words(const uint32_t* p, int rank) {
  uint32_t a;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Copy kept rows [r0, r1) of a unit.
__device__ __forceinline__ void gather_rows(const EvictParams& p, const EvictSeq& sq, int h, int r0, int r1, int t) {
  constexpr int kBlock = 1 << 16;  // rows whose pieces an int counts
  const int per = p.row_bytes / 16;
  for (int64_t rb = r0; rb < r1; rb += kBlock) {
    const int64_t base = sq.out_row + (int64_t)h * sq.keep + rb;
    const int n = (int)min((int64_t)kBlock, r1 - rb) * per;
    for (int i0 = t; i0 < n; i0 += 4 * kSelThreads) {
      uint4 a[4], b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kSelThreads;
        if (i < n) {
          const int r = i / per, c = (i - r * per) * 16;
          const int64_t tok = (int64_t)sq.start + p.index[base + r];
          a[e] = __ldcs(reinterpret_cast<const uint4*>(p.k + tok * p.k_ts + (int64_t)h * p.k_hs + c));
          b[e] = __ldcs(reinterpret_cast<const uint4*>(p.v + tok * p.v_ts + (int64_t)h * p.v_hs + c));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kSelThreads;
        if (i < n) {
          const int r = i / per, c = (i - r * per) * 16;
          *reinterpret_cast<uint4*>(p.k_out + (base + r) * p.row_bytes + c) = a[e];
          *reinterpret_cast<uint4*>(p.v_out + (base + r) * p.row_bytes + c) = b[e];
        }
      }
    }
  }
}

// CLUSTER: a cluster a unit; else one CTA.
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint8_t sel_smem[];
  SelShared& sh = *reinterpret_cast<SelShared*>(sel_smem);
  uint32_t* run = reinterpret_cast<uint32_t*>(sel_smem + sizeof(SelShared));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int size = CLUSTER ? gridDim.x : 1, rank = CLUSTER ? blockIdx.x : 0, h = blockIdx.y;  // a cluster is one unit
  const EvictSeq sq = p.seq[blockIdx.z];
  int32_t* out = p.index + sq.out_row + (int64_t)h * sq.keep;
  sh.hist[0][t] = 0;  // 1024 counters
  if (t < 256) sh.sums[t] = 0;
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
      for (int i0 = t; i0 < n; i0 += 8 * kSelThreads) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = i0 + e * kSelThreads < n ? __ldcs(w + i0 + e * kSelThreads) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = i0 + e * kSelThreads;
          if (i < n) {
            const uint32_t o = order_bits(x[e]);
            if (cached) run[i] = o;
            atomicAdd(&sh.hist[0][o >> 24], 1u);
          }
        }
      }
      uint32_t prefix = 0, need = left;
#pragma unroll 1
      for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        uint32_t* hist = sh.hist[pass];
        if (pass > 0) {
          auto count = [&](uint32_t x) {
            if (x >> (shift + 8) == prefix) atomicAdd(&hist[(x >> shift) & 255u], 1u);
          };
          const int fours = cached ? n / 4 : 0;
#pragma unroll 2
          for (int i = t; i < fours; i += kSelThreads) {
            const uint4 x = reinterpret_cast<const uint4*>(run)[i];
            count(x.x);
            count(x.y);
            count(x.z);
            count(x.w);
          }
          for (int i = 4 * fours + t; i < n; i += kSelThreads) count(word(i));
        }
        unit_barrier<CLUSTER>();
        const uint32_t* sums = hist;
        if (CLUSTER) {
          // 64 threads a rank, four counters each
          if (t < 64 * size) {
            const uint4 c = peer_words(hist + 4 * (t & 63), t >> 6);
            if (c.x) atomicAdd(&sh.sums[4 * (t & 63)], c.x);
            if (c.y) atomicAdd(&sh.sums[4 * (t & 63) + 1], c.y);
            if (c.z) atomicAdd(&sh.sums[4 * (t & 63) + 2], c.z);
            if (c.w) atomicAdd(&sh.sums[4 * (t & 63) + 3], c.w);
          }
          __syncthreads();
          sums = sh.sums;
        }
        if (warp == 0) {
          // lane l holds digits 255 - 8 l .. 248 - 8 l; find where the count from the top passes the rank
          uint32_t c[8], mine = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) mine += c[e] = sums[255 - 8 * lane - e];
          uint32_t incl = mine;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
          }
          uint32_t before = incl - mine;
          if (before < need && need <= incl) {
            int digit = 255 - 8 * lane;
#pragma unroll
            for (int e = 0; e < 7; ++e) {
              if (digit == 255 - 8 * lane - e && before + c[e] < need) {
                before += c[e];
                --digit;
              }
            }
            sh.digit = (uint32_t)digit;
            sh.rank = need - before;
          }
        }
        __syncthreads();
        prefix = prefix << 8 | sh.digit;
        need = sh.rank;
        if (t < 256) sh.sums[t] = 0;  // warp 0 is done with them, and the next pass adds behind a barrier
      }
      // Words above the left-th largest stay, and the first ``need`` equal to
      // it.  A thread counts a stretch of the run (of odd length: no two lanes on
      // one bank), then writes its kept tokens from where those before it end.
      const int stretch = (n + kSelThreads - 1) / kSelThreads | 1, s0 = min(n, t * stretch), s1 = min(n, s0 + stretch);
      // (of at most 64 words it remembers which, and need not look at the others again)
      uint32_t above = 0, equal = 0;
      uint64_t ups = 0, ties = 0;
      const bool remember = stretch <= 64;
      if (remember) {
#pragma unroll 4
        for (int i = s0; i < s1; ++i) {
          const uint32_t x = word(i);
          ups |= (uint64_t)(x > prefix) << (i - s0);
          ties |= (uint64_t)(x == prefix) << (i - s0);
        }
        above = (uint32_t)__popcll(ups);
        equal = (uint32_t)__popcll(ties);
      } else {
        for (int i = s0; i < s1; ++i) {
          const uint32_t x = word(i);
          above += x > prefix;
          equal += x == prefix;
        }
      }
      uint32_t n_above = above, n_equal = equal;  // running sums over the threads, this one's included
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t ya = __shfl_up_sync(0xffffffffu, n_above, d), ye = __shfl_up_sync(0xffffffffu, n_equal, d);
        if (lane >= d) {
          n_above += ya;
          n_equal += ye;
        }
      }
      if (lane == 31) {
        sh.above[warp] = n_above;
        sh.equal[warp] = n_equal;
      }
      __syncthreads();
      uint32_t wa = sh.above[lane], we = sh.equal[lane];
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
      wa = __shfl_sync(0xffffffffu, wa, max(warp - 1, 0));
      we = __shfl_sync(0xffffffffu, we, max(warp - 1, 0));
      n_above += (warp > 0 ? wa : 0u) - above;
      n_equal += (warp > 0 ? we : 0u) - equal;
      if (CLUSTER) {
        unit_barrier<CLUSTER>();
        uint32_t ra = lane < rank ? peer_word(&sh.totals[0], lane) : 0u, re = lane < rank ? peer_word(&sh.totals[1], lane) : 0u;
        n_above += __reduce_add_sync(0xffffffffu, ra);
        n_equal += __reduce_add_sync(0xffffffffu, re);
      }
      auto give = [&](int i, bool up, bool tie) {
        if (up || (tie && n_equal < need)) out[lo + n_above + min(n_equal, need)] = r0 + i;
        n_above += up;
        n_equal += tie;
      };
      if (remember) {
        for (uint64_t left_of = ups | ties; left_of; left_of &= left_of - 1) {
          const int e = __ffsll((long long)left_of) - 1;
          give(s0 + e, ups >> e & 1u, ties >> e & 1u);
        }
      } else if (above + equal > 0) {
        for (int i = s0; i < s1; ++i) {
          const uint32_t x = word(i);
          give(i, x > prefix, x == prefix);
        }
      }
    }
  }
  unit_barrier<CLUSTER>();  // the indices are written, and no rank reads another's counts any more
  gather_rows(p, sq, h, (int)((int64_t)sq.keep * rank / size), (int)((int64_t)sq.keep * (rank + 1) / size), t);
}

}  // namespace

// Clusters of ``size`` choosing CTAs that run at once with one CTA an SM; asked
// of the driver once a device and size.
static int active_clusters(int size) {
  static std::atomic<int> known[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][size].load();
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kSelSmemMax;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, evict_kernel<true>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[dev][size].store(n);
  return n;
}

cudaError_t launch_evict(const EvictParams& p, int32_t max_len, int32_t max_keep, cudaStream_t s) {
  // the largest cluster that lets every unit run at once and still leaves each
  // CTA 8192 tokens to choose from or 64 KB of rows to copy; more units than that
  // fill the GPU with one CTA each
  int size = 1;
  const int64_t units = (int64_t)p.Hkv * p.n_seqs, bytes = 2 * (int64_t)max_keep * p.row_bytes;
  if (max_len >= 2 * 8192 || bytes >= 2 * 65536) {
    cudaError_t e = cudaFuncSetAttribute(evict_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmemMax);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    for (int c : {2, 4, 8, 12, 16})
      if ((max_len >= c * 8192 || bytes >= c * 65536) && units <= active_clusters(c)) size = c;
  }
  const int share = (max_len + size - 1) / size;
  const size_t smem = sizeof(SelShared) + (size_t)std::min(share, kCached) * sizeof(uint32_t);
  const auto kernel = size > 1 ? evict_kernel<true> : evict_kernel<false>;
  cudaError_t e = cudaSuccess;
  if (size == 1) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmemMax);
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
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace kvq
