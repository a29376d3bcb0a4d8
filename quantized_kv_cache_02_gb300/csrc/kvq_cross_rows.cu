// Cross attention of few queries (kvq_cross_attention): one new token a sequence, a
// short turn.  bf16, head_dim 64 or 128.
//
// A tile is up to 16 rows (floor(16 / g) tokens times the g query heads of a KV head),
// the height of an mma.sync operand, so shared heads cost nothing extra.  Its
// states are split over the warps of a cluster of CTAs: each warp streams runs of 16
// states through shared memory of its own (TMA, a few runs ahead) and keeps a running
// maximum, sum and 16 x d output of what it has seen:
//
//   S = Q K^T   16 x 16, d / 16 steps        m, l: per row, over the run
//   O += P V    16 x d, one step             P = 2^(S c - m), rounded to bf16
//
// The partials meet in shared memory (m_w, l_w, O_w of warp w):
//   m = max m_w,  l = sum 2^(m_w - m) l_w,  out = sum 2^(m_w - m) O_w / l,
// each CTA of the cluster joining its share of the elements in the same order of
// warps, so no workspace, no atomics and the same bits each time
// ("KV Cache 与自回归视频生成" section 05, FlashDecoding).
//
// An MMA takes operands of one type, so weights meet bf16 Values as bf16: off by at most
// 2^-8 of each, the output by 2.3e-3 (relative norm) where fp32 weights leave its own rounding's 1.7e-3.
// (A second product on what the rounding leaves would hide under the copies, but
// turn an infinite Value into NaN.)
//
// Bound: HBM, the states read once.  mma.sync and not tcgen05: 16 rows would leave
// seven eighths of a 128-row accumulator empty, and the copies take longer than these.

#include "kvq_cluster.cuh"
#include "kvq_prompt.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kRun = 16, kWarps = 4, kRowsThreads = 32 * kWarps;
constexpr float kSlack = 8.f;  // the maximum moves only past 2^8

template <int D>
struct RowsLayout {
  static constexpr uint32_t kChunk = kRun * 128;              // 16 states of 64 channels
  static constexpr uint32_t kHalf = kChunk * (D / 64);        // a run's Keys, or Values
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kWarpBytes = kStages * kStage;    // 24 KB: then the warp's 16 x D partial
  static constexpr int kOut = D + 4;                          // floats of a partial's row
  static constexpr uint32_t kBars = kWarps * kWarpBytes;
  static constexpr uint32_t kMl = kBars + kWarps * kStages * 8;  // [warp][16] float2
  static constexpr size_t kSmem = kMl + kWarps * 16 * 8 + 1024;
  static_assert(16 * kOut * 4 <= kWarpBytes, "a partial takes the place of the runs");
};

struct RowsMaps {
  CUtensorMap k, v;
};

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int D>
__global__ void __launch_bounds__(kRowsThreads, 2)
    cross_rows_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ RowsMaps maps) {
  using L = RowsLayout<D>;
  extern __shared__ uint8_t rows_raw[];
  uint8_t* smem = rows_raw + ((1024u - (smem_u32(rows_raw) & 1023u)) & 1023u);  // (the same in every CTA)
  const uint32_t sbase = smem_u32(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int rank = blockIdx.x % p.split;
  const Tile tile = tile_at(p.tiles, blockIdx.x / p.split);
  const CrossSeq sq = tile.seq;
  const int tok0 = tile.level * p.tiles.step, n_rows = min(p.tiles.step, sq.q_len - tok0) * p.g;
  const int n_runs = (sq.kv_len + kRun - 1) / kRun, stride = p.split * kWarps;
  const uint32_t ring = sbase + warp * L::kWarpBytes, bars = sbase + L::kBars + warp * L::kStages * 8;

  auto load = [&](int run, int stage) {  // by one lane
    const uint32_t dst = ring + stage * L::kStage, bar = bars + 8 * stage;
    bar_expect(bar, L::kStage);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      tma_load3(dst + c * L::kChunk, &maps.k, 64 * c, sq.kv_start + run * kRun, tile.head, bar);
      tma_load3(dst + L::kHalf + c * L::kChunk, &maps.v, 64 * c, sq.kv_start + run * kRun, tile.head, bar);
    }
  };
  int next = rank * kWarps + warp, issued = 0;  // the run to load next
  if (lane == 0) {
    for (int s = 0; s < L::kStages; ++s) bar_init(bars + 8 * s, 1);
    bar_init_fence();
  }
  __syncwarp();
  pdl_wait();
  pdl_release();
  for (; issued < L::kStages && next < n_runs; ++issued, next += stride)
    if (lane == 0) load(next, issued);

  // Q as the A operand: rows gid and gid + 8, two channels a register
  uint32_t q[D / 16][4];
  {
    const __nv_bfloat16* rows[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = gid + 8 * i, t = r / p.g;
      rows[i] = r < n_rows ? static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(sq.q_start + tok0 + t) * p.q_ts +
                                 (int64_t)(tile.head * p.g + r - t * p.g) * p.q_hs
                           : nullptr;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat16* row = rows[e & 1];
        q[ks][e] = row ? *reinterpret_cast<const uint32_t*>(row + 16 * ks + 2 * tig + 8 * (e >> 1)) : 0u;
      }
  }

  float o[D / 8][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int run = rank * kWarps + warp; run < n_runs; run += stride) {
    if (!(ok = warp_wait(bars + 8 * stage, phase, nullptr))) break;
    const uint32_t kt = ring + stage * L::kStage, vt = kt + L::kHalf;
    const int limit = sq.kv_len - run * kRun;
    if (limit < kRun) {
      // Values behind the last state: a weight of 0 does not silence their infinities and NaN
      for (int x = 8 * limit + lane; x < 8 * kRun; x += 32)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          reinterpret_cast<uint4*>(smem + (vt - sbase) + c * L::kChunk)[x] = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
    }
    float s[2][4] = {};
    // states 0-7 and 8-15, channels 16 ks .. + 15 (a matrix of 8 states by 8 channels each)
    const int kr = (lane & 7) + 8 * (lane >> 4), kc = lane >> 3 & 1;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b[4];
      ldm4(b, kt + (ks / 4) * L::kChunk + kr * 128 + (((2 * (ks % 4) + kc) ^ (kr & 7)) << 4));
      mma16(s[0], q[ks], b[0], b[1]);
      mma16(s[1], q[ks], b[2], b[3]);
    }
    uint32_t pa[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // row gid + 8 i: states 2 tig, 2 tig + 1 and those + 8
      float x[4] = {s[0][2 * i], s[0][2 * i + 1], s[1][2 * i], s[1][2 * i + 1]};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= p.scale2;
      if (limit < kRun) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (2 * tig + (e & 1) + 8 * (e >> 1) >= limit) x[e] = -INFINITY;
      }
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool up = top > (m[i] == -INFINITY ? m[i] : m[i] + kSlack);
      if (__any_sync(0xffffffffu, up)) {
        const float a = up ? ex2(m[i] - top) : 1.f;  // (from minus infinity: 0)
        if (up) m[i] = top;
        l[i] *= a;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          o[c][2 * i] *= a;
          o[c][2 * i + 1] *= a;
        }
      }
      const float base = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = ex2(x[e] - base);
      l[i] += (x[0] + x[1]) + (x[2] + x[3]);
      pa[i] = pack_bf16(x[0], x[1]);
      pa[2 + i] = pack_bf16(x[2], x[3]);
    }
    // (transposed) states 0-7 and 8-15 of channels 16 c .. + 7, then of the next 8
    const int vr = lane & 15, vc = lane >> 4;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t b[4];
      ldm4t(b, vt + (c / 4) * L::kChunk + vr * 128 + (((2 * (c % 4) + vc) ^ (vr & 7)) << 4));
      mma16(o[2 * c], pa, b[0], b[1]);
      mma16(o[2 * c + 1], pa, b[2], b[3]);
    }
    __syncwarp();  // the run has been read
    if (next < n_runs) {
      if (lane == 0) load(next, stage);
      next += stride;
      ++issued;
    }
    if (++stage == L::kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (!ok) {
    if (p.status && lane == 0) atomicOr(p.status, kStatusPromptTimeout);
    // nothing in flight when the memory is used again, or the CTA ends
    for (int x = max(0, issued - L::kStages); x < issued; ++x)
      bar_drain(bars + 8 * (x % L::kStages), (uint32_t)(x / L::kStages) & 1u);
  }

  // the warps' partials meet
  __syncwarp();
  float* part = reinterpret_cast<float*>(smem + warp * L::kWarpBytes);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMl) + warp * 16;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float sum = l[i];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (tig == 0) ml[gid + 8 * i] = make_float2(m[i], sum);
    if (gid + 8 * i < n_rows) {
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<float2*>(part + (gid + 8 * i) * L::kOut + 8 * c + 2 * tig) =
            make_float2(o[c][2 * i], o[c][2 * i + 1]);
    }
  }
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  for (int x = rank * kRowsThreads + threadIdx.x; x < n_rows * (D / 4); x += p.split * kRowsThreads) {
    const int r = x / (D / 4), col = 4 * (x % (D / 4));
    const uint32_t at_ml = sbase + L::kMl + r * 8, at_o = sbase + (r * L::kOut + col) * 4;
    float top = -INFINITY;
    for (int k = 0; k < p.split; ++k)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, peer_load2(peer_addr(at_ml, k) + w * 16 * 8).x);
    const float base = top == -INFINITY ? 0.f : top;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float lr = 0.f;
    for (int k = 0; k < p.split; ++k) {
      const uint32_t pm = peer_addr(at_ml, k), po = peer_addr(at_o, k);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 part_ml = peer_load2(pm + w * 16 * 8);
        const float4 v = peer_load4(po + w * L::kWarpBytes);
        const float a = ex2(part_ml.x - base);
        lr = fmaf(part_ml.y, a, lr);
        sum.x = fmaf(v.x, a, sum.x);
        sum.y = fmaf(v.y, a, sum.y);
        sum.z = fmaf(v.z, a, sum.z);
        sum.w = fmaf(v.w, a, sum.w);
      }
    }
    const float inv = sq.kv_len == 0 ? 0.f : 1.f / lr;  // over no states: zeros, and lse minus infinity
    const int t = r / p.g, head = tile.head * p.g + r - t * p.g;
    const int64_t token = sq.q_start + tok0 + t;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + token * p.o_ts + (int64_t)head * p.o_hs + col) =
        make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
    if (p.lse && col == 0) p.lse[(int64_t)head * p.n_tokens + token] = (top + log2f(lr)) * 0.69314718055994530942f;
  }
  if (p.split > 1) cluster_sync();  // no CTA ends while another reads its partials
}

template <int D>
cudaError_t launch_rows(const CrossParams& p, const RowsMaps& maps, int64_t tiles, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(cross_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)RowsLayout<D>::kSmem);
  if (e != cudaSuccess) return e;
  if (p.split > 8) {
    const cudaError_t wide =
        cudaFuncSetAttribute(cross_rows_kernel<D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (wide != cudaSuccess) return wide;
    if (active_clusters<cross_rows_kernel<D>>(p.split, kRowsThreads, RowsLayout<D>::kSmem) < tiles) {
      CrossParams q = p;
      q.split = 8;
      return launch_rows<D>(q, maps, tiles, s);
    }
  }
  return launch_cluster(cross_rows_kernel<D>, tiles, p.split, kRowsThreads, RowsLayout<D>::kSmem, s, p, maps);
}

}  // namespace

int cross_rows_tokens(int g) { return 16 / g; }

// One tile: with two, their CTAs read the states twice (8 prompts of 32 rows over 4096
// states 37 us, the tensor-memory kernel 43; 128 channels; at 64 channels 45 and 35).
int cross_few_tokens(int g) { return 16 / g; }

// CTAs of a cluster that share a tile: until the SMs are full, each with some runs to
// stream.  Clusters of 16 where all of them run at once (8 tiles of 16384 states 24.3 ->
// 19.2 us); 16 tiles would be 20.8 -> 26 us.
int cross_rows_split(int64_t tiles, int32_t max_kv, int n_sm) {
  int split = 1;
  while (split < 8 && tiles * split < 2 * (int64_t)n_sm && max_kv >= 2 * split * 8 * kRun) split *= 2;
  return split == 8 && tiles * 16 <= n_sm && max_kv >= 16 * 8 * kRun ? 16 : split;
}

cudaError_t launch_cross_rows(const CrossParams& p, int64_t tiles, cudaStream_t s) {
  RowsMaps maps;
  // dims (channel, token, head)
  if (!tma_map3(&maps.k, p.k, p.D, p.n_kv_tokens, p.Hkv, p.k_ts, p.k_hs, kRun, 1) ||
      !tma_map3(&maps.v, p.v, p.D, p.n_kv_tokens, p.Hkv, p.v_ts, p.v_hs, kRun, 1))
    return cudaErrorInvalidValue;
  return p.D == 128 ? launch_rows<128>(p, maps, tiles, s) : launch_rows<64>(p, maps, tiles, s);
}

}  // namespace kvq
