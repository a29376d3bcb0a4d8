// Cross attention of few queries on CUDA cores (kvq_cross_attention): fp32, and the
// head_dims that the tensor-core kernels do not take.
//
// A tile is up to 8 rows, the g query heads of a KV head times floor(8 / g) tokens.
// Its states are split over a cluster of CTAs, which take steps of 32 states in
// turn, the next step's Keys and Values in flight (cp.async) under the current one:
//
//   scores   thread (state, quarter of the channels): its part of q . k of every row,
//            each Key read from shared memory once for all rows
//   softmax  a row a warp, a state a lane: running maximum m and sum l
//   output   thread (four channels, share of the states): o += p v of every row
//
// Then the shares meet, and the CTAs through distributed shared memory in rank order
// (m = max m_k, l = sum 2^(m_k - m) l_k, out = sum 2^(m_k - m) o_k / l), so no
// workspace, no atomics, and the same bits each time.
//
// Bound: HBM for one row, then shared memory and the FMA pipe: a state of 128 fp32
// channels is 1 KB to read and 5 + 2 R wavefronts for R rows.

#include <cuda_bf16.h>

#include "kvq_cluster.cuh"
#include "kvq_prompt.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kKeys = 32, kThreads = 128, kFewRows = 8;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}
// 16 bytes, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// Bytes of shared memory: two steps of Keys and Values (rows padded by 16 bytes), the
// queries, then partial scores, weights, factors and the rows' (m, l).
template <typename T>
__host__ __device__ constexpr size_t few_row_bytes(int d) {
  return (size_t)d * sizeof(T) + 16;
}
// (then the shares' sums take the steps' place)
template <typename T>
__host__ __device__ constexpr size_t few_step_bytes(int d) {
  const size_t steps = 4 * kKeys * few_row_bytes<T>(d), sums = sizeof(float) * 4 * kThreads * kFewRows;
  return steps > sums ? steps : sums;
}
template <typename T>
size_t few_smem(int d) {
  return few_step_bytes<T>(d) +
         sizeof(float) * ((size_t)kFewRows * d + 4 * kFewRows * kKeys + kFewRows * kKeys + 3 * kFewRows);
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads) cross_few_kernel(const __grid_constant__ CrossParams p) {
  extern __shared__ __align__(16) uint8_t few_raw[];
  const int D = p.D, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row_bytes = (int)few_row_bytes<T>(D), half = kKeys * row_bytes;  // of a step's Keys, or Values
  float* qs = reinterpret_cast<float*>(few_raw + few_step_bytes<T>(D));      // [R][D]
  float* parts = qs + kFewRows * D;                                          // [4][R][32] scores
  float* ps = parts + 4 * kFewRows * kKeys;                                  // [32][R]
  float* factor = ps + kFewRows * kKeys;                                     // [R]
  float2* ml = reinterpret_cast<float2*>(factor + kFewRows);                 // [R]
  const int rank = blockIdx.x % p.split;
  const Tile tile = tile_at(p.tiles, blockIdx.x / p.split);
  const CrossSeq sq = tile.seq;
  const int tok0 = tile.level * p.tiles.step, n_rows = min(p.tiles.step, sq.q_len - tok0) * p.g;
  const T* k = static_cast<const T*>(p.k) + (int64_t)sq.kv_start * p.k_ts + (int64_t)tile.head * p.k_hs;
  const T* v = static_cast<const T*>(p.v) + (int64_t)sq.kv_start * p.v_ts + (int64_t)tile.head * p.v_hs;
  pdl_wait();
  pdl_release();

  const int pieces = D * (int)sizeof(T) / 16;  // of a row
  auto load = [&](int k0, int buf) {
    const uint32_t dst = smem_u32(few_raw) + buf * 2 * half;
    for (int x = tid; x < kKeys * pieces; x += kThreads) {
      const int r = x / pieces, c = x - r * pieces;
      const bool real = k0 + r < sq.kv_len;
      const int64_t row = real ? k0 + r : 0;  // (an address that is there: nothing is read)
      copy16(dst + r * row_bytes + 16 * c, reinterpret_cast<const uint8_t*>(k + row * p.k_ts) + 16 * c, real);
      copy16(dst + half + r * row_bytes + 16 * c, reinterpret_cast<const uint8_t*>(v + row * p.v_ts) + 16 * c, real);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int first = rank * kKeys, stride = p.split * kKeys;
  if (first < sq.kv_len) load(first, 0);
  for (int x = tid; x < R * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = 4 * (x - r * (D / 4)), t = r / p.g;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n_rows)
      q = load4(static_cast<const T*>(p.q) + (int64_t)(sq.q_start + tok0 + t) * p.q_ts +
                (int64_t)(tile.head * p.g + r - t * p.g) * p.q_hs + c);
    *reinterpret_cast<float4*>(qs + r * D + c) = q;
  }

  // the output: groups of four channels times shares of the states
  const int groups = D / 4, shares = kThreads / groups, share = tid / groups, col = 4 * (tid - share * groups);
  const bool owns = share < shares;
  float2 o[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) o[r][0] = o[r][1] = make_float2(0.f, 0.f);
  constexpr int kMine = (R + 3) / 4;  // rows of a warp: warp, warp + 4
  float m[kMine], l[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  int buf = 0;
  for (int k0 = first; k0 < sq.kv_len; k0 += stride, buf ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the step is here, and the other buffer has been read
    if (k0 + stride < sq.kv_len) load(k0 + stride, buf ^ 1);
    const uint8_t* kt = few_raw + buf * 2 * half;
    const uint8_t* vt = kt + half;
    {
      const int quarter = D / 4;
      const T* row = reinterpret_cast<const T*>(kt + lane * row_bytes) + warp * quarter;
      const float* qr = qs + warp * quarter;
      float2 acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < quarter; c += 4) {
        const float4 x = load4(row + c);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 q = load4(qr + r * D + c);
          acc[r] = fma2(make_float2(q.x, q.y), make_float2(x.x, x.y), acc[r]);
          acc[r] = fma2(make_float2(q.z, q.w), make_float2(x.z, x.w), acc[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) parts[(warp * R + r) * kKeys + lane] = acc[r].x + acc[r].y;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = warp + 4 * i;
      if (r >= R) break;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) s += parts[(w * R + r) * kKeys + lane];
      s = k0 + lane < sq.kv_len ? s * p.scale2 : -INFINITY;
      float top = s;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      top = fmaxf(top, m[i]);
      const float base = top == -INFINITY ? 0.f : top, a = exp2f(m[i] - base), e = exp2f(s - base);
      float sum = e;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      m[i] = top;
      l[i] = fmaf(l[i], a, sum);
      ps[lane * R + r] = e;
      if (lane == 0) factor[r] = a;
    }
    __syncthreads();
    if (owns) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 a = make_float2(factor[r], factor[r]);
        o[r][0] = mul2(o[r][0], a);
        o[r][1] = mul2(o[r][1], a);
      }
      const int end = min(kKeys, sq.kv_len - k0);
#pragma unroll 4
      for (int n = share; n < end; n += shares) {
        const float4 x = load4(reinterpret_cast<const T*>(vt + n * row_bytes) + col);
        float w[R];
        if constexpr (R % 4 == 0) {
#pragma unroll
          for (int r = 0; r < R; r += 4) *reinterpret_cast<float4*>(w + r) = load4(ps + n * R + r);
        } else {
#pragma unroll
          for (int r = 0; r < R; ++r) w[r] = ps[n * R + r];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 e = make_float2(w[r], w[r]);
          o[r][0] = fma2(e, make_float2(x.x, x.y), o[r][0]);
          o[r][1] = fma2(e, make_float2(x.z, x.w), o[r][1]);
        }
      }
    }
  }

  // the shares meet: [share][R][D] in place of the steps, their sum in place of the queries
  __syncthreads();
  float* sums = reinterpret_cast<float*>(few_raw);
  if (owns) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      *reinterpret_cast<float4*>(sums + (share * R + r) * D + col) =
          make_float4(o[r][0].x, o[r][0].y, o[r][1].x, o[r][1].y);
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (warp + 4 * i < R) ml[warp + 4 * i] = make_float2(m[i], l[i]);
  }
  __syncthreads();
  for (int x = tid; x < R * D; x += kThreads) {
    float sum = 0.f;
    for (int n = 0; n < shares; ++n) sum += sums[n * R * D + x];
    qs[x] = sum;
  }
  // (a warp's lanes meet inside)
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  for (int x = rank * kThreads + tid; x < n_rows * groups; x += p.split * kThreads) {
    const int r = x / groups, c = 4 * (x - r * groups);
    const uint32_t at_ml = smem_u32(ml + r), at_o = smem_u32(qs + r * D + c);
    float top = -INFINITY;
    for (int n = 0; n < p.split; ++n) top = fmaxf(top, peer_load2(peer_addr(at_ml, n)).x);
    const float base = top == -INFINITY ? 0.f : top;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float lr = 0.f;
    for (int n = 0; n < p.split; ++n) {
      const float2 part = peer_load2(peer_addr(at_ml, n));
      const float4 y = peer_load4(peer_addr(at_o, n));
      const float a = exp2f(part.x - base);
      lr = fmaf(part.y, a, lr);
      sum.x = fmaf(y.x, a, sum.x);
      sum.y = fmaf(y.y, a, sum.y);
      sum.z = fmaf(y.z, a, sum.z);
      sum.w = fmaf(y.w, a, sum.w);
    }
    const float inv = sq.kv_len == 0 ? 0.f : 1.f / lr;  // over no states: zeros, and lse minus infinity
    const int t = r / p.g, head = tile.head * p.g + r - t * p.g;
    const int64_t token = sq.q_start + tok0 + t;
    store4(static_cast<T*>(p.out) + token * p.o_ts + (int64_t)head * p.o_hs + c,
           make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
    if (p.lse && c == 0) p.lse[(int64_t)head * p.n_tokens + token] = (top + log2f(lr)) * 0.69314718055994530942f;
  }
  if (p.split > 1) cluster_sync();  // no CTA ends while another reads its sums
}

template <typename T, int R>
cudaError_t launch_r(const CrossParams& p, int64_t tiles, cudaStream_t s) {
  // the most that any head_dim takes: the limit is a state that all host threads share
  const cudaError_t e = cudaFuncSetAttribute(cross_few_kernel<T, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)few_smem<T>(kMaxDim));
  if (e != cudaSuccess) return e;
  if (p.split > 8) {
    const cudaError_t wide =
        cudaFuncSetAttribute(cross_few_kernel<T, R>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (wide != cudaSuccess) return wide;
    if (active_clusters<cross_few_kernel<T, R>>(p.split, kThreads, few_smem<T>(p.D), p.D / 16) < tiles) {
      CrossParams q = p;
      q.split = 8;
      return launch_r<T, R>(q, tiles, s);
    }
  }
  return launch_cluster(cross_few_kernel<T, R>, tiles, p.split, kThreads, few_smem<T>(p.D), s, p);
}

template <typename T>
cudaError_t launch_t(const CrossParams& p, int rows, int64_t tiles, cudaStream_t s) {
  return rows <= 1 ? launch_r<T, 1>(p, tiles, s)
         : rows <= 2 ? launch_r<T, 2>(p, tiles, s)
         : rows <= 4 ? launch_r<T, 4>(p, tiles, s)
                     : launch_r<T, 8>(p, tiles, s);
}

}  // namespace

int cross_few_simt_step(int g) { return kFewRows / g; }

// Up to 64 rows, though every 8 read the states again: eight prompts of 64 fp32 rows over
// 1000 states 49 us, on the 64-row tiles 75.
int cross_few_simt_tokens(int g) { return 64 / g; }

// CTAs of a cluster that share a tile: until the SMs are full, each with some steps to stream
int cross_few_simt_split(int64_t tiles, int32_t max_kv, int n_sm) {
  int split = 1;
  while (split < 8 && tiles * split < 2 * (int64_t)n_sm && max_kv >= 2 * split * 2 * kKeys) split *= 2;
  return split == 8 && tiles * 16 <= n_sm && max_kv >= 16 * 2 * kKeys ? 16 : split;
}

cudaError_t launch_cross_few_simt(const CrossParams& p, int dtype, int rows, int64_t tiles, cudaStream_t s) {
  return dtype == 0 ? launch_t<__nv_bfloat16>(p, rows, tiles, s) : launch_t<float>(p, rows, tiles, s);
}

}  // namespace kvq
