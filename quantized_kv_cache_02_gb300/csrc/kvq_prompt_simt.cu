// CUDA-core kernels of the prompt operators: any supported shape and dtype
// (the tensor-core kernels take bf16 with head_dim 64 and 128).
//
// Both work on tiles of 64 rows x 64 keys in fp32.  A row is a (token, query
// head) pair of one KV head, token major, so the heads that share a KV head
// share its tiles: 64 / g tokens a tile.  256 threads as 16 x 16; thread
// (ty, tx) holds rows 4 ty .. 4 ty + 3 and keys tx, tx + 16, tx + 32, tx + 48.
//
//   attention:  o_i = sum_{j <= i} p_ij v_j / l_i,  p_ij = 2^(s_ij - m_i),
//               s_ij = q_i . k_j log2(e) / sqrt(d), one pass over the keys with
//               the running maximum m and sum l ("KV Cache 与自回归视频生成",
//               attn_full in section 04's appendix, softmax(QK^T / sqrt(d) + M) V)
//   weights:    w_j = sum over the last queries i >= j of 2^(s_ij - lse_i)
//
// Bound: shared loads and the FMA pipe together.  Per four channels a warp takes
// 24 wavefronts (a 16-byte load of 32 rows is 4, of two broadcast rows 2) and, as
// packed pairs (two channels of a score, two columns of the output; half the
// issue slots of single products), 32 cycles of FMA for each of the SM's four
// schedulers.  Few tiles are split along the keys over a cluster (``split`` CTAs
// take the key steps in turn) and joined through distributed shared memory in rank
// order; a causal prompt's last tiles are otherwise what everything waits for.
// 1999 fp32 tokens, 8/2 heads of 128: 252 us, 286 us without either.  Tiles of 128
// x 128 with 8 x 8 a thread halve the loads but leave two warps a scheduler
// to hide them (285 us); a second buffer for V changes nothing.

#include <cuda_bf16.h>

#include "kvq_prompt.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kPStride = kPromptKeys + 4;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// Rows [0, 64) of K or V (keys ``key0`` on of one head) into shared memory as
// fp32 rows of ``stride`` floats; keys at or past ``end`` and channels past D are 0.
// CLEAN: infinities and NaN too; returns whether there were any.
template <bool CLEAN, typename T>
__device__ __forceinline__ bool load_keys(float* dst, int stride, int cols, const T* base, int64_t ts, int key0,
                                          int end, int D) {
  bool dirty = false;
  const int per = cols / 4;
  for (int i = threadIdx.x; i < kPromptKeys * per; i += kThreads) {
    const int r = i / per, c = (i - r * per) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (key0 + r < end && c < D) x = load4(base + (int64_t)(key0 + r) * ts + c);
    if (CLEAN && !(finite(x.x) && finite(x.y) && finite(x.z) && finite(x.w))) {
      dirty = true;
      x = make_float4(finite(x.x) ? x.x : 0.f, finite(x.y) ? x.y : 0.f, finite(x.z) ? x.z : 0.f, finite(x.w) ? x.w : 0.f);
    }
    *reinterpret_cast<float4*>(dst + r * stride + c) = x;
  }
  return dirty;
}

// Row r of a query tile is token tok0 + r / g, head h * g + r % g; rows past
// the tile's tokens or the sequence are 0.
template <typename T>
__device__ __forceinline__ void load_queries(float* dst, int stride, const PromptParams& p, const T* q, int tok0,
                                             int tile_tok, int len, int h) {
  const int per = p.D / 4;
  for (int i = threadIdx.x; i < kPromptRows * per; i += kThreads) {
    const int r = i / per, c = (i - r * per) * 4, t = r / p.g;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < tile_tok && tok0 + t < len)
      x = load4(q + (int64_t)(tok0 + t) * p.q_ts + (int64_t)(h * p.g + r - t * p.g) * p.q_hs + c);
    *reinterpret_cast<float4*>(dst + r * stride + c) = x;
  }
}

__device__ __forceinline__ void scores(float (&s)[4][4], const float* qs, const float* ks, int stride, int D, int ty,
                                       int tx) {
  float2 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = load4(qs + (4 * ty + i) * stride + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = load4(ks + (tx + 16 * j) * stride + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), acc[i][j]);
        acc[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = acc[i][j].x + acc[i][j].y;
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 peer_load4(const float* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_addr(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_load2(const float2* p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}

// NC: 64-channel column groups of the output (D <= 64 NC).
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads, NC == 4 ? 1 : 2) prompt_simt_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ __align__(16) float simt_smem[];
  constexpr int kStride = 64 * NC + 4;
  float* qs = simt_smem;                        // [64][kStride]
  float* ks = qs + kPromptRows * kStride;       // K, then V
  float* ps = ks + kPromptKeys * kStride;       // [64][kPStride]
  int si, h, level;
  const int rank = blockIdx.x % p.split;  // clusters are ``split`` CTAs in a row
  prompt_tile(p.tiles, blockIdx.x / p.split, &si, &h, &level);
  const PromptSeq sq = p.tiles.seq[si];
  const int tile_tok = p.tiles.step, tok0 = level * tile_tok;
  const T* q = static_cast<const T*>(p.q) + (int64_t)sq.start * p.q_ts;
  const T* k = static_cast<const T*>(p.k) + (int64_t)sq.start * p.k_ts + (int64_t)h * p.k_hs;
  const T* v = static_cast<const T*>(p.v) + (int64_t)sq.start * p.v_ts + (int64_t)h * p.v_hs;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  pdl_wait();
  pdl_release();
  load_queries(qs, kStride, p, q, tok0, tile_tok, sq.len, h);
  const int end = min(sq.len, tok0 + tile_tok);  // keys some row sees
  float2 o[NC][4][2];
  float m[4], l[4];
  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    pos[i] = tok0 + (4 * ty + i) / p.g;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) o[c][i][0] = o[c][i][1] = make_float2(0.f, 0.f);
  }
  int dirty = 0;
  for (int k0 = rank * kPromptKeys; k0 < end; k0 += p.split * kPromptKeys) {
    __syncthreads();  // the previous step's V has been read
    load_keys<false>(ks, kStride, p.D, k, p.k_ts, k0, end, p.D);
    __syncthreads();
    float s[4][4];
    scores(s, qs, ks, kStride, p.D, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 16 * j;
        s[i][j] = key <= pos[i] && key < end ? s[i][j] * p.scale2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      // (a row may see none of a later rank's keys)
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn, a = exp2f(m[i] - base);
      m[i] = mn;
      float sum = 0.f;
      float* row = ps + (4 * ty + i) * kPStride;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - base);
        sum += e;
        row[tx + 16 * j] = e;
      }
      l[i] = fmaf(l[i], a, sum);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        o[c][i][0] = mul2(o[c][i][0], make_float2(a, a));
        o[c][i][1] = mul2(o[c][i][1], make_float2(a, a));
      }
    }
    __syncthreads();  // K has been read; P is complete
    // A weight of 0 does not silence an infinite or NaN Value: in blocks with keys
    // that some row does not see they are taken out, and given back at the end.
    if (k0 + kPromptKeys - 1 > tok0) dirty |= __syncthreads_or(load_keys<true>(ks, kStride, 64 * NC, v, p.v_ts, k0, end, p.D));
    else {
      load_keys<false>(ks, kStride, 64 * NC, v, p.v_ts, k0, end, p.D);
      __syncthreads();
    }
#pragma unroll 2
    for (int n = 0; n < kPromptKeys; n += 4) {
      float4 pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = load4(ps + (4 * ty + i) * kPStride + n);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int nn = 0; nn < 4; ++nn) {
          const float4 vv = load4(ks + (n + nn) * kStride + 64 * c + 4 * tx);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pp = nn == 0 ? pr[i].x : nn == 1 ? pr[i].y : nn == 2 ? pr[i].z : pr[i].w;
            o[c][i][0] = fma2(make_float2(pp, pp), make_float2(vv.x, vv.y), o[c][i][0]);
            o[c][i][1] = fma2(make_float2(pp, pp), make_float2(vv.z, vv.w), o[c][i][1]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
  }
  if (dirty) {
    // a weight times an infinity or NaN is one
    for (int key = tok0 / kPromptKeys * kPromptKeys; key < end; ++key) {
      if (key / kPromptKeys % p.split != rank) continue;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (64 * c + 4 * tx >= p.D) continue;
        const float4 x = load4(v + (int64_t)key * p.v_ts + 64 * c + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (key > pos[i]) continue;
          if (!finite(x.x)) o[c][i][0].x += x.x;
          if (!finite(x.y)) o[c][i][0].y += x.y;
          if (!finite(x.z)) o[c][i][1].x += x.z;
          if (!finite(x.w)) o[c][i][1].y += x.w;
        }
      }
    }
  }
  auto finish = [&](int r, int col, float4 sum, float mr, float lr, bool first) {  // row r, columns col .. col + 3
    const int t = r / p.g, head = h * p.g + r - t * p.g;
    if (t >= tile_tok || tok0 + t >= sq.len) return;
    const float inv = 1.f / lr;
    T* dst = static_cast<T*>(p.out) + (int64_t)(sq.start + tok0 + t) * p.o_ts + (int64_t)head * p.o_hs;
    if (col < p.D) store4(dst + col, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
    if (p.lse && first)
      p.lse[(int64_t)head * p.n_tokens + sq.start + tok0 + t] = (mr + log2f(lr)) * 0.69314718055994530942f;
  };
  if (p.split == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        finish(4 * ty + i, 64 * c + 4 * tx, make_float4(o[c][i][0].x, o[c][i][0].y, o[c][i][1].x, o[c][i][1].y), m[i],
               l[i], c == 0 && tx == 0);
    return;
  }
  // the ranks' partials meet: each puts its own in its shared memory, and joins its share of the rows
  __syncthreads();  // V has been read
  float2* ml = reinterpret_cast<float2*>(ps);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (tx == 0) ml[4 * ty + i] = make_float2(m[i], l[i]);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      *reinterpret_cast<float4*>(ks + (4 * ty + i) * kStride + 64 * c + 4 * tx) =
          make_float4(o[c][i][0].x, o[c][i][0].y, o[c][i][1].x, o[c][i][1].y);
  }
  cluster_sync();
  const int rows = kPromptRows / p.split;
  for (int x = threadIdx.x; x < rows * 16 * NC; x += kThreads) {
    const int r = rank * rows + x / (16 * NC), col = 4 * (x % (16 * NC));
    float top = -INFINITY;
    for (int k = 0; k < p.split; ++k) top = fmaxf(top, peer_load2(ml + r, k).x);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float lr = 0.f;
    for (int k = 0; k < p.split; ++k) {
      const float2 part = peer_load2(ml + r, k);
      const float4 v = peer_load4(ks + r * kStride + col, k);
      const float a = exp2f(part.x - top);  // rank 0 holds key 0: top is finite
      lr = fmaf(part.y, a, lr);
      sum.x = fmaf(v.x, a, sum.x);
      sum.y = fmaf(v.y, a, sum.y);
      sum.z = fmaf(v.z, a, sum.z);
      sum.w = fmaf(v.w, a, sum.w);
    }
    finish(r, col, sum, top, lr, col == 0);
  }
  cluster_sync();  // no rank ends while another reads its partials
}

// One CTA per 64 keys of a KV head: the column sums stay in registers while
// the counted queries pass, so no partial leaves the CTA and the order of
// every sum is fixed.
template <typename T>
__global__ void __launch_bounds__(kThreads) weights_simt_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ __align__(16) float simt_smem[];
  const int stride = p.D + 4;
  float* qs = simt_smem;
  float* ks = qs + kPromptRows * stride;
  float* red = ks + kPromptKeys * stride;  // [16][64]
  int si, h, level;
  prompt_tile(p.tiles, blockIdx.x, &si, &h, &level);
  const PromptSeq sq = p.tiles.seq[si];
  const int k0 = (prompt_blocks(sq.len, kPromptKeys) - 1 - level) * kPromptKeys;
  const int tile_tok = kPromptRows / p.g;
  const T* q = static_cast<const T*>(p.q) + (int64_t)sq.start * p.q_ts;
  const T* k = static_cast<const T*>(p.k) + (int64_t)sq.start * p.k_ts + (int64_t)h * p.k_hs;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  pdl_wait();
  pdl_release();
  load_keys<false>(ks, stride, p.D, k, p.k_ts, k0, sq.len, p.D);
  RunningSum total[4] = {};
  const int64_t back = sq.len - p.last;
  const int t_first = (int)(back > k0 ? back : k0);
  for (int t0 = t_first; t0 < sq.len; t0 += tile_tok) {
    __syncthreads();
    load_queries(qs, stride, p, q, t0, tile_tok, sq.len, h);
    __syncthreads();
    float s[4][4];
    scores(s, qs, ks, stride, p.D, ty, tx);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i, t = r / p.g, pos = t0 + t;
      if (t < tile_tok && pos < sq.len) {
        // lse in the scores' units as a float and the factor that makes up for its
        // rounding (from 2^24 on a weight is 0 or infinite with or without it, and an infinity has none)
        const float e = p.lse[(int64_t)(h * p.g + r - t * p.g) * p.n_tokens + sq.start + pos];
        const float lse2 = __fmul_rn(e, p.lse_hi);
        const float f = fabsf(lse2) < 0x1p24f ? exp2f(-(fmaf(e, p.lse_hi, -lse2) + e * p.lse_lo)) : 1.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k0 + tx + 16 * j <= pos) sum[j] = fmaf(exp2f(fmaf(s[i][j], p.scale2, -lse2)), f, sum[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) total[j].add(sum[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) red[ty * 64 + tx + 16 * j] = total[j].sum;
  __syncthreads();
  if (threadIdx.x < kPromptKeys && k0 + threadIdx.x < sq.len) {
    float w = 0.f;
#pragma unroll
    for (int y = 0; y < 16; ++y) w += red[y * 64 + threadIdx.x];
    p.weights[(int64_t)h * p.n_tokens + sq.start + k0 + threadIdx.x] = w;
  }
}

// ``most``: the shared memory of the kernel's largest head_dim.  The limit is a
// state of the kernel that all host threads share: set to one call's size, it
// would refuse a larger call that another thread is about to launch.
template <typename K>
cudaError_t launch_sized(K kernel, size_t most, size_t smem, int64_t tiles, const PromptParams& p, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, tiles, p.split, kThreads, smem, s, p);
}

template <typename T>
cudaError_t launch_attention_t(const PromptParams& p, int64_t tiles, cudaStream_t s) {
  auto smem = [](int nc) {
    return ((size_t)(kPromptRows + kPromptKeys) * (64 * nc + 4) + kPromptRows * kPStride) * sizeof(float);
  };
  if (p.D <= 64) return launch_sized(prompt_simt_kernel<T, 1>, smem(1), smem(1), tiles, p, s);
  if (p.D <= 128) return launch_sized(prompt_simt_kernel<T, 2>, smem(2), smem(2), tiles, p, s);
  return launch_sized(prompt_simt_kernel<T, 4>, smem(4), smem(4), tiles, p, s);
}

}  // namespace

int prompt_simt_split(int64_t tiles, int32_t max_len, int n_sm) {
  int split = 1;
  while (split < 4 && tiles * split < 3 * (int64_t)n_sm && max_len >= 8 * split * kPromptKeys) split *= 2;
  return split;
}

cudaError_t launch_prompt_simt(const PromptParams& p, int dtype, int64_t tiles, cudaStream_t s) {
  return dtype == 0 ? launch_attention_t<__nv_bfloat16>(p, tiles, s) : launch_attention_t<float>(p, tiles, s);
}

cudaError_t launch_weights_simt(const PromptParams& p, int dtype, int64_t tiles, cudaStream_t s) {
  auto smem = [](int d) { return ((size_t)(kPromptRows + kPromptKeys) * (d + 4) + 16 * 64) * sizeof(float); };
  return dtype == 0 ? launch_sized(weights_simt_kernel<__nv_bfloat16>, smem(kMaxDim), smem(p.D), tiles, p, s)
                    : launch_sized(weights_simt_kernel<float>, smem(kMaxDim), smem(p.D), tiles, p, s);
}

}  // namespace kvq
