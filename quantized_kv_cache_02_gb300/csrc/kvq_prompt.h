// Internal definitions of the prompt operators (kvq_prompt_attention,
// kvq_prompt_weights, kvq_evict) and of the cross attention (kvq_cross_attention): launch parameter blocks, the order in which
// a launch takes its tiles, and the launchers.
#pragma once

#include <cuda.h>

#include <atomic>

#include "kvq_internal.h"

namespace kvq {

// Device status word bit of the prompt kernels.
constexpr int32_t kStatusPromptTimeout = 0x102;  // a bounded mbarrier wait gave up

struct PromptSeq {
  int32_t start;  // first token row
  int32_t len;
};

// Tiles of one launch.  Sequence s (sorted by falling length) is cut into
// nb[s] = ceil(len / step) blocks of ``step`` tokens.  Block costs grow along a
// sequence (causal), so tiles are taken level by level from the top: level l
// holds block l of every sequence that has one, times the KV heads.  Segment k
// is the levels that exactly the first k + 1 sequences reach; first[k] is its
// first tile.
struct PromptTiles {
  int32_t n_seqs, Hkv, step;
  int64_t first[kMaxSeqsPerLaunch + 1];
  PromptSeq seq[kMaxSeqsPerLaunch];
};

__host__ __device__ inline int prompt_blocks(int len, int step) { return (int)(((int64_t)len + step - 1) / step); }

// Tile x: its sequence (index into seq), KV head and level.
__host__ __device__ inline void prompt_tile(const PromptTiles& t, int64_t x, int* seq, int* head, int* level) {
  int lo = 0, hi = t.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  const int64_t off = x - t.first[lo], per = (int64_t)(lo + 1) * t.Hkv;
  const int down = (int)(off / per), rem = (int)(off - down * per);
  *level = prompt_blocks(t.seq[lo].len, t.step) - 1 - down;
  *seq = rem / t.Hkv;
  *head = rem - *seq * t.Hkv;
}

// Tiles of a cross attention: sequence s (sorted by falling number of states) is
// cut into nb[s] = ceil(q_len / step) blocks; its tiles, from first[s] on, are
// its blocks of KV head 0, then of head 1 and so on.
struct CrossSeq {
  int32_t q_start, q_len;      // rows of q and out
  int32_t kv_start, kv_len;    // rows of k and v
};

struct CrossTiles {
  int32_t n_seqs, Hkv, step;
  int64_t first[kMaxSeqsPerLaunch + 1];
  CrossSeq seq[kMaxSeqsPerLaunch];
};

// What a tile's kernel needs to know: its sequence, KV head and block of tokens.
struct Tile {
  CrossSeq seq;
  int head, level;
};
__host__ __device__ inline Tile tile_at(const PromptTiles& t, int64_t x) {
  Tile r;
  int s;
  prompt_tile(t, x, &s, &r.head, &r.level);
  r.seq = {t.seq[s].start, t.seq[s].len, t.seq[s].start, t.seq[s].len};
  return r;
}
__host__ __device__ inline Tile tile_at(const CrossTiles& t, int64_t x) {
  int lo = 0, hi = t.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  Tile r;
  r.seq = t.seq[lo];
  const int64_t off = x - t.first[lo];
  const int nb = prompt_blocks(r.seq.q_len, t.step);
  r.head = (int)(off / nb);
  r.level = (int)(off - (int64_t)r.head * nb);
  return r;
}

// What causal and cross attention share.
struct AttentionParams {
  int32_t D, Hq, Hkv, g;
  float scale2;                // log2(e) / sqrt(D): scores are kept in base 2
  const void* q;               // element (token, head, c) at token * q_ts + head * q_hs + c
  const void* k;
  const void* v;
  void* out;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
  float* lse;                  // [Hq][n_tokens] (attention: written if non-null; weights: read)
  int64_t n_tokens;            // rows of q (and, causal, of k and v)
  int32_t split;               // CTAs of a cluster that share a tile (of queries, or a pair of key tiles)
  int32_t* status;
};

struct PromptParams : AttentionParams {
  static constexpr bool kCausal = true;
  float* weights;              // [Hkv][n_tokens]
  int64_t last;                // weights: queries counted back from each sequence's end
  float lse_hi, lse_lo;        // weights: lse times their sum is in the scores' units
  PromptTiles tiles;
};

struct CrossParams : AttentionParams {
  static constexpr bool kCausal = false;
  int64_t n_kv_tokens;         // rows of k and v
  CrossTiles tiles;
};

struct EvictSeq {
  int64_t out_row;             // rows (of every KV head) before this sequence's
  int32_t start, len, keep;
};

struct EvictParams {
  int32_t Hkv, row_bytes;      // bytes of one token's head
  int32_t first, recent;
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_ts, k_hs, v_ts, v_hs;  // bytes
  const float* weights;        // [Hkv][n_tokens]
  int64_t n_tokens;
  uint8_t* k_out;              // per sequence [Hkv][keep][row_bytes]
  uint8_t* v_out;
  int32_t* index;              // per sequence [Hkv][keep]
  int32_t n_seqs;
  EvictSeq seq[kMaxSeqsPerLaunch];
};

// A sum that keeps what its additions round off (Kahan, "Further remarks on
// reducing truncation errors", 1965): thousands of tiles may meet in one weight.
struct RunningSum {
  float sum, rest;
  __device__ __forceinline__ void add(float x) {
    const float y = __fsub_rn(x, rest), next = __fadd_rn(sum, y);
    const float lost = __fsub_rn(__fsub_rn(next, sum), y);
    rest = fabsf(lost) < INFINITY ? lost : 0.f;  // an infinite sum stays infinite
    sum = next;
  }
};

// Launch with clusters of ``split`` CTAs in a row a tile.
template <typename... Params, typename... Args>
cudaError_t launch_cluster(void (*kernel)(Params...), int64_t tiles, int split, int threads, size_t smem, cudaStream_t s,
                           const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Clusters of ``size`` CTAs of a kernel that run at once on the current device, asked
// for once a size and ``kind`` (0..16: calls of one kind have the same shared memory);
// 0 if unknown.
template <auto KERNEL>
int active_clusters(int size, int threads, size_t smem, int kind = 0) {
  static std::atomic<int> known[64][17][17];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || size > 16 || kind > 16) return 0;
  int n = known[dev][size][kind].load();
  if (n) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[dev][size][kind].store(n + 1);
  return n;
}

// Launchers (return the launch's error code).
cudaError_t launch_prompt_simt(const PromptParams& p, int dtype, int64_t tiles, cudaStream_t s);
cudaError_t launch_cross_simt(const CrossParams& p, int dtype, int64_t tiles, cudaStream_t s);
// CTAs that share a tile of the CUDA-core attention
int prompt_simt_split(int64_t tiles, int32_t max_len, int n_sm);
int cross_simt_split(int64_t tiles, int32_t max_kv, int n_sm);
cudaError_t launch_weights_simt(const PromptParams& p, int dtype, int64_t tiles, cudaStream_t s);
cudaError_t launch_evict(const EvictParams& p, int32_t max_len, int32_t max_keep, cudaStream_t s);

// the tensor-core attention (bf16, head_dim 64 or 128); a tile of its order is
// prompt_tc_tokens(g) tokens
cudaError_t launch_prompt_tc(const PromptParams& p, int64_t tiles, cudaStream_t s);
int prompt_tc_tokens(int g);

// the tensor-core weights: ``pairs`` pairs of 128-key tiles (KV heads counted)
// and at most most_tokens counted tokens a sequence; a CTA takes ``chunk``
// pairs, or a cluster of ``split`` CTAs one pair
void weights_tc_plan(int64_t pairs, int64_t most_tokens, int g, int n_sm, int* chunk, int* split);
cudaError_t launch_weights_tc(const PromptParams& p, int64_t tiles, cudaStream_t s);

// the tensor-core cross attention (bf16, head_dim 64 or 128): tiles of
// prompt_tc_tokens(g) tokens, taken by at most n_sm CTAs or each by a cluster of p.split
int cross_tc_split(int d, int64_t tiles, int32_t max_kv, int n_sm);
cudaError_t launch_cross_tc(const CrossParams& p, int64_t tiles, int n_sm, cudaStream_t s);

// the cross attention of few queries (bf16, head_dim 64 or 128): tiles of
// cross_rows_tokens(g) tokens, a cluster of p.split CTAs each; and up to how many
// tokens a sequence goes there
cudaError_t launch_cross_rows(const CrossParams& p, int64_t tiles, cudaStream_t s);
int cross_rows_tokens(int g);
int cross_rows_split(int64_t tiles, int32_t max_kv, int n_sm);
int cross_few_tokens(int g);

// the same on CUDA cores: tiles of cross_few_simt_step(g) tokens, at most ``rows`` rows each
cudaError_t launch_cross_few_simt(const CrossParams& p, int dtype, int rows, int64_t tiles, cudaStream_t s);
int cross_few_simt_step(int g);
int cross_few_simt_tokens(int g);
int cross_few_simt_split(int64_t tiles, int32_t max_kv, int n_sm);

// what the tensor cores' rounding takes from a score
double rounding_loss(double sums);

// TMA map of a bf16 tensor (channel, d1, d2) with strides s1, s2 (elements) and
// boxes of 64 channels x b1 x b2, 128-byte swizzled; false if the driver refuses it.
bool tma_map3(CUtensorMap* map, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t s1, int64_t s2, int b1,
              int b2);

constexpr int kMaxDim = 256;  // head_dim

// Rows of a CUDA-core attention tile and keys of one of its steps.
constexpr int kPromptRows = 64, kPromptKeys = 64;

}  // namespace kvq
