// Internal definitions of the prompt operators (kvq_prompt_attention,
// kvq_prompt_weights, kvq_evict): launch parameter blocks, the order in which
// a launch takes its tiles, and the launchers.
#pragma once

#include <cuda.h>

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

struct PromptParams {
  int32_t D, Hq, Hkv, g;
  float scale2;                // log2(e) / sqrt(D): scores are kept in base 2
  const void* q;               // element (token, head, c) at token * q_ts + head * q_hs + c
  const void* k;
  const void* v;
  void* out;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
  float* lse;                  // [Hq][n_tokens] (attention: written if non-null; weights: read)
  float* weights;              // [Hkv][n_tokens]
  int64_t n_tokens;
  int64_t last;                // weights: queries counted back from each sequence's end
  float lse_hi, lse_lo;        // weights: lse times their sum is in the scores' units
  int32_t split;               // CTAs of a cluster that share a tile (of queries, or a pair of key tiles)
  int32_t* status;
  PromptTiles tiles;
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

// Launchers (return the launch's error code).
cudaError_t launch_prompt_simt(const PromptParams& p, int dtype, int64_t tiles, cudaStream_t s);
// CTAs that share a tile of the CUDA-core attention
int prompt_simt_split(int64_t tiles, int32_t max_len, int n_sm);
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

// TMA map of a bf16 tensor (channel, d1, d2) with strides s1, s2 (elements) and
// boxes of 64 channels x b1 x b2, 128-byte swizzled; false if the driver refuses it.
bool tma_map3(CUtensorMap* map, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t s1, int64_t s2, int b1,
              int b2);

constexpr int kMaxDim = 256;  // head_dim

// Rows of a CUDA-core attention tile and keys of one of its steps.
constexpr int kPromptRows = 64, kPromptKeys = 64;

}  // namespace kvq
