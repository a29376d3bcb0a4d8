// Host side of kvq_cross_attention: argument checks, tile order and launches.
// Lengths live on the host and travel in the launch parameter block, so the call
// neither synchronizes with the device nor needs a workspace.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "kvq_args.h"
#include "kvq_prompt.h"

namespace {

using kvq::check_floats;
using kvq::check_on_device;
using kvq::check_out_tensor;
using kvq::check_tensor;
using kvq::CrossSeq;
using kvq::cuda_fail;
using kvq::fail;
using kvq::kMaxTiles;
using kvq::kMaxTokens;

kvq_status check_cross(const kvq_cross* c) {
  if (!c) return fail(KVQ_EINVAL, "cross is NULL");
  if (c->n_seqs < 1) return fail(KVQ_EINVAL, "n_seqs must be >= 1 (got %d)", c->n_seqs);
  if (c->n_kv_heads < 1) return fail(KVQ_EINVAL, "n_kv_heads must be >= 1");
  if (c->n_kv_heads > 65535) return fail(KVQ_EUNSUPPORTED, "n_kv_heads must be <= 65535");
  if (c->n_q_heads < 1 || c->n_q_heads % c->n_kv_heads != 0)
    return fail(KVQ_EINVAL, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", c->n_q_heads,
                c->n_kv_heads);
  if (c->n_q_heads / c->n_kv_heads > kvq::kMaxGqa)
    return fail(KVQ_EUNSUPPORTED, "query heads per KV head must be <= %d", kvq::kMaxGqa);
  if (c->head_dim < 16 || c->head_dim > kvq::kMaxDim || c->head_dim % 16 != 0)
    return fail(KVQ_EUNSUPPORTED, "head_dim must be a multiple of 16 in [16, %d] (got %d)", kvq::kMaxDim, c->head_dim);
  if (c->dtype != KVQ_BF16 && c->dtype != KVQ_FP32) return fail(KVQ_EINVAL, "unknown dtype %d", c->dtype);
  if (!c->q_lens || !c->kv_lens) return fail(KVQ_EINVAL, "q_lens / kv_lens is NULL");
  if (c->n_q_tokens < 0 || c->n_q_tokens > kMaxTokens || c->n_kv_tokens < 0 || c->n_kv_tokens > kMaxTokens)
    return fail(KVQ_EINVAL, "n_q_tokens and n_kv_tokens must be in [0, 2^30] (got %lld and %lld)",
                (long long)c->n_q_tokens, (long long)c->n_kv_tokens);
  return KVQ_OK;
}

// The sequences with queries; *any_kv: one of them has states.
kvq_status sequences_of(const kvq_cross* c, std::vector<CrossSeq>* out, bool* any_kv) {
  int64_t q = 0, kv = 0;
  *any_kv = false;
  for (int i = 0; i < c->n_seqs; ++i) {
    const int64_t n = c->q_lens[i], m = c->kv_lens[i];
    if (n < 0 || n > c->n_q_tokens - q)
      return fail(KVQ_EINVAL, "query length %lld of sequence %d is negative or goes past the %lld rows", (long long)n, i,
                  (long long)c->n_q_tokens);
    const int64_t at = c->kv_starts ? c->kv_starts[i] : kv;
    if (at < 0 || at > c->n_kv_tokens || m < 0 || m > c->n_kv_tokens - at)
      return fail(KVQ_EINVAL, "states [%lld, %lld + %lld) of sequence %d are not within the %lld rows", (long long)at,
                  (long long)at, (long long)m, i, (long long)c->n_kv_tokens);
    if (n > 0) {
      out->push_back({(int32_t)q, (int32_t)n, (int32_t)at, (int32_t)m});
      *any_kv |= m > 0;
    }
    q += n;
    kv += m;
  }
  return KVQ_OK;
}

// Tiles of ``step`` tokens over seqs[at, at + n), longest states first; returns their number.
int64_t fill_tiles(std::vector<CrossSeq>& seqs, size_t at, int n, int hkv, int step, kvq::CrossTiles* t) {
  std::stable_sort(seqs.begin() + at, seqs.begin() + at + n,
                   [](const CrossSeq& a, const CrossSeq& b) { return a.kv_len > b.kv_len; });
  t->n_seqs = n;
  t->Hkv = hkv;
  t->step = step;
  int64_t x = 0;
  for (int k = 0; k < n; ++k) {
    t->seq[k] = seqs[at + k];
    t->first[k] = x;
    x += (int64_t)kvq::prompt_blocks(t->seq[k].q_len, step) * hkv;
  }
  t->first[n] = x;
  return x;
}

kvq_status cross_attention(const kvq_cross* c, const void* q, const void* k, const void* v, void* out, float* lse,
                           void* stream) {
  KVQ_TRY(check_cross(c));
  std::vector<CrossSeq> seqs;
  bool any_kv;
  KVQ_TRY(sequences_of(c, &seqs, &any_kv));
  if (seqs.empty()) return KVQ_OK;
  const int es = c->dtype == KVQ_BF16 ? 2 : 4, d = c->head_dim;
  KVQ_TRY(check_tensor("q", q, es, c->n_q_tokens, c->n_q_heads, d, c->q_token_stride, c->q_head_stride));
  if (any_kv) {
    KVQ_TRY(check_tensor("k", k, es, c->n_kv_tokens, c->n_kv_heads, d, c->k_token_stride, c->k_head_stride));
    KVQ_TRY(check_tensor("v", v, es, c->n_kv_tokens, c->n_kv_heads, d, c->v_token_stride, c->v_head_stride));
  }
  KVQ_TRY(check_out_tensor("out", out, es, c->n_q_tokens, c->n_q_heads, d, c->out_token_stride, c->out_head_stride));
  KVQ_TRY(check_on_device("q", q));
  if (any_kv) {
    KVQ_TRY(check_on_device("k", k));
    KVQ_TRY(check_on_device("v", v));
  }
  KVQ_TRY(check_on_device("out", out));
  if (lse) KVQ_TRY(check_floats("lse", lse));
  if (c->status) KVQ_TRY(check_floats("status", c->status));
  int n_sm = 0;
  KVQ_TRY(kvq::sm_count(&n_sm));
  kvq::CrossParams p;
  p.D = d;
  p.Hq = c->n_q_heads;
  p.Hkv = c->n_kv_heads;
  p.g = c->n_q_heads / c->n_kv_heads;
  const bool tc = c->dtype == KVQ_BF16 && (d == 64 || d == 128) && any_kv;
  // (the tensor cores: d / 16 partial sums that grow evenly)
  p.scale2 = (float)(1.4426950408889634 / std::sqrt((double)d) *
                     (tc ? 1.0 + kvq::rounding_loss((d / 16 + 1) / 2.0) : 1.0));
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.q_ts = c->q_token_stride;
  p.q_hs = c->q_head_stride;
  p.k_ts = c->k_token_stride;
  p.k_hs = c->k_head_stride;
  p.v_ts = c->v_token_stride;
  p.v_hs = c->v_head_stride;
  p.o_ts = c->out_token_stride;
  p.o_hs = c->out_head_stride;
  p.lse = lse;
  p.n_tokens = c->n_q_tokens;
  p.n_kv_tokens = c->n_kv_tokens;
  p.status = c->status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // sequences of few queries apart from the others
  const int few = tc ? kvq::cross_few_tokens(p.g) : kvq::cross_few_simt_tokens(p.g);
  const auto many =
      std::stable_partition(seqs.begin(), seqs.end(), [few](const CrossSeq& x) { return x.q_len <= few; });
  const int dtype = c->dtype == KVQ_BF16 ? 0 : 1;
  struct Part {
    std::vector<CrossSeq> seqs;
    int step;
  } parts[2] = {{{seqs.begin(), many}, tc ? kvq::cross_rows_tokens(p.g) : kvq::cross_few_simt_step(p.g)},
                {{many, seqs.end()}, tc ? kvq::prompt_tc_tokens(p.g) : kvq::kPromptRows / p.g}};
  // every refusal before the first launch
  for (const Part& part : parts) {
    int64_t tiles = 0;
    for (size_t at = 0; at < part.seqs.size(); ++at) {
      if (at % kvq::kMaxSeqsPerLaunch == 0) tiles = 0;
      tiles += (int64_t)kvq::prompt_blocks(part.seqs[at].q_len, part.step) * p.Hkv;
      if (tiles > kMaxTiles / 16) return fail(KVQ_EUNSUPPORTED, "too many tiles for one launch");
    }
  }
  for (Part& part : parts) {
    for (size_t at = 0; at < part.seqs.size(); at += kvq::kMaxSeqsPerLaunch) {
      const int n = (int)std::min<size_t>(kvq::kMaxSeqsPerLaunch, part.seqs.size() - at);
      const int64_t tiles = fill_tiles(part.seqs, at, n, p.Hkv, part.step, &p.tiles);
      const int32_t most = p.tiles.seq[0].kv_len;
      cudaError_t e;
      if (&part == parts && tc) {
        p.split = kvq::cross_rows_split(tiles, most, n_sm);
        e = kvq::launch_cross_rows(p, tiles, s);
      } else if (&part == parts) {
        int32_t tokens = 0;
        for (int k = 0; k < n; ++k) tokens = std::max(tokens, p.tiles.seq[k].q_len);
        p.split = kvq::cross_few_simt_split(tiles, most, n_sm);
        e = kvq::launch_cross_few_simt(p, dtype, std::min(tokens, part.step) * p.g, tiles, s);
      } else if (tc) {
        p.split = kvq::cross_tc_split(d, tiles, most, n_sm);
        e = kvq::launch_cross_tc(p, tiles, n_sm, s);
      } else {
        p.split = kvq::cross_simt_split(tiles, most, n_sm);
        e = kvq::launch_cross_simt(p, dtype, tiles, s);
      }
      if (e != cudaSuccess) return cuda_fail(e, "cross attention launch");
      kvq::count_launches(1);
    }
  }
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_cross_attention(const kvq_cross* cross, const void* q, const void* k, const void* v, void* out,
                               float* lse, void* stream) {
  try {
    return cross_attention(cross, q, k, v, out, lse, stream);
  } catch (const std::bad_alloc&) {
    return fail(KVQ_ENOMEM, "out of host memory");
  }
}

}  // extern "C"
