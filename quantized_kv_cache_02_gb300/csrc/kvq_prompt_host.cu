// Host side of the prompt operators: argument checks, tile order and launches
// of kvq_prompt_attention, kvq_prompt_weights and kvq_evict.  Sequence lengths
// live on the host and travel in the launch parameter block, so no call
// synchronizes with the device or needs a workspace.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "kvq_host.h"
#include "kvq_prompt.h"

namespace kvq {

bool tma_map3(CUtensorMap* map, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t s1, int64_t s2, int b1,
              int b2) {
  // the driver's encoder, looked up once (the library does not link libcuda)
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  // the stride of a dimension of one entry is not used: any legal one
  const cuuint64_t strides[2] = {(cuuint64_t)(d1 > 1 ? s1 : d0) * 2, (cuuint64_t)(d2 > 1 ? s2 : d0) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kvq

namespace {

using kvq::cuda_fail;
using kvq::fail;

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // positions and tile ends stay within 32 bits
constexpr int64_t kMaxTiles = (int64_t(1) << 31) - 1;

int esize_of(const kvq_prompt* p) { return p->dtype == KVQ_BF16 ? 2 : 4; }

// Shapes and lengths; *total receives the sum of the lengths.
kvq_status check_prompt(const kvq_prompt* p, int64_t* total) {
  if (!p) return fail(KVQ_EINVAL, "prompt is NULL");
  if (p->n_seqs < 1) return fail(KVQ_EINVAL, "n_seqs must be >= 1 (got %d)", p->n_seqs);
  if (p->n_kv_heads < 1) return fail(KVQ_EINVAL, "n_kv_heads must be >= 1");
  if (p->n_kv_heads > 65535) return fail(KVQ_EUNSUPPORTED, "n_kv_heads must be <= 65535");
  if (p->n_q_heads < 1 || p->n_q_heads % p->n_kv_heads != 0)
    return fail(KVQ_EINVAL, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", p->n_q_heads,
                p->n_kv_heads);
  if (p->n_q_heads / p->n_kv_heads > kvq::kMaxGqa)
    return fail(KVQ_EUNSUPPORTED, "query heads per KV head must be <= %d", kvq::kMaxGqa);
  if (p->head_dim < 16 || p->head_dim > kvq::kMaxDim || p->head_dim % 16 != 0)
    return fail(KVQ_EUNSUPPORTED, "head_dim must be a multiple of 16 in [16, %d] (got %d)", kvq::kMaxDim, p->head_dim);
  if (p->dtype != KVQ_BF16 && p->dtype != KVQ_FP32) return fail(KVQ_EINVAL, "unknown dtype %d", p->dtype);
  if (!p->seq_lens) return fail(KVQ_EINVAL, "seq_lens is NULL");
  if (p->n_tokens < 0 || p->n_tokens > kMaxTokens)
    return fail(KVQ_EINVAL, "n_tokens must be in [0, 2^30] (got %lld)", (long long)p->n_tokens);
  int64_t sum = 0;
  for (int i = 0; i < p->n_seqs; ++i) {
    if (p->seq_lens[i] < 0 || p->seq_lens[i] > p->n_tokens - sum)
      return fail(KVQ_EINVAL, "length %lld of sequence %d is negative or goes past the %lld token rows",
                  (long long)p->seq_lens[i], i, (long long)p->n_tokens);
    sum += p->seq_lens[i];
  }
  *total = sum;
  return KVQ_OK;
}

// A [tokens][heads][head_dim] tensor: strides in elements, 16-byte steps.
kvq_status check_tensor(const kvq_prompt* p, const char* name, const void* ptr, int64_t ts, int64_t hs, int heads) {
  if (!ptr || ((uintptr_t)ptr & 15u))
    return fail(KVQ_EINVAL, "%s must be a non-NULL 16-byte aligned device pointer", name);
  const int64_t step = 16 / esize_of(p);
  if ((p->n_tokens > 1 && (ts < p->head_dim || ts % step)) || (heads > 1 && (hs < p->head_dim || hs % step)))
    return fail(KVQ_EINVAL, "%s strides (token %lld, head %lld) must be multiples of %lld elements and at least head_dim",
                name, (long long)ts, (long long)hs, (long long)step);
  const int64_t most = (int64_t(1) << 40) / esize_of(p);
  if ((p->n_tokens > 1 && ts >= most) || (heads > 1 && hs >= most))
    return fail(KVQ_EUNSUPPORTED, "%s strides must be below 2^40 bytes", name);
  return KVQ_OK;
}

// No two of out's rows may share memory.
kvq_status check_out(const kvq_prompt* p, const void* ptr) {
  const int64_t ts = p->out_token_stride, hs = p->out_head_stride, d = p->head_dim;
  const kvq_status st = check_tensor(p, "out", ptr, ts, hs, p->n_q_heads);
  if (st != KVQ_OK) return st;
  if (p->n_tokens > 1 && p->n_q_heads > 1 && hs * (p->n_q_heads - 1) + d > ts && ts * (p->n_tokens - 1) + d > hs)
    return fail(KVQ_EINVAL, "out strides (token %lld, head %lld) make its rows overlap", (long long)ts, (long long)hs);
  return KVQ_OK;
}

// Kernels launch on the current device: every tensor has to live there.
kvq_status check_on_device(const char* name, const void* ptr) {
  int cur = -1;
  cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  cudaPointerAttributes attr;
  e = cudaPointerGetAttributes(&attr, ptr);
  if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes");
  if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
    return fail(KVQ_EINVAL, "%s is not device memory", name);
  if (attr.type == cudaMemoryTypeDevice && attr.device != cur)
    return fail(KVQ_EINVAL, "the current device is %d but %s lives on device %d", cur, name, attr.device);
  return KVQ_OK;
}

kvq_status check_floats(const char* name, const void* ptr) {
  if (!ptr || ((uintptr_t)ptr & 3u)) return fail(KVQ_EINVAL, "%s must be a non-NULL 4-byte aligned device pointer", name);
  return check_on_device(name, ptr);
}

kvq_status check_status_word(const kvq_prompt* p) { return p->status ? check_floats("status", p->status) : KVQ_OK; }

#define KVQ_TRY(x)                       \
  do {                                   \
    const kvq_status st_ = (x);          \
    if (st_ != KVQ_OK) return st_;       \
  } while (0)

// The sequences of the prompt that hold tokens, in launches of at most
// kMaxSeqsPerLaunch, each sorted by falling length.
std::vector<std::vector<kvq::PromptSeq>> launches_of(const kvq_prompt* p) {
  std::vector<std::vector<kvq::PromptSeq>> out;
  int64_t start = 0;
  for (int i = 0; i < p->n_seqs; ++i) {
    const int64_t n = p->seq_lens[i];
    if (n > 0) {
      if (out.empty() || (int)out.back().size() == kvq::kMaxSeqsPerLaunch) out.emplace_back();
      out.back().push_back({(int32_t)start, (int32_t)n});
    }
    start += n;
  }
  for (auto& l : out)
    std::stable_sort(l.begin(), l.end(), [](const kvq::PromptSeq& a, const kvq::PromptSeq& b) { return a.len > b.len; });
  return out;
}

// The tensor-core kernels' shapes.
bool tensor_cores(const kvq_prompt* p) {
  return p->dtype == KVQ_BF16 && (p->head_dim == 64 || p->head_dim == 128);
}

kvq_status sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? KVQ_OK : cuda_fail(e, "cudaDeviceGetAttribute");
}

// Tiles of ``step`` tokens over the sequences; returns their number.
int64_t fill_tiles(const std::vector<kvq::PromptSeq>& seqs, int hkv, int step, kvq::PromptTiles* t) {
  t->n_seqs = (int32_t)seqs.size();
  t->Hkv = hkv;
  t->step = step;
  int64_t x = 0;
  for (int k = 0; k < t->n_seqs; ++k) {
    t->seq[k] = seqs[k];
    t->first[k] = x;
    const int64_t below = k + 1 < t->n_seqs ? kvq::prompt_blocks(seqs[k + 1].len, step) : 0;
    x += (kvq::prompt_blocks(seqs[k].len, step) - below) * (int64_t)(k + 1) * hkv;
  }
  t->first[t->n_seqs] = x;
  return x;
}

// The tensor cores round every accumulation toward zero (Fasi, Higham, Mikaitis
// and Pranesh, "Numerical behavior of NVIDIA tensor cores", 2021): a score loses
// half a step of each partial sum on average, and a step is 2^-23 / (2 ln 2) of
// its number on average.  The relative loss of a score whose partial sums add up to
// ``sums`` times its size, by which its factor is raised.
// An estimate, for channels whose products are spread in size and sign.  Measured
// on normal queries and Keys (1024 tokens, d = 128, all weights' sum off by; without
// the factor in brackets): plain 0.5e-7 (1.3e-7), a heavy channel in every 16 0.8e-7
// (10e-7), the heavy ones all first 0.8e-7 (5.8e-7), all last 1.6e-7 (3.4e-7).
// Where nothing is rounded off (products of one sign, close in size) the factor
// itself is left over, 0.9e-7 of the score; where small products of one sign follow
// one heavy step, each loses its own low bits, and 5e-7 of the score stay lost.
double rounding_loss(double sums) { return 0.5 * sums * std::ldexp(1.0, -23) / (2.0 * std::log(2.0)); }

// sqrt(d) for the scores: their factor, and lse in their units -- on the tensor
// cores before the factor, else after it -- as a factor in two floats.
void set_scale(const kvq_prompt* p, double loss, kvq::PromptParams* pp) {
  const double root = std::sqrt((double)p->head_dim);
  pp->scale2 = (float)(1.4426950408889634 / root * (1.0 + loss));
  const double r = tensor_cores(p) ? root / (1.0 + loss) : root * (double)pp->scale2;
  pp->lse_hi = (float)r;
  pp->lse_lo = (float)(r - (double)pp->lse_hi);
}

void base_params(const kvq_prompt* p, kvq::PromptParams* pp) {
  memset(pp, 0, sizeof *pp);
  pp->D = p->head_dim;
  pp->Hq = p->n_q_heads;
  pp->Hkv = p->n_kv_heads;
  pp->g = p->n_q_heads / p->n_kv_heads;
  pp->q_ts = p->q_token_stride;
  pp->q_hs = p->q_head_stride;
  pp->k_ts = p->k_token_stride;
  pp->k_hs = p->k_head_stride;
  pp->v_ts = p->v_token_stride;
  pp->v_hs = p->v_head_stride;
  pp->o_ts = p->out_token_stride;
  pp->o_hs = p->out_head_stride;
  pp->n_tokens = p->n_tokens;
  pp->status = p->status;
}

kvq_status prompt_attention(const kvq_prompt* p, const void* q, const void* k, const void* v, void* out, float* lse,
                            void* stream) {
  int64_t total = 0;
  KVQ_TRY(check_prompt(p, &total));
  if (total == 0) return KVQ_OK;
  KVQ_TRY(check_tensor(p, "q", q, p->q_token_stride, p->q_head_stride, p->n_q_heads));
  KVQ_TRY(check_tensor(p, "k", k, p->k_token_stride, p->k_head_stride, p->n_kv_heads));
  KVQ_TRY(check_tensor(p, "v", v, p->v_token_stride, p->v_head_stride, p->n_kv_heads));
  KVQ_TRY(check_out(p, out));
  KVQ_TRY(check_on_device("q", q));
  KVQ_TRY(check_on_device("k", k));
  KVQ_TRY(check_on_device("v", v));
  KVQ_TRY(check_on_device("out", out));
  if (lse) KVQ_TRY(check_floats("lse", lse));
  KVQ_TRY(check_status_word(p));
  kvq::PromptParams pp;
  base_params(p, &pp);
  pp.q = q;
  pp.k = k;
  pp.v = v;
  pp.out = out;
  pp.lse = lse;
  // D / 16 partial sums that grow evenly
  set_scale(p, tensor_cores(p) ? rounding_loss((p->head_dim / 16 + 1) / 2.0) : 0.0, &pp);
  const bool tc = tensor_cores(p);
  const int step = tc ? kvq::prompt_tc_tokens(pp.g) : kvq::kPromptRows / pp.g;
  int n_sm = 0;
  KVQ_TRY(sm_count(&n_sm));
  const auto launches = launches_of(p);
  for (const auto& l : launches)
    if (fill_tiles(l, pp.Hkv, step, &pp.tiles) > kMaxTiles / 4) return fail(KVQ_EUNSUPPORTED, "too many tiles for one launch");
  for (const auto& l : launches) {
    const int64_t tiles = fill_tiles(l, pp.Hkv, step, &pp.tiles);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    pp.split = tc ? 1 : kvq::prompt_simt_split(tiles, l[0].len, n_sm);
    const cudaError_t e = tc ? kvq::launch_prompt_tc(pp, tiles, s)
                             : kvq::launch_prompt_simt(pp, p->dtype == KVQ_BF16 ? 0 : 1, tiles, s);
    if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
    kvq::count_launches(1);
  }
  return KVQ_OK;
}

kvq_status prompt_weights(const kvq_prompt* p, const void* q, const void* k, const float* lse, int64_t last,
                          float* weights, void* stream) {
  int64_t total = 0;
  KVQ_TRY(check_prompt(p, &total));
  if (last < 1) return fail(KVQ_EINVAL, "last must be >= 1 (got %lld)", (long long)last);
  if (total == 0) return KVQ_OK;
  KVQ_TRY(check_tensor(p, "q", q, p->q_token_stride, p->q_head_stride, p->n_q_heads));
  KVQ_TRY(check_tensor(p, "k", k, p->k_token_stride, p->k_head_stride, p->n_kv_heads));
  KVQ_TRY(check_on_device("q", q));
  KVQ_TRY(check_on_device("k", k));
  KVQ_TRY(check_floats("lse", lse));
  KVQ_TRY(check_floats("weights", weights));
  KVQ_TRY(check_status_word(p));
  kvq::PromptParams pp;
  base_params(p, &pp);
  pp.q = q;
  pp.k = k;
  pp.lse = const_cast<float*>(lse);
  pp.weights = weights;
  pp.last = last;
  // Two halves of D / 32 partial sums that grow to half the score; the second
  // ends with lse taken off, which leaves about minus half the score of a heavy
  // weight and loses the other way.
  set_scale(p, tensor_cores(p) ? rounding_loss((p->head_dim / 32 + 1) / 2.0 - 0.5) : 0.0, &pp);
  pp.split = 1;
  const bool tc = tensor_cores(p);
  int n_sm = 0;
  if (tc) KVQ_TRY(sm_count(&n_sm));
  const auto launches = launches_of(p);
  auto step_of = [&](const std::vector<kvq::PromptSeq>& l) {
    if (!tc) return kvq::kPromptKeys;
    int64_t pairs = 0;
    for (const kvq::PromptSeq& q1 : l) pairs += (int64_t)kvq::prompt_blocks(q1.len, 256) * pp.Hkv;
    int chunk;
    kvq::weights_tc_plan(pairs, std::min<int64_t>(last, l[0].len), pp.g, n_sm, &chunk, &pp.split);
    return 256 * chunk;
  };
  for (const auto& l : launches) {
    const int step = step_of(l);  // sets pp.split
    if (fill_tiles(l, pp.Hkv, step, &pp.tiles) > kMaxTiles / pp.split)
      return fail(KVQ_EUNSUPPORTED, "too many tiles for one launch");
  }
  for (const auto& l : launches) {
    const int64_t tiles = fill_tiles(l, pp.Hkv, step_of(l), &pp.tiles);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = tc ? kvq::launch_weights_tc(pp, tiles, s)
                             : kvq::launch_weights_simt(pp, p->dtype == KVQ_BF16 ? 0 : 1, tiles, s);
    if (e != cudaSuccess) return cuda_fail(e, "prompt weights launch");
    kvq::count_launches(1);
  }
  return KVQ_OK;
}

kvq_status evict(const kvq_prompt* p, const void* k, const void* v, const float* weights, const int64_t* keep,
                 int64_t first, int64_t recent, void* k_out, void* v_out, int32_t* index, void* stream) {
  int64_t total = 0;
  KVQ_TRY(check_prompt(p, &total));
  if (!keep) return fail(KVQ_EINVAL, "keep is NULL");
  if (first < 0 || recent < 0)
    return fail(KVQ_EINVAL, "first (%lld) and recent (%lld) must not be negative", (long long)first, (long long)recent);
  int64_t kept = 0;
  for (int i = 0; i < p->n_seqs; ++i) {
    if (keep[i] < 0 || keep[i] > p->seq_lens[i])
      return fail(KVQ_EINVAL, "keep[%d] = %lld is outside [0, %lld]", i, (long long)keep[i], (long long)p->seq_lens[i]);
    if (keep[i] < p->seq_lens[i] && (first > keep[i] || recent > keep[i] - first))
      return fail(KVQ_EINVAL, "sequence %d keeps %lld tokens, fewer than its first %lld and last %lld", i,
                  (long long)keep[i], (long long)first, (long long)recent);
    kept += keep[i];
  }
  if (kept == 0) return KVQ_OK;
  KVQ_TRY(check_tensor(p, "k", k, p->k_token_stride, p->k_head_stride, p->n_kv_heads));
  KVQ_TRY(check_tensor(p, "v", v, p->v_token_stride, p->v_head_stride, p->n_kv_heads));
  if (!k_out || !v_out || ((uintptr_t)k_out & 15u) || ((uintptr_t)v_out & 15u))
    return fail(KVQ_EINVAL, "k_out / v_out must be non-NULL 16-byte aligned device pointers");
  KVQ_TRY(check_on_device("k", k));
  KVQ_TRY(check_on_device("v", v));
  KVQ_TRY(check_on_device("k_out", k_out));
  KVQ_TRY(check_on_device("v_out", v_out));
  KVQ_TRY(check_floats("weights", weights));
  KVQ_TRY(check_floats("index", index));
  const int es = esize_of(p);
  kvq::EvictParams ep;
  memset(&ep, 0, sizeof ep);
  ep.Hkv = p->n_kv_heads;
  ep.row_bytes = p->head_dim * es;
  // neither can pass a length that evicts, and a sequence that keeps everything reads neither
  ep.first = (int32_t)std::min<int64_t>(first, p->n_tokens);
  ep.recent = (int32_t)std::min<int64_t>(recent, p->n_tokens);
  ep.k = static_cast<const uint8_t*>(k);
  ep.v = static_cast<const uint8_t*>(v);
  ep.k_ts = p->k_token_stride * es;
  ep.k_hs = p->k_head_stride * es;
  ep.v_ts = p->v_token_stride * es;
  ep.v_hs = p->v_head_stride * es;
  ep.weights = weights;
  ep.n_tokens = p->n_tokens;
  ep.k_out = static_cast<uint8_t*>(k_out);
  ep.v_out = static_cast<uint8_t*>(v_out);
  ep.index = index;
  int64_t start = 0, row = 0;
  for (int i = 0; i < p->n_seqs;) {
    ep.n_seqs = 0;
    int32_t max_len = 0, max_keep = 0;
    for (; i < p->n_seqs && ep.n_seqs < kvq::kMaxSeqsPerLaunch; ++i) {
      if (keep[i] > 0) {
        ep.seq[ep.n_seqs++] = {row, (int32_t)start, (int32_t)p->seq_lens[i], (int32_t)keep[i]};
        max_len = std::max(max_len, (int32_t)p->seq_lens[i]);
        max_keep = std::max(max_keep, (int32_t)keep[i]);
      }
      start += p->seq_lens[i];
      row += keep[i] * p->n_kv_heads;
    }
    if (ep.n_seqs == 0) continue;
    const cudaError_t e = kvq::launch_evict(ep, max_len, max_keep, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "evict launch");
    kvq::count_launches(1);
  }
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_prompt_attention(const kvq_prompt* prompt, const void* q, const void* k, const void* v, void* out,
                                float* lse, void* stream) {
  try {
    return prompt_attention(prompt, q, k, v, out, lse, stream);
  } catch (const std::bad_alloc&) {
    return fail(KVQ_ENOMEM, "out of host memory");
  }
}

kvq_status kvq_prompt_weights(const kvq_prompt* prompt, const void* q, const void* k, const float* lse, int64_t last,
                              float* weights, void* stream) {
  try {
    return prompt_weights(prompt, q, k, lse, last, weights, stream);
  } catch (const std::bad_alloc&) {
    return fail(KVQ_ENOMEM, "out of host memory");
  }
}

kvq_status kvq_evict(const kvq_prompt* prompt, const void* k, const void* v, const float* weights, const int64_t* keep,
                     int64_t first, int64_t recent, void* k_out, void* v_out, int32_t* index, void* stream) {
  return evict(prompt, k, v, weights, keep, first, recent, k_out, v_out, index, stream);
}

}  // extern "C"
