// Rotary positions with several axes (kvq_rotary): pair i of a head, at
// frequency f_i on the axis a_i of the token's position, is turned by the angle
// t = position[a_i] f_i,
//   y1 = x1 cos t - x2 sin t,   y2 = x1 sin t + x2 cos t   (-t when inverse).
//
// Angles.  A position of 2^20 at f = 1 leaves an fp32 angle 4 of its bits behind
// the point.  Here f / 2 pi is a fraction of 2^64, so that position times
// fraction, modulo 2^64, is the angle in turns with its whole turns gone: off by
// at most |position| 2^-65 turns, in three integer multiplies and without fp64.  The
// upper 32 bits are split into a quadrant and an eighth of a turn to either side
// of it, where sincospif keeps the fp32 step of small arguments.
//
// Bound: HBM, each element read and written once.  A block takes a few tokens with all
// their q and k heads, so each angle is computed once (its table entry is a
// divergent constant load and its sine and cosine some 60 instructions: computed by
// every thread for its own pieces they took as long as the copies).  A thread keeps a
// 16-byte piece's place (or the two that hold the halves of its pairs) and its sines
// through a run of heads, the next heads' loads in flight while it turns the last.
// ("KV Cache 与自回归视频生成": the cache holds Keys after their positions.)

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "kvq_args.h"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kMaxPairs = 128, kMaxAxes = 4;
constexpr int kRotaryThreads = 256, kMaxAngles = 2048;
constexpr int kAhead = 4;  // heads loaded at once
// Blocks an SM below which a block takes fewer tokens (14400 tokens of 32 + 8 heads of 128 in
// us: 4 48.8, 6 46.4, 16 51.5, 32 63.7; 4096 tokens: 14.0, 14.0, 21.2, 21.3).
constexpr int kBlocksPerSm = 6;

struct RotaryTensor {
  const void* in;
  void* out;
  int64_t in_ts, in_hs, out_ts, out_hs;  // elements
  int32_t heads;
};

struct RotaryParams {
  int32_t D, pairs, items, n_tensors;
  int32_t heads;               // of all tensors
  int32_t tokens, lanes;       // of a block: tokens, and heads taken side by side
  int32_t run;                 // heads a block takes
  int32_t inverse, wide;       // wide: 8-byte positions
  int64_t n_tokens;
  const void* positions;
  int64_t p_ts, p_as;          // elements
  RotaryTensor t[2];
  uint64_t turns[kMaxPairs];   // f / 2 pi, modulo 1, in units of 2^-64
  uint8_t axis[kMaxPairs];
};

__device__ __forceinline__ void sincos_turns(uint64_t turns, float* c, float* s) {
  const uint32_t at = (uint32_t)((turns + 0x80000000u) >> 32);
  const uint32_t quadrant = (at + 0x20000000u) >> 30;
  float a, b;
  sincospif((float)(int32_t)(at - (quadrant << 30)) * 0x1p-31f, &a, &b);  // sine, cosine
  const bool swap = quadrant & 1u;
  const float cc = swap ? a : b, ss = swap ? b : a;
  *c = (quadrant == 1u || quadrant == 2u) ? -cc : cc;
  *s = (quadrant & 2u) ? -ss : ss;
}

// A thread's share of a head: one 16-byte piece of E elements at A (and, for halves, one at B).
enum Shape { kHalves, kAdjacent, kRows };

template <typename T, int SHAPE>
struct Share {
  static constexpr int E = 16 / (int)sizeof(T);
  static constexpr int kAngles = SHAPE == kAdjacent ? E / 2 : E;
  T a[E], b[SHAPE == kAdjacent ? 1 : E];
};

template <typename T>
__device__ __forceinline__ void move_piece(T* dst, const T* src) {
  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16(x);
  else return x;
}

// [token][pair]: cosine and sine.  A warp's lanes lie along the tokens, so that few of its
// table entries differ.
__device__ __forceinline__ void fill_angles(const RotaryParams& p, int64_t first, int n_tok, float2* turned) {
  for (int y = threadIdx.x; y < n_tok * p.pairs; y += kRotaryThreads) {
    const int pair = y / n_tok, t = y - pair * n_tok;
    const int64_t at = (first + t) * p.p_ts + p.axis[pair] * p.p_as;
    const int64_t pos = p.wide ? static_cast<const int64_t*>(p.positions)[at]
                               : (int64_t)static_cast<const int32_t*>(p.positions)[at];
    float2 cs;
    sincos_turns((uint64_t)pos * p.turns[pair], &cs.x, &cs.y);
    if (p.inverse) cs.y = -cs.y;
    turned[t * p.pairs + pair] = cs;
  }
}

// Head ``head`` of all tensors' heads, of a token.
template <typename T>
__device__ __forceinline__ const T* head_in(const RotaryParams& p, int64_t token, int head) {
  const RotaryTensor& t = p.t[head >= p.t[0].heads];
  return static_cast<const T*>(t.in) + token * t.in_ts + (head - (head >= p.t[0].heads ? p.t[0].heads : 0)) * t.in_hs;
}
template <typename T>
__device__ __forceinline__ T* head_out(const RotaryParams& p, int64_t token, int head) {
  const RotaryTensor& t = p.t[head >= p.t[0].heads];
  return static_cast<T*>(t.out) + token * t.out_ts + (head - (head >= p.t[0].heads ? p.t[0].heads : 0)) * t.out_hs;
}

// x1, x2 by the angle of cs, rounded once.
template <typename T>
__device__ __forceinline__ void turn(T& u, T& v, float2 cs) {
  const float x1 = to_float(u), x2 = to_float(v);
  u = from_float<T>(fmaf(x1, cs.x, -x2 * cs.y));
  v = from_float<T>(fmaf(x1, cs.y, x2 * cs.x));
}

template <typename T, int SHAPE>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using S = Share<T, SHAPE>;
  __shared__ __align__(16) float2 turned[kMaxAngles];  // [token][pair]: cosine, sine
  const int tid = threadIdx.x, slot = tid / p.items, item = tid - slot * p.items;
  const int lane = slot / p.tokens, own = slot - lane * p.tokens;
  const int64_t first = (int64_t)blockIdx.x * p.tokens, token = first + own;
  const int n_tok = (int)min((int64_t)p.tokens, p.n_tokens - first);
  pdl_wait();
  pdl_release();

  // where the share lies, its pairs, and whether it only passes through
  int at_a, at_b = 0, pair0;
  bool through = false;
  if (SHAPE == kAdjacent) {
    at_a = item * S::E;
    pair0 = at_a / 2;
    through = pair0 >= p.pairs;
  } else {
    const int pieces = p.pairs / S::E;
    through = item >= pieces;
    at_a = through ? 2 * p.pairs + (item - pieces) * S::E : item * S::E;
    at_b = at_a + p.pairs;
    pair0 = at_a;
  }
  const int h1 = min(p.heads, (int)(blockIdx.y + 1) * p.run);
  int h = lane < p.lanes && own < n_tok ? blockIdx.y * p.run + lane : h1;  // (threads past the last lane have no work)

  S x[kAhead];
  auto load = [&] {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (h + e * p.lanes >= h1) break;
      const T* in = head_in<T>(p, token, h + e * p.lanes);
      move_piece(x[e].a, in + at_a);
      if (SHAPE != kAdjacent && !through) move_piece(x[e].b, in + at_b);
    }
  };
  load();
  fill_angles(p, first, n_tok, turned);  // under the first loads
  __syncthreads();
  if (h >= h1) return;
  float2 cs[S::kAngles];
#pragma unroll
  for (int i = 0; i < S::kAngles; ++i) {
    const bool real = !through && pair0 + i < p.pairs;
    cs[i] = real ? turned[own * p.pairs + pair0 + i] : make_float2(1.f, 0.f);
  }
  while (true) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (h + e * p.lanes >= h1) break;
      if (!through) {
#pragma unroll
        for (int i = 0; i < S::kAngles; ++i) {
          T& u = SHAPE == kAdjacent ? x[e].a[2 * i] : x[e].a[i];
          T& v = SHAPE == kAdjacent ? x[e].a[2 * i + 1] : x[e].b[i];
          if (SHAPE == kAdjacent && pair0 + i >= p.pairs) continue;  // as it is, infinities too
          turn(u, v, cs[i]);
        }
      }
      T* out = head_out<T>(p, token, h + e * p.lanes);
      move_piece(out + at_a, x[e].a);
      if (SHAPE != kAdjacent && !through) move_piece(out + at_b, x[e].b);
    }
    h += kAhead * p.lanes;
    if (h >= h1) break;
    load();
  }
}

// Halves whose second one starts off a 16-byte step: a warp takes whole heads through
// shared memory, 2 KB at a time, and turns them there.
template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotary_rows_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kPieces = 32 * kAhead, kE = 16 / (int)sizeof(T);
  __shared__ __align__(16) float2 turned[kMaxAngles];
  __shared__ uint4 pieces[kRotaryThreads / 32][kPieces];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = (int64_t)blockIdx.x * p.tokens;
  const int n_tok = (int)min((int64_t)p.tokens, p.n_tokens - first);
  pdl_wait();
  pdl_release();
  fill_angles(p, first, n_tok, turned);
  __syncthreads();
  const int per_head = p.D / kE, at_once = kPieces / per_head;  // heads in the warp's pieces
  const int h0 = blockIdx.y * p.run, heads = min(p.heads - h0, p.run), all = n_tok * heads;
  uint4* mine = pieces[warp];
  for (int r0 = warp * at_once; r0 < all; r0 += kRotaryThreads / 32 * at_once) {
    const int n = min(at_once, all - r0);
    uint4 x[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int y = lane + 32 * e, r = y / per_head, t = (r0 + r) / heads;
      if (r < n)
        x[e] = reinterpret_cast<const uint4*>(head_in<T>(p, first + t, h0 + r0 + r - t * heads))[y - r * per_head];
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) mine[lane + 32 * e] = x[e];  // (past the heads: not looked at)
    __syncwarp();
    for (int y = lane; y < n * p.pairs; y += 32) {
      const int r = y / p.pairs, pair = y - r * p.pairs, t = (r0 + r) / heads;
      T* row = reinterpret_cast<T*>(mine) + r * p.D;
      turn(row[pair], row[pair + p.pairs], turned[t * p.pairs + pair]);
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int y = lane + 32 * e, r = y / per_head, t = (r0 + r) / heads;
      if (r < n)
        reinterpret_cast<uint4*>(head_out<T>(p, first + t, h0 + r0 + r - t * heads))[y - r * per_head] = mine[y];
    }
    __syncwarp();
  }
}

template <typename T>
cudaError_t launch_t(const RotaryParams& p, Shape shape, dim3 grid, cudaStream_t s) {
  const dim3 block(kRotaryThreads);
  return shape == kHalves     ? launch_pdl(rotary_kernel<T, kHalves>, grid, block, 0, s, p)
         : shape == kAdjacent ? launch_pdl(rotary_kernel<T, kAdjacent>, grid, block, 0, s, p)
                              : launch_pdl(rotary_rows_kernel<T>, grid, block, 0, s, p);
}

// f / 2 pi modulo 1 in units of 2^-64: the quotient in two doubles (its product
// with the rest of 1 / 2 pi and the product's own rounding in the second), each
// rounded to an integer.
uint64_t turns_of(double f) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvRest = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
  const double hi = f * kInv, lo = std::fma(f, kInv, -hi) + f * kInvRest;
  double part = hi - std::nearbyint(hi);  // exact, in [-1/2, 1/2]
  if (part == 0.5) part = -0.5;           // the same angle, and 2^63 would not fit
  auto fixed = [](double x) { return (uint64_t)(int64_t)std::nearbyint(std::ldexp(x, 64)); };
  return fixed(part) + fixed(lo);
}

kvq_status rotary(const kvq_rotary_plan* plan, const void* positions, int32_t position_bytes,
                  int64_t position_token_stride, int64_t position_axis_stride, int64_t n_tokens, int32_t dtype,
                  const kvq_rotary_tensor* tensors, int32_t n_tensors, int32_t inverse, void* stream) {
  if (!plan) return fail(KVQ_EINVAL, "plan is NULL");
  const int d = plan->head_dim;
  if (d < 16 || d > 2 * kMaxPairs || d % 16 != 0)
    return fail(KVQ_EUNSUPPORTED, "head_dim must be a multiple of 16 in [16, %d] (got %d)", 2 * kMaxPairs, d);
  if (plan->n_axes < 1 || plan->n_axes > kMaxAxes)
    return fail(KVQ_EINVAL, "n_axes must be in [1, %d] (got %d)", kMaxAxes, plan->n_axes);
  if (plan->n_pairs < 1 || plan->n_pairs > d / 2)
    return fail(KVQ_EINVAL, "n_pairs must be in [1, head_dim / 2] (got %d)", plan->n_pairs);
  if (!plan->frequency || !plan->axis) return fail(KVQ_EINVAL, "the plan's frequency or axis is NULL");
  RotaryParams p;
  memset(&p, 0, sizeof p);
  for (int i = 0; i < plan->n_pairs; ++i) {
    if (!(std::fabs(plan->frequency[i]) <= 0x1p20))
      return fail(KVQ_EINVAL, "frequency %g of pair %d is not within 2^20 of 0", plan->frequency[i], i);
    if (plan->axis[i] < 0 || plan->axis[i] >= plan->n_axes)
      return fail(KVQ_EINVAL, "axis %d of pair %d is outside [0, %d)", plan->axis[i], i, plan->n_axes);
    p.turns[i] = turns_of(plan->frequency[i]);
    p.axis[i] = (uint8_t)plan->axis[i];
  }
  if (dtype != KVQ_BF16 && dtype != KVQ_FP32) return fail(KVQ_EINVAL, "unknown dtype %d", dtype);
  if (position_bytes != 4 && position_bytes != 8)
    return fail(KVQ_EINVAL, "position_bytes must be 4 or 8 (got %d)", position_bytes);
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return fail(KVQ_EINVAL, "n_tokens must be in [0, 2^30] (got %lld)", (long long)n_tokens);
  if (!tensors) return fail(KVQ_EINVAL, "tensors is NULL");
  if (n_tensors < 1 || n_tensors > 2) return fail(KVQ_EINVAL, "n_tensors must be 1 or 2 (got %d)", n_tensors);
  constexpr int64_t kMaxStride = int64_t(1) << 30;  // (a position's offset stays within 63 bits)
  if ((n_tokens > 1 && (position_token_stride < 0 || position_token_stride > kMaxStride)) ||
      (plan->n_axes > 1 && (position_axis_stride < 0 || position_axis_stride > kMaxStride)))
    return fail(KVQ_EINVAL, "position strides (token %lld, axis %lld) must be in [0, 2^30]",
                (long long)position_token_stride, (long long)position_axis_stride);
  if (n_tokens == 0) return KVQ_OK;
  if (!positions || ((uintptr_t)positions & (position_bytes - 1)))
    return fail(KVQ_EINVAL, "positions must be a non-NULL device pointer, aligned to its elements");
  const int es = dtype == KVQ_BF16 ? 2 : 4;
  static const char* const kIn[2] = {"q", "k"};
  static const char* const kOut[2] = {"q_out", "k_out"};
  p.D = d;
  p.n_tensors = n_tensors;
  for (int n = 0; n < n_tensors; ++n) {
    const kvq_rotary_tensor& t = tensors[n];
    if (t.n_heads < 1 || t.n_heads > 65535)
      return fail(KVQ_EINVAL, "%s must have 1 to 65535 heads (got %d)", kIn[n], t.n_heads);
    KVQ_TRY(check_tensor(kIn[n], t.input, es, n_tokens, t.n_heads, d, t.in_token_stride, t.in_head_stride));
    KVQ_TRY(check_out_tensor(kOut[n], t.out, es, n_tokens, t.n_heads, d, t.out_token_stride, t.out_head_stride));
    // in place a thread reads what it writes, and nothing else, only if every row stays where it is
    if (t.input == t.out && ((n_tokens > 1 && t.in_token_stride != t.out_token_stride) ||
                          (t.n_heads > 1 && t.in_head_stride != t.out_head_stride)))
      return fail(KVQ_EINVAL, "%s in place must have the strides of %s", kOut[n], kIn[n]);
    p.t[n] = {t.input, t.out, t.in_token_stride, t.in_head_stride, t.out_token_stride, t.out_head_stride, t.n_heads};
    p.heads += t.n_heads;
  }
  for (int n = 0; n < n_tensors; ++n) {
    KVQ_TRY(check_on_device(kIn[n], tensors[n].input));
    if (tensors[n].out != tensors[n].input) KVQ_TRY(check_on_device(kOut[n], tensors[n].out));
  }
  KVQ_TRY(check_on_device("positions", positions));
  p.pairs = plan->n_pairs;
  p.inverse = inverse != 0;
  p.wide = position_bytes == 8;
  p.n_tokens = n_tokens;
  p.positions = positions;
  p.p_ts = position_token_stride;
  p.p_as = position_axis_stride;
  const int piece = 16 / es;
  const Shape shape = plan->interleaved ? kAdjacent : p.pairs % piece == 0 ? kHalves : kRows;
  p.items = shape == kHalves ? d / piece - p.pairs / piece : d / piece;
  int n_sm = 0;
  KVQ_TRY(sm_count(&n_sm));
  // As many tokens a block as leave enough blocks (and its threads fit), then the heads
  // side by side; with few tokens the heads are split among blocks too.
  p.tokens = 1;
  while (2 * p.tokens * p.items <= kRotaryThreads && 2 * p.tokens * p.pairs <= kMaxAngles &&
         n_tokens >= 2 * p.tokens * kBlocksPerSm * (int64_t)n_sm)
    p.tokens *= 2;
  p.lanes = std::min(p.heads, kRotaryThreads / (p.tokens * p.items));
  const int64_t blocks = (n_tokens + p.tokens - 1) / p.tokens;
  if (blocks > kMaxTiles) return fail(KVQ_EUNSUPPORTED, "too many tokens for one launch");
  p.run = p.heads;
  while (p.run > p.lanes && blocks * ((p.heads + p.run - 1) / p.run) < 2 * (int64_t)n_sm) p.run = (p.run + 1) / 2;
  p.run = std::max(p.run, (p.heads + 65534) / 65535);
  const dim3 grid((unsigned)blocks, (unsigned)((p.heads + p.run - 1) / p.run));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == KVQ_BF16 ? launch_t<__nv_bfloat16>(p, shape, grid, s) : launch_t<float>(p, shape, grid, s);
  if (e != cudaSuccess) return cuda_fail(e, "rotary launch");
  count_launches(1);
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" {

kvq_status kvq_rotary(const kvq_rotary_plan* plan, const void* positions, int32_t position_bytes,
                      int64_t position_token_stride, int64_t position_axis_stride, int64_t n_tokens, int32_t dtype,
                      const kvq_rotary_tensor* tensors, int32_t n_tensors, int32_t inverse, void* stream) {
  return kvq::rotary(plan, positions, position_bytes, position_token_stride, position_axis_stride, n_tokens, dtype,
                     tensors, n_tensors, inverse, stream);
}

}  // extern "C"
