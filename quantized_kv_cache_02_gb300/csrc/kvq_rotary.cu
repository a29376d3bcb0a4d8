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
// Bound: HBM, each element read and written once.  A thread takes one 16-byte
// piece (or the two that hold the halves of its pairs) of one token, computes its
// sines once and walks a run of the q and then of the k heads, the next heads'
// loads in flight while it turns the last.
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
constexpr int kRotaryThreads = 256;
constexpr int kAhead = 4;  // heads loaded at once

struct RotaryTensor {
  const void* in;
  void* out;
  int64_t in_ts, in_hs, out_ts, out_hs;  // elements
  int32_t heads;
};

struct RotaryParams {
  int32_t D, pairs, items, n_tensors;
  int32_t heads;               // of all tensors
  int32_t run;                 // heads a thread takes
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

// A thread's share of a head: one 16-byte piece of E elements at A (and one at B), or single elements.
enum Shape { kHalves, kAdjacent, kSingle };

template <typename T, int SHAPE>
struct Share {
  static constexpr int E = SHAPE == kSingle ? 1 : 16 / (int)sizeof(T);
  static constexpr int kAngles = SHAPE == kAdjacent ? E / 2 : E;
  T a[E], b[SHAPE == kAdjacent ? 1 : E];
};

template <int E, typename T>
__device__ __forceinline__ void load_piece(T* dst, const T* src) {
  if constexpr (E == 1) *dst = *src;
  else *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
}
template <int E, typename T>
__device__ __forceinline__ void store_piece(T* dst, const T* src) {
  if constexpr (E == 1) *dst = *src;
  else *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16(x);
  else return x;
}

template <typename T, int SHAPE>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using S = Share<T, SHAPE>;
  const int64_t idx = (int64_t)blockIdx.x * kRotaryThreads + threadIdx.x;
  const int64_t token = idx / p.items;
  const int item = (int)(idx - token * p.items);
  pdl_wait();
  pdl_release();
  if (token >= p.n_tokens) return;

  // where the share lies, its pairs, and whether it only passes through
  int at_a, at_b = 0, pair0;
  bool through = false;
  if (SHAPE == kAdjacent) {
    at_a = item * S::E;
    pair0 = at_a / 2;
    through = pair0 >= p.pairs;
  } else {
    const int turned = p.pairs / S::E;
    through = item >= turned;
    at_a = through ? 2 * p.pairs + (item - turned) * S::E : item * S::E;
    at_b = at_a + p.pairs;
    pair0 = at_a;
  }
  const int h0 = blockIdx.y * p.run, h1 = min(p.heads, h0 + p.run);

  float c[S::kAngles], s[S::kAngles];
  bool ready = false;
  auto angles = [&] {
    ready = true;
    if (through) return;
    const int64_t row = token * p.p_ts;
#pragma unroll
    for (int i = 0; i < S::kAngles; ++i) {
      const int pair = pair0 + i;
      if (SHAPE == kAdjacent && pair >= p.pairs) {
        c[i] = 1.f;
        s[i] = 0.f;
        continue;
      }
      const int64_t at = row + p.axis[pair] * p.p_as;
      const int64_t pos = p.wide ? static_cast<const int64_t*>(p.positions)[at]
                                 : (int64_t)static_cast<const int32_t*>(p.positions)[at];
      sincos_turns((uint64_t)pos * p.turns[pair], &c[i], &s[i]);
      if (p.inverse) s[i] = -s[i];
    }
  };
  auto turn = [&](S& x) {
    if (through) return;
#pragma unroll
    for (int i = 0; i < S::kAngles; ++i) {
      T& u = SHAPE == kAdjacent ? x.a[2 * i] : x.a[i];
      T& v = SHAPE == kAdjacent ? x.a[2 * i + 1] : x.b[i];
      if (SHAPE == kAdjacent && pair0 + i >= p.pairs) continue;  // as it is, infinities too
      const float x1 = to_float(u), x2 = to_float(v);
      u = from_float<T>(fmaf(x1, c[i], -x2 * s[i]));
      v = from_float<T>(fmaf(x1, s[i], x2 * c[i]));
    }
  };

  int before = 0;
  for (int n = 0; n < p.n_tensors; ++n) {
    const RotaryTensor& t = p.t[n];
    const int first = max(h0 - before, 0), last = min(h1 - before, t.heads);
    before += t.heads;
    const T* in = static_cast<const T*>(t.in) + token * t.in_ts;
    T* out = static_cast<T*>(t.out) + token * t.out_ts;
    if (first >= last || (through && in == out)) continue;
    S x[kAhead];
    for (int h = first; h < last; h += kAhead) {
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (h + e >= last) break;
        load_piece<S::E>(x[e].a, in + (h + e) * t.in_hs + at_a);
        if (SHAPE != kAdjacent && !through) load_piece<S::E>(x[e].b, in + (h + e) * t.in_hs + at_b);
      }
      if (!ready) angles();  // under the first loads
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (h + e >= last) break;
        turn(x[e]);
        store_piece<S::E>(out + (h + e) * t.out_hs + at_a, x[e].a);
        if (SHAPE != kAdjacent && !through) store_piece<S::E>(out + (h + e) * t.out_hs + at_b, x[e].b);
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const RotaryParams& p, Shape shape, dim3 grid, cudaStream_t s) {
  const dim3 block(kRotaryThreads);
  return shape == kHalves     ? launch_pdl(rotary_kernel<T, kHalves>, grid, block, 0, s, p)
         : shape == kAdjacent ? launch_pdl(rotary_kernel<T, kAdjacent>, grid, block, 0, s, p)
                              : launch_pdl(rotary_kernel<T, kSingle>, grid, block, 0, s, p);
}

// f / 2 pi modulo 1 in units of 2^-64: the quotient in two doubles (its product
// with the rest of 1 / 2 pi and the product's own rounding in the second), each
// rounded to an integer.
uint64_t turns_of(double f) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvRest = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
  const double hi = f * kInv, lo = std::fma(f, kInv, -hi) + f * kInvRest;
  double part = hi - std::nearbyint(hi);  // exact, in [-1/2, 1/2]
  if (part == 0.5) part = -0.5;           // the same angle, and 2^63 would not fit
  return (uint64_t)(int64_t)std::nearbyint(std::ldexp(part, 64)) + (uint64_t)(int64_t)std::nearbyint(std::ldexp(lo, 64));
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
  // halves whose second one starts off a 16-byte step go element by element
  const int piece = 16 / es;
  const Shape shape = plan->interleaved ? kAdjacent : p.pairs % piece == 0 ? kHalves : kSingle;
  p.items = shape == kAdjacent ? d / piece : shape == kHalves ? d / piece - p.pairs / piece : d - p.pairs;
  int n_sm = 0;
  KVQ_TRY(sm_count(&n_sm));
  const int64_t threads = n_tokens * p.items, blocks = (threads + kRotaryThreads - 1) / kRotaryThreads;
  if (blocks > kMaxTiles) return fail(KVQ_EUNSUPPORTED, "too many tokens for one launch");
  p.run = p.heads;
  while (p.run > 1 && blocks * ((p.heads + p.run - 1) / p.run) < 8 * (int64_t)n_sm) p.run = (p.run + 1) / 2;
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
