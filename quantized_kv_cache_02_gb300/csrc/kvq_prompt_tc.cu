// Prompt attention on the fifth-generation tensor cores: bf16, head_dim 64 or
// 128 (kvq_prompt_attention).
//
// A row is a (token, query head) pair of one KV head, token major: the heads
// that share a KV head share its Key and Value tiles and the causal boundary.
// A CTA holds two tiles of 128 rows (floor(128 / g) tokens each) and walks the
// keys in blocks of 128, both tiles on the same Key and Value tile:
//
//   S_i = Q_i K^T       128 x 128, fp32 in tensor memory (Q, K from shared memory)
//   P_i = 2^(S_i c - m) bf16, in tensor memory
//   O_i += P_i V        128 x d, fp32 in tensor memory (P from tensor memory)
//
// Warps 0-3 and 4-7 run the softmax of tile 0 and 1, one row a thread, so
// maxima and sums need no exchange; warp 8 issues the MMAs, warp 9 the TMA
// copies, and with 10 and 11 it cleans the Values that some row does not see.
// At d = 128 tensor memory holds S, with P over it, and O: the tiles alternate,
// one's MMAs run under the other's softmax.  At d = 64 P has columns of its own,
// S_i is free once its rows are in registers, and the next block's Q K^T runs
// under the same tile's softmax too.
//
// Bound at d = 128: the MMAs, 2048 cycles for two tiles and a block, measured
// some 2600 with the waits between them: 4096 tokens of 32/8 heads 96 us (1.43
// PFLOP/s), 16384 tokens 1.27 ms (1.73 PFLOP/s, what a library product sustains at
// the power limit).  At d = 64 the softmax: 256 exponentials a scheduler for a
// block, measured some 2400 cycles with the maxima, sums and conversions.  Tried:
// the block's maximum beside the first half's exponentials (105 us for 4096
// tokens), half a row a thread on sixteen warps (113 us; at d = 64 30 us where 27
// are taken), a MMA warp a tile (116 us: the tiles fall into step).
//
// P is rounded to bf16 because V is bf16 and an MMA takes operands of one type: a
// second MMA on what the rounding leaves would double the P V.  It is off by at
// most 2^-8 of each weight, as the output's own rounding is of the output: against
// 64 bits the output is off by 2.1e-3 where fp32 weights leave 1.7e-3 (4096
// tokens).  The sum l, and lse with it, takes the weights before that rounding.
//
// One pass with a running maximum and sum is Milakov and Gimelshein's ("Online
// normalizer calculation for softmax", 2018).  Here the maximum moves only when a
// score passes it by 2^8, a published refinement, so O is rescaled rarely and by
// the softmax threads themselves.  A maximum that lags scales all terms of a row by
// one factor of at most 2^8: the relative roundings stay as they are, and 8 bits of
// the exponent's range go (kvq.h on the size of Values).
// ("KV Cache 与自回归视频生成", softmax(Q K^T / sqrt(d) + M) V.)

#include <cfloat>

#include "kvq_prompt.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kMmaWarp = 8, kCopyWarp = 9, kTcThreads = 384;
// Registers a thread after the split of the launch's 3 x 168: a softmax thread
// holds a whole row of scores.
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr float kSlack = 8.f;

template <int D>
struct TcLayout {
  static constexpr int kSlots = D == 128 ? 2 : 4;         // (V_j, K_j+1) pairs in flight
  static constexpr uint32_t kChunk = 128 * 128;           // 128 rows of 64 channels
  static constexpr uint32_t kTile = kChunk * (D / 64);    // a Q, K or V tile
  static constexpr uint32_t kQ = 0, kK0 = 2 * kTile, kRing = 3 * kTile, kBars = kRing + 2 * kSlots * kTile;
  // barriers: full and empty per slot, K_0, cleaned Values (two), then per tile: Q, S, P (two halves), O, S read
  static constexpr int kNBars = 2 * kSlots + 3 + 12;
  static constexpr bool kApart = D == 64;                 // P beside S, not over it
  static constexpr size_t kSmem = kBars + kNBars * 8 + 32 + 1024;  // + alignment
  // S_i at 128 i, O_i at 256 + D i, P_i over S_i or at 384 + 64 i
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = kApart ? 384 : 0, kStepP = kApart ? 64 : 128;
};

__device__ __forceinline__ __nv_bfloat162 times_zero(uint32_t w, __nv_bfloat162 sum) {
  return __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w), __nv_bfloat162{}, sum);
}

// The infinities and NaN that were taken out, to the rows that see them: a weight
// times one is one.  (By the softmax warps; all rows have been written.)
template <int D>
__device__ __forceinline__ void give_back(const PromptParams& p, int si, int h, int level) {
  const PromptSeq sq = p.tiles.seq[si];
  const int tok0 = level * p.tiles.step, end = min(sq.len, tok0 + p.tiles.step), lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < (end - tok0) * p.g; r += kMmaWarp) {
    const int pos = tok0 + r / p.g;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (int64_t)(sq.start + pos) * p.o_ts +
                         (int64_t)(h * p.g + r % p.g) * p.o_hs;
    for (int c = lane; c < D; c += 32) {
      float o = __bfloat162float(dst[c]);
      for (int key = tok0 + 1; key <= pos; ++key) {
        const float x = __bfloat162float(
            static_cast<const __nv_bfloat16*>(p.v)[(int64_t)(sq.start + key) * p.v_ts + (int64_t)h * p.v_hs + c]);
        if (!isfinite(x)) o += x;
      }
      dst[c] = __float2bfloat16(o);
    }
  }
}

struct TcMaps {
  CUtensorMap q, k, v;
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    prompt_tc_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ TcMaps maps) {
  using L = TcLayout<D>;
  extern __shared__ uint8_t tc_raw[];
  uint8_t* smem = tc_raw + ((1024u - (smem_u32(tc_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t bar_full = sbase + L::kBars, bar_empty = bar_full + 8 * L::kSlots;
  const uint32_t bar_k0 = bar_empty + 8 * L::kSlots, bar_clean = bar_k0 + 8, bar_q = bar_clean + 16, bar_s = bar_q + 16,
                 bar_p = bar_s + 16, bar_o = bar_p + 32, bar_r = bar_o + 16;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::kBars + 8 * L::kNBars);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  volatile int* dirty = abort + 1;  // then the tile, kept here and not in registers

  int si, h, level;
  prompt_tile(p.tiles, blockIdx.x, &si, &h, &level);
  const PromptSeq sq = p.tiles.seq[si];
  const int tile_tok = p.tiles.step / 2;            // tokens of a tile
  const int tok0 = level * p.tiles.step;            // of tile 0
  // key blocks of each tile: through its last token
  const int end0 = min(sq.len, tok0 + tile_tok), end1 = min(sq.len, tok0 + 2 * tile_tok);
  const int n0 = (end0 + kKeys - 1) / kKeys, n1 = tok0 + tile_tok < sq.len ? (end1 + kKeys - 1) / kKeys : 0;
  const int nmax = max(n0, n1);
  // A weight of 0 does not silence an infinite or NaN Value.  Blocks from
  // ``own`` on (two at most) hold Values that some row does not see: later
  // tokens', whose infinities and NaN are taken out and given back at the end to
  // the rows that see them, and in a last k-step of 16 other sequences', cleared.
  const int own = tok0 / kKeys;

  // the copies: Q_0, K_0, Q_1, then the pairs V_j, K_j+1
  auto load_q = [&](int i) {
    bar_expect(bar_q + 8 * i, (uint32_t)(tile_tok * p.g) * 128u * (D / 64));
    for (int c = 0; c < D / 64; ++c)
      tma_load3(sbase + L::kQ + i * L::kTile + c * L::kChunk, &maps.q, 64 * c, h * p.g, sq.start + tok0 + i * tile_tok,
                bar_q + 8 * i);
  };
  auto load_kv = [&](const CUtensorMap* m, uint32_t dst, int blk, uint32_t bar) {
    for (int c = 0; c < D / 64; ++c)
      tma_load3(sbase + dst + c * L::kChunk, m, 64 * c, sq.start + blk * kKeys, h, bar);
  };
  auto load_pair = [&](int j) {
    const int s = j % L::kSlots;
    const bool more = j + 1 < nmax;
    bar_expect(bar_full + 8 * s, L::kTile * (more ? 2 : 1));
    load_kv(&maps.v, L::kRing + 2 * s * L::kTile, j, bar_full + 8 * s);
    if (more) load_kv(&maps.k, L::kRing + (2 * s + 1) * L::kTile, j + 1, bar_full + 8 * s);
  };

  if (warp == kMmaWarp) tm_alloc<512>(smem_u32(tslot));
  if (t == 32 * kCopyWarp) {
    // the first copies fly while the rest of the CTA sets up
    *abort = 0;
    *dirty = 0;
    dirty[1] = si;
    dirty[2] = h;
    dirty[3] = level;
    for (int s = 0; s < L::kSlots; ++s) {
      bar_init(bar_full + 8 * s, 1);
      bar_init(bar_empty + 8 * s, 1);
    }
    bar_init(bar_k0, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(bar_clean + 8 * i, 3);
      bar_init(bar_q + 8 * i, 1);
      bar_init(bar_s + 8 * i, 1);
      bar_init(bar_p + 16 * i, 4);  // a warp arrives once, by one lane
      bar_init(bar_p + 16 * i + 8, 4);
      bar_init(bar_o + 8 * i, 1);
      bar_init(bar_r + 8 * i, 4);
    }
    bar_init_fence();
    pdl_wait();
    load_q(0);
    bar_expect(bar_k0, L::kTile);
    load_kv(&maps.k, L::kK0, 0, bar_k0);
    if (n1 > 0) load_q(1);
    for (int j = 0; j < min(nmax, L::kSlots); ++j) load_pair(j);
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *tslot;
  pdl_wait();
  pdl_release();

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    int issued = 0;
    if (warp == kCopyWarp) {
      // ============ copies (lane 0) ==================================================
      issued = min(nmax, L::kSlots);
      if (lane == 0) {
        for (; issued < nmax; ++issued) {
          if (!bar_wait(bar_empty + 8 * (issued % L::kSlots), (uint32_t)(issued / L::kSlots - 1) & 1u, abort)) {
            *abort = 1;
            if (p.status) atomicOr(p.status, kStatusPromptTimeout);
            break;
          }
          load_pair(issued);
        }
      }
      issued = __shfl_sync(0xffffffffu, issued, 0);
      // nothing in flight when the CTA ends
      for (int x = max(0, issued - L::kSlots); x < min(issued, own); ++x)
        bar_drain(bar_full + 8 * (x % L::kSlots), (uint32_t)(x / L::kSlots) & 1u);
    }
    if (warp >= kCopyWarp) {
      // ============ Values that some row does not see (keys past tok0 that a k-step
      // of a tile covers), by the three warps that issue no MMA, under the softmax: the
      // check costs 0.7 us of a short call, nothing at 4096 tokens.  (After an early
      // stop this runs on whatever is there.)
      for (int j = own; j < nmax; ++j) {
        if (warp == kCopyWarp && j < issued) bar_drain(bar_full + 8 * (j % L::kSlots), (uint32_t)(j / L::kSlots) & 1u);
        asm volatile("bar.sync 1, 96;" ::: "memory");  // the copy warp has seen it land
        const int mine = t - 32 * kCopyWarp;
        uint8_t* v = smem + L::kRing + 2 * (j % L::kSlots) * L::kTile;
        const int len = min(sq.len - j * kKeys, kKeys), first = max(0, tok0 + 1 - j * kKeys);
        const int last = min(len, ((n1 > 0 ? end1 : end0) - j * kKeys + 15) & ~15);
        __nv_bfloat162 sum[2] = {};  // NaN once an infinity or a NaN came
        for (int c = 0; c < D / 64; ++c) {
          uint4* rows = reinterpret_cast<uint4*>(v + c * L::kChunk);
          for (int x = 8 * len + mine; x < 8 * ((len + 15) & ~15); x += 96) rows[x] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
          for (int x = 8 * first + mine; x < 8 * last; x += 96) {
            const uint4 w = rows[x];
            sum[0] = times_zero(w.x, sum[0]);
            sum[1] = times_zero(w.y, sum[1]);
            sum[0] = times_zero(w.z, sum[0]);
            sum[1] = times_zero(w.w, sum[1]);
          }
        }
        const float2 any = __bfloat1622float2(__hadd2(sum[0], sum[1]));
        if (any.x + any.y != 0.f) {
          auto finite = [](uint32_t w) {
            return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) |
                   ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
          };
          for (int c = 0; c < D / 64; ++c) {
            uint32_t* words = reinterpret_cast<uint32_t*>(v + c * L::kChunk);
#pragma unroll 1
            for (int x = 8 * first + mine; x < 8 * last; x += 96)
#pragma unroll 1
              for (int y = 0; y < 4; ++y) words[4 * x + y] = finite(words[4 * x + y]);
          }
          *dirty = 1;
        }
        async_proxy_fence();
        warp_arrive(bar_clean + 8 * (j - own));
      }
      if (warp == kCopyWarp) {
        bar_drain(bar_k0, 0);
        bar_drain(bar_q, 0);
        if (n1 > 0) bar_drain(bar_q + 8, 0);
      }
    } else {
      // ============ MMAs, all issued by one lane ======================================
      // With P over S, Q K^T of the next block overwrites P right behind the P V
      // that reads it.  They have different accumulators, for which the instruction
      // set promises no order by itself: a tcgen05.fence between them, which orders
      // the asynchronous tcgen05 instructions before it ahead of those behind it.
      // The arrival for S_j then also says that the P V of block j - 1 is done.  With
      // P apart, O's barrier says so, once a block.  (For 4096 tokens the fence takes
      // nothing, a wait for the P V's completion 9 us of 104, and one S that the tiles
      // share beside two P 14 us of 110.)
      constexpr uint32_t idesc_s = bf16_idesc(kRows, kKeys, false), idesc_o = bf16_idesc(kRows, D, true);
      const bool one = elect_one();
      auto scores = [&](int i, uint32_t kaddr) {
        const uint64_t a = sw128_desc(sbase + L::kQ + i * L::kTile, 0), b = sw128_desc(kaddr, 0);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks / 4) * (L::kChunk >> 4) + (ks % 4) * 2;
          if (one) mma_ss(tm + L::kColS + 128 * i, a + off, b + off, idesc_s, ks > 0);
        }
        if (one) mma_commit(bar_s + 8 * i);
      };
      auto landed = [&](int j) -> bool {
        return bar_wait(bar_full + 8 * (j % L::kSlots), (uint32_t)(j / L::kSlots) & 1u, abort);
      };
      bool ok = bar_wait(bar_k0, 0, abort) && bar_wait(bar_q, 0, abort);
      if (ok) scores(0, sbase + L::kK0);
      if (ok && n1 > 0) {
        ok = bar_wait(bar_q + 8, 0, abort);
        if (ok) scores(1, sbase + L::kK0);
      }
      if (ok) ok = landed(0);
      for (int j = 0; j < nmax && ok; ++j) {
        const int s = j % L::kSlots;
        const uint32_t vaddr = sbase + L::kRing + 2 * s * L::kTile, kaddr = vaddr + L::kTile;
        if (L::kApart) {
          for (int i = 0; i < 2 && ok; ++i) {
            if (j + 1 >= (i ? n1 : n0)) continue;
            if (!(ok = bar_wait(bar_r + 8 * i, (uint32_t)j & 1u, abort))) break;
            tm_fence_after();
            scores(i, kaddr);
          }
        }
        for (int i = 0; i < 2 && ok; ++i) {
          const int ni = i ? n1 : n0;
          if (j >= ni) continue;
          const uint64_t b = sw128_desc(vaddr, L::kChunk);
          const int steps = min(8, ((i ? end1 : end0) - j * kKeys + 15) / 16);
          auto values = [&](int ks) {
            if (one) mma_ts(tm + L::kColO + D * i, tm + L::kColP + L::kStepP * i + 8 * ks, b + ks * (2048 >> 4), idesc_o,
                            j > 0 || ks > 0);
          };
          if (!(ok = bar_wait(bar_p + 16 * i, (uint32_t)j & 1u, abort))) break;
          if (j >= own && !(ok = bar_wait(bar_clean + 8 * (j - own), 0, abort))) break;
          tm_fence_after();
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            if (ks < steps) values(ks);
          if (!(ok = bar_wait(bar_p + 16 * i + 8, (uint32_t)j & 1u, abort))) break;
          tm_fence_after();
#pragma unroll
          for (int ks = 4; ks < 8; ++ks)
            if (ks < steps) values(ks);
          if (one && (L::kApart || j + 1 == ni)) mma_commit(bar_o + 8 * i);
          // the next pair's wait passes while MMAs are queued
          if (i == (n1 > 0) && j + 1 < nmax) ok = landed(j + 1);
          if (!L::kApart && j + 1 < ni) {
            tm_fence_before();
            scores(i, kaddr);
          }
        }
        if (ok && one) mma_commit(bar_empty + 8 * s);
      }
      if (!ok) {
        // stopped early: nothing in flight when the CTA ends (bar_k0's one phase is over, unless K_0 never came)
        *abort = 1;
        if (one) {
          if (p.status) atomicOr(p.status, kStatusPromptTimeout);
          mma_commit(bar_k0);
          bar_drain(bar_k0, 1);
        }
      }
    }
  } else {
    // ============ softmax: tile i, one row a thread ===================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2, r = t & 127;
    const int n = i ? n1 : n0;
    const int tt = r / p.g, pos = tok0 + i * tile_tok + tt;
    const bool live = tt < tile_tok && pos < sq.len;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tm + L::kColS + 128 * i + lanes, to = tm + L::kColO + D * i + lanes,
                   tp = tm + L::kColP + L::kStepP * i + lanes;
    const float2 sc = make_float2(p.scale2, p.scale2);
    float m = -FLT_MAX, l = 0.f;  // (not -INFINITY: scores of minus infinity may come first)
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!(ok = warp_wait(bar_s + 8 * i, (uint32_t)j & 1u, abort))) break;
      if (warp_live) {
        tm_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tm_ld32(ts + 32 * c, s + 32 * c);
        tm_wait_ld();
        if (L::kApart) {
          tm_fence_before();
          warp_arrive(bar_r + 8 * i);
        }
        const int limit = pos - j * kKeys;  // the last key of the block this row sees
        if (__any_sync(0xffffffffu, limit < kKeys - 1)) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > limit) s[c] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[c + e], s[c + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[124 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale2;
        const bool up = top > m + kSlack;
        if (L::kApart && j > 0) {  // the last block's P V is done with P and with O
          if (!(ok = warp_wait(bar_o + 8 * i, (uint32_t)(j - 1) & 1u, abort))) break;
          tm_fence_after();
        }
        if (__any_sync(0xffffffffu, up)) {
          const float a = up ? ex2(m - top) : 1.f;
          if (up) m = top;
          l *= a;
          if (j > 0) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tm_ld32(to + 32 * c, o);
              tm_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= a;
              tm_st32(to + 32 * c, o);
            }
          }
        }
        const float2 nm = make_float2(-m, -m);
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 128; c += 64) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float2 x = fma2(make_float2(s[c + e], s[c + e + 1]), sc, nm);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum[(e >> 1) & 3] = add2(sum[(e >> 1) & 3], x);
            w[e / 2] = pack_bf16(x.x, x.y);
          }
          tm_st32(tp + c / 2, reinterpret_cast<const float*>(w));
          tm_wait_st();
          tm_fence_before();
          if (c == 0) warp_arrive(bar_p + 16 * i);  // the first 64 keys' weights: their P V may start
        }
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
      } else {
        if (L::kApart) {
          // like the others, so that no arrival counts for the block before
          warp_arrive(bar_r + 8 * i);
          if (j > 0 && !(ok = warp_wait(bar_o + 8 * i, (uint32_t)(j - 1) & 1u, abort))) break;
        }
        warp_arrive(bar_p + 16 * i);
      }
      warp_arrive(bar_p + 16 * i + 8);
    }
    if (ok && n > 0) ok = warp_wait(bar_o + 8 * i, L::kApart ? (uint32_t)(n - 1) & 1u : 0u, abort);
    if (!ok) {
      *abort = 1;
      if (p.status && lane == 0) atomicOr(p.status, kStatusPromptTimeout);
    } else if (n > 0 && warp_live) {
      tm_fence_after();
      const float inv = 1.f / l;
      const int head = h * p.g + r - tt * p.g;
      __nv_bfloat16* dst =
          static_cast<__nv_bfloat16*>(p.out) + (int64_t)(sq.start + pos) * p.o_ts + (int64_t)head * p.o_hs;
      // through the tile's Q buffer (no MMA reads it any more), 16-byte pieces
      // swizzled by row, so that the warp stores whole rows: one row a thread
      // took a memory transaction a piece, 2 us a CTA
      constexpr int kPieces = D / 8;
      uint8_t* stage = smem + L::kQ + i * L::kTile + (warp & 3) * 32 * (2 * D);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tm_ld32(to + 32 * c, o);
        tm_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4*>(stage + lane * (2 * D) + ((4 * c + e / 8) ^ (lane & (kPieces - 1))) * 16) =
              make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                         pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
      }
      __syncwarp();
      const uint32_t rows_live = __ballot_sync(0xffffffffu, live);
#pragma unroll 4
      for (int x = lane; x < 32 * kPieces; x += 32) {
        const int row = x / kPieces, c = x % kPieces;
        const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), row);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + row * (2 * D) + (c ^ (row & (kPieces - 1))) * 16);
        if (rows_live >> row & 1u) *reinterpret_cast<uint4*>(at + 16 * c) = v;
      }
      if (live && p.lse)
        p.lse[(int64_t)head * p.n_tokens + sq.start + pos] = (m + log2f(l)) * 0.69314718055994530942f;
    }
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    tm_free<512>(tm);
  }
  if (warp < kMmaWarp && *dirty) give_back<D>(p, dirty[1], dirty[2], dirty[3]);
}

template <int D>
cudaError_t launch_tc(const PromptParams& p, const TcMaps& maps, int64_t tiles, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)TcLayout<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_tc_kernel<D>, dim3((unsigned)tiles), dim3(kTcThreads), TcLayout<D>::kSmem, s, p, maps);
}

}  // namespace

int prompt_tc_tokens(int g) { return 2 * (kRows / g); }

cudaError_t launch_prompt_tc(const PromptParams& p, int64_t tiles, cudaStream_t s) {
  TcMaps maps;
  // dims (channel, head, token) for the queries, (channel, token, head) for Keys and Values
  if (!tma_map3(&maps.q, p.q, p.D, p.Hq, p.n_tokens, p.q_hs, p.q_ts, p.g, kRows / p.g) ||
      !tma_map3(&maps.k, p.k, p.D, p.n_tokens, p.Hkv, p.k_ts, p.k_hs, kKeys, 1) ||
      !tma_map3(&maps.v, p.v, p.D, p.n_tokens, p.Hkv, p.v_ts, p.v_hs, kKeys, 1))
    return cudaErrorInvalidValue;
  return p.D == 128 ? launch_tc<128>(p, maps, tiles, s) : launch_tc<64>(p, maps, tiles, s);
}

}  // namespace kvq
