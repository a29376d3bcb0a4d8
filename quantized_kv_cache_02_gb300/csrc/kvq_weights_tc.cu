// Gathered prompt weights on the fifth-generation tensor cores: bf16, head_dim
// 64 or 128 (kvq_prompt_weights).
//
//   w_j = sum over the counted rows r of 2^(s_jr - L_r),  s_jr = k_j . q_r log2(e) / sqrt(d)
//
// A row r is a (token, query head) pair of the KV head, token major; a query
// tile is 128 rows (floor(128 / g) tokens).  Keys are the M side of the MMA,
//
//   S^T = K Q^T    128 keys x 128 rows, fp32 in tensor memory,
//
// so a thread owns one key and its sum never leaves a register.  A CTA takes
// pairs of key tiles: warps 0-3 sum the first, warps 4-7 the second, and both
// use every query tile that arrives.  Each key tile has its own MMA warp, so
// MMAs, exponentials and the waits overlap.  With few
// counted queries (at most two tiles) the query tiles stay in shared memory
// and a run of pairs streams past them; else a CTA has one pair, which stays
// while the queries stream.  ``split`` CTAs of a cluster take a pair's query
// tiles in turn and rank 0 adds their sums in rank order, so a short prompt
// fills the GPU and the result has the same bits every time.
//
// The row's L_r enters in the MMA: one more k-step of 16 takes it off every
// score, as four bf16 pieces against a column of ones, so an element costs one
// multiplication, one exponential and one addition, and no load of its own.
// (Read per column from shared memory instead, the loads took the bandwidth that
// the MMAs' operands need: 123 us, then 80 us, for 4096 whole tokens, 32/8 heads
// of 128; 63 us with a MMA warp a tile and no more CTAs a pair than fill the SMs.)
//
// A score is two sums, over the first and the last half of the channels, added by
// the thread: the tensor cores round every accumulation toward zero, by more the
// larger the sum, and four steps of half the size lose less than half of eight.
// It adds them before anything else, so both buffers fill with the next tile's
// during this one's exponentials.  It took 12 of the 75 us of 4096 whole tokens
// and on one input the error there from 1.6e-6 to 1.0e-6 of the weights; a running
// sum over the tiles that keeps what it rounds off, no longer, to 0.5e-6.  Over ten
// inputs it is 0.44e-6 to 0.9e-6 (the sums' mean off by at most 1.5e-7) where sums in
// fp32 throughout are at 0.27e-6 to 0.46e-6 and their single weights up to 6e-6 off
// (here 2.2e-6).
//
// Bound: per pair and query tile 9/8 of 1024 cycles of MMA and 1024 of
// exponentials on each scheduler; measured, some 1800: a scheduler's two summing
// warps also read 256 columns of tensor memory each, 512 cycles, and hide little of
// that under the other's exponentials.
// ("KV Cache 与自回归视频生成", softmax(Q K^T / sqrt(d) + M).)

#include <algorithm>
#include <type_traits>

#include "kvq_prompt.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kKeys = 128, kRows = 128;
constexpr int kMmaWarp = 8, kCopyWarp = 10, kWThreads = 384;  // MMA warps 8 and 9; 11 only fills the warpgroup
constexpr int kSumRegs = 216, kOtherRegs = 72;              // a thread, out of the launch's 3 x 168
constexpr int kQStages = 4, kStayTiles = 2;

template <int D>
struct WLayout {
  static constexpr uint32_t kChunk = 128 * 128;
  static constexpr uint32_t kTile = kChunk * (D / 64);
  // what streams, and what stays: two key pairs past two query tiles, or four query tiles past one key pair
  static constexpr uint32_t kStream = 0, kStay = 4 * kTile;
  // the last k-step's operands, 8 rows x 16 bytes a core matrix: columns 0-7 of
  // -L per query tile and of ones, and the zeros of columns 8-15 of both
  static constexpr uint32_t kL = kStay + 2 * kTile, kOnes = kL + kQStages * 2048, kZero = kOnes + 2048;
  static constexpr uint32_t kRed = kZero + 2048;                 // [8 ranks][256 keys]
  static constexpr uint32_t kBars = kRed + 8 * 256 * 4;
  // K full / empty (2 each), Q full / empty, S full / empty (tile, half of the channels)
  static constexpr int kNBars = 4 + 2 * kQStages + 8;
  static constexpr size_t kSmem = kBars + kNBars * 8 + 16 + 1024;
};

struct WMaps {
  CUtensorMap q, k;
};

template <int D>
__global__ void __launch_bounds__(kWThreads, 1)
    weights_tc_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ WMaps maps) {
  using L = WLayout<D>;
  extern __shared__ uint8_t w_raw[];
  uint8_t* smem = w_raw + ((1024u - (smem_u32(w_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t bar_kf = sbase + L::kBars, bar_ke = bar_kf + 16, bar_qf = bar_ke + 16,
                 bar_qe = bar_qf + 8 * kQStages, bar_sf = bar_qe + 8 * kQStages, bar_se = bar_sf + 32;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::kBars + 8 * L::kNBars);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);

  int si, h, level;
  const int rank = blockIdx.x % p.split;  // clusters are ``split`` CTAs in a row
  prompt_tile(p.tiles, blockIdx.x / p.split, &si, &h, &level);
  const PromptSeq sq = p.tiles.seq[si];
  const int run0 = (prompt_blocks(sq.len, p.tiles.step) - 1 - level) * p.tiles.step;  // first key
  const int pairs = min(p.tiles.step / (2 * kKeys), (sq.len - run0 + 2 * kKeys - 1) / (2 * kKeys));
  const int tile_tok = kRows / p.g;
  const int tok0 = (int)max((int64_t)0, sq.len - p.last);  // first counted token
  const int nq = (sq.len - tok0 + tile_tok - 1) / tile_tok;
  const bool resident = p.split == 1 && nq <= kStayTiles;
  auto k_tile = [&](int pr, int w) { return (resident ? L::kStream + 2 * (pr & 1) * L::kTile : L::kStay) + w * L::kTile; };
  auto q_tile = [&](int s) { return (resident ? L::kStay : L::kStream) + s * L::kTile; };
  // the first query tile that sees a key of the pair; this CTA takes every split-th from there
  auto q_first = [&](int pair) {
    const int key = run0 + pair * 2 * kKeys;
    return (resident || key < tok0 ? 0 : (key - tok0) / tile_tok) + rank;
  };

  // the copies: key pairs and query tiles
  auto load_pair = [&](int pr) {
    const int s = pr & 1, key = run0 + pr * 2 * kKeys, both = key + kKeys < sq.len;
    bar_expect(bar_kf + 8 * s, L::kTile * (both ? 2 : 1));
    for (int w = 0; w < 1 + both; ++w)
      for (int c = 0; c < D / 64; ++c)
        tma_load3(sbase + k_tile(pr, w) + c * L::kChunk, &maps.k, 64 * c, sq.start + key + w * kKeys, h, bar_kf + 8 * s);
  };
  auto load_q = [&](int i, int s) {
    bar_expect(bar_qf + 8 * s, (uint32_t)(tile_tok * p.g) * 128u * (D / 64));
    for (int c = 0; c < D / 64; ++c)
      tma_load3(sbase + q_tile(s) + c * L::kChunk, &maps.q, 64 * c, h * p.g, sq.start + tok0 + i * tile_tok,
                bar_qf + 8 * s);
  };
  // those that wait for nothing: the first pair's query tiles that have a stage, and the pairs that have a place
  const int q_early = max(0, min(kQStages, (nq - q_first(0) + p.split - 1) / p.split));
  const int k_early = min(pairs, resident ? 2 : 1);

  if (warp == kMmaWarp) tm_alloc<512>(smem_u32(tslot));
  if (t == 32 * kCopyWarp) {
    // they fly while the rest of the CTA sets up
    *abort = 0;
    for (int i = 0; i < 2; ++i) {
      bar_init(bar_kf + 8 * i, 1);
      bar_init(bar_ke + 8 * i, 2);  // both MMA warps
    }
    for (int i = 0; i < kQStages; ++i) {
      bar_init(bar_qf + 8 * i, 2);  // the copy, and the warp that wrote -L
      bar_init(bar_qe + 8 * i, 2);  // both MMA warps
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(bar_sf + 8 * i, 1);
      bar_init(bar_se + 8 * i, 4);  // a warp arrives once, by one lane
    }
    bar_init_fence();
    pdl_wait();
    for (int pr = 0; pr < k_early; ++pr) load_pair(pr);
    for (int x = 0; x < q_early; ++x) load_q(q_first(0) + x * p.split, x);
  }
  if (t < 256) {
    *reinterpret_cast<uint4*>(smem + L::kOnes + t * 16) =
        t < 128 ? make_uint4(0x3f803f80u, 0x3f803f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    async_proxy_fence();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *tslot;
  if (p.split > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_release();

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kCopyWarp) {
      // ============ copies; the lanes turn lse into -L =================================
      // the lane's four rows of a tile: their first tile's lse and how many tokens come before the sequence's end
      // (worked out once: this warp shares its scheduler with two of the summing warps)
      const float* src[4];
      int room[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 32 * e + lane, tt = r / p.g;
        src[e] = p.lse + (int64_t)(h * p.g + r - tt * p.g) * p.n_tokens + sq.start + tok0 + tt;
        room[e] = tt < tile_tok ? sq.len - tok0 - tt : 0;
      }
      float ahead[4];
      int ahead_tile = -1;
      auto fetch_lse = [&](int i) {
        const int at = i * tile_tok;
#pragma unroll
        for (int e = 0; e < 4; ++e) ahead[e] = at < room[e] ? src[e][at] : 0.f;
        ahead_tile = i;
      };
      int issued = 0;
      bool go = true;
      auto give_q = [&](int i, int then) {  // tile i; its successor's lse is fetched under it
        const int s = issued % kQStages;
        if (issued >= q_early) {
          if (!(go = warp_wait(bar_qe + 8 * s, (uint32_t)(issued / kQStages - 1) & 1u, abort))) return;
          if (lane == 0) load_q(i, s);
        }
        if (ahead_tile != i) fetch_lse(i);
        float now[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) now[e] = ahead[e];
        if (then >= 0) fetch_lse(then);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // -L = -lse * lse_hi - lse * lse_lo, cut into four pieces of 8 bits; an infinity is one piece
          const float hi = __fmul_rn(-now[e], p.lse_hi), b0 = __bfloat162float(__float2bfloat16_rn(hi));
          const bool whole = !(fabsf(b0) < INFINITY);
          const float rest = whole ? 0.f : fmaf(-now[e], p.lse_hi, -hi) - now[e] * p.lse_lo;
          const float left = whole ? 0.f : hi - b0;
          const float b1 = __bfloat162float(__float2bfloat16_rn(left)), last = left - b1 + rest;
          const float b2 = __bfloat162float(__float2bfloat16_rn(last));
          *reinterpret_cast<uint4*>(smem + L::kL + s * 2048 + (32 * e + lane) * 16) =
              make_uint4(pack_bf16(b0, b1), pack_bf16(b2, last - b2), 0u, 0u);
        }
        async_proxy_fence();
        warp_arrive(bar_qf + 8 * s);
        ++issued;
      };
      int kpairs = k_early;
      for (int pr = 0; pr < pairs && go; ++pr) {
        if (pr >= k_early) {
          if (!(go = warp_wait(bar_ke + 8 * (pr & 1), (uint32_t)(pr / 2 - 1) & 1u, abort))) break;
          if (lane == 0) load_pair(pr);
          ++kpairs;
        }
        if (pr == 0 || !resident)
          for (int i = q_first(pr); i < nq && go; i += p.split) give_q(i, i + p.split < nq ? i + p.split : -1);
      }
      if (!go) {
        *abort = 1;
        if (p.status && lane == 0) atomicOr(p.status, kStatusPromptTimeout);
        for (; issued < q_early; ++issued) warp_arrive(bar_qf + 8 * issued);  // complete but for the copy
      }
      // nothing in flight when the CTA ends
      for (int x = max(0, kpairs - 2); x < kpairs; ++x) bar_drain(bar_kf + 8 * (x & 1), (uint32_t)(x / 2) & 1u);
      for (int x = max(0, issued - kQStages); x < issued; ++x)
        bar_drain(bar_qf + 8 * (x % kQStages), (uint32_t)(x / kQStages) & 1u);
    } else if (warp < kCopyWarp) {
      // ============ MMAs of key tile w, issued by one lane ==============================
      // a warp a tile: one waits while the other issues
      const bool one = elect_one();
      constexpr uint32_t idesc = bf16_idesc(kKeys, kRows, false);
      const int w = warp - kMmaWarp;
      int taken = 0, n_s = 0;
      bool ok = true;
      for (int pr = 0; pr < pairs && ok; ++pr) {
        const bool active = run0 + (2 * pr + w) * kKeys < sq.len;
        ok = bar_wait(bar_kf + 8 * (pr & 1), (uint32_t)(pr / 2) & 1u, abort);
        for (int i = q_first(pr); i < nq && ok; i += p.split) {
          const int s = resident ? i : taken % kQStages;
          ok = bar_wait(bar_qf + 8 * s, resident ? 0u : (uint32_t)(taken / kQStages) & 1u, abort);
          ++taken;
          if (ok && active) {
            const uint64_t da = sw128_desc(sbase + k_tile(pr, w), 0), db = sw128_desc(sbase + q_tile(s), 0);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int b = 2 * w + half;
              if (n_s > 0 && !(ok = bar_wait(bar_se + 8 * b, (uint32_t)(n_s - 1) & 1u, abort))) break;
              tm_fence_after();
#pragma unroll
              for (int ks = half * D / 32; ks < (half + 1) * D / 32; ++ks) {
                const uint32_t off = (ks / 4) * (L::kChunk >> 4) + (ks % 4) * 2;
                if (one) mma_ss(tm + 128 * b, da + off, db + off, idesc, ks > half * D / 32);
              }
              if (one && half)
                mma_ss(tm + 128 * b, plain_desc(sbase + L::kOnes, 2048),
                       plain_desc(sbase + L::kL + s * 2048, L::kZero - L::kL - s * 2048), idesc, 1);
              if (one) mma_commit(bar_sf + 8 * b);
            }
            if (!ok) break;
            ++n_s;
          }
          if (ok && one && !resident) mma_commit(bar_qe + 8 * s);
        }
        if (one) mma_commit(bar_ke + 8 * (pr & 1));
      }
      if (!ok) {
        *abort = 1;
        if (one && p.status) atomicOr(p.status, kStatusPromptTimeout);
      }
      // nothing in flight when the CTA ends
      for (int half = 0; half < 2 && n_s > 0; ++half) bar_drain(bar_sf + 8 * (2 * w + half), (uint32_t)(n_s - 1) & 1u);
    }
  } else {
    // ============ sums: key tile w, one key a thread ==================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int w = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float2 sc = make_float2(p.scale2, p.scale2);
    int n_s = 0;
    bool ok = true;
    for (int pr = 0; pr < pairs && ok; ++pr) {
      const int tile_key = run0 + pr * 2 * kKeys + w * kKeys, key = tile_key + (t & 127);
      const bool active = tile_key < sq.len;
      RunningSum total[2] = {};
      for (int i = q_first(pr); i < nq && active; i += p.split) {
        const uint32_t parity = (uint32_t)n_s++ & 1u, ts = tm + 256 * w + lanes;
        if (!(ok = warp_wait(bar_sf + 16 * w, parity, abort))) break;
        tm_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tm_ld32(ts + 32 * c, x + 32 * c);
        tm_wait_ld();
        tm_fence_before();
        warp_arrive(bar_se + 16 * w);
        if (!(ok = warp_wait(bar_sf + 16 * w + 8, parity, abort))) break;
        tm_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float y[32];
          tm_ld32(ts + 128 + 32 * c, y);
          tm_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 z = add2(make_float2(x[32 * c + e], x[32 * c + e + 1]), make_float2(y[e], y[e + 1]));
            x[32 * c + e] = z.x;
            x[32 * c + e + 1] = z.y;
          }
        }
        tm_fence_before();
        warp_arrive(bar_se + 16 * w + 8);
        // rows [lo, hi) of the tile count for this key
        const int pos0 = tok0 + i * tile_tok;
        const int lo = max(0, key - pos0) * p.g, hi = min(tile_tok, sq.len - pos0) * p.g;
        const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < kRows);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto add_tile = [&](auto with_mask) {
#pragma unroll
          for (int r = 0; r < kRows; r += 2) {
            float2 y = mul2(make_float2(x[r], x[r + 1]), sc);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            if (decltype(with_mask)::value) {
              y.x = r >= lo && r < hi ? y.x : 0.f;
              y.y = r + 1 >= lo && r + 1 < hi ? y.y : 0.f;
            }
            sum[(r >> 1) & 1] = add2(sum[(r >> 1) & 1], y);
          }
        };
        if (masked) add_tile(std::true_type());
        else add_tile(std::false_type());
        sum[0] = add2(sum[0], sum[1]);
        total[0].add(sum[0].x);
        total[1].add(sum[0].y);
      }
      if (!ok) break;
      const float mine = total[0].sum + total[1].sum;
      if (p.split > 1) {
        // into rank 0's shared memory (one pair a CTA; every rank runs: it arrived)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        uint32_t dst = sbase + L::kRed + (uint32_t)(rank * 256 + t) * 4, remote;
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(dst));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(mine) : "memory");
      } else if (key < sq.len) {
        p.weights[(int64_t)h * p.n_tokens + sq.start + key] = mine;
      }
    }
    if (!ok) {
      *abort = 1;
      if (p.status && lane == 0) atomicOr(p.status, kStatusPromptTimeout);
      if (p.split > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
  }
  __syncwarp();
  if (p.split > 1 && warp >= kMmaWarp) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    tm_free<512>(tm);
  }
  if (p.split > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && t < 2 * kKeys && run0 + t < sq.len) {
      const float* red = reinterpret_cast<const float*>(smem + L::kRed);
      float sum = red[t];
      for (int r = 1; r < p.split; ++r) sum += red[256 * r + t];
      p.weights[(int64_t)h * p.n_tokens + sq.start + run0 + t] = sum;
    }
  }
}

template <int D>
cudaError_t launch_w(const PromptParams& p, const WMaps& maps, int64_t tiles, cudaStream_t s) {
  const size_t smem = WLayout<D>::kSmem;
  const cudaError_t e =
      cudaFuncSetAttribute(weights_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(weights_tc_kernel<D>, tiles, p.split, kWThreads, smem, s, p, maps);
}

}  // namespace

void weights_tc_plan(int64_t pairs, int64_t most_tokens, int g, int n_sm, int* chunk, int* split) {
  *chunk = *split = 1;
  const int64_t tiles = (most_tokens + kRows / g - 1) / (kRows / g);  // query tiles of a pair, at most
  if (tiles <= kStayTiles) {
    *chunk = (int)std::min<int64_t>(1024, std::max<int64_t>(1, (pairs + n_sm - 1) / n_sm));
  } else {
    while (*split < 8 && pairs * *split < n_sm && tiles >= 8 * *split) *split *= 2;
  }
}

cudaError_t launch_weights_tc(const PromptParams& p, int64_t tiles, cudaStream_t s) {
  WMaps maps;
  if (!tma_map3(&maps.q, p.q, p.D, p.Hq, p.n_tokens, p.q_hs, p.q_ts, p.g, kRows / p.g) ||
      !tma_map3(&maps.k, p.k, p.D, p.n_tokens, p.Hkv, p.k_ts, p.k_hs, kKeys, 1))
    return cudaErrorInvalidValue;
  return p.D == 128 ? launch_w<128>(p, maps, tiles, s) : launch_w<64>(p, maps, tiles, s);
}

}  // namespace kvq
