// Cross attention on the fifth-generation tensor cores: bf16, head_dim 64 or 128,
// sequences of many queries (kvq_cross_attention).
//
// A row is a (token, query head) pair of one KV head, token major.  A CTA holds
// two tiles of 128 rows (floor(128 / g) tokens each) and walks the states in blocks
// of 128, both tiles on the same Key and Value tile:
//
//   S_i = Q_i K^T       128 x 128, fp32 in tensor memory (Q, K from shared memory)
//   P_i = 2^(S_i c - m) bf16, in tensor memory
//   O_i += P_i V        128 x d, fp32 in tensor memory (P from tensor memory)
//
// Warps 0-3 and 4-7 run the softmax of tile 0 and 1, one row a thread; warp 8
// issues the MMAs, warp 9 the TMA copies (two more fill the warpgroup, whose registers
// go to the softmax).  Encoders' states are few (a text's 512 are four blocks), so what
// surrounds the blocks counts: the CTAs stay and take item after item, and the ends
// overlap.  The next item's queries and first states are copied while the last
// blocks run, and its first Q K^T follows a tile's last P V at once.  At d = 128 warps
// 12-15 write the outputs under the next item's blocks (14400 tokens over 512 states of
// 32/8 heads 120 -> 111 us, 1.09 PFLOP/s); at d = 64, bound by the softmax, its warps do it
// themselves (they are slower with the registers that four more warps leave them: 2048
// states 171 us, 160 without).
//
// Bound: an item of one block takes 4.9 us (its two tiles' scores, softmax, output and
// copies, one after the other with little under them), a further block 1.5 to 1.7 us: the
// tiles' softmax and MMAs in turn, with 64 KB of Keys and Values an SM out of L2 (6 TB/s).
// Tried: the next queries prefetched into L2 (512 states 115 us), or copied into ring
// slots as they come free, a block or more earlier (114); the next Keys waited for
// earlier (114).
//
// Few items of many states are split over a cluster (p.split CTAs, an equal run of
// blocks each), whose outputs, maxima and sums meet through distributed shared
// memory, in rank order.
// Tensor memory, the running maximum that moves only past 2^8, and what is rounded
// where are as in the causal kernel (kvq_prompt_tc.cu).
// ("KV Cache 与自回归视频生成", softmax(Q K^T / sqrt(d)) V.)

#include <cfloat>

#include "kvq_cluster.cuh"
#include "kvq_prompt.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kMmaWarp = 8, kCopyWarp = 9, kOutWarp = 12;
// Warps that write outputs.
template <int D, bool SPLIT>
constexpr bool kOutWarps = D == 128 && !SPLIT;
// Registers a thread after the split of the launch's 4 x 128 (3 x 168 without output
// warps): a softmax thread holds a whole row of scores.
template <bool OUT>
constexpr int kTcThreads = OUT ? 512 : 384;
template <bool OUT>
constexpr int kSoftmaxRegs = OUT ? 176 : 216;
template <bool OUT>
constexpr int kOtherRegs = OUT ? 88 : 72;
constexpr int kOutRegs = 72;
constexpr float kSlack = 8.f;

// 16 consecutive 32-bit columns of this thread's lane, times a.
__device__ __forceinline__ void tm_scale16(uint32_t at, float a) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
  tm_wait_ld();
#pragma unroll
  for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * a);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <int D>
struct TcLayout {
  static constexpr int kSlots = D == 128 ? 4 : 8;         // Key and Value tiles in flight
  static constexpr uint32_t kChunk = 128 * 128;           // 128 rows of 64 channels
  static constexpr uint32_t kTile = kChunk * (D / 64);    // a Q, K or V tile
  static constexpr uint32_t kStageWarp = 32 * 128;        // 32 rows of 64 output channels
  static constexpr uint32_t kQ = 0, kRing = 2 * kTile, kStage = kRing + kSlots * kTile, kBars = kStage + 8 * kStageWarp;
  static constexpr uint32_t kMl = kStage + 4 * kStageWarp;  // [tile][row] (m, l), behind four output warps' stages
  // barriers: full and empty per slot, the end, then per tile: Q full, Q empty, S, P (two halves), O after a block, S
  // read, O after an item, (m, l) written, O read
  static constexpr int kNBars = 2 * kSlots + 1 + 20;
  static constexpr bool kApart = D == 64;                 // P beside S, not over it
  static constexpr uint32_t kBriefs = kBars + kNBars * 8 + 8;  // behind the tensor memory's address and the abort word
  static constexpr size_t kSmem = kBriefs + 16 + 1024;    // + alignment
  // S_i at 128 i, O_i at 256 + D i, P_i over S_i or at 384 + 64 i
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = kApart ? 384 : 0, kStepP = kApart ? 64 : 128;
};

struct TcMaps {
  CUtensorMap q, k, v;
};

// An item: one KV head of one sequence, the tokens of two tiles.
struct Item {
  CrossSeq seq;
  int head, tok0, n;   // first token of tile 0; blocks of states
  bool two;            // tile 1 has tokens
};

template <bool SPLIT>
__device__ __forceinline__ Item item_at(const CrossParams& p, int x) {
  const Tile t = tile_at(p.tiles, x);
  Item r;
  r.seq = t.seq;
  r.head = t.head;
  r.tok0 = t.level * p.tiles.step;
  r.n = (t.seq.kv_len + kKeys - 1) / kKeys;
  if (SPLIT) {  // this CTA's run of the blocks
    const int per = (r.n + p.split - 1) / p.split, first = min(r.n, per * (int)(blockIdx.x % p.split));
    r.n = min(per, r.n - first);
    r.seq.kv_start += first * kKeys;
    r.seq.kv_len = min(r.seq.kv_len - first * kKeys, r.n * kKeys);
  }
  r.two = r.tok0 + p.tiles.step / 2 < t.seq.q_len;
  return r;
}

// What the MMA warp needs of an item, written by the copy warp before the
// item's first copy: registers that the MMA warp does not have.
struct Brief {
  int n;
  uint32_t info;  // states of the last block, tile 1 has tokens (bit 8), another item follows (bit 9)
};

// A warp's rows of an item's output, from tensor memory at ``to``, 64 channels at a time
// through shared memory, 16-byte pieces swizzled by row, so that it stores whole rows.
// free_bar (or 0): told once tensor memory has been read.
template <int D>
__device__ __forceinline__ void write_rows(const CrossParams& p, const Item& it, int pos, int head, bool live,
                                           uint32_t rows_live, uint32_t to, uint8_t* stage, float inv, float lse,
                                           uint32_t free_bar) {
  const int lane = threadIdx.x & 31;
  __nv_bfloat16* dst =
      static_cast<__nv_bfloat16*>(p.out) + (int64_t)(it.seq.q_start + pos) * p.o_ts + (int64_t)head * p.o_hs;
#pragma unroll 1
  for (int half = 0; half < D / 64; ++half) {
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      float o[32];
      tm_ld32(to + 64 * half + 32 * c, o);  // (without states anything, and not used)
      tm_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = it.n > 0 ? o[e] * inv : 0.f;
#pragma unroll
      for (int e = 0; e < 32; e += 8)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((4 * c + e / 8) ^ (lane & 7)) * 16) =
            make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]), pack_bf16(o[e + 4], o[e + 5]),
                       pack_bf16(o[e + 6], o[e + 7]));
    }
    tm_fence_before();
    if (half == D / 64 - 1 && free_bar) warp_arrive(free_bar);
    __syncwarp();
#pragma unroll
    for (int y = lane; y < 32 * 8; y += 32) {
      const int row = y / 8, c = y % 8;
      const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), row);
      const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 128 + (c ^ (row & 7)) * 16);
      if (rows_live >> row & 1u) *reinterpret_cast<uint4*>(at + 128 * half + 16 * c) = v;
    }
    __syncwarp();
  }
  if (live && p.lse) p.lse[(int64_t)head * p.n_tokens + it.seq.q_start + pos] = lse;
}

// SPLIT: a cluster of p.split CTAs an item, one item a cluster; else items in turn.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kTcThreads<kOutWarps<D, SPLIT>>, 1)
    cross_tc_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ TcMaps maps, int n_items) {
  using L = TcLayout<D>;
  constexpr bool OUT = kOutWarps<D, SPLIT>;
  extern __shared__ uint8_t tc_raw[];
  uint8_t* smem = tc_raw + ((1024u - (smem_u32(tc_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t bar_full = sbase + L::kBars, bar_empty = bar_full + 8 * L::kSlots;
  const uint32_t bar_end = bar_empty + 8 * L::kSlots, bar_q = bar_end + 8, bar_qfree = bar_q + 16,
                 bar_s = bar_qfree + 16, bar_p = bar_s + 16, bar_o = bar_p + 32, bar_r = bar_o + 16, bar_e = bar_r + 16,
                 bar_l = bar_e + 16, bar_free = bar_l + 16;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::kBars + 8 * L::kNBars);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  Brief* briefs = reinterpret_cast<Brief*>(smem + L::kBriefs);
  const int tile_tok = p.tiles.step / 2;  // tokens of a tile
  const int x0 = SPLIT ? blockIdx.x / p.split : blockIdx.x, dx = SPLIT ? n_items : gridDim.x;

  if (warp == kMmaWarp) tm_alloc<512>(smem_u32(tslot));
  if (t == 32 * kCopyWarp) {
    *abort = 0;
    for (int s = 0; s < L::kSlots; ++s) {
      bar_init(bar_full + 8 * s, 1);
      bar_init(bar_empty + 8 * s, 1);
    }
    bar_init(bar_end, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(bar_q + 8 * i, 1);
      bar_init(bar_qfree + 8 * i, 1);
      bar_init(bar_s + 8 * i, 1);
      bar_init(bar_p + 16 * i, 4);  // a warp arrives once, by one lane
      bar_init(bar_p + 16 * i + 8, 4);
      bar_init(bar_o + 8 * i, 1);
      bar_init(bar_r + 8 * i, 4);
      bar_init(bar_e + 8 * i, 1);
      bar_init(bar_l + 8 * i, 4);
      bar_init(bar_free + 8 * i, 4);
    }
    bar_init_fence();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *tslot;
  pdl_wait();
  pdl_release();

  if (warp >= kMmaWarp && warp < kOutWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<OUT>));
    if (warp == kCopyWarp) {
      // ============ copies (lane 0): per item Q_0, Q_1, then K_0, V_0, K_1, V_1 ... ====
      if (lane == 0) {
        uint32_t ring = 0, n_q[2] = {0, 0};
        bool ok = true;
        // the first item with states from x on, or past the end
        auto find = [&](int x, Item* it) {
          for (; x < n_items; x += dx) {
            *it = item_at<SPLIT>(p, x);
            if (it->n > 0) break;
          }
          return x;
        };
        Item it, next;
        for (int x = find(x0, &it), after, k = 0; x < n_items && ok; x = after, it = next, ++k) {
          after = find(x + dx, &next);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || (i == 1 && !it.two)) break;
            if (n_q[i] > 0 && !(ok = bar_wait(bar_qfree + 8 * i, (n_q[i] - 1) & 1u, abort))) break;
            ++n_q[i];
            // (the item before the last, whose place it takes, is done: its last Q K^T was)
            if (i == 0)
              briefs[k & 1] = {it.n, (uint32_t)(it.seq.kv_len - (it.n - 1) * kKeys) | (it.two ? 0x100u : 0u) |
                                         (after < n_items ? 0x200u : 0u)};
            bar_expect(bar_q + 8 * i, (uint32_t)(tile_tok * p.g) * 128u * (D / 64));
            for (int c = 0; c < D / 64; ++c)
              tma_load3(sbase + L::kQ + i * L::kTile + c * L::kChunk, &maps.q, 64 * c, it.head * p.g,
                        it.seq.q_start + it.tok0 + i * tile_tok, bar_q + 8 * i);
          }
          for (int b = 0; b < 2 * it.n && ok; ++b) {
            const uint32_t s = ring % L::kSlots;
            if (ring >= L::kSlots && !(ok = bar_wait(bar_empty + 8 * s, (ring / L::kSlots - 1) & 1u, abort))) break;
            ++ring;
            bar_expect(bar_full + 8 * s, L::kTile);
            for (int c = 0; c < D / 64; ++c)
              tma_load3(sbase + L::kRing + s * L::kTile + c * L::kChunk, b & 1 ? &maps.v : &maps.k, 64 * c,
                        it.seq.kv_start + (b >> 1) * kKeys, it.head, bar_full + 8 * s);
          }
        }
        if (!ok) {
          *abort = 1;
          if (p.status) atomicOr(p.status, kStatusPromptTimeout);
        }
        // nothing in flight when the CTA ends
        for (uint32_t r = ring > L::kSlots ? ring - L::kSlots : 0; r < ring; ++r)
          bar_drain(bar_full + 8 * (r % L::kSlots), (r / L::kSlots) & 1u);
        for (int i = 0; i < 2; ++i)
          if (n_q[i] > 0) bar_drain(bar_q + 8 * i, (n_q[i] - 1) & 1u);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ============ MMAs, all issued by one lane ======================================
      // With P over S, the next Q K^T overwrites P right behind the P V that reads it; a
      // tcgen05.fence orders the two (different accumulators have no order of their own).
      // The lanes wait each for itself and meet before anything is issued that lets a phase
      // that they waited for be followed by its next: a lane that lags behind that
      // would miss the one it waits for.
      constexpr uint32_t idesc_s = bf16_idesc(kRows, kKeys, false), idesc_o = bf16_idesc(kRows, D, true);
      const bool one = elect_one();
      auto meet = [](bool ok) -> bool { return __all_sync(0xffffffffu, ok); };
      uint32_t ring = 0;                                  // of the current item's K_0
      uint32_t ph_q = 0, ph_p = 0, ph_r = 0, ph_f = 0;    // the phase to wait for, bit i for tile i
      uint32_t used = 0;                                  // bit i: O_i holds an item's output
      bool ok = true;
      // Block -1 stands for the end of an item before the first (items come by falling
      // number of states).
      Brief cur = {0, item_at<SPLIT>(p, x0).n > 0 ? 0x200u : 0u}, next = {};
      int j = -1, begun = 0;
      for (;;) {
        const int rest = cur.info & 0xff;
        for (; j < cur.n && ok; ++j) {
          const bool end = j + 1 == cur.n;
          const uint32_t rk = ring + 2 * (j + 1), kslot = rk % L::kSlots;
          const uint64_t bk = sw128_desc(sbase + L::kRing + kslot * L::kTile, 0);
          // the scores that follow tile i's block j: of the next block, or of the next item
          auto ahead = [&](int i) {
            if (!ok || (end && !(cur.info & 0x200u))) return;
            if (i == 1 && !((end ? next.info : cur.info) & 0x100u)) return;
            if (end) {
              ok = bar_wait(bar_q + 8 * i, ph_q >> i & 1u, abort);
              ph_q ^= 1u << i;
              if (i == 0) next = briefs[begun++ & 1];
            }
            const bool two = (end ? next.info : cur.info) & 0x100u, last = end ? next.n == 1 : j + 2 == cur.n;
            if (i == 0) ok = ok && bar_wait(bar_full + 8 * kslot, (rk / L::kSlots) & 1u, abort);
            if (!(ok = meet(ok))) return;
            uint32_t qaddr;  // (computed here: descriptors kept over the blocks would be spilled)
            asm volatile("add.u32 %0, %1, %2;" : "=r"(qaddr) : "r"(sbase), "r"(L::kQ + i * L::kTile));
            const uint64_t a = sw128_desc(qaddr, 0);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = (ks / 4) * (L::kChunk >> 4) + (ks % 4) * 2;
              if (one) mma_ss(tm + L::kColS + 128 * i, a + off, bk + off, idesc_s, ks > 0);
            }
            if (one) mma_commit(bar_s + 8 * i);
            if (one && last) mma_commit(bar_qfree + 8 * i);
            if (one && (i == 1 || !two)) mma_commit(bar_empty + 8 * kslot);
          };
          if (L::kApart || j < 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // the rows have been read (every block's, so that no phase is missed)
              if (L::kApart && j >= 0 && (i == 0 || cur.info & 0x100u)) {
                ok = meet(ok && bar_wait(bar_r + 8 * i, ph_r >> i & 1u, abort));
                ph_r ^= 1u << i;
                tm_fence_after();
              }
              ahead(i);
            }
          }
          if (j < 0) continue;
          const uint32_t rv = ring + 2 * j + 1, vslot = rv % L::kSlots;
          const uint64_t bv = sw128_desc(sbase + L::kRing + vslot * L::kTile, L::kChunk);
          const int steps = end ? (rest + 15) / 16 : 8;
          ok = ok && bar_wait(bar_full + 8 * vslot, (rv / L::kSlots) & 1u, abort);
          if (end && rest % 16 != 0) {
            // Values behind the last state, in the last k-step of 16: other sequences', whose
            // infinities and NaN a weight of 0 does not silence
            for (int c = 0; c < D / 64; ++c) {
              uint4* rows = reinterpret_cast<uint4*>(smem + L::kRing + vslot * L::kTile + c * L::kChunk);
              for (int y = 8 * rest + lane; y < 8 * ((rest + 15) & ~15); y += 32) rows[y] = make_uint4(0u, 0u, 0u, 0u);
            }
            async_proxy_fence();
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i == 0 || cur.info & 0x100u) {
              auto values = [&](int ks) {
                if (one)
                  mma_ts(tm + L::kColO + D * i, tm + L::kColP + L::kStepP * i + 8 * ks, bv + ks * (2048 >> 4), idesc_o,
                         j > 0 || ks > 0);
              };
              ok = ok && bar_wait(bar_p + 16 * i, ph_p >> i & 1u, abort);
              if (OUT && j == 0) {  // O_i has been read
                if (used >> i & 1u) {
                  ok = ok && bar_wait(bar_free + 8 * i, ph_f >> i & 1u, abort);
                  ph_f ^= 1u << i;
                }
                used |= 1u << i;
              }
              tm_fence_after();
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                if (ok && ks < steps) values(ks);
              ok = ok && bar_wait(bar_p + 16 * i + 8, ph_p >> i & 1u, abort);
              ph_p ^= 1u << i;
              if (!(ok = meet(ok))) break;
              tm_fence_after();
#pragma unroll
              for (int ks = 4; ks < 8; ++ks)
                if (ks < steps) values(ks);
              if (one && (L::kApart || end)) mma_commit((end ? bar_e : bar_o) + 8 * i);
            }
            if (!L::kApart) {
              tm_fence_before();
              ahead(i);
            }
          }
          if (ok && one) mma_commit(bar_empty + 8 * vslot);
        }
        if (!ok || !(cur.info & 0x200u)) break;
        ring += 2 * cur.n;
        cur = next;
        j = 0;
      }
      if (!ok) {
        *abort = 1;
        if (one && p.status) atomicOr(p.status, kStatusPromptTimeout);
      }
      // no MMA in flight, and no arrival to come, when the CTA ends
      __syncwarp();
      if (one) {
        mma_commit(bar_end);
        bar_drain(bar_end, 0);
      }
      __syncwarp();
    }
    if constexpr (SPLIT) {  // (the softmax warps join the outputs in between)
      cluster_sync();
      cluster_sync();
    }
  } else if (warp < kMmaWarp) {
    // ============ softmax: tile i, one row a thread ===================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<OUT>));
    const int i = warp >> 2, r = t & 127;
    const int tt = r / p.g;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tm + L::kColS + 128 * i + lanes, to = tm + L::kColO + D * i + lanes,
                   tp = tm + L::kColP + L::kStepP * i + lanes;
    const float2 sc = make_float2(p.scale2, p.scale2);
    float2* ml = reinterpret_cast<float2*>(smem + (SPLIT ? L::kStage : L::kMl));
    uint32_t n_s = 0, n_o = 0, n_e = 0;
    bool ok = true;
    for (int x = x0; x < n_items && ok; x += dx) {
      int n, kv_len;
      bool warp_live;
      {
        const Item it = item_at<SPLIT>(p, x);
        if (i == 1 && !it.two) continue;
        n = it.n;
        kv_len = it.seq.kv_len;
        warp_live = __any_sync(0xffffffffu, tt < tile_tok && it.tok0 + i * tile_tok + tt < it.seq.q_len);
      }
      if (n == 0 && OUT) continue;
      float m = -FLT_MAX, l = 0.f;  // (not -INFINITY: scores of minus infinity may come first)
      auto before_weights = [&](int j) {  // the last block's P V, or the last item's, is done with P (and with O)
        bool done = true;
        if (j > 0) done = warp_wait(bar_o + 8 * i, n_o++ & 1u, abort);
        else if (n_e > 0) done = warp_wait(bar_e + 8 * i, (n_e - 1) & 1u, abort);
        tm_fence_after();
        return done;
      };
      for (int j = 0; j < n; ++j, ++n_s) {
        if (!(ok = warp_wait(bar_s + 8 * i, n_s & 1u, abort))) break;
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
          const int limit = kv_len - j * kKeys;  // states of the block
          if (limit < kKeys) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= limit) s[c] = -INFINITY;
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
          if (L::kApart && !(ok = before_weights(j))) break;
          if (__any_sync(0xffffffffu, up)) {
            const float a = up ? ex2(m - top) : 1.f;
            if (up) m = top;
            l *= a;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 16) tm_scale16(to + c, a);
            }
          }
          const float2 nm = make_float2(-m, -m);
          float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 128; c += 64) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float2 y = fma2(make_float2(s[c + e], s[c + e + 1]), sc, nm);
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              sum[(e >> 1) & 3] = add2(sum[(e >> 1) & 3], y);
              w[e / 2] = pack_bf16(y.x, y.y);
            }
            tm_st32(tp + c / 2, reinterpret_cast<const float*>(w));
            tm_wait_st();
            tm_fence_before();
            if (c == 0) warp_arrive(bar_p + 16 * i);  // the first 64 states' weights: their P V may start
          }
          sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l += sum[0].x + sum[0].y;
        } else {
          if (L::kApart) {
            // like the others, so that no arrival counts for the block before
            warp_arrive(bar_r + 8 * i);
            if (!(ok = before_weights(j))) break;
          }
          warp_arrive(bar_p + 16 * i);
        }
        warp_arrive(bar_p + 16 * i + 8);
      }
      if (!ok) break;
      if constexpr (SPLIT) {
        if (n > 0 && !(ok = warp_wait(bar_e + 8 * i, 0, abort))) break;
        tm_fence_after();
        ml[t] = make_float2(m, l);
      } else if constexpr (OUT) {
        // the last item's have been read (else its phase of bar_l could pass unseen, too)
        if (n_e > 0 && !(ok = warp_wait(bar_free + 8 * i, (n_e - 1) & 1u, abort))) break;
        ml[t] = make_float2(m, l);
        warp_arrive(bar_l + 8 * i);
      } else {
        if (n > 0 && !(ok = warp_wait(bar_e + 8 * i, n_e & 1u, abort))) break;
        if (warp_live) {
          tm_fence_after();
          const Item it = item_at<SPLIT>(p, x);  // (again: kept over the blocks it would cost them registers)
          const int pos = it.tok0 + i * tile_tok + tt, head = it.head * p.g + r - tt * p.g;
          const bool live = tt < tile_tok && pos < it.seq.q_len;
          write_rows<D>(p, it, pos, head, live, __ballot_sync(0xffffffffu, live), to,
                        smem + L::kStage + warp * L::kStageWarp, 1.f / l,
                        n > 0 ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY, 0u);
        }
        if (n == 0) continue;  // (no phase of this item)
      }
      ++n_e;
    }
    if (!ok) {
      *abort = 1;
      if (p.status && lane == 0) atomicOr(p.status, kStatusPromptTimeout);
    }
    if constexpr (SPLIT) {
      // Both tiles' MMAs are done: the ring takes the outputs, D floats a row, 16-byte
      // pieces swizzled by row.
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const Item it = item_at<SPLIT>(p, x0);
      const int rank = blockIdx.x % p.split, rows = min(2 * tile_tok, it.seq.q_len - it.tok0);
      constexpr int kPieces = D / 4;
      float* part = reinterpret_cast<float*>(smem + L::kRing);
      if (__any_sync(0xffffffffu, tt < tile_tok && i * tile_tok + tt < rows)) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tm_ld32(to + 32 * c, o);
          tm_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part + t * D + 4 * ((8 * c + e / 4) ^ (t & (kPieces - 1)))) =
                it.n > 0 ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        tm_fence_before();
      }
      cluster_sync();
      const int kv_len = tile_at(p.tiles, x0).seq.kv_len;  // all ranks'
      for (int y = rank * 256 + t; y < rows * p.g * kPieces; y += p.split * 256) {
        const int live_row = y / kPieces, c = y % kPieces;
        const int token = live_row / p.g, at_tile = token / tile_tok;
        const int row = 128 * at_tile + live_row - at_tile * tile_tok * p.g;  // (a tile's last rows may be idle)
        const uint32_t at_ml = sbase + L::kStage + row * 8,
                       at_o = sbase + L::kRing + (row * D + 4 * (c ^ (row & (kPieces - 1)))) * 4;
        float top = -FLT_MAX;
        for (int k = 0; k < p.split; ++k) top = fmaxf(top, peer_load2(peer_addr(at_ml, k)).x);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float lr = 0.f;
        for (int k = 0; k < p.split; ++k) {
          const float2 part_ml = peer_load2(peer_addr(at_ml, k));
          const float4 v = peer_load4(peer_addr(at_o, k));
          const float a = ex2(part_ml.x - top);
          lr = fmaf(part_ml.y, a, lr);
          sum.x = fmaf(v.x, a, sum.x);
          sum.y = fmaf(v.y, a, sum.y);
          sum.z = fmaf(v.z, a, sum.z);
          sum.w = fmaf(v.w, a, sum.w);
        }
        const float inv = kv_len == 0 ? 0.f : 1.f / lr;  // over no states: zeros, and lse minus infinity
        const int64_t pos = it.seq.q_start + it.tok0 + token;
        const int head = it.head * p.g + live_row - token * p.g;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + pos * p.o_ts + (int64_t)head * p.o_hs + 4 * c) =
            make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
        if (p.lse && c == 0)
          p.lse[(int64_t)head * p.n_tokens + pos] =
              kv_len == 0 ? -INFINITY : (top + log2f(lr)) * 0.69314718055994530942f;
      }
      cluster_sync();  // no CTA ends while another reads its outputs
    }
  } else {
    // ============ outputs (OUT): an item's O_0, then its O_1, one row a thread ============
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    const int r = t & 127, tt = r / p.g, member = r - tt * p.g;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    uint8_t* stage = smem + L::kStage + (warp & 3) * L::kStageWarp;
    const float2* ml = reinterpret_cast<const float2*>(smem + L::kMl);
    uint32_t done = 0;  // bit i: the phase to wait for of tile i
    bool ok = true;
    for (int x = x0; x < n_items && ok; x += dx) {
      const Item it = item_at<SPLIT>(p, x);
#pragma unroll 1
      for (int i = 0; i < (it.two ? 2 : 1); ++i) {
        const int pos = it.tok0 + i * tile_tok + tt, head = it.head * p.g + member;
        const bool live = tt < tile_tok && pos < it.seq.q_len;
        const uint32_t rows_live = __ballot_sync(0xffffffffu, live), phase = done >> i & 1u;
        float inv = 0.f, lse = -INFINITY;  // without states
        if (it.n > 0) {
          if (!(ok = warp_wait(bar_l + 8 * i, phase, abort) && warp_wait(bar_e + 8 * i, phase, abort))) break;
          done ^= 1u << i;
          tm_fence_after();
          const float2 row = ml[128 * i + r];
          inv = 1.f / row.y;
          lse = (row.x + log2f(row.y)) * 0.69314718055994530942f;
        }
        if (rows_live) {
          write_rows<D>(p, it, pos, head, live, rows_live, tm + L::kColO + D * i + lanes, stage, inv, lse,
                        it.n > 0 ? bar_free + 8 * i : 0u);
        } else if (it.n > 0) {
          warp_arrive(bar_free + 8 * i);
        }
      }
    }
    if (!ok) {
      *abort = 1;
      if (p.status && lane == 0) atomicOr(p.status, kStatusPromptTimeout);
    }
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    tm_free<512>(tm);
  }
}

template <int D, bool SPLIT>
cudaError_t launch_tc(const CrossParams& p, const TcMaps& maps, int64_t tiles, int n_sm, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(cross_tc_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)TcLayout<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_cluster(cross_tc_kernel<D, SPLIT>, SPLIT || tiles < n_sm ? tiles : n_sm, p.split,
                        kTcThreads<kOutWarps<D, SPLIT>>, TcLayout<D>::kSmem, s, p, maps, (int)tiles);
}

template <int D>
int split_of(int64_t tiles, int32_t max_kv, int n_sm) {
  if (cudaFuncSetAttribute(cross_tc_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)TcLayout<D>::kSmem) != cudaSuccess)
    return 1;
  const int64_t blocks = (max_kv + kKeys - 1) / kKeys;
  for (int split = 8; split > 1; --split)
    if (tiles * split <= n_sm && blocks >= 2 * split &&
        tiles <= active_clusters<cross_tc_kernel<D, true>>(split, kTcThreads<false>, TcLayout<D>::kSmem))
      return split;
  return 1;
}

}  // namespace

// CTAs of a cluster that share an item's blocks: while all clusters run at once, each
// CTA with two blocks or more (256 rows over 16384 states: 150 us with one, 27 with 8).
int cross_tc_split(int d, int64_t tiles, int32_t max_kv, int n_sm) {
  return d == 128 ? split_of<128>(tiles, max_kv, n_sm) : split_of<64>(tiles, max_kv, n_sm);
}

cudaError_t launch_cross_tc(const CrossParams& p, int64_t tiles, int n_sm, cudaStream_t s) {
  TcMaps maps;
  // dims (channel, head, token) for the queries, (channel, token, head) for Keys and Values
  if (!tma_map3(&maps.q, p.q, p.D, p.Hq, p.n_tokens, p.q_hs, p.q_ts, p.g, kRows / p.g) ||
      !tma_map3(&maps.k, p.k, p.D, p.n_kv_tokens, p.Hkv, p.k_ts, p.k_hs, kKeys, 1) ||
      !tma_map3(&maps.v, p.v, p.D, p.n_kv_tokens, p.Hkv, p.v_ts, p.v_hs, kKeys, 1))
    return cudaErrorInvalidValue;
  if (p.split > 1)
    return p.D == 128 ? launch_tc<128, true>(p, maps, tiles, n_sm, s) : launch_tc<64, true>(p, maps, tiles, n_sm, s);
  return p.D == 128 ? launch_tc<128, false>(p, maps, tiles, n_sm, s) : launch_tc<64, false>(p, maps, tiles, n_sm, s);
}

}  // namespace kvq
