// Dequantize a cache into dense Key/Value tensors (kvq_restore): the first
// half of the dequantize-to-HBM read path ("KV Cache 量化与压缩" section 06,
// path (a)), kept as the measured foil of the fused decode kernel.
//
// Row t < quantized of a unit is restore(code, scale) = code / max(scale, eps)
// in fp32 ("54. KV Cache Quantization Strategies", restore): Key codes over the
// page's per-channel scales, Value codes over the per-token scales; rows from
// quantized to total are the residual window as held.  A CTA per (run of up to four
// pages, unit) stages its pages in shared memory with cp.async, the next page
// in flight while the current one is decoded, decodes the
// offset-binary codes of the layout in kvq.h (the channel-major Value codes
// through a shared [G][D] tile) and writes 8 channels per thread (16- or
// 32-byte stores); the last grid columns copy the window rows.

#include <cuda_bf16.h>

#include <algorithm>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kRestoreThreads = 256;
constexpr int kRestorePages = 4;  // most pages per CTA, double-buffered
constexpr int kWindowItems = 4 * kRestoreThreads;  // eight-channel pieces of the window per CTA

__device__ __forceinline__ void cpa16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cpa_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cpa_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// Key codes of channels c8 .. c8 + 7 of token t, offset binary as stored.
template <int BITS>
__device__ __forceinline__ void key_codes8(const uint8_t* page, int t, int c8, int D, uint32_t (&code)[8]) {
  if constexpr (BITS == 2) {
    const uint32_t v = *reinterpret_cast<const uint16_t*>(page + t * (D / 4) + c8 / 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = (v >> (2 * e)) & 0x3;
  } else if constexpr (BITS == 4) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(page + t * (D / 2) + c8 / 2);
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = (v >> (4 * e)) & 0xF;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(page + t * D + c8);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      code[e] = (v.x >> (8 * e)) & 0xFF;
      code[4 + e] = (v.y >> (8 * e)) & 0xFF;
    }
  }
}

__device__ __forceinline__ void store8(void* out, int64_t elem, const float (&x)[8], int out_dtype) {
  if (out_dtype == 0) {
    uint4 w;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      u[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + elem) = w;
  } else {
    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + elem);
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

__device__ __forceinline__ void load8(const void* in, int64_t elem, float (&x)[8], int in_dtype) {
  if (in_dtype == 0) {
    const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(in) + elem);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(h[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(in) + elem);
    const float4 a = f[0], b = f[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

// Entries of a scale's table of restored values: one for each stored code, or (any group:
// a large one leaves no room) one for each magnitude.  8-bit codes have none.
template <int BITS, bool FULL>
constexpr int kEntries = (BITS == 2 ? 2 : BITS == 4 ? 8 : 0) * (FULL ? 2 : 1);

// DC, GC: head_dim and group, or 0 for any.  Bound: instructions.  With both and the code
// width known at compile time index arithmetic is shifts, and a table entry for each
// stored code leaves three instructions an element: 300 a thread and page where the
// general form of all widths took 1320 (seven copies of 8192 tokens, 235 MB: 76 us, 153).
template <int BITS, int DC, int GC>
__global__ void __launch_bounds__(kRestoreThreads) restore_kernel(const __grid_constant__ RestoreParams p) {
  extern __shared__ __align__(16) uint8_t page[];
  pdl_wait();
  pdl_release();
  const int n_units = p.n_seqs * p.Hkv;
  const int col = blockIdx.x / n_units;
  const int u = blockIdx.x - col * n_units;
  const int i = u / p.Hkv, h = u - i * p.Hkv;
  const int b = p.seq_begin + i;
  const int D = DC ? DC : p.D, G = GC ? GC : p.G;
  const int T0 = p.ctr[i].total, Q0 = p.ctr[i].quantized;
  const int64_t out_unit = ((int64_t)i * p.Hkv + h) * p.t_stride;  // first row of the unit in the output
  const int per_row = D / 8;

  if (col >= p.page_cols) {
    // the window rows, as held in the ring, by as many columns as the longest window fills
    const int64_t unit = (int64_t)b * p.Hkv + h;
    const int esz = p.in_dtype == 0 ? 2 : 4;
    const uint8_t* rk = reinterpret_cast<const uint8_t*>(p.ring_k) + unit * p.Rcap * D * esz;
    const uint8_t* rv = reinterpret_cast<const uint8_t*>(p.ring_v) + unit * p.Rcap * D * esz;
    const int begin = (col - p.page_cols) * kWindowItems, end = min((T0 - Q0) * per_row, begin + kWindowItems);
    for (int idx = begin + threadIdx.x; idx < end; idx += kRestoreThreads) {
      const int r = idx / per_row, c8 = (idx - r * per_row) * 8;
      const int t = Q0 + r;
      const int64_t src = (int64_t)(t % p.Rcap) * D + c8;
      float x[8], y[8];
      load8(rk, src, x, p.in_dtype);
      load8(rv, src, y, p.in_dtype);
      store8(p.k_out, (out_unit + t) * D + c8, x, p.out_dtype);
      store8(p.v_out, (out_unit + t) * D + c8, y, p.out_dtype);
    }
    return;
  }
  const int P = Q0 / G;
  const int pg_begin = col * p.run;
  if (pg_begin >= P) return;
  const int pg_end = min(P, pg_begin + p.run);
  constexpr int kZero = BITS == 2 ? 2 : BITS == 4 ? 8 : 128, kN = kEntries<BITS, (GC > 0)>;
  const PageGeom geom = make_geom(G, D, BITS);
  const int pbytes = (int)geom.page_bytes;  // a multiple of 16

  uint8_t* buf[2] = {page, page + pbytes};
  float* vtile = reinterpret_cast<float*>(page + 2 * pbytes);  // [G][D]
  // Restored values (code - zero) / max(scale, eps).  IEEE division is sign-symmetric, so a
  // magnitude's quotient serves both signs.  8-bit codes divide directly.
  float* ktab = vtile + G * D;  // [kN][D], channel c at (c % 8) (D / 8) + c / 8: the lanes' eight-channel steps
                                // then lie in neighbouring banks
  float* vtab = ktab + kN * D;  // [G][kN]
  auto look_up = [&](const float* tab, int step, uint32_t code) {  // the table's entry of a stored code
    if (GC) return tab[code * step];
    const int signed_code = (int)code - kZero;
    const float q = tab[(signed_code < 0 ? -signed_code : signed_code) * step];
    return signed_code < 0 ? -q : q;
  };
  auto issue = [&](int pg, uint8_t* dst) {
    const uint8_t* src = p.pages + page_offset(p.map, pbytes, b, h, pg);
    for (int o = threadIdx.x * 16; o < pbytes; o += kRestoreThreads * 16) cpa16(dst + o, src + o);
    cpa_commit();
  };
  issue(pg_begin, buf[0]);
  for (int pg = pg_begin; pg < pg_end; ++pg) {
    uint8_t* cur = buf[(pg - pg_begin) & 1];
    if (pg + 1 < pg_end) {
      issue(pg + 1, buf[(pg + 1 - pg_begin) & 1]);
      cpa_wait<1>();
    } else {
      cpa_wait<0>();
    }
    __syncthreads();
    const float* ks = reinterpret_cast<const float*>(cur + geom.kscale_off);
    const float* vs = reinterpret_cast<const float*>(cur + geom.vscale_off);
    const uint8_t* vbase = cur + geom.code_bytes;
    if constexpr (kN > 0) {
      for (int idx = threadIdx.x; idx < kZero * D; idx += kRestoreThreads) {
        const int m = idx / D, at = idx - m * D, c = at % per_row * 8 + at / per_row;
        const float q = __fdiv_rn((float)m, fmaxf(ks[c], p.eps));
        ktab[(GC ? kZero + m : m) * D + at] = q;
        if (GC && m > 0) ktab[(kZero - m) * D + at] = -q;
      }
      for (int idx = threadIdx.x; idx < kZero * G; idx += kRestoreThreads) {
        const int t = idx / kZero, m = idx - t * kZero;
        const float q = __fdiv_rn((float)m, fmaxf(vs[t], p.eps));
        vtab[t * kN + (GC ? kZero + m : m)] = q;
        if (GC && m > 0) vtab[t * kN + kZero - m] = -q;
      }
      __syncthreads();
    }
    const int64_t row0 = out_unit + (int64_t)pg * G;
    // Value codes: one thread per (channel, 8-token unit of its sub-tile row: a
    // 32-bit word at 4 bits, a 16-bit piece at 2 bits; 4 tokens a word at 8
    // bits), the unit's tokens restored into a [G][D] tile (consecutive
    // threads, consecutive channels: no bank conflicts on the tile)
    constexpr int kTpu = BITS == 8 ? 4 : 8;  // tokens per unit
    for (int idx = threadIdx.x; idx < G * D / kTpu; idx += kRestoreThreads) {
      const int ui = idx / D, c = idx - ui * D;
      const int t0 = ui * kTpu;
      const int st = t0 / 32, n_st = min(32, G - 32 * st);
      const uint8_t* row = vbase + (size_t)st * 32 * D * BITS / 8 + (size_t)c * (n_st * BITS / 8);
      const int uo = (t0 - 32 * st) / kTpu;
      const uint32_t unit = BITS == 2 ? (uint32_t)reinterpret_cast<const uint16_t*>(row)[uo]
                                      : reinterpret_cast<const uint32_t*>(row)[uo];
#pragma unroll
      for (int j = 0; j < kTpu; ++j) {
        int t;
        uint32_t code;
        if (BITS == 2) {
          t = t0 + 2 * (j & 3) + (j >> 2);
          code = (unit >> ((j >> 2) * 8 + 2 * (j & 3))) & 0x3;
        } else if (BITS == 4) {
          t = t0 + (j < 4 ? 2 * j : 2 * (j - 4) + 1);
          code = (unit >> (4 * j)) & 0xF;
        } else {
          t = t0 + j;
          code = (unit >> (8 * j)) & 0xFF;
        }
        vtile[t * D + c] = kN > 0 ? look_up(vtab + t * kN, 1, code) : __fdiv_rn((float)((int)code - kZero), fmaxf(vs[t], p.eps));
      }
    }
    __syncthreads();
    // Key codes: one thread per (token, 8 channels); both rows go out as
    // 16-byte (bf16) or 32-byte (fp32) stores
    for (int idx = threadIdx.x; idx < G * per_row; idx += kRestoreThreads) {
      const int t = idx / per_row, c8 = (idx - t * per_row) * 8;
      uint32_t code[8];
      key_codes8<BITS>(cur, t, c8, D, code);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = kN > 0 ? look_up(ktab + e * per_row + c8 / 8, D, code[e])
                      : __fdiv_rn((float)((int)code[e] - kZero), fmaxf(ks[c8 + e], p.eps));
      store8(p.k_out, (row0 + t) * D + c8, x, p.out_dtype);
      const float4 a = *reinterpret_cast<const float4*>(vtile + t * D + c8);
      const float4 b4 = *reinterpret_cast<const float4*>(vtile + t * D + c8 + 4);
      const float y[8] = {a.x, a.y, a.z, a.w, b4.x, b4.y, b4.z, b4.w};
      store8(p.v_out, (row0 + t) * D + c8, y, p.out_dtype);
    }
    __syncthreads();  // the tables, the tile and this buffer are rewritten next
  }
}

template <int BITS, int DC, int GC>
cudaError_t launch_t(const RestoreParams& p, unsigned blocks, cudaStream_t s) {
  const size_t smem = 2 * (size_t)p.geom.page_bytes +
                      ((size_t)p.G * p.D + (size_t)kEntries<BITS, (GC > 0)> * (p.D + p.G)) * sizeof(float);
  if (smem > 48 * 1024) {
    // all there is, not this cache's need: the limit is a state of the kernel that all caches and threads share
    const cudaError_t e = cudaFuncSetAttribute(restore_kernel<BITS, DC, GC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               227 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(restore_kernel<BITS, DC, GC>, dim3(blocks), dim3(kRestoreThreads), smem, s, p);
}

template <int BITS>
cudaError_t launch_bits(const RestoreParams& p, unsigned blocks, cudaStream_t s) {
  return p.D == 128 && p.G == 32   ? launch_t<BITS, 128, 32>(p, blocks, s)
         : p.D == 128 && p.G == 64 ? launch_t<BITS, 128, 64>(p, blocks, s)
         : p.D == 64 && p.G == 32  ? launch_t<BITS, 64, 32>(p, blocks, s)
                                   : launch_t<BITS, 0, 0>(p, blocks, s);
}

}  // namespace

cudaError_t launch_restore(const RestoreParams& p, cudaStream_t s) {
  RestoreParams q = p;
  // runs of four pages, or shorter ones while they fill the SMs (four sequences of 2100 tokens 21.3 -> 12.7 us)
  q.run = kRestorePages;
  while (q.run > 1 && (int64_t)p.page_cols * p.n_seqs * p.Hkv < 8 * (int64_t)p.n_sm * q.run) q.run /= 2;
  q.page_cols = (p.page_cols + q.run - 1) / q.run;  // page-run columns
  int window = 0;
  for (int i = 0; i < p.n_seqs; ++i) window = std::max(window, p.ctr[i].total - p.ctr[i].quantized);
  const int64_t items = (int64_t)window * (p.D / 8), cols = std::max<int64_t>(1, (items + kWindowItems - 1) / kWindowItems);
  const unsigned blocks = (unsigned)((q.page_cols + cols) * p.n_seqs * p.Hkv);
  return p.bits == 2 ? launch_bits<2>(q, blocks, s) : p.bits == 4 ? launch_bits<4>(q, blocks, s) : launch_bits<8>(q, blocks, s);
}

}  // namespace kvq
