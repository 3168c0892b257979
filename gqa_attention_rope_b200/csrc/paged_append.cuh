// paged_append.cuh -- appends new keys and values to a paged KV cache, the
// keys rotated on the way (RoPE at each row's cache position), into bf16 pages
// or into E4M3 pages with one scale per block (page) and KV head.
//
// Mathematics. Row p of a sequence goes to row p % page_size of the page of
// logical block p / page_size. With (c, s) = table row p, the pair (x0, x1) of
// a key becomes (x0 c - x1 s, x0 s + x1 c), every product and the sum rounded
// to float32 once, then once more to the cache's type.
// E4M3 pages: a block's scale is 2^e with the least e for which
// amax <= 448 * 2^e over its rows, so x / 2^e is exact and a code carries one
// rounding. A power of two also makes growing a block cheap to get right: when
// a later row raises the scale, the codes already there are divided by a power
// of two, which is exact except where they fall below 2^-6 of the new scale
// (E4M3's subnormals, off by at most half a subnormal step, 2^-10 scales).
// With scale = amax / 448 every such growth would round every code again.
// Key bounds: per block, head and channel the least and the greatest rotated
// key, in bf16 (rounding is monotone, so it commutes with min and max).
//
// Work split: one CTA owns one (sequence, logical block, KV head), so the
// block's amax, scale and bounds need no atomics. Half of its threads take K,
// the other half V, 16 threads per row with 16 bytes each. The bound is the
// memory traffic: 512 bytes read and 256 (E4M3) or 512 (bf16) written per token
// and head; up to 8 rows per thread wait in registers for the block's scale.
#pragma once

#include "ptx.cuh"

namespace la {
namespace pap {

constexpr int kMaxRowsPerThread = 8;
constexpr int kMinExp = -100, kMaxExp = 119;  // exponents of the block scales

struct Params {
  const uint16_t* k;       // row t of sequence b, head h: k + b * batch_stride + t * row_stride + h * 128
  const uint16_t* v;
  int64_t row_stride, batch_stride;
  void* kpages;            // [n_pages, Hkv, page_size, 128] bf16 or E4M3
  void* vpages;
  float* kscales;          // [n_pages, Hkv], E4M3 only
  float* vscales;
  uint16_t* kbounds;       // [n_pages, Hkv, 2, 128] bf16 (min, max) or null
  const int32_t* block_table;
  const int32_t* lens;
  const int32_t* new_lens;  // null: every sequence gets T rows
  int32_t* out_lens;        // null, or the lengths after the append
  const float4* tab;        // RoPE table rows as float4 (two pairs each)
  int T, Hkv, page_size, max_blocks, n_pages;
};

// Least exponent e (within [kMinExp, kMaxExp]) with amax <= 448 * 2^e, read off
// the float32 bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(v);
}

// Every code of the 4 in `w` multiplied by r and rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(w & 0xFFFFu));
  const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(w >> 16));
  return e4m3x2(a.x * r, a.y * r) | (e4m3x2(b.x * r, b.y * r) << 16);
}

// Eight values of one row (this thread's channels) in float32.
__device__ __forceinline__ void load_row(const uint16_t* src, float (&x)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(src));
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}
// The four pairs of this thread turned by the table row (no contraction into
// FMA: the rounding is the one stated above on every path).
__device__ __forceinline__ void rotate_row(const float4* tab_row, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 cs = __ldg(tab_row + i);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float c = j ? cs.z : cs.x, s = j ? cs.w : cs.y;
      const float a = x[4 * i + 2 * j], b = x[4 * i + 2 * j + 1];
      x[4 * i + 2 * j] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
      x[4 * i + 2 * j + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    }
  }
}

// grid (block slots, Hkv, B), kThreads threads. A page of more than
// kThreads / 32 * 8 new rows is read twice (the second time from L2).
template <bool kE4M3, int kThreads>
__global__ void __launch_bounds__(kThreads) kv_append_paged_kernel(const Params p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kRowsPerPass = kThreads / 32;  // per half: (kThreads / 2) / 16
  constexpr int kTile = kRowsPerPass * kMaxRowsPerThread;
  __shared__ float s_amax[kWarps];
  __shared__ float s_bound[kWarps / 2][2][128];

  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t len = p.lens[b];
  const int64_t n_new = p.new_lens ? p.new_lens[b] : p.T;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.page_size;
  const bool ok = len >= 0 && n_new >= 0 && n_new <= p.T && len + n_new <= cap;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    if (!ok) raise_error(LLAMA_ATTN_DEVERR_CACHE_LEN);
    if (p.out_lens) p.out_lens[b] = static_cast<int32_t>(ok ? len + n_new : len);
  }
  if (!ok) return;
  const int64_t blk = len / p.page_size + blockIdx.x;
  const int64_t first = blk * p.page_size;                   // the block's first position
  const int64_t r0 = len > first ? len : first;
  const int64_t r1 = min(len + n_new, first + p.page_size);
  if (r0 >= r1) return;
  const int page = p.block_table[static_cast<int64_t>(b) * p.max_blocks + blk];
  if (page < 0 || page >= p.n_pages) {
    if (threadIdx.x == 0) raise_error(LLAMA_ATTN_DEVERR_BLOCK_TABLE);
    return;
  }
  const int64_t ph = static_cast<int64_t>(page) * p.Hkv + h;
  const int was = static_cast<int>(r0 - first);              // rows the block already holds
  const int n = static_cast<int>(r1 - r0);

  const bool is_v = threadIdx.x >= kThreads / 2;
  const int tid = threadIdx.x - (is_v ? kThreads / 2 : 0);
  const int row0 = tid >> 4, ch = (tid & 15) * 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint16_t* src = (is_v ? p.v : p.k) + b * p.batch_stride + (r0 - len) * p.row_stride + h * 128 + ch;
  const float4* tab = p.tab + r0 * 32 + ch / 4;

  auto fetch = [&](int r, float (&x)[8]) {
    load_row(src + r * p.row_stride, x);
    if (!is_v) rotate_row(tab + static_cast<int64_t>(r) * 32, x);
  };
  auto store_bf16 = [&](int r, const float (&x)[8]) {
    uint16_t* dst = static_cast<uint16_t*>(is_v ? p.vpages : p.kpages) + (ph * p.page_size + was + r) * 128 + ch;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  };
  auto store_e4m3 = [&](int r, const float (&x)[8], float inv) {
    uint8_t* dst = static_cast<uint8_t*>(is_v ? p.vpages : p.kpages) + (ph * p.page_size + was + r) * 128 + ch;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16),
                   e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16));
  };

  float keep[kMaxRowsPerThread][8];
  float lo[8], hi[8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  for (int t0 = 0; t0 < n; t0 += kTile) {
#pragma unroll
    for (int i = 0; i < kMaxRowsPerThread; ++i) {
      const int r = t0 + row0 + i * kRowsPerPass;
      if (r < n) fetch(r, keep[i]);
    }
#pragma unroll
    for (int i = 0; i < kMaxRowsPerThread; ++i) {
      const int r = t0 + row0 + i * kRowsPerPass;
      if (r < n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          lo[j] = fminf(lo[j], keep[i][j]);
          hi[j] = fmaxf(hi[j], keep[i][j]);
        }
        if constexpr (!kE4M3) store_bf16(r, keep[i]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(-lo[j], hi[j]));  // no row: -inf, -inf

  float old_scale = 0.f;
  float* scales = nullptr;
  if constexpr (kE4M3) {
    scales = (is_v ? p.vscales : p.kscales) + ph;
    if (was > 0) old_scale = *scales;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_amax[warp] = amax;
  }
  if (p.kbounds && !is_v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], 16));
      hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 16));
      if (lane < 16) s_bound[warp][0][ch + j] = lo[j], s_bound[warp][1][ch + j] = hi[j];
    }
  }
  __syncthreads();
  if (p.kbounds) {
    for (int i = threadIdx.x; i < 256; i += kThreads) {  // 128 minima, then 128 maxima
      const int m = i >> 7, c = i & 127;
      float x = s_bound[0][m][c];
      for (int w = 1; w < kWarps / 2; ++w) x = m ? fmaxf(x, s_bound[w][m][c]) : fminf(x, s_bound[w][m][c]);
      uint16_t* dst = p.kbounds + ph * 256 + i;
      if (was > 0) {
        const float old = __uint_as_float(static_cast<uint32_t>(*dst) << 16);
        x = m ? fmaxf(x, old) : fminf(x, old);
      }
      const __nv_bfloat16 y = __float2bfloat16_rn(x);
      *dst = *reinterpret_cast<const uint16_t*>(&y);
    }
  }
  if constexpr (kE4M3) {
    float a = 0.f;
    for (int w = 0; w < kWarps / 2; ++w) a = fmaxf(a, s_amax[(is_v ? kWarps / 2 : 0) + w]);
    float scale = exp2i(scale_exp(a));
    if (was > 0) scale = fmaxf(scale, old_scale);
    if (was > 0 && scale != old_scale) {  // the rows already there follow the block's scale
      const float r = old_scale / scale;
      uint4* codes = reinterpret_cast<uint4*>(static_cast<uint8_t*>(is_v ? p.vpages : p.kpages) +
                                              ph * p.page_size * 128);
      for (int i = tid; i < was * 8; i += kThreads / 2) {
        const uint4 c = codes[i];
        codes[i] = make_uint4(rescale4(c.x, r), rescale4(c.y, r), rescale4(c.z, r), rescale4(c.w, r));
      }
    }
    if (tid == 0) *scales = scale;
    const float inv = 1.f / scale;
    for (int t0 = 0; t0 < n; t0 += kTile) {
#pragma unroll
      for (int i = 0; i < kMaxRowsPerThread; ++i) {
        const int r = t0 + row0 + i * kRowsPerPass;
        if (r < n) {
          if (n > kTile) fetch(r, keep[i]);
          store_e4m3(r, keep[i], inv);
        }
      }
    }
  }
}

}  // namespace pap
}  // namespace la
