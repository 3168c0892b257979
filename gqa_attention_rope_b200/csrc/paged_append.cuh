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
// Work split: one CTA owns K or V of one (sequence, logical block, KV head),
// so the block's amax, scale and bounds need no atomics. 16 threads take a row,
// 16 bytes each, and a thread up to 8 rows. All loads of a thread are issued before
// the first is used, and before the page is looked up (rows past the end read
// the last row again instead of branching). bf16 pages are bound by the memory
// traffic (512 bytes read and 512 written per token and head): four 8192-token
// prompts of 8 KV heads 49 us in a CUDA graph, 50 as calls (5730 GB/s of the bytes
// it cannot do without, 87% of a copy's rate).
// E4M3 pages (256 bytes written) are bound by waiting: a 131072-token prompt into
// 128-row pages takes 193 us in a graph, 200 as calls (4380 GB/s; K and V in one CTA
// of 512 threads took 704 us), with 49% of the DRAM rate, 45% of the issue slots
// and 36% of the warps. The keys alone take 140 us and the values 78: a key row is
// copied to shared memory, read, turned, written back as float32 until its block's
// scale is known, and read again, and 64 KB for that leave three CTAs on an SM.
// Pages of 64 rows 184 us, of 256 265 (every key fetched and turned twice). A
// persistent form that loads the next head's rows while one is coded was 4%
// faster on 64-row pages and slower on others.
#pragma once

#include "ptx.cuh"

namespace la {
namespace pap {

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

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, u;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 u, %4, %3;\n\tmov.b32 %0, {l, u};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Every code of the 4 in `w` multiplied by r and rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(w & 0xFFFFu));
  const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(w >> 16));
  return e4m3x2(a.x * r, a.y * r) | (e4m3x2(b.x * r, b.y * r) << 16);
}

__device__ __forceinline__ uint4 load_row(const uint16_t* src) {
  uint4 u;  // read once: not kept in L1
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(src));
  return u;
}
__device__ __forceinline__ void unpack_row(const uint4& u, float (&x)[8]) {
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}
// The four pairs of this thread turned by its part of the table row (no
// contraction into FMA: the rounding is the one stated above on every path).
__device__ __forceinline__ void rotate_row(const float4 (&cs)[2], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float c = j ? cs[i].z : cs[i].x, s = j ? cs[i].w : cs[i].y;
      const float a = x[4 * i + 2 * j], b = x[4 * i + 2 * j + 1];
      x[4 * i + 2 * j] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
      x[4 * i + 2 * j + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    }
  }
}

// 16 bytes from global to this thread's own place in shared memory, asynchronously.
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// What one CTA does: rows [r0, r0 + n) of sequence b, all in logical block
// blk, which holds `was` rows already; K or V of KV head h.
struct Job {
  int b, h, blk, len, r0, n, was;
};

// The page of the job's block times Hkv plus its head, or -1 with the error raised.
__device__ __forceinline__ int64_t page_head(const Params& p, const Job& j) {
  const int page = p.block_table[static_cast<int64_t>(j.b) * p.max_blocks + j.blk];
  if (page < 0 || page >= p.n_pages) {
    if (threadIdx.x == 0) raise_error(LLAMA_ATTN_DEVERR_BLOCK_TABLE);
    return -1;
  }
  return static_cast<int64_t>(page) * p.Hkv + j.h;
}
__device__ __forceinline__ const uint16_t* first_row(const Params& p, const Job& j, const uint16_t* x) {
  return x + j.b * p.batch_stride + (j.r0 - j.len) * p.row_stride + j.h * 128 + (threadIdx.x & 15) * 8;
}
// Row of a thread's i-th slot; past the end the last row again (it changes no range and is not stored).
template <int kRowsPerPass>
__device__ __forceinline__ int64_t slot_row(int t0, int i, int n) {
  return min(t0 + static_cast<int>(threadIdx.x >> 4) + i * kRowsPerPass, n - 1);
}

// The block's new scale from this thread's greatest magnitude; codes that the
// block holds already follow it. All threads of the CTA; s_amax: one per warp.
template <int kThreads>
__device__ __forceinline__ float settle_scale(const Job& j, float amax, float old_scale, float* scale_at, uint8_t* codes,
                                              float* s_amax) {
  const uint32_t a = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));  // magnitudes order like their bits
  if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = __uint_as_float(a);
  __syncthreads();
  float m = s_amax[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, s_amax[w]);
  float scale = exp2i(scale_exp(m));
  if (j.was > 0) scale = fmaxf(scale, old_scale);
  if (j.was > 0 && scale != old_scale) {
    const float r = old_scale / scale;
    uint4* at = reinterpret_cast<uint4*>(codes);
    const int64_t n = static_cast<int64_t>(j.was) * 8;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
      const uint4 c = at[i];
      at[i] = make_uint4(rescale4(c.x, r), rescale4(c.y, r), rescale4(c.z, r), rescale4(c.w, r));
    }
  }
  if (threadIdx.x == 0) *scale_at = scale;
  return scale;
}
// A warp's channel-wise ranges into shared memory, and (after a barrier) the
// CTA's into the block's bounds, which they widen where the block had rows.
__device__ __forceinline__ void gather_bounds(float (&lo)[8], float (&hi)[8], float (*s_bound)[2][128]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    lo[c] = fminf(lo[c], __shfl_xor_sync(0xffffffffu, lo[c], 16));
    hi[c] = fmaxf(hi[c], __shfl_xor_sync(0xffffffffu, hi[c], 16));
  }
  const bool upper = lane >= 16;  // lanes 0-15 write the minima, 16-31 the maxima
  float4* at = reinterpret_cast<float4*>(&s_bound[threadIdx.x >> 5][upper][(lane & 15) * 8]);
  at[0] = upper ? make_float4(hi[0], hi[1], hi[2], hi[3]) : make_float4(lo[0], lo[1], lo[2], lo[3]);
  at[1] = upper ? make_float4(hi[4], hi[5], hi[6], hi[7]) : make_float4(lo[4], lo[5], lo[6], lo[7]);
}
template <int kThreads>
__device__ __forceinline__ void store_bounds(uint16_t* bounds, bool widen, float (*s_bound)[2][128]) {
  for (int i = threadIdx.x; i < 256; i += kThreads) {  // 128 minima, then 128 maxima
    const int m = i >> 7, c = i & 127;
    const float sign = m ? -1.f : 1.f;  // max x = -min(-x)
    float x = sign * s_bound[0][m][c];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) x = fminf(x, sign * s_bound[w][m][c]);
    if (widen) x = fminf(x, sign * __uint_as_float(static_cast<uint32_t>(bounds[i]) << 16));
    const __nv_bfloat16 y = __float2bfloat16_rn(sign * x);
    bounds[i] = *reinterpret_cast<const uint16_t*>(&y);
  }
}
__device__ __forceinline__ void store_codes(uint8_t* dst, float (&x)[8], uint64_t inv) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), inv), x[j], x[j + 1]);
  *reinterpret_cast<uint2*>(dst) = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
}

// Values: copied, or coded once the scale is known from rows kept in registers.
template <bool kE4M3, int kThreads, int kRows>
__device__ __forceinline__ void append_values(const Params& p, const Job& j, float* s_amax) {
  constexpr int kRowsPerPass = kThreads / 16;
  constexpr int kHeld = kRowsPerPass * kRows;
  const int n = j.n, row0 = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8;
  const uint16_t* src = first_row(p, j, p.v);
  uint4 raw[kRows];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) raw[i] = load_row(src + slot_row<kRowsPerPass>(t0, i, n) * p.row_stride);
  };
  fetch(0);  // on their way before the page is looked up
  const int64_t ph = page_head(p, j);
  if (ph < 0) return;
  const int64_t dst0 = (ph * p.page_size + j.was) * 128 + ch;
  if constexpr (!kE4M3) {
    for (int t0 = 0; t0 < n; t0 += kHeld) {
      if (t0 > 0) fetch(t0);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = t0 + row0 + i * kRowsPerPass;
        if (r < n) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.vpages) + dst0 + static_cast<int64_t>(r) * 128) = raw[i];
      }
    }
  } else {
    const float old_scale = j.was > 0 ? p.vscales[ph] : 0.f;
    uint32_t m = 0u;  // greatest magnitudes of even and odd channels, as bf16 bits
    for (int t0 = 0; t0 < n; t0 += kHeld) {
      if (t0 > 0) fetch(t0);
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu)));
    }
    const float amax = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    uint8_t* pages = static_cast<uint8_t*>(p.vpages);
    const float scale = settle_scale<kThreads>(j, amax, old_scale, p.vscales + ph, pages + ph * p.page_size * 128, s_amax);
    const uint64_t inv = f2_pack(1.f / scale, 1.f / scale);
    for (int t0 = 0; t0 < n; t0 += kHeld) {
      if (n > kHeld) fetch(t0);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        float x[8];
        unpack_row(raw[i], x);
        const int r = t0 + row0 + i * kRowsPerPass;
        if (r < n) store_codes(pages + dst0 + static_cast<int64_t>(r) * 128, x, inv);
      }
    }
  }
}

// Keys. Table rows come along in registers, half of a thread's rows at a time.
// bf16: rotated and stored. E4M3: all rows are first copied into shared memory,
// each thread its own 16 bytes of a row; the rotated row takes the copy's place
// and waits there for the scale.
template <bool kE4M3, int kThreads, int kRows>
__device__ __forceinline__ void append_keys(const Params& p, const Job& j, float* s_amax, float (*s_bound)[2][128]) {
  constexpr int kRowsPerPass = kThreads / 16;
  constexpr int kStep = kRows / 2;
  constexpr int kHeld = kRowsPerPass * kRows;
  extern __shared__ float4 s_keep[];  // [row slot][half][thread]
  const int n = j.n, row0 = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8;
  const uint16_t* src = first_row(p, j, p.k);
  const float4* tab = p.tab + static_cast<int64_t>(j.r0) * 32 + ch / 4;
  auto row = [&](int t0, int i) { return slot_row<kRowsPerPass>(t0, i, n); };
  auto kept = [&](int i) { return s_keep + 2 * kThreads * i + threadIdx.x; };

  uint4 raw[kStep];
  auto fetch = [&](int t0, int i0) {  // E4M3: the tile; bf16: a step of it from slot i0
#pragma unroll
    for (int i = 0; i < (kE4M3 ? kRows : kStep); ++i) {
      if constexpr (kE4M3)
        copy_async16(kept(i), src + row(t0, i) * p.row_stride);
      else
        raw[i] = load_row(src + row(t0, i0 + i) * p.row_stride);
    }
  };
  fetch(0, 0);  // on their way before the page is looked up
  const int64_t ph = page_head(p, j);
  if (ph < 0) {
    if constexpr (kE4M3) copy_async_wait();
    return;
  }
  const int64_t dst0 = (ph * p.page_size + j.was) * 128 + ch;
  const float old_scale = kE4M3 && j.was > 0 ? p.kscales[ph] : 0.f;
  const bool ranges = kE4M3 || p.kbounds;
  float lo[8], hi[8];  // of the thread's channels
#pragma unroll
  for (int c = 0; c < 8; ++c) lo[c] = INFINITY, hi[c] = -INFINITY;
  auto rotate_tile = [&](int t0) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if constexpr (!kE4M3) {
        if (t0 + half > 0) fetch(t0, half * kStep);
      }
      float4 cs[kStep][2];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const float4* c = tab + row(t0, half * kStep + i) * 32;
        cs[i][0] = c[0];
        cs[i][1] = c[1];
      }
      if constexpr (kE4M3) {
        if (half == 0) copy_async_wait();
      }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int s = half * kStep + i;
        float x[8];
        if constexpr (kE4M3)
          unpack_row(*reinterpret_cast<const uint4*>(kept(s)), x);
        else
          unpack_row(raw[i], x);
        rotate_row(cs[i], x);
        if (ranges) {
#pragma unroll
          for (int c = 0; c < 8; ++c) lo[c] = fminf(lo[c], x[c]), hi[c] = fmaxf(hi[c], x[c]);
        }
        if constexpr (kE4M3) {
          kept(s)[0] = make_float4(x[0], x[1], x[2], x[3]);
          kept(s)[kThreads] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          const int r = t0 + row0 + s * kRowsPerPass;
          if (r < n)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.kpages) + dst0 + static_cast<int64_t>(r) * 128) =
                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                           pack_bf16x2(x[6], x[7]));
        }
      }
    }
  };
  for (int t0 = 0; t0 < n; t0 += kHeld) {
    if (kE4M3 && t0 > 0) fetch(t0, 0);
    rotate_tile(t0);
  }
  if (!ranges) return;
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fmaxf(-lo[c], hi[c]));
  if (p.kbounds) gather_bounds(lo, hi, s_bound);
  float scale = 1.f;
  uint8_t* pages = static_cast<uint8_t*>(p.kpages);
  if constexpr (kE4M3)
    scale = settle_scale<kThreads>(j, amax, old_scale, p.kscales + ph, pages + ph * p.page_size * 128, s_amax);
  else
    __syncthreads();
  if (p.kbounds) store_bounds<kThreads>(p.kbounds + ph * 256, j.was > 0, s_bound);
  if constexpr (kE4M3) {
    const uint64_t inv = f2_pack(1.f / scale, 1.f / scale);
    for (int t0 = 0; t0 < n; t0 += kHeld) {
      if (n > kHeld) {  // a page of more rows than are held: once more, from L2
        fetch(t0, 0);
        rotate_tile(t0);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float4 u = kept(i)[0], w = kept(i)[kThreads];
        float x[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
        const int r = t0 + row0 + i * kRowsPerPass;
        if (r < n) store_codes(pages + dst0 + static_cast<int64_t>(r) * 128, x, inv);
      }
    }
  }
}

// Rows that slot `slot` (the slot-th block that sequence b's new rows touch)
// and KV head h get; n <= 0: none. `first_cta`: this CTA reports for the sequence.
__device__ __forceinline__ Job job_of(const Params& p, int b, int slot, int h, bool first_cta) {
  Job j;
  j.b = b;
  j.h = h;
  j.len = p.lens[b];
  j.n = 0;
  j.blk = j.r0 = j.was = 0;
  const int n_new = p.new_lens ? p.new_lens[b] : p.T;
  const int cap = p.max_blocks * p.page_size;  // below 2^31
  const bool ok = j.len >= 0 && n_new >= 0 && n_new <= p.T && j.len <= cap && n_new <= cap - j.len;
  if (first_cta && threadIdx.x == 0) {
    if (!ok) raise_error(LLAMA_ATTN_DEVERR_CACHE_LEN);
    if (p.out_lens) p.out_lens[b] = ok ? j.len + n_new : j.len;
  }
  if (!ok) return j;
  j.blk = j.len / p.page_size + slot;
  if (j.blk >= p.max_blocks) return j;
  const int first = j.blk * p.page_size;  // the block's first position
  j.r0 = max(j.len, first);
  j.n = min(j.len + n_new - j.r0, first + p.page_size - j.r0);
  j.was = j.r0 - first;
  return j;
}

// One block and K or V of one head per CTA: grid (2 * Hkv, block slots, B).
template <bool kE4M3, int kThreads, int kRows>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 6) kv_append_paged_kernel(const Params p) {
  __shared__ float s_amax[kThreads / 32];
  __shared__ __align__(16) float s_bound[kThreads / 32][2][128];
  grid_launch_dependents();
  grid_dependency_wait();
  const Job j = job_of(p, blockIdx.z, blockIdx.y, blockIdx.x >> 1, blockIdx.x == 0 && blockIdx.y == 0);
  if (j.n <= 0) return;
  if (blockIdx.x & 1)
    append_values<kE4M3, kThreads, kRows>(p, j, s_amax);
  else
    append_keys<kE4M3, kThreads, kRows>(p, j, s_amax, s_bound);
}

}  // namespace pap
}  // namespace la
