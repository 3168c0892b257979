// select_blocks.cuh -- chooses, for each (sequence, KV head) of a single-token
// decode over a paged cache, the blocks worth reading.
//
// Mathematics. A block's key bounds (channel-wise least and greatest rotated
// key) bound any of its keys' products with a query: q . k <= sum_d max(q_d
// lo_d, q_d hi_d). The heads of a KV group share the rows they read, so a
// block is scored by the sum of its bounds over the group, which needs no
// loop over the heads:
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = sum_d up_d hi_d + down_d lo_d,
//   up_d = sum_h max(q_hd, 0), down_d = sum_h min(q_hd, 0).
// The choice is defined by float64 scores: it is an order, and sums in float32
// would let the order of additions decide between near blocks. Of the others
// than the first n_first and the last n_last blocks those with the greatest
// scores are taken, of equal scores the lower index.
//
// Most blocks are far from the border, so the scores are first formed on the
// tensor cores: 16 blocks are the rows of an m16n8k16 product over the 256
// bounds, and three of its 8 columns carry the weights as three bf16 terms (24
// bits), which costs nothing next to one. Products of bf16 are exact; the 16
// accumulations in float32 and the residue of the weights stay within
// eps = 2^-15 sum_d |w_d| max |bound| (were each of a product's 17 terms cut
// off at 2^-23 of that sum, 16 products would reach 2^-15). A radix selection
// over these scores finds a range [lo, hi] that holds the one at the border;
// blocks outside [lo - 2 eps, hi + 2 eps] are decided by it, the one or two
// inside get their float64 score and a second selection.
// Measured for 64 sequences of 1024 to 32768 rows (8 KV heads, 64-row blocks,
// 71 MB of bounds): all scores in float64 39 us, three quarters of it
// instructions (400 per warp and 8 blocks); this form: see the table of
// results beside the kernel's launch.
//
// One cluster of CTAs takes one (sequence, KV head): each CTA streams its
// share of the bounds and stores an order-preserving key of every score into
// the first CTA's shared memory, which selects and writes the ids in ascending
// order. What bounds it: HBM for the bounds of large batches, the chain of
// dependent steps for small ones.
#pragma once

#include "ptx.cuh"
#include "rope.cuh"

namespace la {
namespace sel {

constexpr int NTHREADS = 256;
constexpr int NWARPS = NTHREADS / 32;
constexpr int BINS = 1024;
constexpr int MAX_BLOCKS = 24576;  // keys of one (sequence, KV head) in shared memory: 192 KB

struct Params {
  const uint16_t* q;         // [B, Hq, 128] bf16 bits
  const uint16_t* kbounds;   // [n_pages, Hkv, 2, 128] bf16
  const int32_t* block_table;
  const int32_t* lens;
  int32_t* ids;              // [B, Hkv, n_sel]
  int B, Hq, Hkv, G, page_size, max_blocks, n_pages, n_sel, n_first, n_last, q_pos_offset;
  RopeFreqs freqs;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores x at shared address `addr` of the cluster's CTA 0.
__device__ __forceinline__ void store_to_first32(uint32_t addr, uint32_t x) {
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\tst.shared::cluster.u32 [r], %1;\n\t}" ::"r"(addr),
      "r"(x)
      : "memory");
}

// Order-preserving maps of scores to unsigned integers and back; NaN above
// every number, 0 and ~0 left to mark blocks that are decided.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return ~0u - 1;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are one score
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull - 1;
  const long long b = __double_as_longlong(x + 0.0);
  return b < 0 ? ~static_cast<unsigned long long>(b) : static_cast<unsigned long long>(b) | (1ull << 63);
}
constexpr unsigned long long kOut = 0ull, kIn = ~0ull;

// Greater magnitude of each half (the sign of the result means nothing).
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ double bf16_lo(uint32_t u) { return static_cast<double>(__uint_as_float(u << 16)); }
__device__ __forceinline__ double bf16_hi(uint32_t u) { return static_cast<double>(__uint_as_float(u & 0xFFFF0000u)); }

struct RadixShared {
  int hist[BINS];
  int warp[NWARPS];
  unsigned long long lo[NWARPS], hi[NWARPS];
  int bin, above, in_bin;
};

// The `need`-th greatest (1 <= need <= number of keys) of key(j), c0 <= j < c1,
// without those for which key(j) is 0 or ~0: a range [lo, hi] that holds it,
// found 10 bits at a time from the highest bit in which the keys differ. With
// kExact the range is narrowed until `take`, the number of keys within it that
// belong to the `need` greatest, is all of them or lo == hi; without, until one
// window of bits has been looked at. All threads of the CTA.
template <bool kExact, typename K, typename Key>
__device__ __forceinline__ void radix_select(RadixShared& s, Key key, int c0, int c1, int need, K& out_lo, K& out_hi,
                                             int& take) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  K lo = ~K(0), hi = 0;
  for (int j = c0 + threadIdx.x; j < c1; j += NTHREADS) {
    const K k = key(j);
    if (k == 0 || k == ~K(0)) continue;
    lo = k < lo ? k : lo;
    hi = k > hi ? k : hi;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const K a = __shfl_xor_sync(0xffffffffu, lo, o), c = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = a < lo ? a : lo;
    hi = c > hi ? c : hi;
  }
  if (lane == 0) s.lo[warp] = lo, s.hi[warp] = hi;
  for (int i = threadIdx.x; i < BINS; i += NTHREADS) s.hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NWARPS; ++i) {
    lo = s.lo[i] < lo ? static_cast<K>(s.lo[i]) : lo;
    hi = s.hi[i] > hi ? static_cast<K>(s.hi[i]) : hi;
  }
  take = need;
  out_lo = lo;
  out_hi = hi;
  if (lo >= hi) return;  // equal keys
  const int top = 63 - __clzll(static_cast<long long>(static_cast<unsigned long long>(lo ^ hi)));
  constexpr int kBits = static_cast<int>(sizeof(K)) * 8;
  int shift = top > 9 ? top - 9 : 0, bits = 10;
  K prefix = shift + 10 < kBits ? hi >> (shift + 10) : K(0);
  for (;;) {
    for (int j = c0 + threadIdx.x; j < c1; j += NTHREADS) {
      const K k = key(j);
      if (k == 0 || k == ~K(0)) continue;
      const K top_bits = shift + bits < kBits ? k >> (shift + bits) : K(0);
      if (top_bits == prefix) atomicAdd(&s.hist[static_cast<int>((k >> shift) & ((1u << bits) - 1u))], 1);
    }
    __syncthreads();
    // suffix sums over the bins, kPer of them per thread, the highest bins first
    constexpr int kPer = BINS / NTHREADS;
    const int top_bin = BINS - 1 - kPer * static_cast<int>(threadIdx.x);
    int n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      n[i] = s.hist[top_bin - i];
      s.hist[top_bin - i] = 0;  // for the next window
      sum += n[i];
    }
    const int mine = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) s.warp[warp] = sum;
    __syncthreads();
    int above = sum - mine;
#pragma unroll
    for (int i = 0; i < NWARPS; ++i) above += i < warp ? s.warp[i] : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (above < take && above + n[i] >= take) s.bin = top_bin - i, s.above = above, s.in_bin = n[i];
      above += n[i];
    }
    __syncthreads();
    const int in_bin = s.in_bin;
    take -= s.above;
    prefix = (prefix << bits) | static_cast<K>(s.bin);
    out_lo = prefix << shift;
    out_hi = out_lo | ((K(1) << shift) - 1);
    if (!kExact || in_bin == take || shift == 0) return;
    __syncthreads();
    bits = shift < 10 ? shift : 10;
    shift -= bits;
  }
}

// grid (cluster size * B * Hkv): consecutive CTAs form the cluster of one
// (sequence, KV head). Dynamic shared memory: 8 bytes per block of a sequence.
__global__ void __launch_bounds__(NTHREADS, 4) select_blocks_kernel(const Params p) {
  extern __shared__ unsigned long long s_key[];    // first the scores' 32-bit keys, then kIn, kOut or a float64's key
  __shared__ __align__(16) double s_w[256];        // weights of the minima (down), then of the maxima (up)
  __shared__ uint2 s_b[16][32];                    // the same as fragments of the product, three bf16 terms
  __shared__ RadixShared s_radix;
  __shared__ uint32_t s_mag[8 * NWARPS];           // per warp of the cluster: greatest magnitude of a bound, float bits
  __shared__ double s_wsum[4];
  __shared__ int s_count[2][NWARPS];

  const uint32_t rank = cluster_rank(), csize = cluster_size();
  const int64_t bg = blockIdx.x / csize;
  const int b = static_cast<int>(bg / p.Hkv), g = static_cast<int>(bg % p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  int len = p.lens[b];
  if (len < 0 || len > static_cast<int64_t>(p.max_blocks) * p.page_size) {
    if (g == 0 && rank == 0 && threadIdx.x == 0) raise_error(LLAMA_ATTN_DEVERR_CACHE_LEN);
    len = 0;
  }
  const int nb = (len + p.page_size - 1) / p.page_size;
  int32_t* ids = p.ids + bg * p.n_sel;
  if (nb <= p.n_sel) {  // every block; the whole cluster leaves here
    if (rank == 0)
      for (int i = threadIdx.x; i < p.n_sel; i += NTHREADS) ids[i] = i < nb ? i : -1;
    return;
  }

  // ---- the group's weights: up_d, down_d of the query rotated at its position
  if (threadIdx.x < 64) {
    const int k = threadIdx.x;
    double sn, cs;
    sincos(static_cast<double>(len + p.q_pos_offset) * p.freqs.theta[k], &sn, &cs);
    double w[4] = {0.0, 0.0, 0.0, 0.0};
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(b) * p.Hq + g * p.G) * 128) + k;
#pragma unroll 4
    for (int h = 0; h < p.G; ++h) {
      const uint32_t u = q[h * 64];
      const double x0 = bf16_lo(u), x1 = bf16_hi(u);
      const double y0 = x0 * cs - x1 * sn, y1 = x0 * sn + x1 * cs;
      w[0] += fmin(y0, 0.0), w[1] += fmin(y1, 0.0), w[2] += fmax(y0, 0.0), w[3] += fmax(y1, 0.0);
    }
    s_w[2 * k] = w[0], s_w[2 * k + 1] = w[1], s_w[128 + 2 * k] = w[2], s_w[128 + 2 * k + 1] = w[3];
    double sum = (w[2] - w[0]) + (w[3] - w[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_wsum[warp] = sum;
  }
  __syncthreads();
  // Fragments: a thread (row group gq, t) of the product loads 8 neighbouring
  // bounds 32 i + 8 t.. of a block, which are its part of steps 2 i and 2 i + 1.
  for (int e = threadIdx.x; e < 16 * 32; e += NTHREADS) {
    const int st = e >> 5, gq = (e & 31) >> 2, t = e & 3;
    const double* w = s_w + 32 * (st >> 1) + 8 * t + 4 * (st & 1);
    uint32_t r[2] = {0u, 0u};
    if (gq < 3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        double rest = w[i];
        __nv_bfloat16 term = __float2bfloat16_rn(0.f);
        for (int n = 0; n <= gq; ++n) {
          term = __float2bfloat16_rn(static_cast<float>(rest));
          rest -= static_cast<double>(__bfloat162float(term));
        }
        r[i >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&term)) << (16 * (i & 1));
      }
    }
    s_b[st][e & 31] = make_uint2(r[0], r[1]);
  }
  __syncthreads();
  // every CTA of the cluster has started before any of them stores into the first one
  if (csize > 1) cluster_sync();

  // ---- scores, 16 candidates at a time per warp
  const int c0 = p.n_first, c1 = nb - p.n_last;  // candidates [c0, c1); more than n_sel - n_first - n_last of them
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
  {
    const int gq = lane >> 2, t = lane & 3;
    const int step = static_cast<int>(csize) * NWARPS * 16;
    uint32_t mag = 0u;
    int j0 = c0 + (static_cast<int>(rank) * NWARPS + warp) * 16;
    int next = lane < 16 && j0 + lane < c1 ? table[j0 + lane] : 0;
    for (; j0 < c1; j0 += step) {
      int page = next;
      next = lane < 16 && j0 + step + lane < c1 ? table[j0 + step + lane] : 0;
      if (page < 0 || page >= p.n_pages) {
        raise_error(LLAMA_ATTN_DEVERR_BLOCK_TABLE);
        page = -1;
      }
      const int pa = __shfl_sync(0xffffffffu, page, gq), pb = __shfl_sync(0xffffffffu, page, gq + 8);
      const bool ina = j0 + gq < c1 && pa >= 0, inb = j0 + gq + 8 < c1 && pb >= 0;  // others score as zeros
      const uint4* xa = reinterpret_cast<const uint4*>(p.kbounds + (static_cast<int64_t>(pa) * p.Hkv + g) * 256) + t;
      const uint4* xb = reinterpret_cast<const uint4*>(p.kbounds + (static_cast<int64_t>(pb) * p.Hkv + g) * 256) + t;
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4 a[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = c[i] = make_uint4(0u, 0u, 0u, 0u);
          if (ina) a[i] = __ldg(xa + 4 * (4 * half + i));
          if (inb) c[i] = __ldg(xb + 4 * (4 * half + i));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 w0 = s_b[2 * (4 * half + i)][lane], w1 = s_b[2 * (4 * half + i) + 1][lane];
          mma_bf16_16816(s0, a[i].x, c[i].x, a[i].y, c[i].y, w0.x, w0.y);
          mma_bf16_16816(s1, a[i].z, c[i].z, a[i].w, c[i].w, w1.x, w1.y);
          mag = max_abs(max_abs(max_abs(mag, a[i].x), max_abs(a[i].y, a[i].z)),
                        max_abs(max_abs(a[i].w, c[i].x), max_abs(max_abs(c[i].y, c[i].z), c[i].w)));
        }
      }
      // columns 0 and 1 of rows gq and gq + 8 are in lane t = 0, column 2 in lane t = 1
      float u = s0[0] + s1[0], v = s0[2] + s1[2];
      u += __shfl_down_sync(0xffffffffu, u, 1) + (s0[1] + s1[1]);
      v += __shfl_down_sync(0xffffffffu, v, 1) + (s0[3] + s1[3]);
      if (t == 0) {
        if (j0 + gq < c1) store_to_first32(smem_addr(s_key + j0 + gq), order_key(u));
        if (j0 + gq + 8 < c1) store_to_first32(smem_addr(s_key + j0 + gq + 8), order_key(v));
      }
    }
    mag = __reduce_max_sync(0xffffffffu, max((mag << 16) & 0x7FFF0000u, mag & 0x7FFF0000u));  // magnitudes order like their bits
    if (lane == 0) store_to_first32(smem_addr(&s_mag[rank * NWARPS + warp]), mag);
  }
  if (csize > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank != 0) return;

  // ---- the first CTA: which candidates the scores decide
  const int need = p.n_sel - p.n_first - p.n_last;
  auto approx = [&](int j) { return static_cast<uint32_t>(s_key[j]); };
  int n_in = 0, n_near = 0;
  if (need > 0) {
    uint32_t mag = 0u;
    for (int i = 0; i < static_cast<int>(csize) * NWARPS; ++i) mag = max(mag, s_mag[i]);
    const float eps2 = 2.f * 0x1p-15f * static_cast<float>(s_wsum[0] + s_wsum[1]) * __uint_as_float(mag);
    uint32_t klo, khi;
    int unused;
    radix_select<false>(s_radix, approx, c0, c1, need, klo, khi, unused);
    const float lo = score_of(klo) - eps2, hi = score_of(khi) + eps2;
    const int group = lane >> 4, ch = lane & 15;
    for (int j0 = c0 + warp * 32; j0 < c1; j0 += NTHREADS) {
      const int j = j0 + lane;
      const float s = j < c1 ? score_of(approx(j)) : 0.f;
      const bool in = j < c1 && s > hi, out = j < c1 && s < lo;  // a NaN is neither
      if (in || out) s_key[j] = in ? kIn : kOut;
      n_in += __popc(__ballot_sync(0xffffffffu, in));
      unsigned near = __ballot_sync(0xffffffffu, j < c1 && !in && !out);
      n_near += __popc(near);
      for (; near; near &= near - 1) {  // float64, the whole warp
        const int n = j0 + __ffs(near) - 1;
        const int page = table[n];
        double x = 0.0;
        if (page >= 0 && page < p.n_pages) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(p.kbounds + (static_cast<int64_t>(page) * p.Hkv + g) * 256) + lane);
          const double* w = s_w + 128 * group + 8 * ch;
          x = w[0] * bf16_lo(u.x);
          x = fma(w[1], bf16_hi(u.x), x);
          x = fma(w[2], bf16_lo(u.y), x);
          x = fma(w[3], bf16_hi(u.y), x);
          x = fma(w[4], bf16_lo(u.z), x);
          x = fma(w[5], bf16_hi(u.z), x);
          x = fma(w[6], bf16_lo(u.w), x);
          x = fma(w[7], bf16_hi(u.w), x);
        }
        // the same tree for every block, so equal bounds give equal scores
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) s_key[n] = order_key(x);
      }
    }
  } else {
    for (int j = c0 + threadIdx.x; j < c1; j += NTHREADS) s_key[j] = kOut;
  }
  if (lane == 0) s_count[0][warp] = n_in, s_count[1][warp] = n_near;
  __syncthreads();
  n_in = n_near = 0;
#pragma unroll
  for (int i = 0; i < NWARPS; ++i) n_in += s_count[0][i], n_near += s_count[1][i];

  // ---- of the near ones the `take` greatest by float64: those above hi, and of [lo, hi] the first `take`
  unsigned long long lo = 1ull, hi = 1ull;
  int take = need - n_in;
  const bool all = take >= n_near;
  if (!all) {
    auto exact = [&](int j) { return s_key[j]; };
    radix_select<true>(s_radix, exact, c0, c1, take, lo, hi, take);
  }
  // ---- the chosen ids in ascending order: each warp a stretch of the blocks
  const int span = ((nb + NWARPS - 1) / NWARPS + 31) / 32 * 32;
  const int w0 = min(nb, warp * span), w1 = min(nb, w0 + span);
  auto state = [&](int j) {  // 2: chosen, 1: in the range, 0: not
    if (j >= w1) return 0;
    if (j < c0 || j >= c1) return 2;
    const unsigned long long k = s_key[j];
    if (k == kOut) return 0;
    return all || k > hi ? 2 : k >= lo ? 1 : 0;
  };
  auto before = [&](unsigned ball) { return __popc(ball & ((1u << lane) - 1u)); };
  int n_sure = 0, n_eq = 0;
  for (int j = w0; j < w1; j += 32) {
    const int s = state(j + lane);
    n_sure += __popc(__ballot_sync(0xffffffffu, s == 2));
    n_eq += __popc(__ballot_sync(0xffffffffu, s == 1));
  }
  __syncthreads();
  if (lane == 0) s_count[0][warp] = n_sure, s_count[1][warp] = n_eq;
  __syncthreads();
  int sure = 0, eq = 0;
#pragma unroll
  for (int i = 0; i < NWARPS; ++i) sure += i < warp ? s_count[0][i] : 0, eq += i < warp ? s_count[1][i] : 0;
  for (int j = w0; j < w1; j += 32) {
    const int s = state(j + lane);
    const unsigned bs = __ballot_sync(0xffffffffu, s == 2), be = __ballot_sync(0xffffffffu, s == 1);
    const int eq_before = eq + before(be);
    const int at = sure + before(bs) + min(eq_before, take);
    if (s == 2 || (s == 1 && eq_before < take)) ids[at] = j + lane;
    sure += __popc(bs);
    eq += __popc(be);
  }
}

}  // namespace sel
}  // namespace la
