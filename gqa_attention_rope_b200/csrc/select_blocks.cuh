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
// Most blocks are far from the border, so the scores are first formed in
// float32: a weight's rounding, 8 products and sums per lane and 5 sums over
// the lanes stay within eps = 2^-20 sum_d |w_d| max |bound| (14 roundings of
// 2^-24) and, where numbers are below float32's normal range, what that adds: 2^-150
// for each of 256 weights, times max |bound|, and for each of fewer than 2^9 sums;
// together below 2^-141 (max |bound| + 1). A radix selection over these scores finds a range [lo, hi] that holds
// the one at the border; blocks outside [lo - 2 eps, hi + 2 eps] are decided by
// it, and the few inside get their float64 score and are ranked by it.
// For 64 sequences of 1024 to 32768 rows (8 KV heads, 64-row blocks, 71 MB of
// bounds) that takes 28 us; all scores in float64 39 us; scores on the tensor
// cores (three bf16 terms of the weights as columns of one product) 42 us, with
// a bound of 2^-15 only, which left several blocks near.
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

constexpr int kNearCap = 64;  // near blocks that are ranked pair by pair

// grid (cluster size * B * Hkv): consecutive CTAs form the cluster of one
// (sequence, KV head). Dynamic shared memory: 8 bytes per block of a sequence.
__global__ void __launch_bounds__(NTHREADS, 4) select_blocks_kernel(const Params p) {
  extern __shared__ unsigned long long s_key[];  // the scores' 32-bit keys, then (many near blocks) kIn, kOut or a float64's key
  __shared__ __align__(16) double s_w[256];      // weights of the minima (down), then of the maxima (up)
  __shared__ RadixShared s_radix;
  __shared__ uint32_t s_mag[8 * NWARPS];         // per warp of the cluster: greatest magnitude of a bound, float bits
  __shared__ double s_wsum[2];
  __shared__ uint32_t s_in[MAX_BLOCKS / 32], s_eq[MAX_BLOCKS / 32];  // a bit per block: chosen; one of the first `take` of these
  __shared__ int s_near[kNearCap];
  __shared__ unsigned long long s_near_key[kNearCap];
  __shared__ int s_n_in, s_n_near;
  __shared__ int s_scan[2][NWARPS];

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
  const int nb = static_cast<int>((static_cast<unsigned>(len) + p.page_size - 1u) / p.page_size);  // len + page_size may pass 2^31
  int32_t* ids = p.ids + bg * p.n_sel;
  if (nb <= p.n_sel) {  // every block; the whole cluster leaves here
    if (rank == 0)
      for (int i = threadIdx.x; i < p.n_sel; i += NTHREADS) ids[i] = i < nb ? i : -1;
    return;
  }
  const int c0 = p.n_first, c1 = nb - p.n_last;  // candidates [c0, c1); more than n_sel - n_first - n_last of them
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
  const int step = static_cast<int>(csize) * NWARPS * 8;
  const int j_first = c0 + (static_cast<int>(rank) * NWARPS + warp) * 8;
  auto page_at = [&](int j0) { return lane < 8 && j0 + lane < c1 ? table[j0 + lane] : 0; };
  int page = page_at(j_first);
  uint4 u[2][4];  // bounds of 8 blocks: lanes 0-15 minima of channels 8 * lane.., lanes 16-31 maxima
  auto fetch = [&](int half, int pages, int j0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pg = __shfl_sync(0xffffffffu, pages, 4 * half + i);
      u[half][i] = make_uint4(0u, 0u, 0u, 0u);  // a block that is not there scores as zeros
      if (j0 + 4 * half + i < c1) {
        if (pg >= 0 && pg < p.n_pages)
          u[half][i] = *(reinterpret_cast<const uint4*>(p.kbounds + (static_cast<int64_t>(pg) * p.Hkv + g) * 256) + lane);
        else if (lane == 0)
          raise_error(LLAMA_ATTN_DEVERR_BLOCK_TABLE);
      }
    }
  };
  fetch(0, page, j_first);
  fetch(1, page, j_first);
  page = page_at(j_first + step);

  // ---- the group's weights: up_d, down_d of the query rotated at its position
  if (threadIdx.x < 64) {
    const int k = threadIdx.x;
    double sn, cs;
    sincos(static_cast<double>(len + p.q_pos_offset) * p.freqs.theta[k], &sn, &cs);
    double w[4] = {0.0, 0.0, 0.0, 0.0};
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(b) * p.Hq + g * p.G) * 128) + k;
#pragma unroll 4
    for (int h = 0; h < p.G; ++h) {
      const uint32_t x = q[h * 64];
      const double x0 = bf16_lo(x), x1 = bf16_hi(x);
      const double y0 = x0 * cs - x1 * sn, y1 = x0 * sn + x1 * cs;
      w[0] += fmin(y0, 0.0), w[1] += fmin(y1, 0.0), w[2] += fmax(y0, 0.0), w[3] += fmax(y1, 0.0);
    }
    s_w[2 * k] = w[0], s_w[2 * k + 1] = w[1], s_w[128 + 2 * k] = w[2], s_w[128 + 2 * k + 1] = w[3];
    double sum = (w[2] - w[0]) + (w[3] - w[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_wsum[warp] = sum;
  }
  if (threadIdx.x == 64) s_n_in = s_n_near = 0;
  // every CTA of the cluster has started before any of them stores into the first one
  if (csize > 1)
    cluster_sync();
  else
    __syncthreads();

  // ---- scores, 8 candidates at a time per warp, the next ones' bounds on their way
  const double* lane_w = s_w + 8 * lane;
  {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = static_cast<float>(lane_w[i]);
    uint32_t mag = 0u;
    for (int j0 = j_first; j0 < c1; j0 += step) {
      const int page2 = page_at(j0 + 2 * step);
      float v[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = u[half][i];
          const float2 a = unpack_bf16x2(x.x), e = unpack_bf16x2(x.y), f = unpack_bf16x2(x.z), h = unpack_bf16x2(x.w);
          float y = w[0] * a.x;
          y = fmaf(w[1], a.y, y);
          y = fmaf(w[2], e.x, y);
          y = fmaf(w[3], e.y, y);
          y = fmaf(w[4], f.x, y);
          y = fmaf(w[5], f.y, y);
          y = fmaf(w[6], h.x, y);
          v[4 * half + i] = fmaf(w[7], h.y, y);
          mag = max_abs(mag, max_abs(max_abs(x.x, x.y), max_abs(x.z, x.w)));
        }
        fetch(half, page, j0 + step);
      }
      page = page2;
      // Sum each of the 8 over the 32 lanes: three steps that halve the number
      // of sums a lane carries, then two plain ones.
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        const int bit = 16 >> s, n = 4 >> s;
        const bool upper = lane & bit;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float send = upper ? v[i] : v[i + n], mine = upper ? v[i + n] : v[i];
          v[i] = mine + __shfl_xor_sync(0xffffffffu, send, bit);
        }
      }
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
      const int j = j0 + (lane >> 2);  // lane bits 4, 3, 2 = candidate bits 2, 1, 0
      if ((lane & 3) == 0 && j < c1) store_to_first32(smem_addr(s_key + j), order_key(v[0]));
    }
    // magnitudes order like their bits
    mag = __reduce_max_sync(0xffffffffu, max((mag << 16) & 0x7FFF0000u, mag & 0x7FFF0000u));
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
  float lo = INFINITY, hi = INFINITY;  // need == 0: no candidate reaches lo
  if (need > 0) {
    uint32_t mag = lane < static_cast<int>(csize) * NWARPS ? s_mag[lane] : 0u;
    if (lane + 32 < static_cast<int>(csize) * NWARPS) mag = max(mag, s_mag[lane + 32]);
    mag = __reduce_max_sync(0xffffffffu, mag);
    const double bound = __uint_as_float(mag);
    const float eps2 = __double2float_ru(2.0 * (0x1p-20 * (s_wsum[0] + s_wsum[1]) * bound + 0x1p-141 * (bound + 1.0)));
    uint32_t klo, khi;
    int unused;
    radix_select<false>(s_radix, approx, c0, c1, need, klo, khi, unused);
    lo = __fsub_rd(score_of(klo), eps2);
    hi = __fadd_ru(score_of(khi), eps2);
  }
  // 2: chosen, 1: near, 0: not chosen. A NaN is near, whatever else it is.
  auto decide = [&](int j) {
    if (j < c0 || j >= c1) return 2;
    if (need == 0) return 0;
    const float x = score_of(approx(j));
    return x > hi ? 2 : x < lo ? 0 : 1;
  };
  const int nb32 = (nb + 31) & ~31;
  int mine_in = 0;
#pragma unroll 4
  for (int j0 = warp * 32; j0 < nb32; j0 += NTHREADS) {
    const int j = j0 + lane, d = j < nb ? decide(j) : 0;
    const unsigned in = __ballot_sync(0xffffffffu, d == 2), near = __ballot_sync(0xffffffffu, d == 1);
    mine_in += __popc(in);
    if (lane == 0) s_in[j0 >> 5] = in, s_eq[j0 >> 5] = 0u;
    if (near) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_n_near, __popc(near));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(near & ((1u << lane) - 1u));
      if (d == 1 && at < kNearCap) s_near[at] = j;
    }
  }
  if (lane == 0 && mine_in) atomicAdd(&s_n_in, mine_in);
  __syncthreads();
  const int n_near = s_n_near;
  int take = p.n_sel - s_n_in;  // of the near ones
  // float64 score of block j, by a whole warp; the same tree for every block,
  // so equal bounds give equal scores
  auto exact = [&](int j) {
    const int pg = table[j];
    double x = 0.0;
    if (pg >= 0 && pg < p.n_pages) {
      const uint4 y = *(reinterpret_cast<const uint4*>(p.kbounds + (static_cast<int64_t>(pg) * p.Hkv + g) * 256) + lane);
      x = lane_w[0] * bf16_lo(y.x);
      x = fma(lane_w[1], bf16_hi(y.x), x);
      x = fma(lane_w[2], bf16_lo(y.y), x);
      x = fma(lane_w[3], bf16_hi(y.y), x);
      x = fma(lane_w[4], bf16_lo(y.z), x);
      x = fma(lane_w[5], bf16_hi(y.z), x);
      x = fma(lane_w[6], bf16_lo(y.w), x);
      x = fma(lane_w[7], bf16_hi(y.w), x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return order_key(x);
  };
  if (n_near <= kNearCap) {
    if (take < n_near) {
      for (int i = warp; i < n_near; i += NWARPS) {
        const unsigned long long k = exact(s_near[i]);
        if (lane == 0) s_near_key[i] = k;
      }
      __syncthreads();
    }
    if (static_cast<int>(threadIdx.x) < n_near) {
      const int j = s_near[threadIdx.x];
      int above = 0;  // near blocks that come before this one
      if (take < n_near) {
        const unsigned long long k = s_near_key[threadIdx.x];
        for (int i = 0; i < n_near; ++i) above += s_near_key[i] > k || (s_near_key[i] == k && s_near[i] < j) ? 1 : 0;
      }
      if (above < take) atomicOr(&s_in[j >> 5], 1u << (j & 31));
    }
  } else {
    // many near blocks (equal or nearly equal bounds): all their float64 scores, and a second selection
    for (int j0 = c0 + warp * 32; j0 < c1; j0 += NTHREADS) {
      const int j = j0 + lane, d = j < c1 ? decide(j) : 0;
      __syncwarp();
      if (j < c1 && d != 1) s_key[j] = d == 2 ? kIn : kOut;
      for (unsigned near = __ballot_sync(0xffffffffu, d == 1); near; near &= near - 1) {
        const int n = j0 + __ffs(near) - 1;
        const unsigned long long k = exact(n);
        if (lane == 0) s_key[n] = k;
      }
    }
    __syncthreads();
    unsigned long long klo = 1ull, khi = 1ull;
    const bool all = take >= n_near;
    if (!all) radix_select<true>(s_radix, [&](int j) { return s_key[j]; }, c0, c1, take, klo, khi, take);
    for (int j0 = warp * 32; j0 < nb32; j0 += NTHREADS) {
      const int j = j0 + lane;
      const unsigned long long k = j >= c0 && j < c1 ? s_key[j] : kOut;
      const bool near = k != kIn && k != kOut;
      const unsigned in = __ballot_sync(0xffffffffu, near && (all || k > khi));
      const unsigned eq = __ballot_sync(0xffffffffu, near && !all && k >= klo && k <= khi);
      if (lane == 0) s_in[j0 >> 5] |= in, s_eq[j0 >> 5] = eq;
    }
  }
  if (n_near <= kNearCap) take = 0;  // nothing is in s_eq
  __syncthreads();

  // ---- the chosen ids in ascending order: a thread has a stretch of words
  const int words = nb32 >> 5, per = (words + NTHREADS - 1) / NTHREADS;
  const int w0 = min(words, static_cast<int>(threadIdx.x) * per), w1 = min(words, w0 + per);
  int n_in = 0, n_eq = 0;
  for (int w = w0; w < w1; ++w) n_in += __popc(s_in[w]), n_eq += __popc(s_eq[w]);
  int in_before = n_in, eq_before = n_eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, in_before, o), y = __shfl_up_sync(0xffffffffu, eq_before, o);
    if (lane >= o) in_before += x, eq_before += y;
  }
  if (lane == 31) s_scan[0][warp] = in_before, s_scan[1][warp] = eq_before;
  __syncthreads();
  in_before -= n_in;
  eq_before -= n_eq;
  for (int i = 0; i < warp; ++i) in_before += s_scan[0][i], eq_before += s_scan[1][i];
  for (int w = w0; w < w1; ++w) {
    const uint32_t in = s_in[w], eq = s_eq[w];
    for (uint32_t rest = in | eq; rest; rest &= rest - 1) {
      const int bit = __ffs(rest) - 1;
      if (in >> bit & 1) {
        ids[in_before + min(eq_before, take)] = 32 * w + bit;
        ++in_before;
      } else {
        if (eq_before < take) ids[in_before + eq_before] = 32 * w + bit;
        ++eq_before;
      }
    }
  }
}

}  // namespace sel
}  // namespace la
