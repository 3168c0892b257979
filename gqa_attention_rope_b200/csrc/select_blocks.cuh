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
// Everything is float64: the choice is an order, and sums in float32 would
// let the order of additions decide between near blocks. The first n_first and
// the last n_last blocks are always taken; of the others those with the
// greatest scores, of equal scores the lower index.
//
// One cluster of CTAs takes one (sequence, KV head): each CTA streams its
// share of the bounds (512 bytes per block, one 16-byte load per lane) and
// stores an order-preserving 64-bit key of every score into the first CTA's
// shared memory, which then finds the n_sel-th greatest by radix selection,
// 10 bits at a time from the highest bit in which the candidates differ, and
// writes the chosen ids in ascending order. What bounds it: HBM for the bounds
// of large batches, the chain of dependent steps for small ones.
#pragma once

#include "ptx.cuh"

namespace la {
namespace sel {

constexpr int NTHREADS = 512;
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
  double rope_theta;
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
__device__ __forceinline__ void store_to_first(uint32_t addr, unsigned long long x) {
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\tst.shared::cluster.u64 [r], %1;\n\t}" ::"r"(addr),
      "l"(x)
      : "memory");
}

// Order-preserving map of a score; NaN above every number.
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull;
  const long long b = __double_as_longlong(x + 0.0);  // -0 and 0 are one score
  return b < 0 ? ~static_cast<unsigned long long>(b) : static_cast<unsigned long long>(b) | (1ull << 63);
}

__device__ __forceinline__ double bf16_lo(uint32_t u) { return static_cast<double>(__uint_as_float(u << 16)); }
__device__ __forceinline__ double bf16_hi(uint32_t u) { return static_cast<double>(__uint_as_float(u & 0xFFFF0000u)); }

// grid (cluster size * B * Hkv): consecutive CTAs form the cluster of one
// (sequence, KV head). Dynamic shared memory: max_blocks keys.
__global__ void __launch_bounds__(NTHREADS) select_blocks_kernel(const Params p) {
  extern __shared__ unsigned long long s_key[];
  __shared__ double s_w[2][128];   // down (for the minima), up (for the maxima)
  __shared__ int s_hist[BINS];
  __shared__ int s_warp[2][NWARPS];
  __shared__ unsigned long long s_lo[NWARPS], s_hi[NWARPS];
  __shared__ int s_bin, s_above;

  const uint32_t rank = cluster_rank(), csize = cluster_size();
  const int64_t bg = blockIdx.x / csize;
  const int b = static_cast<int>(bg / p.Hkv), g = static_cast<int>(bg % p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    const double freq = pow(p.rope_theta, -2.0 * static_cast<double>(k) / 128.0);
    double sn, cs;
    sincos(static_cast<double>(len + p.q_pos_offset) * freq, &sn, &cs);
    double w[4] = {0.0, 0.0, 0.0, 0.0};
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(b) * p.Hq + g * p.G) * 128) + k;
    for (int h = 0; h < p.G; ++h) {
      const uint32_t u = q[h * 64];
      const double x0 = bf16_lo(u), x1 = bf16_hi(u);
      const double y0 = x0 * cs - x1 * sn, y1 = x0 * sn + x1 * cs;
      w[0] += fmin(y0, 0.0), w[1] += fmin(y1, 0.0), w[2] += fmax(y0, 0.0), w[3] += fmax(y1, 0.0);
    }
    s_w[0][2 * k] = w[0], s_w[0][2 * k + 1] = w[1], s_w[1][2 * k] = w[2], s_w[1][2 * k + 1] = w[3];
  }
  __syncthreads();
  // every CTA of the cluster has started before any of them stores into the first one
  if (csize > 1) cluster_sync();

  // ---- scores: 8 candidates at a time per warp
  const int c0 = p.n_first, c1 = nb - p.n_last;  // candidates [c0, c1); more than n_sel - n_first - n_last of them
  {
    double w[8];  // lanes 0-15: minima of channels 8 * lane.., lanes 16-31: maxima
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = s_w[lane >> 4][(lane & 15) * 8 + j];
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    const int step = static_cast<int>(csize) * NWARPS * 8;
    for (int j0 = c0 + (static_cast<int>(rank) * NWARPS + warp) * 8; j0 < c1; j0 += step) {
      int page = -1;
      if (lane < 8 && j0 + lane < c1) {
        page = table[j0 + lane];
        if (page < 0 || page >= p.n_pages) {
          raise_error(LLAMA_ATTN_DEVERR_BLOCK_TABLE);
          page = -1;
        }
      }
      uint4 u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, i);
        u[i] = make_uint4(0u, 0u, 0u, 0u);  // a block that is not there scores as zeros
        if (pg >= 0)
          u[i] = __ldg(reinterpret_cast<const uint4*>(p.kbounds + (static_cast<int64_t>(pg) * p.Hkv + g) * 256) + lane);
      }
      double v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        double x = w[0] * bf16_lo(u[i].x);
        x = fma(w[1], bf16_hi(u[i].x), x);
        x = fma(w[2], bf16_lo(u[i].y), x);
        x = fma(w[3], bf16_hi(u[i].y), x);
        x = fma(w[4], bf16_lo(u[i].z), x);
        x = fma(w[5], bf16_hi(u[i].z), x);
        x = fma(w[6], bf16_lo(u[i].w), x);
        v[i] = fma(w[7], bf16_hi(u[i].w), x);
      }
      // Sum each of the 8 over the 32 lanes: three steps that halve the number
      // of sums a lane carries, then two plain ones. Every candidate's sum is
      // taken over the same tree, so equal bounds give equal scores.
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        const int bit = 16 >> s, n = 4 >> s;
        const bool upper = lane & bit;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const double send = upper ? v[i] : v[i + n], mine = upper ? v[i + n] : v[i];
          v[i] = mine + __shfl_xor_sync(0xffffffffu, send, bit);
        }
      }
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
      if ((lane & 3) == 0) {
        const int j = j0 + (lane >> 2);  // lane bits 4, 3, 2 = candidate bits 2, 1, 0
        if (j < c1) store_to_first(smem_addr(s_key + j), order_key(v[0]));
      }
    }
  }
  if (csize > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank != 0) return;

  // ---- the first CTA: threshold of the `need` greatest candidates
  int need = p.n_sel - p.n_first - p.n_last;
  unsigned long long lo = ~0ull, hi = 0ull;
  for (int j = c0 + threadIdx.x; j < c1; j += NTHREADS) {
    const unsigned long long k = s_key[j];
    lo = k < lo ? k : lo;
    hi = k > hi ? k : hi;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long a = __shfl_xor_sync(0xffffffffu, lo, o), c = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = a < lo ? a : lo;
    hi = c > hi ? c : hi;
  }
  if (lane == 0) s_lo[warp] = lo, s_hi[warp] = hi;
  __syncthreads();
  for (int i = 0; i < NWARPS; ++i) {
    lo = s_lo[i] < lo ? s_lo[i] : lo;
    hi = s_hi[i] > hi ? s_hi[i] : hi;
  }
  // Keys above `thr` are chosen, and of those equal to it the first `need`
  // (all of them where take_equal).
  unsigned long long thr = lo;
  bool take_equal = false;
  if (need == 0) {
    thr = ~0ull;
  } else if (lo != hi) {
    const int top = 63 - __clzll(static_cast<long long>(lo ^ hi));
    int shift = top > 9 ? top - 9 : 0;
    unsigned long long prefix = shift + 10 < 64 ? hi >> (shift + 10) : 0ull;
    int bits = 10;
    for (;;) {
      for (int i = threadIdx.x; i < BINS; i += NTHREADS) s_hist[i] = 0;
      __syncthreads();
      for (int j = c0 + threadIdx.x; j < c1; j += NTHREADS) {
        const unsigned long long k = s_key[j];
        const unsigned long long top_bits = shift + bits < 64 ? k >> (shift + bits) : 0ull;
        if (top_bits == prefix) atomicAdd(&s_hist[static_cast<int>((k >> shift) & ((1u << bits) - 1u))], 1);
      }
      __syncthreads();
      // suffix sums over the bins, two bins per thread, the highest bins first
      const int i0 = BINS - 1 - 2 * static_cast<int>(threadIdx.x), i1 = i0 - 1;
      const int n0 = s_hist[i0], n1 = s_hist[i1];
      int sum = n0 + n1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) s_warp[0][warp] = sum;
      __syncthreads();
      int above = sum - n0 - n1;
      for (int i = 0; i < warp; ++i) above += s_warp[0][i];
      if (above < need && above + n0 >= need) s_bin = i0, s_above = above;
      if (above + n0 < need && above + n0 + n1 >= need) s_bin = i1, s_above = above + n0;
      __syncthreads();
      const int bin = s_bin, in_bin = s_hist[bin];
      need -= s_above;
      prefix = (prefix << bits) | static_cast<unsigned long long>(bin);
      __syncthreads();
      if (in_bin == need) {  // the whole bin
        thr = prefix << shift;
        take_equal = true;
        break;
      }
      if (shift == 0) {  // equal keys: the first `need` of them
        thr = prefix;
        break;
      }
      bits = shift < 10 ? shift : 10;
      shift -= bits;
    }
  }

  // ---- the chosen ids in ascending order: each warp a stretch of the blocks
  const int span = ((nb + NWARPS - 1) / NWARPS + 31) / 32 * 32;
  const int w0 = min(nb, warp * span), w1 = min(nb, w0 + span);
  auto state = [&](int j) {  // 2: chosen, 1: at the threshold, 0: not
    if (j >= w1) return 0;
    if (j < c0 || j >= c1) return 2;
    const unsigned long long k = s_key[j];
    if (need == 0 && !take_equal) return 0;
    return k > thr || (take_equal && k == thr) ? 2 : k == thr ? 1 : 0;
  };
  auto chosen_in = [&](unsigned ball) { return __popc(ball & ((1u << lane) - 1u)); };
  int n_sure = 0, n_eq = 0;
  for (int j = w0; j < w1; j += 32) {
    const int s = state(j + lane);
    n_sure += __popc(__ballot_sync(0xffffffffu, s == 2));
    n_eq += __popc(__ballot_sync(0xffffffffu, s == 1));
  }
  if (lane == 0) s_warp[0][warp] = n_sure, s_warp[1][warp] = n_eq;
  __syncthreads();
  int sure = 0, eq = 0;
  for (int i = 0; i < warp; ++i) sure += s_warp[0][i], eq += s_warp[1][i];
  for (int j = w0; j < w1; j += 32) {
    const int s = state(j + lane);
    const unsigned bs = __ballot_sync(0xffffffffu, s == 2), be = __ballot_sync(0xffffffffu, s == 1);
    const int eq_before = eq + chosen_in(be);
    const int at = sure + chosen_in(bs) + min(eq_before, need);
    if (s == 2 || (s == 1 && eq_before < need)) ids[at] = j + lane;
    sure += __popc(bs);
    eq += __popc(be);
  }
}

}  // namespace sel
}  // namespace la
