// decode_paged.cuh -- single-token GQA decode over a paged cache of E4M3 codes
// with a scale per (page, KV head), and over chosen blocks of a paged cache
// (E4M3 or bf16): the work of the whole batch is cut into runs of equal cost, one per
// resident CTA.
//
// Mathematics, for the query heads h of a KV group and the cache rows n that
// the call names (all rows below len, or those of the chosen blocks):
//   s_hn = (q_h . k_n) ks_n / sqrt(128) in log2 units,  o_h = sum_n 2^(s_hn - M) vs_n v_n / sum_n 2^(s_hn - M)
// with k_n, v_n the codes and ks_n, vs_n the scales of row n's block (1 for
// bf16). A row's value scale is put into its exponent: P_hn = 2^(s_hn + log2
// vs_n - m) with m a running bound of the whole exponent, so P stays within
// range of 16 bits whatever the scales are. The denominator is a sum of its own:
// where value scales differ by 2^100 and more, a row may vanish as P and still have
// most of the weight (a block of zeros, which the append gives the scale 2^-100,
// next to one of scale 2^40). It adds 2^(s_hn + log2 vs_n - m + d - log2 vs_n), with
// d such that m - d is a running bound of the scores alone, and the result is
// O 2^d / L. On bf16 pages all scales are 1, d is 0 and P serves both sums. The
// second exponential costs two tiles of heads 6% (one 131072-row sequence under
// 128 heads 55.2 -> 58.6 us) and one tile 1%; forming it only where scales are far
// apart took more (registers of the rare path spill: 59 to 64 us).
//
// What bounds it: HBM. A row of an E4M3 cache is 256 bytes for 4 * 128 * G
// flop. Times here are of a call in a CUDA graph of ten; a program's calls one after
// another take 0.5 us (short ones) to 3% more. 64 sequences of 1024 to 32768 rows,
// 64 heads over 8: 342 us, 6480 GB/s (99% of a copy's rate; 350 us and 97% as calls);
// two tiles of heads (G > 8) 58 us for 131072 rows, 4630 GB/s, bound by a warp's
// chain of conversions, products and exponentials (168 registers, 60 to 88 bytes
// spilled); short caches by latency (one sequence of 1000 rows, 32 heads: 5.6 us).
// The products run on mma.sync m16n8k16 with the 16 cache rows of a warp as M
// and the heads of the group as N (8 or 16): S^T = K Q^T, O^T = V^T P^T.
// With heads as M, groups of 8 heads would leave half of each product empty.
// E4M3 codes become f16 exactly (cvt.rn.f16x2.e4m3x2), so K and V carry no
// rounding beyond their own; Q is rounded to f16 after its row is brought to
// [0.5, 1) by a power of two (2^-11 relative; bf16 would be 2^-8), P to f16.
// On bf16 pages the products are bf16: Q and P are sums of two bf16 terms (2^-16
// relative). With one term for P (2^-8) the error to float64 was 2.3e-3 of the
// outputs' size instead of the 1.7e-3 of the output's own rounding (16 sequences of
// 8192-32768 rows, 64 blocks); the second term costs under 1% of the time.
// The 8-bit rows are loaded with the 16-bit ldmatrix: each 32-bit register
// then holds 4 neighbouring codes of a key, or 2 codes of 2 neighbouring rows
// of V (transposed form). The products sum over d in any order, so Q is laid
// out to match, and V's even and odd channels go to rows i and i + 8 of a tile.
//
// Work split: a unit is one 64-row stage of one (sequence, KV head). All units
// of the batch in the order (sequence, head, stage) are cut into gridDim.x
// runs of equal cost, so ragged lengths leave no CTA idle and the ring of
// stages never drains between sequences. A unit costs 1, and each (sequence,
// head) PAIR_COST more ahead of its first one: its query, and the join of the
// warps. 64 sequences of 1 to 4000 rows (log-uniform), 8 KV heads, with 0, 3, 6
// and 10 for that: 67, 53, 51 and 52 us; 40 sequences of 1 to 1000: 27, 16, 16
// and 16; equal lengths the same with each. A (sequence, head) inside one run is written to
// the output directly; one that spans several leaves partial results (at most
// two per CTA: its first and its last), which decode_join_kernel merges in
// the order of the runs: the result does not depend on timing.
// Short batches have a second form: a cluster of CTAs per (sequence, head), which
// cut its stages among themselves and join their results through one another's
// shared memory; no kernel follows (one sequence of 1000 rows 5.6 us, 8.0 as runs).
// The block table's width decides, since the host does not know the lengths: under
// a table of many blocks short sequences run in the first form.
#pragma once

#include <cuda_fp16.h>

#include "ptx.cuh"
#include "rope.cuh"
#include "runs.cuh"

namespace la {
namespace dpg {

constexpr int ROWS = 64;                  // cache rows of a stage
constexpr int NRW = 4;                    // row groups: 16 rows of a stage each
constexpr float kLift = 7.f;              // P of the greatest row: 2^7
constexpr float kSlack = 8.f;             // the bounds move when a row passes them by more: P <= 2^15, weights <= 2^8
constexpr int MAX_CLUSTER = 16;
constexpr int MAX_CTAS = 512;             // runs (and twice as many partial results) the workspace holds

// kWide: more than 8 query heads per KV head, two tiles of 8 (NT). Four compute
// warps have 16 rows of a stage each, one more warp loads.
template <bool kE4M3, bool kWide>
struct Tile {
  static constexpr int NT = kWide ? 2 : 1;
  static constexpr int NCW = NRW;
  static constexpr int NTHREADS = (NCW + 1) * 32;
  // Both tiles in one warp, 2 CTAs per SM, query in registers: one 131072-row
  // sequence under 128 heads 58.5 us (all of these with one exponential for both
  // sums, in its first form); 3 CTAs with the query in shared memory
  // (128 registers) 76 us; a tile per warp and eight compute warps (every code
  // converted twice) 63 us; the next stage's scores formed before this one's
  // values (spills) 80 us. One tile for 64 heads over 8: 341 us for the 70B
  // batch, 391 us when the empty second tile is computed along.
  static constexpr int CTAS = 2;
  static constexpr bool Q_REGS = kE4M3 || !kWide;  // query fragments in registers (two tiles of two bf16 terms: 64)
  static constexpr uint32_t HALF = ROWS * 128;                    // 64 rows x 128 bytes
  static constexpr uint32_t TENSOR = kE4M3 ? HALF : 2 * HALF;     // K or V of a stage
  static constexpr uint32_t STAGE = 2 * TENSOR;
  static constexpr int NSTAGE = kE4M3 ? 6 : 3;                    // 192 KB of stages per SM
  // One region for two uses that never overlap in time: the query rows (f16,
  // or two bf16 terms) until a segment's last product, and the merge scratch
  // (two warps x 8 heads x 64 channels, float) behind it.
  static constexpr uint32_t OFF_Q = NSTAGE * STAGE;
  static constexpr uint32_t OFF_SCR = OFF_Q;
  static constexpr uint32_t Q_ROW = 264;                          // bytes: 128 16-bit values, 8 bytes of padding
  static constexpr uint32_t OFF_META = OFF_Q + (kE4M3 || !kWide ? 16 : 32) * Q_ROW;
  static constexpr uint32_t OFF_BAR = OFF_META + NSTAGE * 16;
  static constexpr uint32_t OFF_ML = OFF_BAR + 128;               // per warp and head: m, d, l
  static constexpr uint32_t OFF_CS = OFF_ML + NCW * 16 * 16;      // (cos, sin) row of the segment
  static constexpr uint32_t OFF_QS = OFF_CS + 64 * 8;             // per head: factor of the query row
  static constexpr uint32_t OFF_D = OFF_QS + 64;                  // per warp and head: d, where it is not in registers
  static constexpr uint32_t SMEM_ALLOC = OFF_D + NCW * 16 * 4 + 1024;
};

struct Params {
  int B, Hq, Hkv, G, page_size, max_blocks, n_pages;
  const int32_t* lens;
  const int32_t* block_table;
  const int32_t* block_ids;   // [B, Hkv, n_sel], chosen blocks only
  int n_sel;
  const uint16_t* q;          // [B, Hq, 128] bf16 bits
  int q_pos_offset;
  const float* kscales;       // [n_pages, Hkv], E4M3 only
  const float* vscales;
  float scale_log2;
  RopeFreqs freqs;
  uint16_t* out;              // [B, Hq, 128] bf16
  float* lse;                 // [B, Hq] or null
  float* part_o;              // [2 * MAX_CTAS][G][128]
  float4* part_ml;            // [2 * MAX_CTAS][G]: m, d, l
  int* prefix;                // [B + 1] cost before each sequence
  int4* ends;                 // [MAX_CTAS] (sequence, KV head, first run) of a pair that ends in a run but began before
  unsigned int epoch;
};

// Stages of one (sequence, KV head).
__device__ __forceinline__ int ceil_div(int a, int b) {  // a + b may pass 2^31
  return static_cast<int>((static_cast<unsigned>(a) + static_cast<unsigned>(b) - 1u) / static_cast<unsigned>(b));
}
template <bool kSparse>
__device__ __forceinline__ int stages_of(const Params& p, int b) {
  const int len = p.lens[b];
  if (len <= 0 || len > static_cast<int64_t>(p.max_blocks) * p.page_size) return 0;
  if constexpr (kSparse) {
    return min(ceil_div(len, p.page_size), p.n_sel) * (p.page_size / ROWS);
  }
  return ceil_div(len, ROWS);
}

template <bool kSparse>
__device__ __forceinline__ void advance(const Params& p, Cursor& c, int by) {
  advance([&](int b) { return stages_of<kSparse>(p, b); }, p.B, p.Hkv, c, by);
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The two codes in the low (high) half of w as f16x2.
__device__ __forceinline__ uint32_t f16x2_of_lo(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t f16x2_of_hi(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The greatest of a warp's values (NaN are passed over).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Factor of a sum whose exponents are relative to x where `top` is the greatest
// such reference; a sum of no row is 0 (or a NaN).
__device__ __forceinline__ float rebase(float x, float top) { return x == -INFINITY ? 1.f : ex2_approx(x - top); }
// The unit m - d of a denominator, relative to M (m = -inf: no row).
__device__ __forceinline__ float unit_of(const float4& v, float M) { return v.x == -INFINITY ? -INFINITY : (v.x - M) - v.y; }
// From O to the output, 2^d / l, for v = (m, d, l). d lies within [-115, 120] (value
// scales within [2^-100, 2^119], m behind the greatest exponent by kLift to kLift +
// kSlack, m - d behind the greatest score by up to kSlack) and l may be as great as
// 2^39 (on bf16 pages d is 0 and l at most 2^46), so neither factor alone leaves
// float32's range.
struct Norm {
  float inv, f;
  __device__ __forceinline__ explicit Norm(const float4& v) : inv(v.z == 0.f ? 0.f : 1.f / v.z), f(v.z == 0.f ? 0.f : ex2_approx(v.y)) {}
  __device__ __forceinline__ float operator()(float x) const { return x * inv * f; }
};
__device__ __forceinline__ float lse_of(const float4& v) {
  return v.z == 0.f ? -INFINITY : (v.x + (log2f(v.z) - v.y)) * 0.6931471805599453f;
}

// Sequences without rows: zeros, dealt out over the CTAs; `n` threads of each.
template <bool kSparse>
__device__ __forceinline__ void clear_empty(const Params& p, int n) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (stages_of<kSparse>(p, b) > 0) continue;
    const int len = p.lens[b];
    if (threadIdx.x == 0 && (len < 0 || len > static_cast<int64_t>(p.max_blocks) * p.page_size))
      raise_error(LLAMA_ATTN_DEVERR_CACHE_LEN);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(b) * p.Hq * 128);
    for (int i = threadIdx.x; i < p.Hq * 64; i += n) dst[i] = 0u;
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += n) p.lse[static_cast<int64_t>(b) * p.Hq + i] = -INFINITY;
  }
}

// kWide: more than 8 query heads per KV head (two tiles of 8).
// kCluster: a cluster of CTAs per (sequence, KV head) instead of runs over the
// batch; they cut the pair's stages among themselves and join their results
// through one another's shared memory, so nothing is left for a second kernel.
template <bool kE4M3, bool kSparse, bool kWide, bool kCluster>
__global__ void __launch_bounds__((Tile<kE4M3, kWide>::NTHREADS), (Tile<kE4M3, kWide>::CTAS))
    decode_runs_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const Params p) {
  using T = Tile<kE4M3, kWide>;
  constexpr int NT = T::NT, NCW = T::NCW, NTHREADS = T::NTHREADS;
  constexpr int NQ = kE4M3 ? 1 : 2, NP = NQ;  // terms of Q and of P
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  auto full = [&](uint32_t s) { return sbase + T::OFF_BAR + 8u * s; };
  auto empty = [&](uint32_t s) { return sbase + T::OFF_BAR + 8u * (T::NSTAGE + s); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{p.epoch};

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::NSTAGE; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), NCW);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  grid_launch_dependents();
  grid_dependency_wait();
  Cut cut(1, 1);
  int u0 = 0, u1 = 0;  // this CTA's units
  int first_cost = 0;  // of the first unit of the pair that this CTA begins in
  Cursor cur;
  const uint32_t rank = kCluster ? cluster_rank() : 0u, csize = kCluster ? cluster_size() : 1u;
  if constexpr (kCluster) {
    const int pair = blockIdx.x / csize;
    cur = Cursor{pair / p.Hkv, pair % p.Hkv, 0, 0};
    cur.nst = stages_of<kSparse>(p, cur.b);
    if (cur.nst == 0) {  // no rows: zeros, and the whole cluster leaves
      if (rank == 0) {
        const int len = p.lens[cur.b];
        if (threadIdx.x == 0 && cur.g == 0 && (len < 0 || len > static_cast<int64_t>(p.max_blocks) * p.page_size))
          raise_error(LLAMA_ATTN_DEVERR_CACHE_LEN);
        const int64_t head = static_cast<int64_t>(cur.b) * p.Hq + cur.g * p.G;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + head * 128);
        for (int i = threadIdx.x; i < p.G * 64; i += NTHREADS) dst[i] = 0u;
        if (p.lse && static_cast<int>(threadIdx.x) < p.G) p.lse[head + threadIdx.x] = -INFINITY;
      }
      return;
    }
    __syncthreads();  // the barriers are there
    const int n_runs = min(static_cast<int>(csize), cur.nst);
    cut = Cut(cur.nst, n_runs);
    if (static_cast<int>(rank) < n_runs) u0 = cut.start(rank), u1 = cut.start(rank + 1);
    cur.s = u0;
  } else {
    __shared__ int4 s_start;
    __shared__ int3 s_range;  // first and last unit, cost of the first pair's first unit
    __shared__ int2 s_part[NTHREADS];
    // Cost and units before this thread's share of the sequences, and the cost
    // in all: thread i takes sequences [i * per, (i + 1) * per).
    const int per = (p.B + NTHREADS - 1) / NTHREADS;
    const int my0 = min(p.B, static_cast<int>(threadIdx.x) * per), my1 = min(p.B, my0 + per);
    {
      int2 sum = make_int2(0, 0);
      for (int b = my0; b < my1; ++b) {
        const int nst = stages_of<kSparse>(p, b);
        sum.x += cost_of(nst) * p.Hkv, sum.y += nst * p.Hkv;
      }
      s_part[threadIdx.x] = sum;
    }
    __syncthreads();
    int2 before = make_int2(0, 0);
    int total = 0, units = 0;
    for (int i = 0; i < NTHREADS && i * per < p.B; ++i) {
      if (i == static_cast<int>(threadIdx.x)) before = make_int2(total, units);
      total += s_part[i].x, units += s_part[i].y;
    }
    if (my0 < p.B && blockIdx.x == 0) {  // the joining kernel reads these
      int at = before.x;
      for (int b = my0; b < my1; ++b) {
        p.prefix[b] = at;
        at += cost_of(stages_of<kSparse>(p, b)) * p.Hkv;
      }
      if (my1 == p.B) p.prefix[p.B] = at;
    }
    if (threadIdx.x == 0) p.ends[blockIdx.x] = make_int4(-1, 0, 0, 0);
    const int n_runs = min(static_cast<int>(gridDim.x), total);
    if (static_cast<int>(blockIdx.x) >= n_runs) {
      clear_empty<kSparse>(p, NTHREADS);
      return;
    }
    cut = Cut(total, n_runs);
    const int c0 = cut.start(blockIdx.x), c1 = cut.start(blockIdx.x + 1) - 1;  // first and last cost
    if (my0 < my1) {  // one thread finds the start, one the end
      int at = before.x, u = before.y;
      const int end = at + s_part[threadIdx.x].x;
      for (int b = my0; b < my1 && at <= c1 && c0 < end; ++b) {
        const int nst = stages_of<kSparse>(p, b), n = cost_of(nst) * p.Hkv;
        if (at <= c0 && c0 < at + n) {
          const RunBegin begin(c0, at, u, nst);
          s_start = make_int4(b, begin.g, begin.s, nst);
          s_range.x = begin.unit;
          s_range.z = begin.first_cost;
        }
        if (c1 < at + n) {
          s_range.y = run_end(c1, at, u, nst);
          break;
        }
        at += n, u += nst * p.Hkv;
      }
    }
    __syncthreads();
    u0 = s_range.x;
    u1 = s_range.y;
    first_cost = s_range.z;
    if (u0 == u1) {  // costs of no unit
      clear_empty<kSparse>(p, NTHREADS);
      return;
    }
    cur = Cursor{s_start.x, s_start.y, s_start.z, s_start.w};
  }

  if (warp == NCW) {
    // ------------------------------------------------------------ producer
    // The lanes resolve 32 units at a time, in three steps that depend on one
    // another's loads: chosen block ids, pages, scales. Each step runs a batch
    // ahead of the next, so that its loads have a batch's time to arrive.
    const int rpp = p.page_size;
    Cursor c = cur;
    int u = u0 + lane;
    if (lane > 0) advance<kSparse>(p, c, lane);
    struct Ids {
      Cursor c;
      int len, id, prev;  // len 0: no unit
    };
    struct Page {
      int g, n, nvalid, page;  // first cache row, rows below len (0: nothing to load)
    };
    struct Unit {
      int row, nvalid;  // first row in the pool
      float ks, vs;
    };
    auto load_ids = [&]() {  // and on to the next batch
      Ids r{c, 0, 0, -2};
      if (u >= u1) return r;
      r.len = p.lens[c.b];
      if constexpr (kSparse) {
        const int e = c.s / (rpp / ROWS);
        const int32_t* ids = p.block_ids + (static_cast<int64_t>(c.b) * p.Hkv + c.g) * p.n_sel;
        r.id = ids[e];
        if (e > 0) r.prev = ids[e - 1];
      }
      u += 32;
      if (u < u1) advance<kSparse>(p, c, 32);
      return r;
    };
    auto load_page = [&](const Ids& a) {
      Page r{a.c.g, 0, 0, 0};
      if (a.len == 0) return r;
      if constexpr (kSparse) {
        const int spp = rpp / ROWS, e = a.c.s / spp, nb = ceil_div(a.len, rpp);
        // ascending, no id twice, -1 only behind the last one
        const bool use = a.id >= 0 && a.id < nb && (e == 0 || (a.prev >= 0 && a.prev < a.id));
        if (!use) {
          if (a.id != -1) raise_error(LLAMA_ATTN_DEVERR_BLOCK_IDS);
          return r;
        }
        r.n = a.id * rpp + (a.c.s - e * spp) * ROWS;
        if (r.n >= a.len) return r;
      } else {
        r.n = a.c.s * ROWS;
      }
      r.nvalid = min(ROWS, a.len - r.n);
      r.page = p.block_table[static_cast<int64_t>(a.c.b) * p.max_blocks + r.n / rpp];
      return r;
    };
    auto load_scales = [&](const Page& a) {
      Unit r{0, a.nvalid, 1.f, 1.f};
      if (a.nvalid == 0) return r;
      if (a.page < 0 || a.page >= p.n_pages) {
        raise_error(LLAMA_ATTN_DEVERR_BLOCK_TABLE);
        r.row = p.n_pages * p.Hkv * rpp;  // past the pool: the copy reads zeros
      } else {
        const int ph = a.page * p.Hkv + a.g;
        r.row = ph * rpp + a.n % rpp;
        if constexpr (kE4M3) {
          r.ks = p.kscales[ph];
          r.vs = p.vscales[ph];
        }
      }
      return r;
    };
    const int n_units = u1 - u0;
    Page page = load_page(load_ids());
    Ids ids = load_ids();
    bool alive = true;
    int done = 0;
    for (int i0 = 0; i0 < n_units && alive; i0 += 32) {
      const Unit now = load_scales(page);
      const int m = min(32, n_units - i0);
      for (int j = 0; j < m; ++j) {
        const int row = __shfl_sync(0xffffffffu, now.row, j);
        const int nvalid = __shfl_sync(0xffffffffu, now.nvalid, j);
        const uint32_t st = static_cast<uint32_t>(i0 + j) % T::NSTAGE;
        const int use = (i0 + j) / T::NSTAGE;
        int ok = 1;
        if (lane == 0) {
          ok = use == 0 || mbar_wait(empty(st), (use - 1) & 1, wc);
          if (ok && nvalid > 0) {
            const uint32_t dst = sbase + st * T::STAGE;
            if constexpr (kE4M3) {
              tma_load_2d(dst, &tm_k, full(st), 0, row);
              tma_load_2d(dst + T::TENSOR, &tm_v, full(st), 0, row);
            } else {
              tma_load_2d(dst, &tm_k, full(st), 0, row);
              tma_load_2d(dst + T::HALF, &tm_k, full(st), 64, row);
              tma_load_2d(dst + T::TENSOR, &tm_v, full(st), 0, row);
              tma_load_2d(dst + T::TENSOR + T::HALF, &tm_v, full(st), 64, row);
            }
          }
        }
        // the scales are needed only now, with the copies on their way; a value
        // scale outside [2^-100, 2^119] would leave the exponent's range (a NaN stays)
        const float ks = __shfl_sync(0xffffffffu, now.ks, j);
        float vs = __shfl_sync(0xffffffffu, now.vs, j);
        vs = vs < 0x1p-100f ? 0x1p-100f : vs > 0x1p119f ? 0x1p119f : vs;
        if (lane == 0 && ok) {
          *reinterpret_cast<float4*>(smem + T::OFF_META + st * 16) =
              make_float4(__int_as_float(nvalid), ks, kE4M3 ? __log2f(vs) : 0.f, 0.f);
          if (nvalid > 0)
            mbar_arrive_expect_tx(full(st), T::STAGE);
          else
            mbar_arrive(full(st));
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          alive = false;
          break;
        }
        ++done;
        if (j == min(3, m - 1)) {  // the steps for the batches to come, behind the first copies
          page = load_page(ids);
          ids = load_ids();
        }
      }
    }
    if (lane == 0)  // copies in flight land before the CTA's shared memory goes
      for (int st = 0; st < T::NSTAGE; ++st)
        if (done > st) mbar_wait(full(st), ((done - 1 - st) / T::NSTAGE) & 1, wc);
    if constexpr (kCluster) {  // with the compute warps: results written, results read
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // -------------------------------------------------------------- compute warps
  const int gq = lane >> 2, t = lane & 3;
  const int G = p.G;
  auto bar = [] { asm volatile("bar.sync 1, %0;" ::"n"(NCW * 32) : "memory"); };
  uint32_t qb[T::Q_REGS ? NQ : 1][T::Q_REGS ? NT : 1][8][2] = {};
  float m[NT][2], l[NT][2];
  // d of a tile's two heads. Two tiles as runs have no registers left for it: one
  // 131072-row sequence under 128 heads takes 61 us with d in registers and 58.5
  // with d in shared memory; as clusters seven sequences up to 9001 rows under 16
  // heads 12.1 and 12.7 us, and a 1000-row sequence under 32 heads 5.5 and 5.7.
  constexpr bool kRegsD = !kWide || kCluster;
  float2 d_regs[kRegsD ? NT : 1] = {};
  float2* const d_smem = reinterpret_cast<float2*>(smem + T::OFF_D + 64 * warp) + t;
  auto get_d = [&](int nt) {
    if constexpr (!kE4M3) return make_float2(0.f, 0.f);
    return kRegsD ? d_regs[kRegsD ? nt : 0] : d_smem[4 * nt];
  };
  auto set_d = [&](int nt, float2 x) {  // all lanes of the warp
    if constexpr (kRegsD) {
      d_regs[nt] = x;
    } else {
      __syncwarp();
      if (gq == 0) d_smem[4 * nt] = x;
      __syncwarp();
    }
  };
  float o[NT][8][4];
  // B fragment of the query for k step c, from shared memory; q_frag: from where the kernel keeps it.
  auto q_read = [&](int term, int nt, int c, uint32_t& b0, uint32_t& b1) {
    const uint8_t* row = smem + T::OFF_Q + (8 * NT * term + 8 * nt + gq) * T::Q_ROW + 32 * c;
    if constexpr (kE4M3) {  // codes 4t .. 4t+3 of a 16-byte chunk
      const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * t);
      b0 = v.x, b1 = v.y;
    } else {
      b0 = *reinterpret_cast<const uint32_t*>(row + 4 * t);
      b1 = *reinterpret_cast<const uint32_t*>(row + 16 + 4 * t);
    }
  };
  auto q_frag = [&](int term, int nt, int c, uint32_t& b0, uint32_t& b1) {
    if constexpr (T::Q_REGS)
      b0 = qb[term][nt][c][0], b1 = qb[term][nt][c][1];
    else
      q_read(term, nt, c, b0, b1);
  };

  // The rotated query rows of (b, g) as B fragments of the score product.
  auto load_query = [&]() {
    float2* cs_row = reinterpret_cast<float2*>(smem + T::OFF_CS);
    uint2 u[2 * NT];  // a warp stages two heads of each tile
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      const int h = warp + i * NCW;
      u[i] = make_uint2(0u, 0u);
      if (h < G)
        u[i] = *reinterpret_cast<const uint2*>(p.q + (static_cast<int64_t>(cur.b) * p.Hq + cur.g * G + h) * 128 + 4 * lane);
    }
    if (threadIdx.x < 64) {
      double sn, cs;
      sincos(static_cast<double>(p.lens[cur.b] + p.q_pos_offset) * p.freqs.theta[threadIdx.x], &sn, &cs);
      cs_row[threadIdx.x] = make_float2(static_cast<float>(cs), static_cast<float>(sn));
    }
    bar();
    const float4 cs = reinterpret_cast<const float4*>(cs_row)[lane];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      const int h = warp + i * NCW;
      const float2 a = unpack_bf16x2(u[i].x), b = unpack_bf16x2(u[i].y);
      const float x[4] = {a.x * cs.x - a.y * cs.y, a.x * cs.y + a.y * cs.x, b.x * cs.z - b.y * cs.w,
                          b.x * cs.w + b.y * cs.z};
      uint8_t* row = smem + T::OFF_Q + h * T::Q_ROW + 8 * lane;
      if constexpr (kE4M3) {
        const float am = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
        // bring the row's greatest magnitude (which orders like its bits) to
        // [0.5, 1): exact, and undone in the scores' factor
        const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
        const int e = bits ? min(max(static_cast<int>(bits >> 23) - 126, -100), 120) : 0;
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        *reinterpret_cast<uint2*>(row) = make_uint2(pack_f16x2(x[0] * f, x[1] * f), pack_f16x2(x[2] * f, x[3] * f));
        if (lane == 0)
          reinterpret_cast<float*>(smem + T::OFF_QS)[h] =
              p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      } else {
        const uint32_t hi[2] = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
        const float2 v = unpack_bf16x2(hi[0]), w = unpack_bf16x2(hi[1]);
        *reinterpret_cast<uint2*>(row) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(row + 8 * NT * T::Q_ROW) =
            make_uint2(pack_bf16x2(x[0] - v.x, x[1] - v.y), pack_bf16x2(x[2] - w.x, x[3] - w.y));
      }
    }
    bar();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
      if constexpr (kE4M3) set_d(nt, make_float2(0.f, 0.f));
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][c][e] = 0.f;
    }
    if constexpr (T::Q_REGS) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int term = 0; term < NQ; ++term) q_read(term, nt, c, qb[term][nt][c][0], qb[term][nt][c][1]);
    }
  };

  // Joins the four warps' results of the segment that ends here, and writes it.
  auto finish = [&](int first_unit, int last_unit, bool last) {  // last: of this run
    float4* ml = reinterpret_cast<float4*>(smem + T::OFF_ML);  // [warp][head]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 d = get_d(nt);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float& s = l[nt][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (gq == 0) ml[warp * 16 + 8 * nt + 2 * t + e] = make_float4(m[nt][e], e ? d.y : d.x, s, 0.f);
      }
    }
    bar();
    const bool whole = first_unit >= u0 && last_unit <= u1;  // the segment lies inside this run
    const int64_t slot = slot_of(blockIdx.x, first_unit >= u0);
    if (!kCluster && first_unit < u0 && last_unit <= u1 && threadIdx.x == 0)
      p.ends[blockIdx.x] = make_int4(cur.b, cur.g, cut.run_of(first_cost), 0);
    // A head's m, and its (m, d, l), over the four warps.
    auto bound_of = [&](int h) {
      float M = ml[h].x;
#pragma unroll
      for (int w = 1; w < NCW; ++w) M = fmaxf(M, ml[w * 16 + h].x);
      return M;
    };
    auto head_of = [&](int h) {
      float4 x = make_float4(bound_of(h), 0.f, 0.f, 0.f);
      float unit[NCW], top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NCW; ++w) top = fmaxf(top, unit[w] = unit_of(ml[w * 16 + h], x.x));
#pragma unroll
      for (int w = 0; w < NCW; ++w) x.z += ml[w * 16 + h].z * rebase(unit[w], top);
      x.y = -top;
      return x;
    };
    auto store_stats = [&](int h, const float4& v) {
      if (!whole)
        p.part_ml[slot * G + h] = v;
      else if (p.lse)
        p.lse[static_cast<int64_t>(cur.b) * p.Hq + cur.g * G + h] = lse_of(v);
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = rebase(m[nt][e], bound_of(8 * nt + 2 * t + e));
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          o[nt][c][e] *= f;
          o[nt][c][2 + e] *= f;
        }
      }
    if (last) {
      // No copy will fill the ring again: all warps put their rows there
      // ([warp][head][channel], rows of 132 floats) and every thread sums a part.
      constexpr int kRow = 132;
      float* ring = reinterpret_cast<float*>(smem);
      static_assert((NCW + 1) * 8 * NT * kRow * 4 <= static_cast<int>(T::OFF_Q), "the partial rows fit into the ring");
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* row = ring + (warp * 8 * NT + 8 * nt + 2 * t + e) * kRow;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if constexpr (kE4M3) {  // channels 16c + 2gq, + 1
              *reinterpret_cast<float2*>(row + 16 * c + 2 * gq) = make_float2(o[nt][c][e], o[nt][c][2 + e]);
            } else {  // channels 16c + gq and 16c + 8 + gq
              row[16 * c + gq] = o[nt][c][e];
              row[16 * c + 8 + gq] = o[nt][c][2 + e];
            }
          }
        }
      bar();
      // kCluster: this CTA's sum of each head, behind the warps' rows
      float* sums = ring + NCW * 8 * NT * kRow;
      for (int h = warp; h < G; h += NCW) {  // a warp a head, a lane 4 channels
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NCW; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(ring + (w * 8 * NT + h) * kRow + 4 * lane);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const float4 v = head_of(h);
        if constexpr (kCluster) {
          *reinterpret_cast<float4*>(sums + h * kRow + 4 * lane) = x;
          if (lane == 0) *reinterpret_cast<float4*>(sums + h * kRow + 128) = v;
          continue;
        }
        if (whole) {
          const Norm norm(v);
          const int64_t head = static_cast<int64_t>(cur.b) * p.Hq + cur.g * G + h;
          *reinterpret_cast<uint2*>(p.out + head * 128 + 4 * lane) =
              make_uint2(pack_bf16x2(norm(x.x), norm(x.y)), pack_bf16x2(norm(x.z), norm(x.w)));
        } else {
          *reinterpret_cast<float4*>(p.part_o + (slot * G + h) * 128 + 4 * lane) = x;
        }
        if (lane == 0) store_stats(h, v);
      }
      return;
    }
    if constexpr (kCluster) return;  // a CTA has one segment
    float4* scr = reinterpret_cast<float4*>(smem + T::OFF_SCR);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // the scratch holds two warps' channels of half the chunks
#pragma unroll
      for (int c0 = 0; c0 < 8; c0 += 4) {
#pragma unroll
        for (int half = NCW / 2; half > 0; half >>= 1) {
          if (nt > 0 || c0 > 0 || half < NCW / 2) bar();  // the scratch of the step before has been read
          if (warp >= half && warp < 2 * half) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float* x = o[nt][c0 + c];
              scr[((warp - half) * 4 + c) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
            }
          }
          bar();
          if (warp < half) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 v = scr[(warp * 4 + c) * 32 + lane];
              float* x = o[nt][c0 + c];
              x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
            }
          }
        }
      }
      if (warp == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = 8 * nt + 2 * t + e;
          if (h >= G) continue;
          const float4 v = head_of(h);
          const int64_t head = static_cast<int64_t>(cur.b) * p.Hq + cur.g * G + h;
          const Norm norm(v);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float x = o[nt][c][e], y = o[nt][c][2 + e];
            if constexpr (kE4M3) {
              if (whole)
                *reinterpret_cast<uint32_t*>(p.out + head * 128 + 16 * c + 2 * gq) = pack_bf16x2(norm(x), norm(y));
              else
                *reinterpret_cast<float2*>(p.part_o + (slot * G + h) * 128 + 16 * c + 2 * gq) = make_float2(x, y);
            } else {
              if (whole) {
                const uint32_t w = pack_bf16x2(norm(x), norm(y));
                p.out[head * 128 + 16 * c + gq] = static_cast<uint16_t>(w & 0xFFFFu);
                p.out[head * 128 + 16 * c + 8 + gq] = static_cast<uint16_t>(w >> 16);
              } else {
                p.part_o[(slot * G + h) * 128 + 16 * c + gq] = x;
                p.part_o[(slot * G + h) * 128 + 16 * c + 8 + gq] = y;
              }
            }
          }
          if (gq == 0) store_stats(h, v);
        }
      }
    }
    bar();  // scratch and the warps' m, d, l may be written again
  };

  if (!kCluster || u1 > u0) load_query();
  const int rbase = 16 * warp;
  const int n_units = u1 - u0;
  int seg_first = u0 - cur.s;  // the segment's first unit (it may lie in an earlier run)
  bool alive = true;  // false once a wait gave up: the barriers of a segment's end are still met
  for (int i = 0; i < n_units; ++i) {
    const uint32_t st = static_cast<uint32_t>(i) % T::NSTAGE;
    if (alive) alive = mbar_wait(full(st), (i / T::NSTAGE) & 1, wc);
    alive = __all_sync(0xffffffffu, alive);
    const float4 meta = *reinterpret_cast<const float4*>(smem + T::OFF_META + st * 16);
    const int nvalid = __float_as_int(meta.x);
    if (alive && rbase < nvalid) {
      const uint32_t kbase = sbase + st * T::STAGE, vbase = kbase + T::TENSOR;
      const int mi = lane >> 3, rr = lane & 7;
      constexpr int kChains = NT == 1 ? 2 : 1;  // two products in flight either way
      float sc[NT][4], sd[kChains == 2 ? NT : 1][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[nt][e] = 0.f;
          if constexpr (kChains == 2) sd[nt][e] = 0.f;
        }
      {
        const int row = rbase + 8 * (mi & 1) + rr;
        uint32_t b0, b1;
        if constexpr (kE4M3) {
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            uint32_t w0, w1, w2, w3;  // rows 0-7 and 8-15 of chunk c, then of chunk c + 1
            ldmatrix_x4(kbase + sw128_off(row, c + (mi >> 1)), w0, w1, w2, w3);
            const uint32_t a[4] = {f16x2_of_lo(w0), f16x2_of_lo(w1), f16x2_of_hi(w0), f16x2_of_hi(w1)};
            const uint32_t b[4] = {f16x2_of_lo(w2), f16x2_of_lo(w3), f16x2_of_hi(w2), f16x2_of_hi(w3)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              q_frag(0, nt, c, b0, b1);
              mma_f16_16816(sc[nt], a, b0, b1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              q_frag(0, nt, c + 1, b0, b1);
              mma_f16_16816(kChains == 2 ? sd[kChains == 2 ? nt : 0] : sc[nt], b, b0, b1);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int d8 = 2 * c + (mi >> 1);  // 16-byte chunk of 8 channels
            uint32_t a0, a1, a2, a3;
            ldmatrix_x4(kbase + (d8 >> 3) * T::HALF + sw128_off(row, d8 & 7), a0, a1, a2, a3);
#pragma unroll
            for (int term = 0; term < NQ; ++term)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                q_frag(term, nt, c, b0, b1);
                mma_bf16_16816(kChains == 2 && term == 1 ? sd[kChains == 2 ? nt : 0] : sc[nt], a0, a1, a2, a3, b0, b1);
              }
          }
        }
      }
      const bool in0 = rbase + gq < nvalid, in1 = rbase + 8 + gq < nvalid;
      const float lv = kE4M3 ? meta.z : 0.f;
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float2 f = make_float2(p.scale_log2, p.scale_log2);
        if constexpr (kE4M3) {
          f = *reinterpret_cast<const float2*>(smem + T::OFF_QS + 4 * (8 * nt + 2 * t));
          f.x *= meta.y, f.y *= meta.y;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float s =
              (kChains == 2 ? sc[nt][e] + sd[kChains == 2 ? nt : 0][e] : sc[nt][e]) * (e & 1 ? f.y : f.x) + lv;
          sc[nt][e] = ((e & 2) ? in1 : in0) ? s : -INFINITY;
        }
        const float2 d = get_d(nt);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = kLift + kSlack;
          if constexpr (kE4M3) top = fminf(top, kSlack + lv - (e ? d.y : d.x));
          top += m[nt][e];
          above |= sc[nt][e] > top || sc[nt][e + 2] > top;
        }
      }
      // m is the exponents' maximum less kLift, m - d that of the scores, and both
      // only have to stay within 2^kSlack of that: they move when some row passes
      // one by more, seldom after the first stages. P then reaches 2^15 at most, and
      // f16 holds P down to 2^-32 of the greatest.
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float2 d = get_d(nt);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(sc[nt][e], sc[nt][e + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float was = m[nt][e], now = fmaxf(mx - kLift, was), alpha = rebase(was, now);
            m[nt][e] = now;
            if constexpr (kE4M3) {
              const float old = e ? d.y : d.x, next = now - fmaxf(was - old, mx - lv);
              l[nt][e] *= ex2_approx((was - now) + (next - old));
              (e ? d.y : d.x) = next;
            } else {
              l[nt][e] *= alpha;
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              o[nt][c][e] *= alpha;
              o[nt][c][2 + e] *= alpha;
            }
          }
          if constexpr (kE4M3) set_d(nt, d);
        }
      }
      uint32_t pb[NT][NP][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[nt][e] -= m[nt][e & 1];
          pr[e] = ex2_approx(sc[nt][e]);
        }
        const float2 d = get_d(nt);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (kE4M3) {
            const float by = (e ? d.y : d.x) - lv;
            l[nt][e] += ex2_approx(sc[nt][e] + by) + ex2_approx(sc[nt][e + 2] + by);
          } else {
            l[nt][e] += pr[e] + pr[e + 2];
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (kE4M3) {
            pb[nt][0][i] = movmatrix_trans(pack_f16x2(pr[2 * i], pr[2 * i + 1]));
          } else {
            const uint32_t hi = pack_bf16x2(pr[2 * i], pr[2 * i + 1]);
            const float2 v = unpack_bf16x2(hi);
            pb[nt][0][i] = movmatrix_trans(hi);
            pb[nt][NP - 1][i] = movmatrix_trans(pack_bf16x2(pr[2 * i] - v.x, pr[2 * i + 1] - v.y));
          }
        }
      }
      // value rows at or past len may hold anything (NaN included): zero them so
      // that P = 0 cannot meet NaN inside the product.
      const bool tail = rbase + 16 > nvalid;
      if (tail) {
        constexpr int kChunks = kE4M3 ? 8 : 16;  // 16-byte chunks of a row
        for (int x = lane; x < 16 * kChunks; x += 32) {
          const int r = rbase + x / kChunks, ch = x % kChunks;
          if (r >= nvalid)
            *reinterpret_cast<uint4*>(smem + st * T::STAGE + T::TENSOR + (ch >> 3) * T::HALF + r * 128 + (ch & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      if constexpr (kE4M3) {
        const int row = rbase + 8 * (mi & 1) + rr;
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          uint32_t w[4];  // keys 0-7 and 8-15 of chunk c, then of chunk c + 1
          ldmatrix_x4_trans(vbase + sw128_off(row, c + (mi >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = __byte_perm(w[k], 0u, 0x3120);  // even channels low, odd high
          const uint32_t a[4] = {f16x2_of_lo(w[0]), f16x2_of_hi(w[0]), f16x2_of_lo(w[1]), f16x2_of_hi(w[1])};
          const uint32_t b[4] = {f16x2_of_lo(w[2]), f16x2_of_hi(w[2]), f16x2_of_lo(w[3]), f16x2_of_hi(w[3])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(o[nt][c], a, pb[nt][0][0], pb[nt][0][1]);
            mma_f16_16816(o[nt][c + 1], b, pb[nt][0][0], pb[nt][0][1]);
          }
        }
      } else {
        const int row = rbase + 8 * (mi >> 1) + rr;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int d8 = 2 * c + (mi & 1);
          uint32_t a0, a1, a2, a3;
          ldmatrix_x4_trans(vbase + (d8 >> 3) * T::HALF + sw128_off(row, d8 & 7), a0, a1, a2, a3);
#pragma unroll
          for (int term = 0; term < NP; ++term)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(o[nt][c], a0, a1, a2, a3, pb[nt][term][0], pb[nt][term][1]);
        }
      }
      if (tail) fence_proxy_async_smem();
    }
    __syncwarp();
    if (alive && lane == 0) mbar_arrive(empty(st));
    if (cur.s + 1 == cur.nst || i + 1 == n_units) {
      finish(seg_first, seg_first + cur.nst, i + 1 == n_units);
      if (i + 1 < n_units) {
        advance<kSparse>(p, cur, 1);
        seg_first = u0 + i + 1;
        load_query();
      }
    } else {
      ++cur.s;
    }
  }
  if constexpr (!kCluster) {
    clear_empty<kSparse>(p, NCW * 32);
  } else {
    // Each head by one warp of the cluster, from the sums of the CTAs that had
    // units, in the order of their ranks.
    cluster_sync();
    constexpr int kRow = 132;
    const uint32_t sums = smem_addr(reinterpret_cast<float*>(smem) + NCW * 8 * NT * kRow);
    const int n = min(static_cast<int>(csize), cur.nst);
    for (int h = static_cast<int>(rank) * NCW + warp; h < G; h += static_cast<int>(csize) * NCW) {
      const uint32_t row = sums + static_cast<uint32_t>(h * kRow * 4);
      float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      if (lane < n) {
        const uint32_t at = peer_addr(row + 128 * 4, lane);
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(ml.x), "=f"(ml.y), "=f"(ml.z), "=f"(ml.w)
                     : "r"(at)
                     : "memory");
      }
      float4 v = make_float4(warp_max(ml.x), 0.f, 0.f, 0.f);
      const float unit = unit_of(ml, v.x), top = warp_max(unit), w = rebase(ml.x, v.x);
      v.y = -top;
      ml.z *= rebase(unit, top);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int r = 0; r < n; ++r) {
        float4 y;
        const uint32_t at = peer_addr(row + 16 * lane, r);
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                     : "r"(at)
                     : "memory");
        const float f = __shfl_sync(0xffffffffu, w, r);
        v.z += __shfl_sync(0xffffffffu, ml.z, r);
        x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
      }
      const Norm norm(v);
      const int64_t head = static_cast<int64_t>(cur.b) * p.Hq + cur.g * G + h;
      *reinterpret_cast<uint2*>(p.out + head * 128 + 4 * lane) =
          make_uint2(pack_bf16x2(norm(x.x), norm(x.y)), pack_bf16x2(norm(x.z), norm(x.w)));
      if (p.lse && lane == 0) p.lse[head] = lse_of(v);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
}

// Merges the partial results of the runs that share a (sequence, KV head), in
// an order fixed by the runs. Heads that one run wrote whole and sequences
// without rows are done already. Latency bounds it (a few dependent loads), so
// there are two layouts:
// kByRun = false: a block per query head, its eight warps share the pair's
// partial rows (one 131072-row sequence of 8 KV heads: 37 of them).
// kByRun = true: a block per run, for the one pair that ends in it and began
// before; a warp takes whole heads. Sparse decode of 64 sequences with 64 heads:
// 4 us, 16 us as 4096 blocks of the first layout.
constexpr int JOIN_WARPS = 8;

// One head's partial rows mine, mine + step .. c1 of c0 .. c1: their sum relative
// to the greatest m of all, and v = (that m, d and l in the greatest unit of all).
// The first rows are on their way while these are found.
template <typename Slot>
__device__ __forceinline__ void join_rows(const Params& p, Slot slot, int c0, int c1, int mine, int step, float4& v,
                                          float4& acc) {
  const int lane = threadIdx.x & 31;
  float4 ml[4], y[4];
  auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ml[i] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + i * step <= c1) {
        const int64_t s = slot(c + i * step);
        ml[i] = p.part_ml[s];
        y[i] = reinterpret_cast<const float4*>(p.part_o + s * 128)[lane];
      }
    }
  };
  fetch(mine);
  // this lane's greatest m and, relative to it, greatest unit
  float4 a = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  for (int c = c0 + lane; c <= c1; c += 32) {
    const float4 x = p.part_ml[slot(c)];
    const float M = fmaxf(a.x, x.x);
    a.y = -fmaxf(unit_of(a, M), unit_of(x, M));
    a.x = M;
  }
  v = make_float4(warp_max(a.x), 0.f, 0.f, 0.f);
  const float top = warp_max(unit_of(a, v.x));
  v.y = -top;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = mine;;) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = rebase(ml[i].x, v.x);
      v.z += ml[i].z * rebase(unit_of(ml[i], v.x), top);
      acc.x += w * y[i].x, acc.y += w * y[i].y, acc.z += w * y[i].z, acc.w += w * y[i].w;
    }
    c += 4 * step;
    if (c > c1) break;
    fetch(c);
  }
}

template <bool kByRun>
__global__ void __launch_bounds__(JOIN_WARPS * 32) decode_join_kernel(const Params p, int max_runs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  if constexpr (kByRun) {
    const int4 end = p.ends[blockIdx.x];
    if (end.x < 0) return;
    const int c0 = end.z, c1 = blockIdx.x;
    for (int h = warp; h < p.G; h += JOIN_WARPS) {
      auto slot = [&](int c) { return static_cast<int64_t>(slot_of(c, c == c0)) * p.G + h; };
      float4 v, a;
      join_rows(p, slot, c0, c1, c0, 1, v, a);
      const int64_t head = static_cast<int64_t>(end.x) * p.Hq + end.y * p.G + h;
      const Norm norm(v);
      *reinterpret_cast<uint2*>(p.out + head * 128 + 4 * lane) =
          make_uint2(pack_bf16x2(norm(a.x), norm(a.y)), pack_bf16x2(norm(a.z), norm(a.w)));
      if (p.lse && lane == 0) p.lse[head] = lse_of(v);
    }
  } else {
    const int head = blockIdx.x, b = head / p.Hq, hq = head - b * p.Hq;
    const int g = hq / p.G, h = hq - g * p.G;
    __shared__ float s_l[JOIN_WARPS];
    __shared__ float4 s_o[JOIN_WARPS][32];
    const int total = p.prefix[p.B], first = p.prefix[b], end = p.prefix[b + 1];
    if (end == first) return;
    const Cut cut(total, min(max_runs, total));
    const int cost = (end - first) / p.Hkv, at = first + g * cost;
    const int c0 = first_run(cut, at), c1 = last_run(cut, at, cost - PAIR_COST);
    if (c0 == c1) return;
    auto slot = [&](int c) { return static_cast<int64_t>(slot_of(c, c == c0)) * p.G + h; };
    float4 v, acc;
    join_rows(p, slot, c0, c1, c0 + warp, JOIN_WARPS, v, acc);
    s_o[warp][lane] = acc;
    if (lane == 0) s_l[warp] = v.z;
    __syncthreads();
    if (threadIdx.x >= 128) return;
    const float* so = reinterpret_cast<const float*>(s_o);
    const int64_t to = static_cast<int64_t>(head) * 128 + threadIdx.x;
    float x = 0.f;
    v.z = 0.f;
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) x += so[128 * w + threadIdx.x], v.z += s_l[w];
    const __nv_bfloat16 y = __float2bfloat16_rn(Norm(v)(x));
    p.out[to] = *reinterpret_cast<const uint16_t*>(&y);
    if (p.lse && threadIdx.x == 0) p.lse[head] = lse_of(v);
  }
}

}  // namespace dpg
}  // namespace la
