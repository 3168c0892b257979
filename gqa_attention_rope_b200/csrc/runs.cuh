// runs.cuh -- how the work of a batch's paged decode is cut into runs, one per
// resident CTA. No CUDA in it: the host compiler takes it too.
//
// A pair is a (sequence, KV head), a unit one stage of a pair; both are counted in
// the order (sequence, KV head, stage). A pair of nst > 0 stages costs PAIR_COST
// for its begin and end, ahead of its first unit, and 1 per unit. The costs of the
// batch are cut into runs of equal length (to one); a run has the units whose cost
// lies in it, and may have none.
#pragma once

#ifdef __CUDACC__
#define LA_BOTH __host__ __device__ __forceinline__
#else
#define LA_BOTH inline
#endif

namespace la {
namespace dpg {

constexpr int PAIR_COST = 6;

LA_BOTH int cost_of(int nst) { return nst > 0 ? nst + PAIR_COST : 0; }

// Position of a unit: stage s of the nst of sequence b's KV head g.
struct Cursor {
  int b, g, s, nst;
};

// The position `by` units further; stages(b): stages of each pair of sequence b.
template <typename Stages>
LA_BOTH void advance(Stages stages, int B, int Hkv, Cursor& c, int by) {
  c.s += by;
  while (c.b < B && c.s >= c.nst) {
    c.s -= c.nst;
    if (c.nst > 0 && ++c.g < Hkv) continue;
    c.g = 0;
    if (++c.b < B) c.nst = stages(c.b);
  }
}

// The cut of `total` costs into n <= total runs: the first total % n of them
// have one more than the others.
struct Cut {
  int q, r;
  LA_BOTH Cut(int total, int n) : q(total / n), r(total - total / n * n) {}
  LA_BOTH int start(int run) const { return q * run + (run < r ? run : r); }
  LA_BOTH int run_of(int cost) const {
    const int big = r * (q + 1);
    return cost < big ? cost / (q + 1) : r + (cost - big) / q;
  }
};

// Where the run begins whose first cost c0 belongs to a sequence whose pairs have
// nst stages, the first of them at cost `at` and unit `u`.
struct RunBegin {
  int g, s;        // the pair's KV head and the stage
  int unit;        // the first unit
  int first_cost;  // of the pair's first unit
  LA_BOTH RunBegin(int c0, int at, int u, int nst) {
    g = (c0 - at) / cost_of(nst);
    const int off = c0 - at - g * cost_of(nst);
    s = off > PAIR_COST ? off - PAIR_COST : 0;
    unit = u + g * nst + s;
    first_cost = c0 - off + PAIR_COST;
  }
};
// The unit behind the run whose last cost is c1, likewise.
LA_BOTH int run_end(int c1, int at, int u, int nst) {
  const int g = (c1 - at) / cost_of(nst), off = c1 - at - g * cost_of(nst);
  return u + g * nst + (off + 1 > PAIR_COST ? off + 1 - PAIR_COST : 0);
}

// A pair within one run is written by it; of others each run has a partial result:
// the first run's lies at 2 * run + 1, those of the runs that the pair enters at
// 2 * run, so a run has one of each at most.
LA_BOTH int slot_of(int run, bool begins) { return 2 * run + (begins ? 1 : 0); }
// The runs of a pair's first and last unit, from the cost at which the pair begins.
LA_BOTH int first_run(const Cut& cut, int pair_at) { return cut.run_of(pair_at + PAIR_COST); }
LA_BOTH int last_run(const Cut& cut, int pair_at, int nst) { return cut.run_of(pair_at + cost_of(nst) - 1); }

}  // namespace dpg
}  // namespace la
