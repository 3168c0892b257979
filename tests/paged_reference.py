"""Plain float64 statements of the paged-cache operators, for the tests: the
append with rotation, attention over named rows of a paged cache, and the
block selection. Written from the formulas, row by row, on CPU tensors."""
import math

import torch

D = 128


def angles(pos, theta):
    k = torch.arange(D // 2, dtype=torch.float64)
    return torch.as_tensor(pos, dtype=torch.float64)[..., None] * theta ** (-2.0 * k / D)


def rotate(x, pos, theta):
    """x [..., D] turned at positions pos (broadcast against x's leading dimensions), float64."""
    a = angles(pos, theta)
    c, s = a.cos(), a.sin()
    x = x.double()
    y = torch.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    y[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    return y


def e4m3_grid(x):
    """x rounded to the nearest E4M3 value (ties to even), saturated at +-448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-5) - 4)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def block_scale(amax):
    """2^e with the least e in [-100, 119] for which amax <= 448 * 2^e."""
    e = -100
    while e < 119 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def codes(pages):
    """Float64 values of E4M3 codes held as uint8."""
    return pages.view(torch.float8_e4m3fn).double()


def append(k, v, pools, scales, bounds, table, lens, new, page, theta):
    """What the append leaves, in float64: pools [K, V] as values (codes without their
    scale), scales [K, V] or None, bounds or None. All given as float64 CPU tensors of
    the state before; returned changed in place."""
    B, T, Hkv, _ = k.shape
    for b in range(B):
        for j in range(lens[b] // page, -(-(lens[b] + new[b]) // page)):
            pg = int(table[b, j])
            r0, r1 = max(lens[b], j * page), min(lens[b] + new[b], (j + 1) * page)
            if r0 >= r1:
                continue
            was = r0 - j * page
            pos = torch.arange(r0, r1)
            rows = [rotate(k[b, r0 - lens[b]:r1 - lens[b]], pos[:, None], theta),
                    v[b, r0 - lens[b]:r1 - lens[b]].double()]
            for h in range(Hkv):
                for c in (0, 1):
                    x = rows[c][:, h]
                    if scales is None:
                        pools[c][pg, h, was:was + r1 - r0] = x
                        continue
                    s = block_scale(float(x.abs().max()))
                    if was:
                        s = max(s, float(scales[c][pg, h]))
                        pools[c][pg, h, :was] = e4m3_grid(pools[c][pg, h, :was] * (float(scales[c][pg, h]) / s))
                    scales[c][pg, h] = s
                    pools[c][pg, h, was:was + r1 - r0] = x / s
                if bounds is not None:
                    lo, hi = rows[0][:, h].amin(0), rows[0][:, h].amax(0)
                    if was:
                        lo, hi = torch.minimum(lo, bounds[pg, h, 0]), torch.maximum(hi, bounds[pg, h, 1])
                    bounds[pg, h, 0], bounds[pg, h, 1] = lo, hi


def attend(q, rows_k, rows_v):
    """q [G, D], rows [n, D], float64: (out, lse, sum_n p |v|, max_n sum_d |q_d k_d| / sqrt(D))."""
    if rows_k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64), z, torch.zeros(q.shape[0])
    s = q @ rows_k.T / math.sqrt(D)
    p = torch.softmax(s, -1)
    return p @ rows_v, torch.logsumexp(s, -1), p @ rows_v.abs(), (q.abs() @ rows_k.abs().T / math.sqrt(D)).amax(-1)


def decode(q, kvals, vvals, table, lens, page, theta, q_pos_offset=0, block_ids=None):
    """kvals, vvals: float64 values of the pools [n_pages, Hkv, page, D]. Returns out, lse and
    the two magnitudes of ``attend`` ([B, Hq, D] and [B, Hq])."""
    B, Hq, _ = q.shape
    Hkv = kvals.shape[1]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    mass = torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    span = torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        n = lens[b]
        qr = rotate(q[b], n + q_pos_offset, theta)
        for g in range(Hkv):
            row = torch.arange(n)
            if block_ids is not None:
                ids = [int(i) for i in block_ids[b, g] if i >= 0]
                row = torch.tensor([r for i in ids for r in range(i * page, min(n, (i + 1) * page))], dtype=torch.long)
            pg = table[b, row // page].long()
            k, v = kvals[pg, g, row % page], vvals[pg, g, row % page]
            hs = slice(g * G, (g + 1) * G)
            out[b, hs], lse[b, hs], mass[b, hs], span[b, hs] = attend(qr[hs], k, v)
    return out, lse, mass, span


def select(q, bounds, table, lens, page, n_sel, n_first, n_last, theta, q_pos_offset=0):
    B, Hq, _ = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    ids = torch.full((B, Hkv, n_sel), -1, dtype=torch.int32)
    for b in range(B):
        nb = -(-lens[b] // page)
        qr = rotate(q[b], lens[b] + q_pos_offset, theta)
        for g in range(Hkv):
            if nb <= n_sel:
                ids[b, g, :nb] = torch.arange(nb)
                continue
            pg = table[b, :nb].long()
            lo, hi = bounds[pg, g, 0].double(), bounds[pg, g, 1].double()
            score = torch.zeros(nb, dtype=torch.float64)
            for h in range(g * G, (g + 1) * G):
                score += torch.maximum(qr[h] * lo, qr[h] * hi).sum(-1)
            mid = range(n_first, nb - n_last)
            best = sorted(mid, key=lambda j: (-float(score[j]), j))[:n_sel - n_first - n_last]
            ids[b, g] = torch.tensor(sorted(list(range(n_first)) + best + list(range(nb - n_last, nb))))
    return ids
