"""Operators of the paged KV cache: append with rotation, decode over an E4M3
cache, and block-sparse decode.

``run`` computes each operator either with elementary torch operations (the
plain form) or, where ``own`` is true, through the package's entry points.
Shapes are the package's own: head size 128, 8 KV heads under 32, 64 or 128
query heads, caches of up to 131072 rows, pages of 64 to 256 rows.
"""
import math

import torch

own = False

D = 128
THETA = 500000.0
E_MIN, E_MAX = -100, 119  # exponent range of the power-of-two block scales


def listed():
    append = dict(op="append", ragged=False, bounds=True)
    decode = dict(op="decode")
    sparse = dict(op="sparse")
    return [
        # one decode step of a 70B server: 64 sequences get one token each
        dict(append, name="append_step_e4m3", cache="e4m3", B=64, T=1, Hkv=8, page=64, lo=1024, hi=4096),
        # packed 8B prompts, four rows of 8192 tokens, into bf16 pages
        dict(append, name="append_prompt_bf16", cache="bf16", B=4, T=8192, Hkv=8, page=64, lo=0, hi=0),
        # a 128K prompt into E4M3 pages
        dict(append, name="append_128k_e4m3", cache="e4m3", B=1, T=131072, Hkv=8, page=128, lo=0, hi=0),
        # prompt chunks of odd lengths that continue partly filled pages
        dict(append, name="append_ragged_e4m3", cache="e4m3", B=5, T=777, Hkv=2, page=64, lo=1, hi=3001, ragged=True),
        # one short chat answer being decoded: latency
        dict(decode, name="decode_e4m3_B1", B=1, Hq=32, Hkv=8, page=64, lo=1000, hi=1000),
        # an odd batch with few KV heads per device and ragged lengths, a length of one among them
        dict(decode, name="decode_e4m3_odd", B=7, Hq=16, Hkv=1, page=256, lo=1, hi=9001),
        # one 128K document under the 405B head layout
        dict(decode, name="decode_e4m3_128k", B=1, Hq=128, Hkv=8, page=128, lo=131072, hi=131072),
        # the 70B decode batch
        dict(decode, name="decode_e4m3_70b", B=64, Hq=64, Hkv=8, page=64, lo=1024, hi=32768),
        # a single long sequence, 64 of its 2048 blocks read
        dict(sparse, name="sparse_e4m3_128k", cache="e4m3", B=1, Hq=32, Hkv=8, page=64, lo=131072, hi=131072, n_sel=64),
        # a small batch over bf16 pages
        dict(sparse, name="sparse_bf16_B5", cache="bf16", B=5, Hq=8, Hkv=2, page=64, lo=700, hi=5003, n_sel=16),
        # bf16 pages, sixteen sequences of the 70B layout
        dict(sparse, name="sparse_bf16_70b", cache="bf16", B=16, Hq=64, Hkv=8, page=64, lo=8192, hi=32768, n_sel=64),
        # the 70B decode batch over E4M3 pages
        dict(sparse, name="sparse_e4m3_70b", cache="e4m3", B=64, Hq=64, Hkv=8, page=64, lo=1024, hi=32768, n_sel=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "sparse"])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([64, 128, 256])
    if op == "append":
        B = _log(rng, 1, 64)
        T = 1 if rng.random() < 0.3 else _log(rng, 2, 131072 // B)
        lo = rng.randrange(0, 4096)
        return dict(op=op, cache=rng.choice(["bf16", "e4m3"]), B=B, T=T, Hkv=Hkv, page=page, lo=lo,
                    hi=lo + rng.randrange(0, 4096), ragged=T > 1 and rng.random() < 0.5, bounds=rng.random() < 0.7)
    B = _log(rng, 1, 64)
    hi = _log(rng, 64, min(131072, 64 * 32768 // B // 2))
    case = dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 3, 4, 8, 16]), Hkv=Hkv, page=page, lo=rng.randrange(1, hi + 1),
                hi=hi)
    if op == "sparse":
        case.update(cache=rng.choice(["bf16", "e4m3"]), n_sel=_log(rng, 3, 128))
        if case["cache"] == "bf16":
            case["hi"] = max(case["lo"], hi // 2)
    return case


def _lengths(case):
    """Per sequence: rows in the cache, spread evenly over [lo, hi], and rows that an append brings."""
    B, lo, hi, T = case["B"], case["lo"], case["hi"], case.get("T", 0)
    return [(hi - (hi - lo) * i // max(1, B - 1), T - (T // 2) * i // B if case.get("ragged") else T)
            for i in range(B)]


def _scale_exp(amax):
    """Least e with amax <= 448 * 2^e, within the range of the scales."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _pool(g, n_pages, Hkv, page, kind, spread):
    """Pages of one of K or V: values in `kind`, and the block scales (E4M3) or None."""
    x = torch.randn(n_pages, Hkv, page, D, generator=g, device="cuda")
    if spread:  # blocks of a real cache differ from each other
        x += spread * torch.randn(n_pages, Hkv, 1, D, generator=g, device="cuda")
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    s = _pow2(_scale_exp(x.abs().amax((2, 3))))
    x /= s[:, :, None, None]
    return x.to(torch.float8_e4m3fn).view(torch.uint8), s


def _values(pages):
    """Float32 values of pages, E4M3 codes without their scale."""
    return (pages.view(torch.float8_e4m3fn) if pages.dtype == torch.uint8 else pages).float()


def _freqs():
    k = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    return THETA ** (-2.0 * k / D)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    pairs = _lengths(case)  # in an order of the seed's
    lens, new = zip(*(pairs[i] for i in torch.randperm(B, generator=g, device="cuda").tolist()))
    need = [-(-(n + t) // page) for n, t in zip(lens, new)]
    blocks = max(1, max(need))
    n_pages = sum(need) + 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(blocks, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[used] = perm[:sum(need)]
    kind = case.get("cache", "e4m3")
    spread = 0.5 if case["op"] == "sparse" else 0.0
    kp, ks = _pool(g, n_pages, Hkv, page, kind, spread)
    vp, vs = _pool(g, n_pages, Hkv, page, kind, 0.0)
    s = dict(op=case["op"], kind=kind, kp=kp, vp=vp, ks=ks, vs=vs, table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), page=page)
    if case["op"] == "append":
        T = case["T"]
        s["k"] = torch.randn(B, T, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        s["v"] = torch.randn(B, T, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda") if case["ragged"] else None
        a = torch.arange(blocks * page, device="cuda", dtype=torch.float64)[:, None] * _freqs()
        s["rope"] = torch.stack([a.cos(), a.sin()], -1).float()
        if case["bounds"]:
            s["bounds"] = _bounds_of(s)
        return s
    Hq = case["Hq"]
    s["q"] = (1.5 * torch.randn(B, Hq, D, generator=g, device="cuda")).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["workspace"] = torch.empty(48 << 20, dtype=torch.uint8, device="cuda")
    if case["op"] == "sparse":
        s["bounds"] = _bounds_of(s)
        s["n_sel"] = case["n_sel"]
        s["ids"] = torch.empty(B, Hkv, case["n_sel"], dtype=torch.int32, device="cuda")
    return s


def _bounds_of(s):
    x = _values(s["kp"])
    if s["ks"] is not None:
        x *= s["ks"][:, :, None, None]
    return torch.stack(torch.aminmax(x, dim=2), 2).to(torch.bfloat16)


# ------------------------------------------------------------- plain forms
def _rotate(x, cos, sin):
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)


def _rotated_query(s, dtype):
    a = s["lens"].double()[:, None, None] * _freqs()
    return _rotate(s["q"].to(dtype), a.cos().to(dtype), a.sin().to(dtype))


def _append(s):
    k, v, lens, page = s["k"], s["v"], s["lens"].long(), s["page"]
    B, T = k.shape[:2]
    new = s["new"].long() if s["new"] is not None else torch.full_like(lens, T)
    t = torch.arange(T, device="cuda")
    pos = lens[:, None] + t
    b, t = torch.nonzero(t[None, :] < new[:, None], as_tuple=True)
    pos = pos[b, t]
    pg, row = s["table"].long()[b, pos // page], pos % page
    cs = s["rope"][pos][:, None]
    kr = _rotate(k[b, t].float(), cs[..., 0], cs[..., 1])
    vn = v[b, t].float()
    fresh = torch.zeros(s["kp"].shape[0], dtype=torch.bool, device="cuda")
    fresh[pg[row == 0]] = True
    out = []
    if s["kind"] == "bf16":
        s["kp"][pg, :, row] = kr.to(torch.bfloat16)
        s["vp"][pg, :, row] = vn.to(torch.bfloat16)
        out += [s["kp"], s["vp"]]
    else:
        # the one page of each sequence that holds older rows: they follow the block's scale
        old = (lens % page > 0) & (new > 0)
        seq = torch.nonzero(old, as_tuple=True)[0]
        old_pg, old_n = s["table"].long()[seq, lens[seq] // page], lens[seq] % page
        older = (torch.arange(page, device="cuda") < old_n[:, None])[:, None, :, None]
        for x, pages, scales in ((kr, s["kp"], s["ks"]), (vn, s["vp"], s["vs"])):
            f8 = pages.view(torch.float8_e4m3fn)
            amax = torch.full_like(scales, -1.0).index_reduce_(0, pg, x.abs().amax(-1), "amax")
            need = _pow2(_scale_exp(amax))
            now = torch.where(amax < 0, scales, torch.where(fresh[:, None], need, torch.maximum(scales, need)))
            kept = f8[old_pg].float() * (scales / now)[old_pg][:, :, None, None]
            f8[old_pg] = torch.where(older, kept, f8[old_pg].float()).to(torch.float8_e4m3fn)
            scales.copy_(now)
            f8[pg, :, row] = (x / now[pg][:, :, None]).to(torch.float8_e4m3fn)
            out += [f8, scales]
    if "bounds" in s:
        lo, hi = s["bounds"][:, :, 0].float(), s["bounds"][:, :, 1].float()
        lo[fresh], hi[fresh] = math.inf, -math.inf
        lo.index_reduce_(0, pg, kr, "amin")
        hi.index_reduce_(0, pg, kr, "amax")
        s["bounds"].copy_(torch.stack([lo, hi], 2))
        out.append(s["bounds"])
    return out


def _attend(s, pages, live):
    """Attention of each query head over the rows of pages [B, Hkv or 1, n] where live [B, Hkv or 1, n * page]."""
    B, Hq, _ = s["q"].shape
    Hkv, page = s["kp"].shape[1], s["page"]
    q = _rotated_query(s, torch.float32).view(B, Hkv, Hq // Hkv, D)
    pages = pages.clamp(min=0).expand(B, Hkv, -1)
    heads = torch.arange(Hkv, device="cuda")[None, :, None]

    def rows(pool, scales):
        x = _values(pool[pages, heads])  # [B, Hkv, n, page, D]
        if scales is not None:
            x *= scales[pages, heads][..., None, None]
        return x.flatten(2, 3)

    sc = torch.matmul(q, rows(s["kp"], s["ks"]).transpose(2, 3)) / math.sqrt(D)
    sc = sc.masked_fill(~live[:, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(sc - m)
    o = torch.matmul(p, rows(s["vp"], s["vs"])) / p.sum(-1, keepdim=True).clamp(min=1e-38)
    return o.view(B, Hq, D).to(torch.bfloat16)


def _decode(s):
    pages = s["table"].long()[:, None, :]
    live = torch.arange(pages.shape[2] * s["page"], device="cuda") < s["lens"][:, None]
    return [_attend(s, pages, live[:, None])]


def _select(s):
    """The first block, the last one and the best-scored others, n_sel in all, ascending, -1 behind them."""
    table, lens, page, n_sel = s["table"].long(), s["lens"].long(), s["page"], s["n_sel"]
    B, nb = table.shape
    Hkv = s["kp"].shape[1]
    q = _rotated_query(s, torch.float64).view(B, Hkv, -1, D)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    bounds = s["bounds"][table.clamp(min=0)].double()  # [B, nb, Hkv, 2, D]
    score = (bounds[:, :, :, 1] * up[:, None] + bounds[:, :, :, 0] * down[:, None]).sum(-1).transpose(1, 2)
    blocks = (lens + page - 1) // page
    j = torch.arange(nb, device="cuda")
    used = (j < blocks[:, None])[:, None]
    forced = ((j < 1) | (j >= blocks[:, None] - 1))[:, None] & used
    score = score.masked_fill(forced, math.inf).masked_fill(~used, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n_sel]
    order = torch.where(order < blocks[:, None, None], order, nb)
    order = torch.sort(order, dim=-1).values
    ids = torch.full((B, Hkv, n_sel), -1, dtype=torch.int32, device="cuda")
    ids[..., :order.shape[-1]] = torch.where(order < nb, order, -1).to(torch.int32)
    return ids


def _sparse(s):
    ids = _select(s)
    at = ids.long().clamp(min=0)
    pages = torch.gather(s["table"].long()[:, None, :].expand(-1, at.shape[1], -1), 2, at)
    row = at[..., None] * s["page"] + torch.arange(s["page"], device="cuda")
    live = (row < s["lens"][:, None, None, None]) & (ids >= 0)[..., None]
    return [ids, _attend(s, pages, live.flatten(2))]


def _own(s):
    import gqa_attention_rope_b200 as la
    e4m3 = s["kind"] == "e4m3"
    if s["op"] == "append":
        more = dict(new_lens=s["new"], kbounds=s.get("bounds"))
        if e4m3:
            la.llama_attn_kv_append_paged_e4m3(s["k"], s["v"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"],
                                               s["lens"], s["rope"], **more)
            out = [s["kp"].view(torch.float8_e4m3fn), s["ks"], s["vp"].view(torch.float8_e4m3fn), s["vs"]]
        else:
            la.llama_attn_kv_append_paged(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], s["rope"], **more)
            out = [s["kp"], s["vp"]]
        return out + ([s["bounds"]] if "bounds" in s else [])
    into = dict(out=s["out"], workspace=s["workspace"], rope_theta=THETA)
    if s["op"] == "decode":
        return [la.llama_attn_decode_paged_e4m3(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["lens"],
                                                **into)]
    ids = la.llama_attn_select_blocks(s["q"], s["bounds"], s["table"], s["lens"], s["page"], s["n_sel"], n_first=1,
                                      n_last=1, block_ids=s["ids"], rope_theta=THETA)
    if e4m3:
        return [ids, la.llama_attn_decode_paged_sparse_e4m3(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"],
                                                            ids, s["lens"], **into)]
    return [ids, la.llama_attn_decode_paged_sparse(s["q"], s["kp"], s["vp"], s["table"], ids, s["lens"], **into)]


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "decode": _decode, "sparse": _sparse}[state["op"]](state)


# ------------------------------------------------------------- work
def work(case):
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    e4m3 = case.get("cache", "e4m3") == "e4m3"
    width = D if e4m3 else 2 * D
    lens, new = zip(*_lengths(case))
    if case["op"] == "append":
        n = sum(new)
        rows = n * Hkv
        b = rows * (4 * D + 2 * width) + n * D * 4
        blocks = -(-n // page) * Hkv
        b += blocks * ((4 * D if case["bounds"] else 0) + (8 if e4m3 else 0))
        return {"bytes": b, "flops": rows * 3 * D}
    Hq = case["Hq"]
    qo = 4 * B * Hq * D
    if case["op"] == "decode":
        rows = sum(lens) * Hkv
        return {"bytes": rows * 2 * width + qo, "flops": rows * (Hq // Hkv) * 4 * D}
    blocks = [-(-n // page) for n in lens]
    rows = sum(min(n, case["n_sel"] * page) for n in lens) * Hkv
    scored = sum(blocks) * Hkv
    return {"bytes": rows * 2 * width + scored * 4 * D + qo + 4 * B * Hkv * case["n_sel"],
            "flops": rows * (Hq // Hkv) * 4 * D + scored * 4 * D}


# ------------------------------------------------------------- 64 bits
def _grid(x):
    """x rounded to the nearest E4M3 value, ties to even."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4
    step = torch.ldexp(torch.ones_like(x), e)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _turn(x, pos):
    """Rows x [..., n, heads, D] in 64 bits turned by their positions [..., n]."""
    z = torch.view_as_complex(x.double().unflatten(-1, (D // 2, 2)).contiguous())
    w = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[..., None] * _freqs())
    return torch.view_as_real(z * w[..., None, :]).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    page, lens, table = s["page"], s["lens"].tolist(), s["table"].long()
    if case["op"] == "append":
        return _exact_append(s, page, lens, table)
    B, Hq, _ = s["q"].shape
    Hkv = s["kp"].shape[1]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    chosen = torch.full((B, Hkv, case.get("n_sel", 1)), -1, dtype=torch.int64, device="cuda")
    for b, n in enumerate(lens):
        nb = -(-n // page)
        pg = table[b, :nb]
        q = _turn(s["q"][b][None], torch.tensor([n], device="cuda"))[0].view(Hkv, -1, D)
        for h in range(Hkv):
            keep = torch.arange(n, device="cuda")
            if case["op"] == "sparse":
                lo, hi = s["bounds"][pg, h, 0].double(), s["bounds"][pg, h, 1].double()
                top = torch.zeros(nb, dtype=torch.float64, device="cuda")
                for g in range(q.shape[1]):
                    top += torch.maximum(q[h, g] * lo, q[h, g] * hi).sum(-1)
                top[0] = top[nb - 1] = math.inf
                best = torch.argsort(-top, stable=True)[:case["n_sel"]].sort().values
                chosen[b, h, :best.numel()] = best
                keep = (best[:, None] * page + torch.arange(page, device="cuda")).flatten()
                keep = keep[keep < n]
            at = pg[keep // page], h, keep % page
            k, v = _values(s["kp"][at]).double(), _values(s["vp"][at]).double()
            if s["ks"] is not None:
                k *= s["ks"][at[0], h].double()[:, None]
                v *= s["vs"][at[0], h].double()[:, None]
            p = torch.softmax(q[h] @ k.T / math.sqrt(D), -1)
            out[b, h * q.shape[1]:(h + 1) * q.shape[1]] = p @ v
    return [out] if case["op"] == "decode" else [chosen.to(torch.int32), out]


def _exact_append(s, page, lens, table):
    B, T = s["k"].shape[:2]
    new = s["new"].tolist() if s["new"] is not None else [T] * B
    pools = [_values(s["kp"]).double(), _values(s["vp"]).double()]
    scales = [s["ks"].double(), s["vs"].double()] if s["kind"] == "e4m3" else None
    bounds = s["bounds"].double() if "bounds" in s else None
    for b in range(B):
        at = torch.arange(lens[b], lens[b] + new[b], device="cuda")
        fresh = [_turn(s["k"][b, :new[b]], at), s["v"][b, :new[b]].double()]
        for j in range(lens[b] // page, -(-(lens[b] + new[b]) // page)):
            pg = int(table[b, j])
            r0, r1 = max(lens[b], j * page), min(lens[b] + new[b], (j + 1) * page)
            was = r0 - j * page
            for c in (0, 1):
                x = fresh[c][r0 - lens[b]:r1 - lens[b]].transpose(0, 1)  # [Hkv, rows, D]
                if scales is None:
                    pools[c][pg, :, was:was + r1 - r0] = x
                else:
                    m, e = torch.frexp(x.abs().amax((1, 2)) / 448.0)
                    e = torch.where(m == 0.5, e - 1, e).clamp(E_MIN, E_MAX)
                    now = torch.ldexp(torch.ones_like(m), e)
                    if was:
                        now = torch.maximum(now, scales[c][pg])
                        pools[c][pg, :, :was] = _grid(pools[c][pg, :, :was] * (scales[c][pg] / now)[:, None, None])
                    scales[c][pg] = now
                    pools[c][pg, :, was:was + r1 - r0] = _grid(x / now[:, None, None])
                if c == 0 and bounds is not None:
                    lo, hi = x.amin(1), x.amax(1)
                    if was:
                        lo, hi = torch.minimum(lo, bounds[pg, :, 0]), torch.maximum(hi, bounds[pg, :, 1])
                    bounds[pg, :, 0], bounds[pg, :, 1] = lo, hi
    out = pools if scales is None else [pools[0], scales[0], pools[1], scales[1]]
    return out + ([bounds] if bounds is not None else [])
