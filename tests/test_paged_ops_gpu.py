"""GPU parity of the paged-cache operators (append with rotation into bf16 and
E4M3 pages, decode over E4M3 pages, block selection, block-sparse decode)
against their float64 statements in paged_reference.py.

Tolerances, derived before the first run (u: half a step of a type, relative:
bf16 2^-8, f16 2^-11, float32 2^-24, E4M3 2^-4 or 2^-10 absolute below 2^-6):

* appended bf16 rows: one bf16 rounding, u |x|, and the float32 rotation: two
  products, a sum and the table's rounding, at most 4 u32 (|x0| + |x1|);
* appended E4M3 rows: one E4M3 rounding of x / scale, plus the same rotation
  error; scales and re-coded older rows exactly;
* attention over E4M3 pages: q carries 1 f16 rounding, so a score is off by at
  most delta = 2^-11 S + 2^-19 (1 + |s|), S = sum_d |q_d k_d| / sqrt(D), and a
  softmax weight by the factor e^(2 delta); the weight itself is rounded to f16
  (2^-11, and 2^-25 of 2^7 absolute: 2^-32 for each of n rows); then one bf16
  rounding of the output. With A = sum_n p_n |v_n|:
  |err| <= u |out| + A (expm1(2 delta) + 2^-10) + n 2^-32 max|v|;
* over bf16 pages: q carries 2^-16 (two bf16 terms: the first leaves at most 2^-8 |x|, of
  which the second leaves 2^-8), a weight 2^-8.
* the log-sum-exp: delta, and float32 rounding.
The 2^-19 (1 + |s|) covers float32 sums of 128 products (their errors are far
below the worst case) and the exponent's and exponential's own rounding.
"""
import math
import threading

import pytest
import torch

import gqa_attention_rope_b200 as la
import paged_reference as R
from gqa_attention_rope_b200 import build as labuild
from guards import check_guard, guarded

pytestmark = pytest.mark.gpu

D = 128
THETA = 500000.0
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    labuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la.lib()
    la.llama_attn_get_device_error()
    yield
    assert la.llama_attn_get_device_error() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_table(g, lens, page, extra=2, slack=0):
    """A block table whose pages lie scattered in the pool; unset entries are -1."""
    need = [-(-n // page) for n in lens]
    blocks = max(1, max(need)) + slack
    n_pages = sum(need) + extra
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), blocks), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, n_pages


def e4m3_pool(g, n_pages, Hkv, page, spread=0):
    """Random codes without NaN, and scales 2^-spread .. 2^spread."""
    x = (torch.randn(n_pages, Hkv, page, D, generator=g) * 64).clamp(-448, 448)
    e = torch.randint(-spread, spread + 1, (n_pages, Hkv), generator=g)
    return x.to(torch.float8_e4m3fn).view(torch.uint8), torch.ldexp(torch.full((n_pages, Hkv), 1 / 64), e)


def poison_tails(pools, table, lens, page, value):
    """Rows at or past each sequence's length, and pages of no sequence, hold ``value``."""
    for pool in pools:
        used = torch.zeros(pool.shape[0], dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                pg = int(table[b, j])
                used[pg] = True
                pool[pg, :, max(0, n - j * page):] = value
        pool[~used] = value


# ---------------------------------------------------------------- append
APPEND = [
    # kind, page, Hkv, T, lens, new_lens (None: all T)
    ("bf16", 64, 2, 1, [0, 1, 63, 64, 200], None),
    ("e4m3", 64, 2, 1, [0, 1, 63, 64, 200], None),
    ("bf16", 64, 1, 130, [0, 5, 64], None),
    ("e4m3", 64, 1, 130, [0, 5, 64], None),
    ("e4m3", 64, 8, 17, [60, 0, 47], [17, 0, 3]),
    ("bf16", 192, 3, 200, [100, 191], [200, 1]),
    ("e4m3", 192, 3, 401, [100, 191, 0], [401, 1, 0]),
    ("e4m3", 256, 2, 300, [0, 255], None),
    ("e4m3", 1024, 1, 1500, [700], None),
]


def append_state(kind, page, Hkv, T, lens, new_lens, seed):
    g = gen(seed)
    B = len(lens)
    new = list(new_lens) if new_lens else [T] * B
    table, n_pages = make_table(g, [n + t for n, t in zip(lens, new)], page)
    if kind == "bf16":
        pools = [torch.randn(n_pages, Hkv, page, D, generator=g).to(torch.bfloat16) for _ in range(2)]
        scales = None
    else:
        pools, scales = zip(*(e4m3_pool(g, n_pages, Hkv, page, 3) for _ in range(2)))
        pools, scales = list(pools), list(scales)
    bounds = torch.randn(n_pages, Hkv, 2, D, generator=g).sort(dim=2).values.to(torch.bfloat16)
    k, v = (torch.randn(B, T, Hkv, D, generator=g).mul(3).to(torch.bfloat16) for _ in range(2))
    for b in range(B):  # rows past new_lens are not read
        k[b, new[b]:] = math.nan
        v[b, new[b]:] = math.nan
    return dict(B=B, new=new, table=table, n_pages=n_pages, pools=pools, scales=scales, bounds=bounds, k=k, v=v)


def run_append(kind, s, lens, rope, k, v, new_lens, bounds=True, **kw):
    d = dict(pools=[p.cuda() for p in s["pools"]],
             scales=[x.cuda() for x in s["scales"]] if s["scales"] else [],
             bounds=s["bounds"].cuda() if bounds else None,
             out_lens=torch.full((s["B"],), -7, dtype=torch.int32, device="cuda"))
    fn = la.llama_attn_kv_append_paged if kind == "bf16" else la.llama_attn_kv_append_paged_e4m3
    got = fn(k, v, *d["pools"], *d["scales"], s["table"].cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
             rope, new_lens=torch.tensor(new_lens, dtype=torch.int32, device="cuda") if new_lens else None,
             kbounds=d["bounds"], out_lens=d["out_lens"], **kw)
    assert got is d["out_lens"]
    return d


@pytest.mark.parametrize("kind,page,Hkv,T,lens,new_lens", APPEND)
def test_append(kind, page, Hkv, T, lens, new_lens):
    s = append_state(kind, page, Hkv, T, lens, new_lens, 11 + T)
    rope = la.llama_attn_rope_table_build(s["table"].shape[1] * page, D, THETA)
    d = run_append(kind, s, lens, rope, s["k"].cuda(), s["v"].cuda(), new_lens)
    torch.cuda.synchronize()
    assert d["out_lens"].tolist() == [n + t for n, t in zip(lens, s["new"])]
    value = (lambda p: p.double()) if kind == "bf16" else R.codes
    ref_pools = [value(p).clone() for p in s["pools"]]
    ref_scales = [x.double().clone() for x in s["scales"]] if s["scales"] else None
    ref_bounds = s["bounds"].double().clone()
    R.append(s["k"], s["v"], ref_pools, ref_scales, ref_bounds, s["table"], lens, s["new"], page, THETA)
    written = torch.zeros(s["n_pages"], page, dtype=torch.bool)
    mag = torch.zeros(s["n_pages"], Hkv, page, D, dtype=torch.float64)  # |x0| + |x1| of each written key
    for b in range(s["B"]):
        for t in range(s["new"][b]):
            p = lens[b] + t
            pg = int(s["table"][b, p // page])
            written[pg, p % page] = True
            x = s["k"][b, t].double().abs().view(Hkv, D // 2, 2).sum(-1, keepdim=True).expand(-1, -1, 2)
            mag[pg, :, p % page] = x.reshape(Hkv, D)
    for c in (0, 1):
        got, ref = value(d["pools"][c].cpu()), ref_pools[c]
        rot = 4 * U["f32"] * mag if c == 0 else torch.zeros_like(mag)
        if kind == "e4m3":
            assert torch.equal(d["scales"][c].cpu().double(), ref_scales[c]), "scales"
            tol = torch.maximum(2.0 ** -4 * ref.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) \
                + 1.07 * rot / ref_scales[c][:, :, None, None]
        else:
            tol = U["bf16"] * ref.abs() + 1.01 * rot
        w = written[:, None, :, None]
        assert torch.all(((got - ref).abs() <= tol) | ~w), "appended rows"
        assert torch.equal(torch.where(w, 0.0, got), torch.where(w, 0.0, ref)), "other rows"
        if kind == "bf16":
            raw, was = d["pools"][c].cpu().view(torch.int16), s["pools"][c].view(torch.int16)
            assert torch.equal(torch.where(w, 0, raw), torch.where(w, 0, was)), "other rows' bits"
    got = d["bounds"].cpu().double()
    top = 3 * 8.0  # |x0| + |x1| of any key here
    assert torch.all((got - ref_bounds).abs() <= U["bf16"] * ref_bounds.abs() + 4 * U["f32"] * top)


def test_append_without_bounds_and_with_fused_projection_strides():
    """k and v as slices of a fused [B, T, (Hq + 2 Hkv) * D] projection, also of a longer batch."""
    page, Hkv, Hq, T, lens = 64, 2, 4, 70, [3, 64]
    s = append_state("e4m3", page, Hkv, T, lens, None, 5)
    W = (Hq + 2 * Hkv) * D
    fused = torch.full((2, T + 9, W), math.nan, dtype=torch.bfloat16)
    fused[:, :T, Hq * D:(Hq + Hkv) * D] = s["k"].reshape(2, T, -1)
    fused[:, :T, (Hq + Hkv) * D:] = s["v"].reshape(2, T, -1)
    f = fused.cuda()
    k = f[:, :T, Hq * D:(Hq + Hkv) * D].view(2, T, Hkv, D)
    v = f[:, :T, (Hq + Hkv) * D:].view(2, T, Hkv, D)
    rope = la.llama_attn_rope_table_build(s["table"].shape[1] * page, D, THETA)
    a = run_append("e4m3", s, lens, rope, k, v, None, bounds=False)
    b = run_append("e4m3", s, lens, rope, s["k"].cuda(), s["v"].cuda(), None)
    for x, y in zip(a["pools"] + a["scales"], b["pools"] + b["scales"]):
        assert torch.equal(x, y)
    # one prompt for every sequence of the batch: batch stride 0
    c = run_append("e4m3", s, lens, rope, k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1), None)
    e = run_append("e4m3", s, lens, rope, k[:1].repeat(2, 1, 1, 1), v[:1].repeat(2, 1, 1, 1), None)
    for x, y in zip(c["pools"] + c["scales"], e["pools"] + e["scales"]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T", [1, 7, 64])
def test_append_steps_equal_one_append_but_for_subnormals(T):
    """An E4M3 block filled T rows at a time: same scales as at once; codes differ at most by
    the second rounding of values below 2^-6 of the final scale (half a subnormal step)."""
    page, Hkv, n = 64, 2, 64
    g = gen(77)
    k, v = ((torch.randn(1, n, Hkv, D, generator=g) * torch.logspace(-3, 3, n, base=2)[None, :, None, None])
            .to(torch.bfloat16).cuda() for _ in range(2))
    rope = la.llama_attn_rope_table_build(page, D, THETA)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")

    def fresh():
        return ([torch.zeros(1, Hkv, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)],
                [torch.full((1, Hkv), math.nan, device="cuda") for _ in range(2)],
                torch.full((1, Hkv, 2, D), math.nan, dtype=torch.bfloat16, device="cuda"))
    p1, s1, b1 = fresh()
    la.llama_attn_kv_append_paged_e4m3(k, v, *p1, *s1, table, torch.zeros(1, dtype=torch.int32, device="cuda"), rope,
                                       kbounds=b1)
    p2, s2, b2 = fresh()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(0, n, T):
        nxt = torch.empty_like(lens)
        la.llama_attn_kv_append_paged_e4m3(k[:, t:t + T], v[:, t:t + T], *p2, *s2, table, lens, rope, kbounds=b2,
                                           out_lens=nxt)
        lens = nxt
    torch.cuda.synchronize()
    assert lens.item() == n and torch.equal(b1, b2)
    for x, y, sx, sy in zip(p1, p2, s1, s2):
        assert torch.equal(sx, sy)
        x, y = R.codes(x.cpu()), R.codes(y.cpu())
        big = x.abs() >= 2.0 ** -5
        assert torch.equal(x[big], y[big])
        assert (x - y).abs().max() <= 2.0 ** -9  # two roundings, half a subnormal step each


@pytest.mark.parametrize("page,Hkv,B,T", [(64, 8, 37, 300), (128, 4, 90, 500), (64, 1, 200, 400), (192, 3, 70, 700), (512, 2, 60, 1500)])
def test_append_of_a_large_batch_equals_its_parts(page, Hkv, B, T):
    """A ragged batch of many blocks at once, and sequence by sequence: the same bits."""
    g = gen(T)
    lens = [int(x) for x in torch.randint(0, 3 * page, (B,), generator=g)]
    new = [int(x) for x in torch.randint(0, T + 1, (B,), generator=g)]
    lens[0], new[0], lens[1], new[1], lens[2], new[2] = 0, 5, 0, T, page, T
    s = append_state("e4m3", page, Hkv, T, lens, new, 12)
    s["table"][5, 0] = -1 if lens[5] < page and new[5] else s["table"][5, 0]
    rope = la.llama_attn_rope_table_build(s["table"].shape[1] * page, D, THETA)
    a = run_append("e4m3", s, lens, rope, s["k"].cuda(), s["v"].cuda(), new)
    bad = la.DEVERR_BLOCK_TABLE if lens[5] < page and new[5] else 0
    assert la.llama_attn_get_device_error() == bad
    out = []
    for b in range(B):
        one = dict(s, B=1, table=s["table"][b:b + 1])
        d = run_append("e4m3", one, lens[b:b + 1], rope, s["k"][b:b + 1].cuda(), s["v"][b:b + 1].cuda(), new[b:b + 1])
        s["pools"], s["scales"] = [x.cpu() for x in d["pools"]], [x.cpu() for x in d["scales"]]
        s["bounds"] = d["bounds"].cpu()
        out += d["out_lens"].tolist()
    assert la.llama_attn_get_device_error() == bad
    assert a["out_lens"].tolist() == out
    for x, y in zip(a["pools"] + a["scales"] + [a["bounds"]], s["pools"] + s["scales"] + [s["bounds"]]):
        assert torch.equal(x.cpu(), y)


def test_append_leaves_refused_sequences_alone():
    page, Hkv, T = 64, 1, 4
    lens, new = [-1, 10, 126, 5], [4, 9, 4, 4]  # negative length, more than T, past the table, fine
    s = append_state("bf16", page, Hkv, T, [0, 0, 0, 5], [4, 4, 4, 4], 3)
    s["table"] = torch.tensor([[0, 1], [2, 3], [4, 5], [1, 9]], dtype=torch.int32)
    s["pools"] = [torch.randn(6, Hkv, page, D).to(torch.bfloat16) for _ in range(2)]
    s["bounds"] = torch.zeros(6, Hkv, 2, D, dtype=torch.bfloat16)
    rope = la.llama_attn_rope_table_build(2 * page, D, THETA)
    d = run_append("bf16", s, lens, rope, s["k"].cuda(), s["v"].cuda(), new)
    assert la.llama_attn_get_device_error() == la.DEVERR_CACHE_LEN
    assert d["out_lens"].tolist() == [-1, 10, 126, 9]
    keep = [0, 2, 3, 4, 5]
    for x, y in zip(d["pools"], s["pools"]):
        assert torch.equal(x.cpu()[keep], y[keep]) and not torch.equal(x.cpu()[1], y[1])
    s["table"][3, 0] = 6  # a page that is not there
    d = run_append("bf16", s, [0, 0, 0, 5], rope, s["k"].cuda().nan_to_num(), s["v"].cuda().nan_to_num(), [0, 0, 0, 4])
    assert la.llama_attn_get_device_error() == la.DEVERR_BLOCK_TABLE
    for x, y in zip(d["pools"], s["pools"]):
        assert torch.equal(x.cpu(), y)


# ---------------------------------------------------------------- attention
def check_attention(kind, out, lse, ref, max_v, n_rows):
    o, ref_lse, mass, span = ref
    u_q, u_p = (2.0 ** -11, 2.0 ** -10) if kind == "e4m3" else (2.0 ** -16, 2.0 ** -8)
    live = torch.isfinite(ref_lse)
    s_abs = torch.where(live, ref_lse.abs(), 0.0) + span  # |s| <= S; the exponent's reference is near the lse
    delta = u_q * span + 2.0 ** -19 * (1 + s_abs)
    tol = U["bf16"] * o.abs() + mass * (torch.expm1(2 * delta) + u_p)[..., None] + n_rows * 2.0 ** -32 * max_v
    err = (out.double().cpu() - o).abs()
    assert torch.all(err <= tol), f"worst error over tolerance: {(err / tol.clamp(min=1e-30)).max():.3g}"
    if lse is not None:
        got = lse.double().cpu()
        assert torch.equal(torch.isinf(got), ~live)
        assert torch.all((got - ref_lse)[live].abs() <= (delta + 2.0 ** -22 * (1 + s_abs))[live])


def attention_state(kind, page, Hq, Hkv, lens, seed, spread=0, q_scale=2.0):
    g = gen(seed)
    table, n_pages = make_table(g, lens, page, slack=1)
    if kind == "e4m3":
        (kp, ks), (vp, vs) = (e4m3_pool(g, n_pages, Hkv, page, spread if c else 0) for c in (0, 1))
        poison_tails([kp, vp], table, lens, page, 0x7F)
        kv = R.codes(kp) * ks.double()[:, :, None, None]
        vv = R.codes(vp) * vs.double()[:, :, None, None]
        scales = [ks, vs]
    else:
        kp, vp = (torch.randn(n_pages, Hkv, page, D, generator=g).to(torch.bfloat16) for _ in range(2))
        poison_tails([kp, vp], table, lens, page, math.nan)
        kv, vv, scales = kp.double(), vp.double(), []
    q = (torch.randn(len(lens), Hq, D, generator=g) * q_scale).to(torch.bfloat16)
    return dict(q=q, kp=kp, vp=vp, kv=kv, vv=vv, scales=scales, table=table, lens=lens, page=page)


def on_gpu(s):
    return dict(q=s["q"].cuda(), pools=(s["kp"].cuda(), s["vp"].cuda()), scales=tuple(x.cuda() for x in s["scales"]),
                table=s["table"].cuda(), lens=torch.tensor(s["lens"], dtype=torch.int32, device="cuda"))


DECODE = [
    # page, Hq, Hkv, lens, spread of the value scales, q_pos_offset
    (64, 32, 8, [1000], 0, 0),
    (64, 8, 1, [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 640], 0, 0),
    (128, 1, 1, [300, 5], 2, -1),
    (256, 6, 2, [256, 255, 257, 0, 1], 4, 0),
    (64, 10, 2, [777, 64], 0, -1),
    (192, 18, 2, [500, 191, 193], 3, 0),
    (64, 32, 2, [2049, 1, 63], 0, 0),
    (64, 13, 13, [90, 200], 0, 0),
    (128, 16, 1, [20000], 1, 0),
    # more pairs than clusters of 8 fit, and caches too long for one
    (64, 24, 8, [0, 1, 64, 65, 777, 2049, 3, 640], 2, 0),
    (64, 96, 8, [700, 1, 130, 2000, 64, 0], 0, -1),
    (64, 3, 1, [9000, 1, 17000], 0, 0),
    # clusters of 1, 3 and 16; more pairs than CTAs are resident, most of a stage or none
    (64, 8, 8, [5, 0, 64, 130, 1, 640, 65, 31, 200, 128, 0, 2, 63, 400, 66, 7, 500, 1, 129, 64, 30, 3, 0, 90], 1, 0),
    (64, 16, 8, [600, 0, 1, 64, 65, 129, 300, 2, 1900, 63], 0, -1),
    (64, 15, 1, [10000, 40], 2, 0),
    (64, 12, 1, [10000, 0, 64, 65], 0, 0),
    (64, 8, 8, [(7 * i * i) % 97 if i % 9 else 70 * i for i in range(64)], 3, 0),
    (128, 40, 4, [1, 0, 2, 700, 1, 1, 130, 1] * 12, 0, 0),
]


@pytest.mark.parametrize("page,Hq,Hkv,lens,spread,off", DECODE)
def test_decode_e4m3(page, Hq, Hkv, lens, spread, off):
    s = attention_state("e4m3", page, Hq, Hkv, lens, 100 + Hq + page, spread)
    d = on_gpu(s)
    buf, out = guarded(s["q"].shape)
    lse = torch.empty(len(lens), Hq, device="cuda")
    ws = torch.full((la.llama_attn_decode_runs_workspace_size(len(lens), Hq, Hkv),), 0xAB, dtype=torch.uint8,
                    device="cuda")
    got = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"], out=out, lse=lse,
                                          workspace=ws, q_pos_offset=off)
    assert got is out
    torch.cuda.synchronize()
    check_guard(buf)
    ref = R.decode(s["q"], s["kv"], s["vv"], s["table"], lens, page, THETA, off)
    max_v = max(float(s["vv"][s["table"][b, j].long()].nan_to_num().abs().max())
                for b, n in enumerate(lens) for j in range(-(-n // page)))
    check_attention("e4m3", out, lse, ref, max_v, max(lens))
    again = la.llama_attn_decode_paged_e4m3(d["q"], d["pools"][0].view(torch.float8_e4m3fn),
                                            d["pools"][1].view(torch.float8_e4m3fn), *d["scales"], d["table"],
                                            d["lens"], q_pos_offset=off)
    assert torch.equal(again, out), "a second call, its own workspace, no lse"


@pytest.mark.parametrize("scale_k,scale_v", [(0.0173, 0.31), (2.0 ** -40, 2.0 ** 90), (3.0e-3, 2.0 ** -95)])
def test_decode_e4m3_any_positive_scale(scale_k, scale_v):
    s = attention_state("e4m3", 64, 8, 2, [130, 64], 9)
    for c, x in enumerate((scale_k, scale_v)):
        s["scales"][c] = (torch.rand(s["scales"][c].shape, generator=gen(c)) + 0.5) * x
    s["kv"] = R.codes(s["kp"]) * s["scales"][0].double()[:, :, None, None]
    s["vv"] = R.codes(s["vp"]) * s["scales"][1].double()[:, :, None, None]
    d = on_gpu(s)
    lse = torch.empty(2, 8, device="cuda")
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"], lse=lse)
    check_attention("e4m3", out, lse, R.decode(s["q"], s["kv"], s["vv"], s["table"], s["lens"], 64, THETA),
                    448 * 1.5 * scale_v, 130)


@pytest.mark.parametrize("scale_v", [2.0 ** -100, 2.0 ** 117])
def test_decode_e4m3_ends_of_the_scale_range_over_many_rows(scale_v):
    """The denominator adds weights divided by the value scale: neither end overflows or vanishes."""
    n = 40000
    s = attention_state("e4m3", 64, 2, 1, [n], 19, q_scale=6.0)
    s["scales"][1] = torch.full_like(s["scales"][1], scale_v)
    s["vv"] = R.codes(s["vp"]) * scale_v
    d = on_gpu(s)
    lse = torch.empty(1, 2, device="cuda")
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"], lse=lse)
    check_attention("e4m3", out, lse, R.decode(s["q"], s["kv"], s["vv"], s["table"], s["lens"], 64, THETA),
                    448 * scale_v, n)


@pytest.mark.parametrize("q_scale", [1e-30, 1e30, 40.0])
def test_decode_e4m3_query_magnitudes(q_scale):
    """Queries far outside f16's range (1e30: the greatest key takes all the weight)."""
    s = attention_state("e4m3", 64, 4, 1, [100], 21, q_scale=q_scale)
    if q_scale == 1e30:  # one key per head stands out, so that rounding cannot change the winner
        s["q"] = (torch.sign(s["q"].double()) * 1e30).to(torch.bfloat16)
        s["kp"][s["table"][0].clamp(min=0).long()] &= 0x80  # +-0 but for one row
        s["kp"][int(s["table"][0, 0]), 0, 7] = 0x38 | (s["kp"][int(s["table"][0, 0]), 0, 7] & 0x80)
        s["kv"] = R.codes(s["kp"]) * s["scales"][0].double()[:, :, None, None]
    d = on_gpu(s)
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"])
    o, l, mass, span = R.decode(s["q"], s["kv"], s["vv"], s["table"], s["lens"], 64, THETA)
    if q_scale == 1e30:
        assert torch.all((out.double().cpu() - o).abs() <= U["bf16"] * o.abs() + 2.0 ** -10 * mass)
    else:
        check_attention("e4m3", out, None, (o, l, mass, span), 448 / 64, 100)


SPARSE = [
    # kind, page, Hq, Hkv, lens, n_sel, n_first, n_last, q_pos_offset
    ("bf16", 64, 8, 2, [0, 1, 64, 65, 1000, 3000], 7, 1, 1, 0),
    ("e4m3", 64, 8, 2, [0, 1, 64, 65, 1000, 3000], 7, 1, 1, 0),
    ("bf16", 128, 32, 2, [5000, 129], 5, 0, 2, -1),
    ("e4m3", 256, 9, 1, [4000, 256, 4097], 3, 1, 2, 0),
    ("bf16", 64, 1, 1, [777], 1, 0, 0, 0),
    ("e4m3", 192, 12, 12, [1000, 10], 40, 1, 1, -1),
    ("e4m3", 64, 16, 1, [70001], 128, 4, 4, 0),
    ("bf16", 64, 4, 4, [20011, 9000], 33, 1, 0, 0),
    ("bf16", 64, 24, 8, [0, 1, 64, 65, 777, 2049, 3, 640], 7, 1, 1, 0),
    ("e4m3", 64, 24, 8, [0, 1, 64, 65, 777, 2049, 3, 640], 7, 1, 1, 0),
    ("bf16", 128, 96, 8, [700, 1, 1300, 2000, 64, 0], 5, 0, 1, -1),
    ("e4m3", 128, 96, 8, [700, 1, 1300, 2000, 64, 0], 5, 0, 1, -1),
    ("bf16", 64, 6, 2, [20011, 9000, 100], 180, 1, 1, 0),
    ("bf16", 64, 24, 2, [20011, 9000, 100], 180, 1, 1, 0),
    # runs over the batch
    ("bf16", 64, 16, 8, [0, 1, 64, 65, 777, 2049, 3, 640] * 6, 7, 1, 1, 0),
    ("e4m3", 64, 16, 8, [0, 1, 64, 65, 777, 2049, 3, 640] * 6, 7, 1, 1, 0),
    ("bf16", 64, 6, 2, [40000, 9000, 100], 560, 1, 1, 0),
    ("e4m3", 64, 24, 2, [40000, 9000, 100], 560, 1, 1, 0),
]


def bounds_of(s, value=None):
    lo, hi = s["kv"].nan_to_num(nan=math.inf).amin(2), s["kv"].nan_to_num(nan=-math.inf).amax(2)
    return torch.stack([lo, hi], 2).clamp(-1e30, 1e30).to(torch.bfloat16)


@pytest.mark.parametrize("kind,page,Hq,Hkv,lens,n_sel,n_first,n_last,off", SPARSE)
def test_select_and_sparse_decode(kind, page, Hq, Hkv, lens, n_sel, n_first, n_last, off):
    s = attention_state(kind, page, Hq, Hkv, lens, 300 + Hq + page)
    d = on_gpu(s)
    bounds = bounds_of(s)
    buf, ids = guarded((len(lens), Hkv, n_sel), torch.int32, 12345)
    got = la.llama_attn_select_blocks(d["q"], bounds.cuda(), d["table"], d["lens"], page, n_sel, n_first, n_last,
                                      block_ids=ids, q_pos_offset=off)
    assert got is ids
    torch.cuda.synchronize()
    check_guard(buf, 12345, "block_ids")
    ref_ids = R.select(s["q"], bounds, s["table"], lens, page, n_sel, n_first, n_last, THETA, off)
    assert torch.equal(ids.cpu(), ref_ids)
    fn = la.llama_attn_decode_paged_sparse if kind == "bf16" else la.llama_attn_decode_paged_sparse_e4m3
    buf, out = guarded(s["q"].shape)
    lse = torch.empty(len(lens), Hq, device="cuda")
    fn(d["q"], *d["pools"], *d["scales"], d["table"], ids, d["lens"], out=out, lse=lse, q_pos_offset=off)
    torch.cuda.synchronize()
    check_guard(buf)
    ref = R.decode(s["q"], s["kv"], s["vv"], s["table"], lens, page, THETA, off, ref_ids)
    check_attention(kind, out, lse, ref, 8.0, n_sel * page)


def test_select_ties_and_equal_scores():
    """Equal blocks: the lowest indices; two values only: all of the greater, then the lowest others."""
    Hq, Hkv, page, nb = 4, 1, 64, 300
    q = torch.randn(1, Hq, D, generator=gen(1)).to(torch.bfloat16)
    table = torch.randperm(nb, generator=gen(2)).to(torch.int32)[None]
    lens = torch.tensor([nb * page], dtype=torch.int32)
    for greater in ([], [7, 100, 298], list(range(40, 90))):
        bounds = torch.ones(nb, Hkv, 2, D, dtype=torch.bfloat16)
        bounds[:, :, 0] = -1
        for j in greater:
            bounds[table[0, j].long()] *= 2
        ids = la.llama_attn_select_blocks(q.cuda(), bounds.cuda(), table.cuda(), lens.cuda(), page, 20, 2, 1)
        best = (greater + [j for j in range(2, nb - 1) if j not in greater])[:17]
        assert ids[0, 0].tolist() == sorted([0, 1] + best + [nb - 1])


@pytest.mark.parametrize("spread", [0, 1])
def test_select_decides_near_scores_in_float64(spread):
    """Blocks whose scores differ by 1e-9 of their size and less: the order is float64's, which the
    reference forms as a sum over heads of maxima."""
    Hq, Hkv, page, nb, n_sel = 8, 2, 64, 700, 40
    g = gen(5)
    q = torch.randn(1, Hq, D, generator=g).to(torch.bfloat16)
    base = torch.randn(Hkv, 2, D, generator=g).sort(dim=1).values.mul(4).to(torch.bfloat16)
    bounds = base.expand(nb, -1, -1, -1).clone()
    bounds[:, :, :, 17] = (torch.randn(nb, Hkv, 2, generator=g).abs() * 2.0 ** -24).to(torch.bfloat16)
    bounds[:, :, 0, 17] *= -1
    if spread:  # and as many far from them on both sides
        bounds[::3] = (bounds[::3].float() * 0.5).to(torch.bfloat16)
        bounds[1::40] = (bounds[1::40].float() * 1.5).to(torch.bfloat16)
    table = torch.randperm(nb, generator=g).to(torch.int32)[None]
    lens = [nb * page - 5]
    ids = la.llama_attn_select_blocks(q.cuda(), bounds.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                      page, n_sel)
    assert torch.equal(ids.cpu(), R.select(q, bounds, table, lens, page, n_sel, 1, 1, THETA))


def test_select_with_values_that_are_not_finite_gives_distinct_ascending_ids():
    nb, page = 500, 64
    g = gen(6)
    table = torch.randperm(nb, generator=g).to(torch.int32)[None].cuda()
    lens = torch.tensor([nb * page], dtype=torch.int32, device="cuda")
    for bad in (math.nan, math.inf, -math.inf, 3.3e38):
        for every in (1, 3, 500):
            bounds = torch.randn(nb, 1, 2, D, generator=g).sort(dim=2).values.to(torch.bfloat16)
            bounds[::every, 0, 0, 5] = bad
            q = torch.randn(1, 4, D, generator=g).to(torch.bfloat16)
            for qq in (q, q * 1e30, torch.full_like(q, bad)):
                for n_sel in (3, 300):
                    buf, ids = guarded((1, 1, n_sel), torch.int32, 12345)
                    la.llama_attn_select_blocks(qq.cuda(), bounds.cuda(), table, lens, page, n_sel, block_ids=ids)
                    torch.cuda.synchronize()
                    check_guard(buf, 12345, "block_ids")
                    i = ids[0, 0].tolist()
                    assert i[0] == 0 and i[-1] == nb - 1 and all(a < b for a, b in zip(i, i[1:]))


@pytest.mark.parametrize("B,Hkv,nb", [(1, 1, 2048), (1, 8, 1000), (40, 8, 129), (2, 2, 24576)])
def test_select_cluster_sizes(B, Hkv, nb):
    """Every cluster width, up to the greatest number of blocks."""
    page, Hq, n_sel = 64, Hkv, 50
    g = gen(nb)
    q = torch.randn(B, Hq, D, generator=g).to(torch.bfloat16)
    n_pages = 256
    bounds = torch.randn(n_pages, Hkv, 2, D, generator=g).sort(dim=2).values.to(torch.bfloat16)
    table = torch.randint(0, n_pages, (B, nb), generator=g, dtype=torch.int32)  # pages shared: many ties
    lens = [nb * page - 63 * (b % 2) for b in range(B)]
    ids = la.llama_attn_select_blocks(q.cuda(), bounds.cuda(), table.cuda(),
                                      torch.tensor(lens, dtype=torch.int32, device="cuda"), page, n_sel)
    assert torch.equal(ids.cpu(), R.select(q, bounds, table, lens, page, n_sel, 1, 1, THETA))


def test_sparse_over_all_blocks_matches_dense_and_paged_decode():
    """Every block chosen: the E4M3 forms agree bit for bit (same units), bf16 with the bf16 decode."""
    s = attention_state("e4m3", 64, 16, 2, [700, 64, 1], 31)
    d = on_gpu(s)
    ids = torch.full((3, 2, 11), -1, dtype=torch.int32)
    for b, n in enumerate(s["lens"]):
        ids[b, :, :-(-n // 64)] = torch.arange(-(-n // 64))
    a = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"])
    b = la.llama_attn_decode_paged_sparse_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], ids.cuda(), d["lens"])
    assert torch.equal(a, b)
    s = attention_state("bf16", 64, 16, 2, [700, 64, 1], 32)
    d = on_gpu(s)
    a = la.llama_attn_decode_paged(d["q"], *d["pools"], d["table"], d["lens"])
    b = la.llama_attn_decode_paged_sparse(d["q"], *d["pools"], d["table"], ids.cuda(), d["lens"])
    assert (a.float() - b.float()).abs().max() <= 1.5e-2  # the bf16 decode's own tolerance


def test_sparse_ids_are_checked_on_the_device():
    s = attention_state("bf16", 64, 4, 1, [200], 41)
    d = on_gpu(s)

    def run(ids):
        out = la.llama_attn_decode_paged_sparse(d["q"], *d["pools"], d["table"],
                                                torch.tensor([[ids]], dtype=torch.int32, device="cuda"), d["lens"])
        return la.llama_attn_get_device_error(), out
    for bad in ([2, 1, -1, -1], [1, 1, -1, -1], [-1, 2, -1, -1], [0, 4, -1, -1], [-5, -1, -1, -1], [0, 1 << 30, -1, -1]):
        err, out = run(bad)
        assert err == la.DEVERR_BLOCK_IDS, bad
        assert torch.isfinite(out.float()).all()
    err, out = run([-1, -1, -1, -1])
    assert err == 0 and not out.any()
    err, out = run([0, 2, 3, -1, 99, 99])  # entries past the sequence's number of blocks are not read
    assert err == 0
    ref = R.decode(s["q"], s["kv"], s["vv"], s["table"], s["lens"], 64, THETA, 0, torch.tensor([[[0, 2, 3]]]))
    check_attention("bf16", out, None, ref, 8.0, 200)


def test_bad_pages_and_lengths_set_the_error_word():
    s = attention_state("e4m3", 64, 4, 1, [100, 100, 100], 51)
    d = on_gpu(s)
    table = d["table"].clone()
    table[0, 1] = s["kp"].shape[0]
    lens = torch.tensor([100, -3, 64 * table.shape[1] + 1], dtype=torch.int32, device="cuda")
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], table, lens)
    assert la.llama_attn_get_device_error() == la.DEVERR_BLOCK_TABLE | la.DEVERR_CACHE_LEN
    assert torch.isfinite(out.float()).all() and not out[1:].any()
    bounds = torch.zeros(s["kp"].shape[0], 1, 2, D, dtype=torch.bfloat16, device="cuda")
    ids = la.llama_attn_select_blocks(d["q"], bounds, table, lens, 64, 1, 0, 0)
    assert la.llama_attn_get_device_error() == la.DEVERR_BLOCK_TABLE | la.DEVERR_CACHE_LEN
    assert ids[1:].eq(-1).all()


# ---------------------------------------------------------------- used as a program uses them
def test_serving_loop_prompt_then_steps():
    """A prompt is appended to E4M3 pages, then tokens one by one: append, choose blocks, attend
    with the token's own key in the cache. The cache and every step against float64."""
    page, Hq, Hkv, steps = 64, 8, 2, 5
    prompt = [150, 1, 64]
    B = len(prompt)
    g = gen(61)
    T = max(prompt)
    k, v = (torch.randn(B, T, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    total = [n + steps for n in prompt]
    table, n_pages = make_table(g, total, page)
    rope = la.llama_attn_rope_table_build(table.shape[1] * page, D, THETA)
    kp, vp = (torch.full((n_pages, Hkv, page, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n_pages, Hkv), math.nan, device="cuda") for _ in range(2))
    kb = torch.full((n_pages, Hkv, 2, D), math.nan, dtype=torch.bfloat16, device="cuda")
    dt = table.cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    after = torch.empty_like(lens)
    la.llama_attn_kv_append_paged_e4m3(k.cuda(), v.cuda(), kp, vp, ks, vs, dt, lens, rope,
                                       new_lens=torch.tensor(prompt, dtype=torch.int32, device="cuda"), kbounds=kb,
                                       out_lens=after)
    hist = [(k[b, :prompt[b]], v[b, :prompt[b]]) for b in range(B)]
    for step in range(steps):
        kn, vn = (torch.randn(B, 1, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
        q = (torch.randn(B, Hq, D, generator=g) * 2).to(torch.bfloat16)
        lens, after = after, torch.empty_like(lens)
        la.llama_attn_kv_append_paged_e4m3(kn.cuda(), vn.cuda(), kp, vp, ks, vs, dt, lens, rope, kbounds=kb,
                                           out_lens=after)
        ids = la.llama_attn_select_blocks(q.cuda(), kb, dt, after, page, 2, 0, 1, q_pos_offset=-1)
        out = la.llama_attn_decode_paged_sparse_e4m3(q.cuda(), kp, vp, ks, vs, dt, ids, after, q_pos_offset=-1)
        hist = [(torch.cat([a, kn[b]]), torch.cat([c, vn[b]])) for b, (a, c) in enumerate(hist)]
        n = [p + step + 1 for p in prompt]
        assert after.tolist() == n
        kv = R.codes(kp.cpu()) * ks.cpu().double()[:, :, None, None]
        vv = R.codes(vp.cpu()) * vs.cpu().double()[:, :, None, None]
        for b in range(B):  # the cache holds the history, rotated, within one rounding (two where a block grew)
            row = torch.arange(n[b])
            pg = table[b, row // page].long()
            want = (R.rotate(hist[b][0], row[:, None], THETA), hist[b][1].double())
            for vals, sc, w in ((kv, ks, want[0]), (vv, vs, want[1])):
                got = vals[pg, :, row % page]
                one = sc.cpu().double()[pg][..., None]
                tol = 1.001 * torch.maximum(2.0 ** -4 * w.abs(), 2.0 ** -10 * one) + 2.0 ** -10 * one + 2.0 ** -20
                assert torch.all((got - w).abs() <= tol)
        bounds = kb.cpu()
        assert torch.equal(ids.cpu(), R.select(q, bounds, table, n, page, 2, 0, 1, THETA, -1))
        ref = R.decode(q, kv, vv, table, n, page, THETA, -1, ids.cpu())
        check_attention("e4m3", out, None, ref, 8.0, 2 * page)


def test_captured_steps_replay_with_new_lengths():
    """Append, selection and decode in one CUDA graph: lengths and inputs are read at replay."""
    page, Hq, Hkv, B = 64, 8, 2, 3
    g = gen(71)
    table, n_pages = make_table(g, [400, 300, 200], page)
    dt = table.cuda()
    rope = la.llama_attn_rope_table_build(table.shape[1] * page, D, THETA)
    kp, vp = (torch.zeros(n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb = torch.zeros(n_pages, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    after, out = torch.empty_like(lens), torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(B, 1, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(B, Hkv, 3, dtype=torch.int32, device="cuda")
    ws = torch.empty(la.llama_attn_decode_runs_workspace_size(B, Hq, Hkv), dtype=torch.uint8, device="cuda")

    def step(out):
        la.llama_attn_kv_append_paged(k, v, kp, vp, dt, lens, rope, kbounds=kb, out_lens=after)
        la.llama_attn_select_blocks(q, kb, dt, after, page, 3, block_ids=ids, q_pos_offset=-1)
        la.llama_attn_decode_paged_sparse(q, kp, vp, dt, ids, after, out=out, workspace=ws, q_pos_offset=-1)
    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    eager = torch.empty_like(out)
    for i, n in enumerate(([0, 0, 0], [1, 63, 64], [399, 130, 199])):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert after.tolist() == [x + 1 for x in n]
        step(eager)
        assert torch.equal(out, eager)


def test_two_streams_at_once():
    """Two decodes that overlap, each with its own workspace, on streams of their own."""
    cases = []
    for i, kind in enumerate(("e4m3", "bf16")):
        s = attention_state(kind, 64, 8, 2, [3000, 1, 2000], 81 + i)
        d = on_gpu(s)
        bounds = bounds_of(s).cuda()
        fn = la.llama_attn_decode_paged_sparse if kind == "bf16" else la.llama_attn_decode_paged_sparse_e4m3

        def one(d=d, bounds=bounds, fn=fn, stream=None):
            ids = la.llama_attn_select_blocks(d["q"], bounds, d["table"], d["lens"], 64, 9, stream=stream)
            return fn(d["q"], *d["pools"], *d["scales"], d["table"], ids, d["lens"], stream=stream)
        cases.append(one)
    want = [one() for one in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, one in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(one())
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_memory_of_a_call_on_a_given_stream_belongs_to_that_stream():
    """A decode without a workspace of the caller's, on a side stream that is busy: what the current
    stream allocates and fills meanwhile is not the decode's working memory."""
    s = attention_state("e4m3", 64, 8, 2, [3000, 900], 97)
    d = on_gpu(s)
    bounds = bounds_of(s).cuda()

    def step(stream):
        ids = la.llama_attn_select_blocks(d["q"], bounds, d["table"], d["lens"], 64, 9, stream=stream)
        return la.llama_attn_decode_paged_sparse_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], ids, d["lens"],
                                                      stream=stream)
    want = step(None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # about 25 ms
    out = step(side)
    sizes = [la.llama_attn_decode_runs_workspace_size(2, 8, 2), 4 * 2 * 2 * 9]
    held = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(x.eq(0x5A).all() for x in held)
    assert torch.equal(out, want)


def test_pool_past_32_bit_offsets():
    """A pool of more than 2^32 bytes per tensor: rows near its end, against the same rows in a small one."""
    page, Hq, Hkv = 64, 8, 1
    n_pages = (1 << 32) // (page * D) + 6
    g = gen(95)
    lens, T = [200, 77], 3
    far = torch.tensor([[n_pages - 1, 3, n_pages - 4, n_pages - 2], [n_pages - 5, n_pages - 3, 0, 1]], dtype=torch.int32)
    near = torch.tensor([[5, 3, 2, 4], [7, 6, 0, 1]], dtype=torch.int32)
    small = [(torch.randn(8, Hkv, page, D, generator=g) * 64).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
             for _ in range(2)]
    k, v = (torch.randn(2, T, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(2, Hq, D, generator=g).to(torch.bfloat16).cuda()
    rope = la.llama_attn_rope_table_build(4 * page, D, THETA)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = []
    for table, n in ((near, 8), (far, n_pages)):
        pools = [torch.zeros(n, Hkv, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.ones(n, Hkv, device="cuda") for _ in range(2)]
        kb = torch.zeros(n, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
        for x, y in zip(pools, small):
            x[table.flatten().long()] = y[near.flatten().long()]
        t, after = table.cuda(), torch.empty_like(ln)
        la.llama_attn_kv_append_paged_e4m3(k, v, *pools, *scales, t, ln, rope, kbounds=kb, out_lens=after)
        dense = la.llama_attn_decode_paged_e4m3(q, *pools, *scales, t, after)
        ids = la.llama_attn_select_blocks(q, kb, t, after, page, 3)
        sparse = la.llama_attn_decode_paged_sparse_e4m3(q, *pools, *scales, t, ids, after)
        got.append([dense, ids, sparse, kb[t.flatten().long()]] + [x[t.flatten().long()] for x in pools + scales])
        del pools, scales, kb
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_binding_checks_every_tensor():
    """One wrong thing at a time: each is refused by name before the library is called."""
    page, Hq, Hkv, B, T, n_pages = 64, 4, 2, 2, 3, 5

    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    good = dict(k=z(B, T, Hkv, D), v=z(B, T, Hkv, D), kpages=z(n_pages, Hkv, page, D, dtype=u8),
                vpages=z(n_pages, Hkv, page, D, dtype=u8), k_scales=z(n_pages, Hkv, dtype=f32),
                v_scales=z(n_pages, Hkv, dtype=f32), block_table=z(B, 2, dtype=i32), cache_lens=z(B, dtype=i32),
                rope_table=z(2 * page, D // 2, 2, dtype=f32), new_lens=z(B, dtype=i32),
                kbounds=z(n_pages, Hkv, 2, D), out_lens=z(B, dtype=i32))
    good["block_table"][1] = 2
    la.llama_attn_kv_append_paged_e4m3(**good)
    read = dict(q=z(B, Hq, D), **{n: good[n] for n in ("kpages", "vpages", "k_scales", "v_scales", "block_table",
                                                       "cache_lens")},
                block_ids=z(B, Hkv, 3, dtype=i32), out=z(B, Hq, D), lse=z(B, Hq, dtype=f32))
    la.llama_attn_decode_paged_sparse_e4m3(**read)
    choose = dict(q=read["q"], kbounds=good["kbounds"], block_table=good["block_table"],
                  cache_lens=good["cache_lens"], block_ids=read["block_ids"])
    la.llama_attn_select_blocks(**choose, page_size=page, n_sel=3)

    def spoiled(t):
        other = torch.float16 if t.dtype == torch.bfloat16 else torch.int64 if t.dtype == i32 else torch.float64
        yield t.to(other)
        yield t.cpu()
        yield torch.cat([t, t])
        yield t[..., None]
        if t.dim() > 1:
            yield t.transpose(0, 1).contiguous().transpose(0, 1)
    for call, args, more in ((la.llama_attn_kv_append_paged_e4m3, good, {}),
                             (la.llama_attn_decode_paged_sparse_e4m3, read, {}),
                             (la.llama_attn_select_blocks, choose, dict(page_size=page, n_sel=3))):
        for name in args:
            for bad in spoiled(args[name]):
                if name in ("k", "v") and bad.dim() == 4 and bad.shape == args[name].shape and bad.is_cuda \
                        and bad.dtype == args[name].dtype:
                    continue  # strides of k and v are free as long as they agree
                if name == "rope_table" and bad.shape[0] > args[name].shape[0]:
                    continue  # a table may have more rows than the cache
                if call is la.llama_attn_select_blocks and name == "kbounds" and bad.shape[0] > n_pages:
                    continue  # the selection knows the pool by its bounds only
                with pytest.raises(ValueError):
                    call(**{**args, name: bad}, **more)
    with pytest.raises(ValueError, match="same strides"):
        la.llama_attn_kv_append_paged_e4m3(**{**good, "v": z(T, B, Hkv, D).transpose(0, 1)})
    with pytest.raises(ValueError, match="heads of a token"):
        la.llama_attn_kv_append_paged_e4m3(**{**good, "v": z(B, T, D, Hkv).transpose(2, 3)})
    with pytest.raises(ValueError, match="bfloat16 pages"):
        la.llama_attn_decode_paged_sparse(**{n: x for n, x in read.items() if n not in ("k_scales", "v_scales")})
    with pytest.raises(la.LlamaAttnError):
        la.llama_attn_select_blocks(**choose, page_size=page, n_sel=3, n_first=4)
    with pytest.raises(la.LlamaAttnError):
        la.llama_attn_decode_paged_sparse_e4m3(**{**read, "out": read["q"]})
    assert la.llama_attn_get_device_error() == 0


def test_many_sequences():
    """More sequences than a CTA has threads, most of them empty or short."""
    g = gen(91)
    B, Hq, Hkv, page = 701, 2, 1, 64
    lens = [int(x) for x in torch.randint(0, 40, (B,), generator=g)]
    lens[3], lens[700] = 500, 129
    s = attention_state("e4m3", page, Hq, Hkv, lens, 92)
    d = on_gpu(s)
    lse = torch.empty(B, Hq, device="cuda")
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"], lse=lse)
    check_attention("e4m3", out, lse, R.decode(s["q"], s["kv"], s["vv"], s["table"], lens, page, THETA), 7.0, 500)
    zero = torch.zeros_like(d["lens"])
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], zero, lse=lse)
    assert not out.any() and torch.isinf(lse).all()


def test_tensors_without_storage_are_refused_and_the_process_goes_on():
    """Under a function transform the binding gets tensors that have no data: a ValueError, and the next call runs."""
    s = attention_state("e4m3", 64, 4, 1, [100], 55)
    d = on_gpu(s)
    bounds = bounds_of(s).cuda()

    def one(q):
        with pytest.raises(ValueError, match="storage"):
            la.llama_attn_select_blocks(q, bounds, d["table"], d["lens"], 64, 1)
        with pytest.raises(ValueError, match="storage"):
            la.llama_attn_decode_paged_e4m3(q, *d["pools"], *d["scales"], d["table"], d["lens"])
        return q
    torch.func.vmap(one)(d["q"][None].repeat(2, 1, 1, 1))
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"])
    check_attention("e4m3", out, None, R.decode(s["q"], s["kv"], s["vv"], s["table"], s["lens"], 64, THETA), 7.0, 100)


def test_sparse_decodes_need_their_block_ids():
    for kind, fn in (("bf16", la.llama_attn_decode_paged_sparse), ("e4m3", la.llama_attn_decode_paged_sparse_e4m3)):
        d = on_gpu(attention_state(kind, 64, 4, 1, [100], 57))
        with pytest.raises(ValueError, match="block_ids: tensor expected"):
            fn(d["q"], *d["pools"], *d["scales"], d["table"], None, d["lens"])


def mixed_reference(s, lens, block_ids=None):
    """out, lse, and the bounds of their errors, per head. The f16 weights are off by 2^-25 at most where the
    greatest product of a weight and its value scale is at least 2^7: 2^-32 of the greatest, for each row, times a
    code of at most 448. An exponent carries the logarithm of the value scale too (up to 119 in magnitude)."""
    B, Hq, _ = s["q"].shape
    Hkv, page = s["kp"].shape[1], s["page"]
    G = Hq // Hkv
    out, tol = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    lse, lse_tol = torch.zeros(B, Hq, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    for b, n in enumerate(lens):
        q = R.rotate(s["q"][b], n, THETA)
        for g in range(Hkv):
            row = torch.arange(n)
            if block_ids is not None:
                row = torch.tensor([r for i in block_ids[b, g].tolist() if i >= 0
                                    for r in range(i * page, min(n, (i + 1) * page))])
            pg = s["table"][b, row // page].long()
            k, v, vs = s["kv"][pg, g, row % page], s["vv"][pg, g, row % page], s["scales"][1][pg, g].double()
            hs = slice(g * G, (g + 1) * G)
            sc = q[hs] @ k.T / math.sqrt(D)
            span = (q[hs].abs() @ k.abs().T / math.sqrt(D)).amax(-1)
            p = torch.softmax(sc, -1)
            out[b, hs], lse[b, hs] = p @ v, torch.logsumexp(sc, -1)
            delta = 2.0 ** -11 * span + 2.0 ** -19 * (1 + sc.abs().amax(-1))
            expo = delta + 2.0 ** -19 * vs.log2().abs().max()
            tol[b, hs] = U["bf16"] * out[b, hs].abs() + (p @ v.abs()) * (torch.expm1(2 * expo) + 2.0 ** -10)[:, None] \
                + len(row) * 2.0 ** -32 * 448 * (p * vs).amax(-1, keepdim=True) + 2.0 ** -133
            lse_tol[b, hs] = delta + 2.0 ** -22 * (1 + sc.abs().amax(-1))
    return out, lse, tol, lse_tol


# value scales (exponents of two) of a sequence's blocks in turn, zeros in the blocks of the least of them
MIXED = [[-100, 40], [40, -100], [-100, -100, 119], [119, -100, -100], [0, -100, 40, -60, 90], [-100, 30, 30, 30],
         [-20, 0, 20]]


@pytest.mark.parametrize("exps", MIXED)
@pytest.mark.parametrize("Hq,Hkv,lens,slack", [
    (4, 1, [128, 74, 640], 1),       # a cluster per pair; a stage of 10 rows in one warp alone
    (24, 2, [128, 74, 640], 1),      # two tiles of heads
    (8, 1, [3000, 128, 74], 1),      # blocks of both kinds in every CTA of a cluster, and CTAs of one kind
    (2, 1, [20000, 700], 1),         # runs, joined by head
    (16, 8, [20000, 128, 700], 1),   # runs, joined by run
    (4, 1, [128, 74], 3000),         # runs for short sequences under a wide table
])
def test_decode_e4m3_value_scales_far_apart(exps, Hq, Hkv, lens, slack):
    """A block counts in the denominator whatever its value scale is next to the others'."""
    s = attention_state("e4m3", 64, Hq, Hkv, lens, 131)
    s["table"] = torch.cat([s["table"], torch.full((len(lens), slack), -1, dtype=torch.int32)], 1)
    for b, n in enumerate(lens):
        for j in range(-(-n // 64)):
            e = exps[j % len(exps)]
            pg = int(s["table"][b, j])
            s["scales"][1][pg] = 2.0 ** e
            if e == -100:
                s["vp"][pg, :, :max(0, min(64, n - 64 * j))] = 0
    s["vv"] = R.codes(s["vp"]) * s["scales"][1].double()[:, :, None, None]
    d = on_gpu(s)
    lse = torch.empty(len(lens), Hq, device="cuda")
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"], lse=lse)
    o, l, tol, lse_tol = mixed_reference(s, lens)
    assert torch.all((lse.double().cpu() - l).abs() <= lse_tol)
    assert torch.all((out.double().cpu() - o).abs() <= tol)
    ids = torch.full((len(lens), Hkv, 6), -1, dtype=torch.int32)
    for b, n in enumerate(lens):  # a few blocks of both kinds
        some = sorted({j * (-(-n // 64) - 1) // 5 for j in range(6)})
        ids[b, :, :len(some)] = torch.tensor(some)
    out = la.llama_attn_decode_paged_sparse_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], ids.cuda(), d["lens"],
                                                 lse=lse)
    o, l, tol, lse_tol = mixed_reference(s, lens, ids)
    assert torch.all((lse.double().cpu() - l).abs() <= lse_tol)
    assert torch.all((out.double().cpu() - o).abs() <= tol)


@pytest.mark.parametrize("order", [0, 1])
def test_decode_e4m3_greatest_score_and_greatest_value_scale_in_different_blocks(order):
    """One block has the scores (they pass the others' by more than 2^130), the other the values: the softmax is the
    first one's, and the second's values still count by what is left of their weights."""
    lens = [128]
    s = attention_state("e4m3", 64, 4, 2, lens, 137)
    big, scored = (int(x) for x in (s["table"][0, :2] if order else s["table"][0, :2].flip(0)))
    s["scales"][1][big], s["scales"][1][scored] = 2.0 ** 119, 2.0 ** -100
    s["scales"][0][big], s["scales"][0][scored] = 2.0 ** -20, 2.0
    s["kv"] = R.codes(s["kp"]) * s["scales"][0].double()[:, :, None, None]
    s["vv"] = R.codes(s["vp"]) * s["scales"][1].double()[:, :, None, None]
    d = on_gpu(s)
    lse = torch.empty(1, 4, device="cuda")
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"], lse=lse)
    o, l, tol, lse_tol = mixed_reference(s, lens)
    assert l.min() > 100  # far above the other block's scores, which are near 0
    assert torch.all((lse.double().cpu() - l).abs() <= lse_tol)
    assert torch.all((out.double().cpu() - o).abs() <= tol)


@pytest.mark.parametrize("q_scale,bound_scale", [(1e-25, 1e-19), (1e-22, 1e-22), (1e-38, 1.0), (1e-40, 1e30), (1.0, 3e-40),
                                                 (1e30, 1e-38), (1e-20, 1e-28)])
def test_select_below_the_normal_range_of_float32(q_scale, bound_scale):
    """Scores, weights or bounds that float32 holds with few bits or none: the order is still float64's."""
    Hq, Hkv, page, nb, B, n_sel = 8, 2, 64, 400, 6, 60
    g = gen(15)
    q = (torch.randn(B, Hq, D, generator=g) * q_scale).to(torch.bfloat16)
    bounds = torch.randn(1, Hkv, 2, D, generator=g).sort(dim=2).values * torch.ones(nb * B, 1, 1, 1)
    bounds[:, :, :, :8] *= 1 + torch.rand(nb * B, Hkv, 2, 8, generator=g) * 2.0 ** -6  # scores near one another
    bounds = (bounds * bound_scale).to(torch.bfloat16)
    table = torch.randperm(nb * B, generator=g).to(torch.int32).view(B, nb)
    lens = [nb * page - b for b in range(B)]
    ids = la.llama_attn_select_blocks(q.cuda(), bounds.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                      page, n_sel)
    assert torch.equal(ids.cpu(), R.select(q, bounds, table, lens, page, n_sel, 1, 1, THETA))


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("Hq,lens", [(4, [200, 64]), (20, [200, 64]), (4, [20000, 300])])
def test_a_scale_that_is_nan_shows_in_its_heads(which, Hq, lens):
    """A page whose scale was never written must not read as zeros: NaN in the heads that use it, nothing elsewhere."""
    s = attention_state("e4m3", 64, Hq, 2, lens, 61)
    d = on_gpu(s)
    want = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"])
    d["scales"][which][int(s["table"][0, (lens[0] - 1) // 64]), 1] = math.nan  # the last page of sequence 0, KV head 1
    lse = torch.empty(2, Hq, device="cuda")
    out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"], lse=lse)
    assert torch.isnan(out[0, Hq // 2:]).all() and torch.isnan(lse[0, Hq // 2:]).all()
    assert torch.equal(out[0, :Hq // 2], want[0, :Hq // 2]) and torch.equal(out[1], want[1])


def test_rope_bases_in_turn_and_from_two_threads():
    """The frequencies follow the base of the call, whatever the call before had, on each host thread."""
    page, Hq, Hkv, lens = 64, 8, 2, [700, 130]
    s = attention_state("e4m3", page, Hq, Hkv, lens, 67)
    d = on_gpu(s)
    bounds = bounds_of(s)
    bases = [10000.0, 500000.0, 1000000.0]
    want_ids = [R.select(s["q"], bounds, s["table"], lens, page, 5, 1, 1, base) for base in bases]
    want = [R.decode(s["q"], s["kv"], s["vv"], s["table"], lens, page, base) for base in bases]
    kb = bounds.cuda()

    def turn(order, results):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for i in order:
                ids = la.llama_attn_select_blocks(d["q"], kb, d["table"], d["lens"], page, 5, rope_theta=bases[i])
                out = la.llama_attn_decode_paged_e4m3(d["q"], *d["pools"], *d["scales"], d["table"], d["lens"],
                                                      rope_theta=bases[i])
                results.append((i, ids, out))
        stream.synchronize()
    torch.cuda.synchronize()
    results = [], []
    threads = [threading.Thread(target=turn, args=([0, 1, 2, 1, 0, 2] * 3, results[0])),
               threading.Thread(target=turn, args=([2, 0, 0, 1, 2, 1] * 3, results[1]))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [len(r) for r in results] == [18, 18]
    for i, ids, out in results[0] + results[1]:
        assert torch.equal(ids.cpu(), want_ids[i])
        check_attention("e4m3", out, None, want[i], 7.0, 700)
    # the append takes its angles from the caller's table
    for base in bases:
        st = append_state("bf16", page, Hkv, 5, [60, 0], None, 68)
        rope = la.llama_attn_rope_table_build(st["table"].shape[1] * page, D, base)
        got = run_append("bf16", st, [60, 0], rope, st["k"].cuda(), st["v"].cuda(), None)
        ref = [p.double().clone() for p in st["pools"]]
        R.append(st["k"], st["v"], ref, None, None, st["table"], [60, 0], st["new"], page, base)
        # one bf16 rounding and 4 u32 (|x0| + |x1|), of values below 3 * 6
        assert torch.all((got["pools"][0].cpu().double() - ref[0]).abs() <= U["bf16"] * ref[0].abs() + 4 * U["f32"] * 36)


@pytest.mark.parametrize("Hq,Hkv,lens,n_sel", [(8, 2, [1000, 64, 3000], 7), (24, 2, [1000, 64, 3000], 7),
                                               (16, 8, [777, 2049, 640] * 16, 7)])
def test_sparse_bf16_weights_carry_16_bits(Hq, Hkv, lens, n_sel):
    """Over bf16 pages a softmax weight is the sum of two bf16 terms (2^-16), as the query is: beyond the output's own
    rounding the error is far below that of one term (2^-8)."""
    s = attention_state("bf16", 64, Hq, Hkv, lens, 141)
    d = on_gpu(s)
    bounds = bounds_of(s)
    ids = la.llama_attn_select_blocks(d["q"], bounds.cuda(), d["table"], d["lens"], 64, n_sel)
    out = la.llama_attn_decode_paged_sparse(d["q"], *d["pools"], d["table"], ids, d["lens"])
    o, lse, mass, span = R.decode(s["q"], s["kv"], s["vv"], s["table"], lens, 64, THETA, 0, ids.cpu())
    delta = 2.0 ** -16 * span + 2.0 ** -19 * (1 + lse.abs() + span)
    # 2^-16 of the weights; 2^-16 more for float32 sums of up to 448 rows in 16-row products (28 roundings of 2^-24)
    # and the exponential's own 2^-22
    tol = U["bf16"] * o.abs() + mass * (torch.expm1(2 * delta) + 2.0 ** -15)[..., None]
    assert torch.all((out.double().cpu() - o).abs() <= tol)


@pytest.mark.parametrize("Hq,Hkv,slack", [
    (8, 2, 0),      # clusters
    (24, 2, 0),     # clusters, two tiles of heads
    (2, 1, 3000),   # runs, joined by head
    (16, 8, 3000),  # runs, joined by run
    (12, 1, 3000),  # runs, two tiles of heads
])
def test_captured_e4m3_decodes_replay_with_new_lengths_on_two_streams(Hq, Hkv, slack):
    """Every form of the decode in a CUDA graph: two graphs with a workspace each, replayed at the same time, take
    lengths, scales and chosen blocks as they are then."""
    page, lens = 64, [900, 64, 300, 1]
    s = attention_state("e4m3", page, Hq, Hkv, lens, 151)
    for b, n in enumerate(lens):  # all rows valid: shorter lengths later leave live rows behind the end
        for j in range(-(-n // page)):
            s["kp"][int(s["table"][b, j])] &= 0x77
            s["vp"][int(s["table"][b, j])] &= 0x77
    s["table"] = torch.cat([s["table"], torch.full((4, slack), -1, dtype=torch.int32)], 1)
    s["kv"] = R.codes(s["kp"]) * s["scales"][0].double()[:, :, None, None]
    d = on_gpu(s)
    sides = []
    for i in range(2):
        stream, lens_d = torch.cuda.Stream(), d["lens"].clone()
        vs = (d["scales"][1] * (i + 1)).contiguous()
        ids = torch.full((4, Hkv, 3), -1, dtype=torch.int32, device="cuda")
        outs = [torch.empty_like(d["q"]) for _ in range(2)]
        ws = torch.empty(la.llama_attn_decode_runs_workspace_size(4, Hq, Hkv), dtype=torch.uint8, device="cuda")
        bounds = bounds_of(s).cuda()

        def step(outs=outs, lens_d=lens_d, vs=vs, ids=ids, ws=ws, bounds=bounds):
            pool = (*d["pools"], d["scales"][0], vs, d["table"])
            la.llama_attn_decode_paged_e4m3(d["q"], *pool, lens_d, out=outs[0], workspace=ws)
            la.llama_attn_select_blocks(d["q"], bounds, d["table"], lens_d, page, 3, block_ids=ids)
            la.llama_attn_decode_paged_sparse_e4m3(d["q"], *pool, ids, lens_d, out=outs[1], workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        sides.append((graph, stream, lens_d, vs, ids, outs, step))
    for now in ([900, 64, 300, 1], [0, 1, 299, 0], [65, 0, 1, 1], [900, 63, 0, 1]):
        for graph, stream, lens_d, *_ in sides:
            lens_d.copy_(torch.tensor(now, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(20):
            for graph, stream, *_ in sides:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for i, (_, _, lens_d, vs, ids, outs, step) in enumerate(sides):
            got = [x.clone() for x in outs] + [ids.clone()]
            vv = R.codes(s["vp"]) * vs.cpu().double()[:, :, None, None]
            for out, chosen in ((got[0], None), (got[1], got[2].cpu())):
                ref = R.decode(s["q"], s["kv"], vv, s["table"], now, page, THETA, 0, chosen)
                check_attention("e4m3", out, None, ref, 2 * 7.0, 900)
            step()  # the same calls outside a graph: the same bits
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, outs + [ids]))
