"""CPU tests of the paged-cache entry points: every bad argument is refused on
the host before anything is launched (this host has no GPU, so a CUDA call
would return LLAMA_ATTN_ERR_CUDA instead), the binding's own checks, and the
float64 statements the GPU tests compare with."""
import ctypes
import math
import types

import pytest
import torch

import gqa_attention_rope_b200 as la
import paged_reference as R
from gqa_attention_rope_b200 import build as labuild

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = ctypes.c_void_p(4096 * 16)   # never dereferenced
P2 = ctypes.c_void_p(4096 * 4096 * 16)
ODD = ctypes.c_void_p(4096 * 16 + 8)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def args(order, base, kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return [a[n] for n in order]


APPEND = dict(k=P, v=P, row=256, batch=2560, kp=P, vp=P, ks=P, vs=P, kb=None, table=P, lens=P, new=None, out_lens=None,
              B=2, T=10, Hkv=2, D=128, page=64, blocks=4, pages=9, rope=P, rows=256)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(rope=None), INVALID),
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(T=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(blocks=0), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
    (dict(D=64), UNSUPPORTED), (dict(page=96), UNSUPPORTED), (dict(page=32), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(Hkv=65536, row=65536 * 128), UNSUPPORTED),
    (dict(row=255), INVALID), (dict(row=260), INVALID), (dict(batch=2561), INVALID), (dict(batch=-8), INVALID),
    (dict(row=1 << 32), UNSUPPORTED),
    (dict(rows=255), INVALID),
    (dict(k=ODD), INVALID), (dict(vp=ODD), INVALID), (dict(rope=ODD), INVALID), (dict(kb=ODD), INVALID),
    (dict(out_lens=P), INVALID), (dict(lens=P, out_lens=ctypes.c_void_p(4096 * 16 + 4)), INVALID),
    (dict(blocks=1 << 25, rows=(1 << 31) - 1), UNSUPPORTED),
    (dict(pages=1 << 24), UNSUPPORTED), (dict(pages=1 << 30, Hkv=2), UNSUPPORTED),
])
def test_append_refuses(lib, kw, expect):
    order = [n for n in APPEND if n not in ("ks", "vs")]
    if not set(kw) & {"ks", "vs"}:
        assert lib.llama_attn_kv_append_paged(*args(order, APPEND, kw), None) == expect
    assert lib.llama_attn_kv_append_paged_e4m3(*args(list(APPEND), APPEND, kw), None) == expect


@pytest.mark.parametrize("off", [0, 4, -4])
def test_append_refuses_new_lengths_that_it_would_overwrite(lib, off):
    """out_lens is written by one CTA of a sequence while others still read new_lens."""
    kw = dict(new=P2, out_lens=ctypes.c_void_p(P2.value + off))
    order = [n for n in APPEND if n not in ("ks", "vs")]
    assert lib.llama_attn_kv_append_paged(*args(order, APPEND, kw), None) == INVALID
    assert lib.llama_attn_kv_append_paged_e4m3(*args(list(APPEND), APPEND, kw), None) == INVALID


def test_append_e4m3_needs_scales(lib):
    for kw in (dict(ks=None), dict(vs=None)):
        assert lib.llama_attn_kv_append_paged_e4m3(*args(list(APPEND), APPEND, kw), None) == INVALID


DECODE = dict(q=P, kp=P, vp=P, ks=P, vs=P, table=P, ids=P, lens=P, out=P2, lse=None, B=2, Hq=8, Hkv=2, D=128, page=64,
              blocks=4, pages=9, n_sel=3, off=0, theta=5e5, ws=P2, ws_bytes=BIG)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(B=0), INVALID), (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=34), UNSUPPORTED),
    (dict(D=64), UNSUPPORTED), (dict(page=65), UNSUPPORTED), (dict(page=0), INVALID), (dict(blocks=0), INVALID),
    (dict(pages=0), INVALID), (dict(theta=0.0), INVALID), (dict(theta=math.inf), INVALID),
    (dict(theta=math.nan), INVALID), (dict(off=1), INVALID), (dict(off=-2), INVALID),
    (dict(q=ODD), INVALID), (dict(out=ODD), INVALID), (dict(kp=ODD), INVALID),
    (dict(out=P), INVALID), (dict(out=ctypes.c_void_p(4096 * 16 + 256)), INVALID),
    (dict(lse=ctypes.c_void_p(4098)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=ctypes.c_void_p(4096 * 4096 * 16 + 128)), WORKSPACE),
    (dict(ws_bytes=1000), WORKSPACE),
    (dict(B=65536), UNSUPPORTED), (dict(blocks=1 << 25), UNSUPPORTED), (dict(pages=1 << 24), UNSUPPORTED),
])
def test_decode_refuses(lib, kw, expect):
    for fn, without in ((lib.llama_attn_decode_paged_e4m3, ("ids", "n_sel")),
                        (lib.llama_attn_decode_paged_sparse, ("ks", "vs")),
                        (lib.llama_attn_decode_paged_sparse_e4m3, ())):
        assert fn(*args([n for n in DECODE if n not in without], DECODE, kw), None) == expect


def test_decode_refuses_missing_scales_and_ids(lib):
    e4m3 = [n for n in DECODE if n not in ("ids", "n_sel")]
    for kw in (dict(ks=None), dict(vs=None)):
        assert lib.llama_attn_decode_paged_e4m3(*args(e4m3, DECODE, kw), None) == INVALID
        assert lib.llama_attn_decode_paged_sparse_e4m3(*args(list(DECODE), DECODE, kw), None) == INVALID
    bf16 = [n for n in DECODE if n not in ("ks", "vs")]
    for kw in (dict(ids=None), dict(n_sel=0), dict(n_sel=-1)):
        assert lib.llama_attn_decode_paged_sparse(*args(bf16, DECODE, kw), None) == INVALID
        assert lib.llama_attn_decode_paged_sparse_e4m3(*args(list(DECODE), DECODE, kw), None) == INVALID


SELECT = dict(q=P, kb=P, table=P, lens=P, ids=P, B=2, Hq=8, Hkv=2, D=128, page=64, blocks=4, pages=9, n_sel=3,
              n_first=1, n_last=1, off=0, theta=5e5)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(kb=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(ids=None), INVALID), (dict(n_sel=0), INVALID), (dict(n_first=-1), INVALID), (dict(n_last=-1), INVALID),
    (dict(n_first=2, n_last=2), INVALID), (dict(n_first=(1 << 31) - 1, n_last=(1 << 31) - 1), INVALID),
    (dict(Hq=7), INVALID), (dict(Hq=0), INVALID), (dict(off=2), INVALID), (dict(theta=-1.0), INVALID),
    (dict(D=32), UNSUPPORTED), (dict(page=63), UNSUPPORTED), (dict(blocks=24577), UNSUPPORTED),
    (dict(Hq=65536), UNSUPPORTED), (dict(kb=ODD), INVALID), (dict(ids=ctypes.c_void_p(4098)), INVALID),
])
def test_select_refuses(lib, kw, expect):
    assert lib.llama_attn_select_blocks(*args(list(SELECT), SELECT, kw), None) == expect


def test_runs_workspace_size(lib):
    f = lib.llama_attn_decode_runs_workspace_size
    assert f(0, 8, 2, 128) == 0 and f(1, 8, 3, 128) == 0 and f(1, 8, 2, 64) == 0 and f(1, 34, 2, 128) == 0
    n = f(64, 64, 8, 128)
    assert n % 256 == 0 and n >= 65 * 8 + 2 * 512 * 8 * (8 + 512)
    assert f(1, 16, 1, 128) < 10 << 20  # whatever the lengths


def test_binding_refuses_before_the_library(lib):
    x = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.llama_attn_kv_append_paged(x, x, x, x, lens[None], lens, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.llama_attn_kv_append_paged_e4m3(x, x, x, x, x, x, lens[None], lens, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.llama_attn_decode_paged_sparse(x[0], x, x, lens[None], lens[None, None], lens)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.llama_attn_decode_paged_e4m3(x[0], x, x, x, x, lens[None], lens, out=x[0], workspace=x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.llama_attn_select_blocks(x[0], x, lens[None], lens, 64, 4)
    with pytest.raises(ValueError, match="k: tensor expected"):
        la.llama_attn_kv_append_paged(None, x, x, x, lens[None], lens, x)
    with pytest.raises(ValueError, match="too few arguments"):
        la._native().append(la._entry["llama_attn_kv_append_paged"], 0, x)


def test_binding_fails_loudly_when_it_is_not_built(lib, monkeypatch, tmp_path):
    la.lib()
    monkeypatch.setattr(la, "_module", None)
    monkeypatch.setattr(la, "_PKG", str(tmp_path))
    with pytest.raises(RuntimeError, match="_binding.so not found"):
        la._native()


def fake_cuda_call():
    """Arguments that pass every check of the binding on a host without a GPU: tensors that say they are on cuda:0,
    and a stream object. Nothing of them is ever read."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    with FakeTensorMode():
        def e(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device="cuda:0")
        table, lens = e(2, 2, dtype=i32), e(2, dtype=i32)
        stream = types.SimpleNamespace(device_index=0, cuda_stream=0)
        scales = dict(k_scales=e(5, 2, dtype=f32), v_scales=e(5, 2, dtype=f32))
        bf16 = dict(kpages=e(5, 2, 64, 128), vpages=e(5, 2, 64, 128))
        e4m3 = dict(kpages=e(5, 2, 64, 128, dtype=u8), vpages=e(5, 2, 64, 128, dtype=u8), **scales)
        both = dict(block_table=table, cache_lens=lens, stream=stream)
        append = dict(k=e(2, 3, 2, 128), v=e(2, 3, 2, 128), rope_table=e(128, 64, 2, dtype=f32),
                      out_lens=e(2, dtype=i32), **both)
        decode = dict(q=e(2, 4, 128), out=e(2, 4, 128), workspace=e(1 << 20, dtype=u8), **both)
        sparse = dict(decode, block_ids=e(2, 2, 3, dtype=i32))
        select = dict(q=e(2, 4, 128), kbounds=e(5, 2, 2, 128), block_ids=e(2, 2, 3, dtype=i32), page_size=64, n_sel=3,
                      **both)
    return [(la.llama_attn_kv_append_paged, dict(append, **bf16)),
            (la.llama_attn_kv_append_paged_e4m3, dict(append, **e4m3)),
            (la.llama_attn_decode_paged_e4m3, dict(decode, **e4m3)),
            (la.llama_attn_decode_paged_sparse, dict(sparse, **bf16)),
            (la.llama_attn_decode_paged_sparse_e4m3, dict(sparse, **e4m3)),
            (la.llama_attn_select_blocks, select)]


@pytest.mark.parametrize("i", range(6))
def test_binding_refuses_tensors_without_storage(lib, i):
    """A tensor of a function transform has no data: refused where the pointers are formed, before
    the device is switched and the interpreter's lock is given up."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    call, args = fake_cuda_call()[i]
    for name in ("k", "q", "block_table", "cache_lens"):
        if name not in args:
            continue
        with FakeTensorMode():
            many = torch.empty(3, *args[name].shape, dtype=args[name].dtype, device="cuda:0")

        def one(x):
            with pytest.raises(ValueError, match="storage"):
                call(**{**args, name: x})
            return x
        torch.func.vmap(one)(many)


@pytest.mark.parametrize("i", range(6))
def test_binding_refuses_none_for_every_tensor_it_needs(lib, i):
    """None is refused by name, not taken for an optional tensor or another call's arguments."""
    call, args = fake_cuda_call()[i]
    needed = [n for n, x in args.items() if isinstance(x, torch.Tensor) and n not in ("out_lens", "out", "workspace")]
    if call is la.llama_attn_select_blocks:
        needed.remove("block_ids")  # made by the call
    assert {"block_table", "cache_lens"} < set(needed)
    for name in needed:
        with pytest.raises(ValueError, match=f"{name}: tensor expected"):
            call(**{**args, name: None})


# ---- the statements the GPU tests rely on
def test_reference_grid_is_the_formats():
    from oracle import fp8 as F
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1), dtype=torch.float64) * 200
    x[:64] = torch.arange(64) * 2.0 ** -11
    got = R.e4m3_grid(x)
    table = torch.from_numpy(F.e4m3_table())
    want = table[torch.from_numpy(F.e4m3_round(x.numpy())).long()]
    assert torch.equal(got, want)


def test_reference_scale_is_least():
    for a in (0.0, 1e-40, 1.0, 447.9, 448.0, 448.0001, 3.3, 896.0, 1e38):
        s = R.block_scale(a)
        assert s == 2.0 ** 119 or a <= 448 * s
        assert s == 2.0 ** -100 or a > 448 * s / 2


def test_reference_selection_bounds_every_key():
    """A block's score is at least the group's summed product with each of its keys."""
    g = torch.Generator().manual_seed(2)
    k = torch.randn(6, 64, 128, generator=g, dtype=torch.float64)
    q = torch.randn(4, 128, generator=g, dtype=torch.float64)
    lo, hi = k.amin(1), k.amax(1)
    score = torch.maximum(q[:, None] * lo, q[:, None] * hi).sum((0, 2))
    both = q.clamp(min=0).sum(0) * hi + q.clamp(max=0).sum(0) * lo
    assert torch.allclose(score, both.sum(-1), rtol=1e-13)
    assert torch.all(score[:, None] >= torch.einsum("hd,jnd->jn", q, k) - 1e-9)


def test_runs_cover_every_unit_once():
    """The cut of the units into runs and its inverse, as the kernels compute them."""
    for total in (1, 2, 5, 100, 296, 297, 1000, 131072):
        for n in (1, 2, 296):
            n = min(n, total)
            at = [total * i // n for i in range(n + 1)]
            assert at[0] == 0 and at[-1] == total and all(a < b for a, b in zip(at, at[1:]))
            for u in {0, total - 1, total // 2, total // 3}:
                i = ((u + 1) * n - 1) // total
                assert at[i] <= u < at[i + 1]
