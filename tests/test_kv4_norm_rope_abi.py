"""Refusals of the norm-with-rotation and 4-bit cache entry points (no GPU):
every bad argument is turned down before anything touches CUDA."""
import ctypes

import pytest
import torch

import exact_attention_134_b200 as attn
from exact_attention_134_b200 import build as attn_build

P = 0x10000  # a fake, 16-byte-aligned "device pointer": never dereferenced on these paths
LL, INT = ctypes.c_longlong, ctypes.c_int


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.lib()


def _rope(lib, bwd=False, t=None, strides=None, wq=P, wk=P, bf16=0, pos=P, pa=0, pb=0, freq=P, sec=(64,), axes=None,
          rot=128, inter=0, B=2, N=100, Hq=4, Hkv=2, d=128, eps=1e-6, dwq=P, dwk=P, ws=P, nbytes=None):
    n = 6 if bwd else 4
    t = [P + 0x1000 * i for i in range(n)] if t is None else t
    strides = [512, 128, 512] * n if strides is None else strides
    s = (LL * len(strides))(*strides) if strides else None
    sec_ = (INT * max(len(sec), 1))(*sec) if sec is not None else None
    axes = len(sec) if axes is None else axes
    tail = [pos, pa, pb, freq, sec_, axes, rot, inter, B, N, Hq, Hkv, d, eps]
    if not bwd:
        return lib.attn_qk_norm_rope(*t, s, wq, wk, bf16, *tail, None)
    if nbytes is None:
        nbytes = lib.attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d)
    return lib.attn_qk_norm_rope_bwd(*t, s, wq, wk, bf16, dwq, dwk, *tail, ws, nbytes, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(Hq=0), 1), (dict(Hkv=-1), 1), (dict(d=0), 1), (dict(strides=[]), 1),
    (dict(wq=None), 1), (dict(wk=None), 1), (dict(bf16=2), 1), (dict(inter=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(d=80), 2), (dict(d=512), 2), (dict(rot=-16), 1), (dict(rot=144), 1),
    (dict(rot=8, sec=(4,)), 1), (dict(pos=None), 1), (dict(freq=None), 1), (dict(sec=None, axes=1), 1),
    (dict(pa=-1), 1), (dict(pb=-1), 1), (dict(axes=0), 1), (dict(sec=(16, 16, 16, 8, 8)), 1), (dict(sec=(63,)), 1),
    (dict(sec=(70, -6)), 1), (dict(Hq=70000), 2), (dict(B=1 << 16, N=1 << 15), 2), (dict(pos=P + 2), 3), (dict(freq=P + 1), 3), (dict(wq=P + 2), 3),
    (dict(wk=P + 1, bf16=1), 3),
])
def test_norm_rope_validation(lib, bwd, kw, code):
    assert _rope(lib, bwd, **kw) == code


def test_norm_rope_in_place_needs_the_same_strides(lib):
    """A result may be the tensor it is made of, with its strides only."""
    for bwd, x, y in ((False, 0, 2), (False, 1, 3), (True, 2, 4), (True, 3, 5)):
        n = 6 if bwd else 4
        t = [P + 0x1000 * i for i in range(n)]
        t[y] = t[x]
        s = [512, 128, 512] * n
        s[3 * y + 1] = 256
        assert _rope(lib, bwd, t=t, strides=s) == 1


def test_calls_are_made_on_the_tensors_device(monkeypatch):
    """With another device current, a call switches to the tensors' one and back."""
    seen, at = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            at[0] = self.index

        def __exit__(self, *exc):
            at[0] = 0

    class Lib:
        @staticmethod
        def entry(*args):
            seen.append((at[0], args))
            return 1 if args[0] == "bad" else 0

    monkeypatch.setattr(attn, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    attn._call("entry", 0, 7)
    attn._call("entry", 3, 8)
    assert seen == [(0, (7, 100)), (3, (8, 103))] and at[0] == 0
    with pytest.raises(attn.AttnError):
        attn._call("entry", 2, "bad")
    assert at[0] == 0


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_rope_tensor_validation(lib, bwd):
    n = 6 if bwd else 4
    for i in range(n):
        t = [P + 0x1000 * i for i in range(n)]
        t[i] = None
        assert _rope(lib, bwd, t=t) == 1
        t[i] = P + 8
        assert _rope(lib, bwd, t=t) == 3
    for i in range(3 * n):
        s = [512, 128, 512] * n
        s[i] = -8
        assert _rope(lib, bwd, strides=s) == 1
        s[i] = 12
        assert _rope(lib, bwd, strides=s) == 3


def test_norm_rope_workspace(lib):
    need = lib.attn_qk_norm_rope_bwd_workspace_size(2, 100, 4, 2, 128)
    assert need >= 2 * 128 * 4 and need % 256 == 0
    assert lib.attn_qk_norm_rope_bwd_workspace_size(2, 100, 4, 2, 80) == 0
    assert lib.attn_qk_norm_rope_bwd_workspace_size(0, 100, 4, 2, 128) == 0
    assert _rope(lib, True, ws=None) == 6 and _rope(lib, True, ws=P + 8) == 6 and _rope(lib, True, nbytes=need - 1) == 6
    assert _rope(lib, True, dwq=None) == 1 and _rope(lib, True, dwk=None) == 1 and _rope(lib, True, dwk=P + 2) == 3


def _append(lib, k=P, v=P, ts=1024, hs=128, vts=1024, vhs=128, pool=P, table=P, lens=P, cu=P, n=3, mp=8, np_=50,
            page=64, total=100, Hkv=8, d=128):
    return lib.attn_kv4_append(k, v, ts, hs, vts, vhs, pool, table, lens, cu, n, mp, np_, page, total, Hkv, d, None)


def _gather(lib, k=P, v=P, pool=P, table=P, lens=P, cu=P, n=3, mp=8, np_=50, page=64, total=100, Hkv=8, d=128):
    return lib.attn_kv4_gather(pool, table, lens, cu, n, mp, np_, page, total, Hkv, d, k, v, None)


def _fwd(lib, q=P, o=P, lse=P, pool=P, table=P, lens=P, cu=P, n=3, mp=8, np_=50, page=64, mq=64, total=100, Hq=16,
         Hkv=8, d=128, causal=1, scale=0.1, ws=P, nbytes=1 << 40):
    return lib.attn_fwd_kv4(q, pool, table, lens, cu, o, lse, n, mp, np_, page, mq, total, Hq, Hkv, d, causal, scale,
                            ws, nbytes, None)


@pytest.mark.parametrize("call", [_append, _gather, _fwd])
@pytest.mark.parametrize("kw,code", [
    (dict(pool=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(n=0), 1), (dict(mp=0), 1),
    (dict(np_=0), 1), (dict(page=0), 1), (dict(page=-16), 1), (dict(total=0), 1), (dict(Hkv=0), 1), (dict(d=0), 1),
    (dict(cu=None), 1),                         # 100 rows of 3 sequences
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=2048), 2), (dict(d=80), 2), (dict(d=32), 2), (dict(n=70000), 2),
    (dict(mp=1 << 25), 2),                      # 2^31 tokens
    (dict(pool=P + 8), 3), (dict(table=P + 2), 3), (dict(lens=P + 1), 3), (dict(cu=P + 2), 3),
])
def test_cache_validation(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_append_and_gather_validation(lib):
    assert _append(lib, k=None) == 1 and _append(lib, v=None) == 1 and _append(lib, ts=-8) == 1 and _append(lib, vhs=-8) == 1
    assert _append(lib, hs=4) == 3 and _append(lib, vts=2) == 3 and _append(lib, k=P + 8) == 3 and _append(lib, v=P + 2) == 3
    assert _gather(lib, k=None) == 1 and _gather(lib, v=None) == 1 and _gather(lib, k=P + 8) == 3
    assert lib.attn_kv4_page_bytes(8, 128, 64) == 8 * 4 * 20 * 128
    for args in ((0, 128, 64), (8, 80, 64), (8, 128, 8), (8, 128, 40), (8, 128, 2048)):
        assert lib.attn_kv4_page_bytes(*args) == 0


def test_fwd_kv4_validation(lib):
    assert _fwd(lib, q=None) == 1 and _fwd(lib, o=None) == 1 and _fwd(lib, lse=None) == 1 and _fwd(lib, Hq=12) == 1
    assert _fwd(lib, mq=0) == 1 and _fwd(lib, causal=2) == 1 and _fwd(lib, scale=0.0) == 1
    assert _fwd(lib, scale=float("inf")) == 1 and _fwd(lib, scale=float("nan")) == 1
    assert _fwd(lib, Hq=80000, Hkv=8) == 2 and _fwd(lib, total=1 << 30, Hq=1600) == 2
    assert _fwd(lib, q=P + 8) == 3 and _fwd(lib, o=P + 8) == 3 and _fwd(lib, lse=P + 4) == 3
    for d in (64, 96, 128, 256):
        for mq in (1, 8, 64):
            need = lib.attn_fwd_kv4_workspace_size(16, 8, mq, d)
            assert 0 < need < 16 << 20 and need % 256 == 0
            kw = dict(d=d, mq=mq, mp=9)  # 576 tokens: partial results are possible
            assert _fwd(lib, ws=P + 8, nbytes=need, d=d, mq=mq) == 6  # one that is given is checked
            assert _fwd(lib, ws=None, **kw) == 6 and _fwd(lib, ws=P + 8, **kw) == 6 and _fwd(lib, nbytes=need - 1, **kw) == 6
    assert lib.attn_fwd_kv4_workspace_size(12, 8, 1, 128) == 0 and lib.attn_fwd_kv4_workspace_size(16, 8, 0, 128) == 0
    assert lib.attn_fwd_kv4_workspace_size(16, 8, 1, 80) == 0


def test_copy_pages_validation(lib):
    def call(pool=P, layers=2, pages=50, nbytes=163840, src=P, dst=P, n=7):
        return lib.attn_kv4_copy_pages(pool, layers, pages, nbytes, src, dst, n, None)
    assert call(pool=None) == 1 and call(src=None) == 1 and call(dst=None) == 1
    assert call(layers=0) == 1 and call(pages=0) == 1 and call(nbytes=0) == 1 and call(n=0) == 1
    assert call(nbytes=24) == 3 and call(pool=P + 8) == 3 and call(src=P + 2) == 3 and call(dst=P + 1) == 3
    assert call(layers=70000) == 2 and call(nbytes=1 << 45, n=1 << 30) == 2


def test_bindings_need_cuda_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros((4, 2, 1, 20 * 64), dtype=torch.uint8)
    for call in (lambda: attn.qk_norm_rope(x, x), lambda: attn.norm_rope(x, x), lambda: attn.qk_norm_rope_bwd(x, x, x, x),
                 lambda: attn.kv4_append(x, x, pool, i[:, None], i), lambda: attn.kv4_gather(pool, i[:, None], i, 4),
                 lambda: attn.kv4_copy_pages(pool, i, i), lambda: attn.attn_fwd_kv4(x, pool, i[:, None], i)):
        with pytest.raises(ValueError):
            call()
    for args in ((4, 2, 80, 16), (4, 2, 64, 24), (4, 0, 64, 16)):
        with pytest.raises(ValueError):
            attn.kv4_alloc(*args, device="cpu")
    assert attn.kv4_alloc(4, 2, 64, 32, device="cpu").shape == (4, 2, 2, 1280)
    assert attn.kv4_alloc(4, 2, 64, 32, num_layers=3, device="cpu").shape == (3, 4, 2, 2, 1280)
