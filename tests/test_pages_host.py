"""Shared blocks, rotary positions and prompt chunks without a GPU: the oracle's pins and the entry points'
refusals."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from gqa_head_gated_gb300 import _lib

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from gqa_head_gated_gb300 import build
        build.build()
    return _lib.load()


def test_oracle_fork_then_free_is_the_identity():
    tables, n, free, shares, lens = [[4, 2, -1], [-1] * 3, [-1] * 3], [2, 0, 0], [1, 3, 5, 0], [0] * 6, [20, 0, 0]
    copies, v = oracle.block_fork([0, 0], [1, 2], None, lens, tables, n, free, shares, 16)
    assert v == ["ok", "ok"] and copies == [[2, 0, 4], [2, 5, 4]] and free == [1, 3]
    assert tables == [[4, 2, -1], [4, 0, -1], [4, 5, -1]] and shares == [0, 0, 0, 0, 2, 0] and lens == [20, 20, 20]
    oracle.block_free([20, 0, 0], tables, n, free, shares, 16)
    assert free == [1, 3, 5, 0] and shares == [0] * 6 and tables == [[4, 2, -1], [-1] * 3, [-1] * 3] and n == [2, 0, 0]


def test_oracle_free_gives_a_shared_block_back_with_its_last_owner():
    tables, n, free, shares = [[3], [3], [3]], [1, 1, 1], [0], [0, 0, 0, 2]
    oracle.block_free([0, 5, 0], tables, n, free, shares, 16)
    assert free == [0] and shares[3] == 0 and tables == [[-1], [3], [-1]]
    oracle.block_free([0, 0, 0], tables, n, free, shares, 16)
    assert free == [0, 3]


def test_oracle_compact_moves_the_high_blocks_down():
    tables, free, shares, index, copies = oracle.block_compact([[5, 1], [1, -1]], [2, 1], [3, 0, 4, 2], [0, 1, 0, 0, 0, 0],
                                                               6, 32)
    assert copies == [[5, 0, 32], [-1, -1, 0], [-1, -1, 0]] and index == [-1, 1, -1, -1, -1, 0]
    assert tables == [[0, 1], [1, -1]] and shares == [0, 1, 0, 0, 0, 0] and free == [5, 4, 3, 2]


def test_oracle_rope_is_a_complex_product_and_its_angles_are_exact():
    rng = np.random.RandomState(0)
    x, f = rng.randn(4, 2, 256), np.array([1.0, 0.25, 0.01, 1e-4, 0.5, 2.0, 0.125, 0.3])
    y = oracle.rope(x, [0, 3, 7, 11], f, True, 1.5)
    z = (x[..., 0:16:2] + 1j * x[..., 1:16:2]) * 1.5 * np.exp(1j * np.array([0, 3, 7, 11])[:, None] * f)[:, None]
    assert np.allclose(y[..., 0:16:2], z.real) and np.allclose(y[..., 1:16:2], z.imag)
    back = oracle.rope(y, [0, 3, 7, 11], f, True, 1 / 1.5, True)
    assert np.allclose(back, x)
    y = oracle.rope(x, [5] * 4, f)
    assert np.allclose(y[..., 0], x[..., 0] * math.cos(5) - x[..., 8] * math.sin(5))
    # 355 / 113 is pi to 8.5e-8 of itself: 2 * 355 = 113 turns + 6.03e-5
    assert abs(oracle.angle(710, 1.0) - 6.028870e-05) < 1e-10
    assert abs(oracle.angle(-710, 1.0) + oracle.angle(710, 1.0) - 2 * math.pi) < 1e-15


def test_rope_frequencies():
    f, s = G.rope_frequencies(64, 1e4, device="cpu")
    assert s == 1.0 and f.dtype == torch.float32 and f[0] == 1 and abs(f[16].item() - 1e-2) < 1e-9
    g, _ = G.rope_frequencies(64, 1e4, "linear", 4.0, device="cpu")
    assert torch.allclose(g, f / 4)
    g, _ = G.rope_frequencies(64, 1e4, "ntk", 4.0, device="cpu")
    assert g[0] == 1 and abs(g[31].item() * 4 / f[31].item() - 1) < 1e-6     # the lowest as in "linear"
    g, s = G.rope_frequencies(64, 1e4, "yarn", 4.0, original_len=4096, device="cpu")
    assert abs(s - (0.1 * math.log(4) + 1)) < 1e-12
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.allclose(g[turns < 0.8], f[turns < 0.8] / 4)
    assert ((g <= f * 1.0000001) & (g >= f / 4.0000004)).all()
    for bad in (dict(rot_dims=60), dict(rot_dims=272), dict(rot_dims=0), dict(rot_dims=64, method="x"),
                dict(rot_dims=64, base=1.0), dict(rot_dims=64, factor=0.5), dict(rot_dims=64, method="yarn", factor=2.0),
                dict(rot_dims=64, method="yarn", factor=2.0, original_len=64, beta_fast=1, beta_slow=1)):
        with pytest.raises(ValueError):
            G.rope_frequencies(device="cpu", **bad)


def _fork(lib, **kw):
    a = dict(src=16, dst=32, lens=48, kv=64, tab=80, nb=96, fl=112, fc=128, sh=144, cp=160, F=2, B=4, mb=4, N=8, bs=16)
    a.update(kw)
    return lib.gqa_block_fork(*(P(a[k]) for k in ("src", "dst", "lens", "kv", "tab", "nb", "fl", "fc", "sh", "cp")),
                              a["F"], a["B"], a["mb"], a["N"], a["bs"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(F=-1), 1), (dict(B=0), 1), (dict(mb=0), 1), (dict(N=0), 1), (dict(bs=24), 1), (dict(src=None), 1),
    (dict(dst=None), 1), (dict(kv=None), 1), (dict(tab=None), 1), (dict(nb=None), 1), (dict(fl=None), 1),
    (dict(fc=None), 1), (dict(sh=None), 1), (dict(cp=None), 1), (dict(lens=50), 1), (dict(cp=162), 1), (dict(B=8193), 2),
    (dict(F=8193), 2), (dict(N=1 << 28, bs=128), 2), (dict(B=4096, mb=1 << 20), 2), (dict(F=2048, mb=1 << 19), 2),
    (dict(F=0, src=None, cp=None), 0),
])
def test_fork_rejects_before_launch(lib, kw, code):
    assert _fork(lib, **kw) == code


def _free(lib, **kw):
    a = dict(kv=16, tab=32, nb=48, fl=64, fc=80, sh=96, B=4, mb=4, N=8, bs=16)
    a.update(kw)
    return lib.gqa_block_free(*(P(a[k]) for k in ("kv", "tab", "nb", "fl", "fc", "sh")), a["B"], a["mb"], a["N"],
                              a["bs"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(mb=0), 1), (dict(N=0), 1), (dict(bs=0), 1), (dict(kv=None), 1), (dict(tab=None), 1),
    (dict(nb=None), 1), (dict(fl=None), 1), (dict(fc=None), 1), (dict(sh=None), 1), (dict(sh=98), 1), (dict(B=8193), 2),
    (dict(mb=1 << 28), 2),
])
def test_free_rejects_before_launch(lib, kw, code):
    assert _free(lib, **kw) == code


def _compact(lib, **kw):
    a = dict(tab=16, nb=32, fl=48, fc=64, sh=80, to=96, fo=112, so=128, ix=144, cp=160, B=4, mb=4, N=8, bs=16)
    a.update(kw)
    return lib.gqa_block_compact(*(P(a[k]) for k in ("tab", "nb", "fl", "fc", "sh", "to", "fo", "so", "ix", "cp")),
                                 a["B"], a["mb"], a["N"], a["bs"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(mb=0), 1), (dict(N=0), 1), (dict(bs=100), 1), (dict(tab=None), 1), (dict(nb=None), 1),
    (dict(fl=None), 1), (dict(fc=None), 1), (dict(sh=None), 1), (dict(to=None), 1), (dict(fo=None), 1),
    (dict(so=None), 1), (dict(ix=None), 1), (dict(cp=None), 1), (dict(to=16), 1), (dict(fo=48), 1), (dict(so=80), 1),
    (dict(ix=146), 1), (dict(B=8193), 2),
])
def test_compact_rejects_before_launch(lib, kw, code):
    assert _compact(lib, **kw) == code


def _copy(lib, **kw):
    a = dict(cp=16, k=32, v=48, ks=64, vs=80, n=2, Hkv=2, N=8, bs=16)
    a.update(kw)
    return lib.gqa_kv8_copy(*(P(a[k]) for k in ("cp", "k", "v", "ks", "vs")), a["n"], a["Hkv"], a["N"], a["bs"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(Hkv=0), 1), (dict(N=0), 1), (dict(bs=12), 1), (dict(cp=None), 1), (dict(k=None), 1),
    (dict(v=56), 1), (dict(ks=None), 1), (dict(vs=81), 1), (dict(N=1 << 27), 2), (dict(Hkv=1 << 14), 2),
    (dict(n=0, cp=None, k=None), 0),
])
def test_copy_rejects_before_launch(lib, kw, code):
    assert _copy(lib, **kw) == code


def _rope(lib, **kw):
    a = dict(q=16, k=32, p=48, f=64, qo=80, ko=96, B=1, L=3, Hq=4, Hkv=2, rot=64, pb=0, s=None)
    a.update(kw)
    s = a["s"] or [0, 1024, 256] * 2 + [0, 512, 256] * 2
    arr = None if s == "none" else (ctypes.c_longlong * 12)(*s)
    return [f(*(P(a[n]) for n in ("q", "k", "p", "f", "qo", "ko")), arr, a["B"], a["L"], a["Hq"], a["Hkv"], a["rot"],
              a["pb"], 0, 0, 1.0, None) for f in (lib.gqa_rope, lib.gqa_rope_f16)]


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(L=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-1), 1), (dict(rot=8), 1), (dict(rot=24), 1),
    (dict(rot=272), 1), (dict(pb=2), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(Hkv=0), 1),
    (dict(p=None), 1), (dict(f=None), 1), (dict(qo=None), 1), (dict(q=24), 1), (dict(ko=100), 1), (dict(p=50), 1),
    (dict(f=66), 1), (dict(s="none"), 1), (dict(s=[0, 1020, 256] + [0, 1024, 256] + [0, 512, 256] * 2), 1),
    (dict(s=[0, -1024, 256] + [0, 1024, 256] + [0, 512, 256] * 2), 1),
    (dict(s=[0, 1024, 256] + [0, 1024, 128] + [0, 512, 256] * 2), 1),      # rows of the output overlap
    (dict(s=[0, 1024, 256] + [0, 0, 256] + [0, 512, 256] * 2), 1),
    (dict(qo=16, s=[0, 2048, 256] + [0, 1024, 256] + [0, 512, 256] * 2), 1),   # in place, other strides
    (dict(B=1 << 16, L=1 << 15), 2), (dict(Hq=1 << 20), 2), (dict(L=1 << 30, Hq=64), 2),
    (dict(L=0, q=None, p=None), 0), (dict(B=0), 0),
])
def test_rope_rejects_before_launch(lib, kw, code):
    assert _rope(lib, **kw) == [code, code]


def _prefill(lib, **kw):
    a = dict(q=16, kp=32, vp=48, ks=64, vs=80, g=96, tab=112, lens=128, cu=144, out=160, lse=None, B=2, T=3, Hq=8, Hkv=2,
             N=8, bs=16, mb=4, mr=2, mk=64, ws=176, wsb=1 << 30)
    a.update(kw)
    return [f(*(P(a[n]) for n in ("q", "kp", "vp", "ks", "vs", "g", "tab", "lens", "cu", "out", "lse")),
              *(a[n] for n in ("B", "T", "Hq", "Hkv", "N", "bs", "mb", "mr", "mk")), P(a["ws"]), a["wsb"], None)
            for f in (lib.gqa_kv8_prefill, lib.gqa_kv8_prefill_f16)]


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(mr=0), 1), (dict(mk=0), 1),
    (dict(mr=65), 1), (dict(bs=20), 1), (dict(N=0), 1), (dict(mb=0), 1), (dict(mk=65), 1), (dict(q=None), 1),
    (dict(kp=None), 1), (dict(vp=40), 1), (dict(ks=None), 1), (dict(vs=82), 1), (dict(g=100), 1), (dict(tab=None), 1),
    (dict(lens=None), 1), (dict(cu=None), 1), (dict(out=None), 1), (dict(lse=2), 1), (dict(ws=None), 5),
    (dict(wsb=1000), 5), (dict(ws=184), 1), (dict(T=1 << 28, Hq=8), 2), (dict(N=1 << 27), 2),
    (dict(mk=1 << 29, mb=1 << 26, mr=1 << 26), 2), (dict(T=0, q=None, out=None), 0),
])
def test_prefill_rejects_before_launch(lib, kw, code):
    assert _prefill(lib, **kw) == [code, code]


def test_prefill_workspace_does_not_grow(lib):
    n = G.kv8_prefill_workspace_size()
    assert 2 * 256 * 1028 < n < 64 << 20 and n == lib.gqa_kv8_prefill_workspace_size()
