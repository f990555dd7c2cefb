"""The paged 8-bit cache without a GPU: the oracle's pins and the entry points' refusals."""
import ctypes
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


def test_e4m3_table_and_rounding_agree_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.E4M3, ref, equal_nan=True)
    gen = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=gen) * 10.0 ** torch.randint(-4, 3, (20000,), generator=gen),
                   torch.from_numpy((oracle.E4M3[:126] + oracle.E4M3[1:127]) / 2).float(),
                   torch.tensor([0.0, -0.0, 448.0, -448.0])]).clamp(-448, 448)
    assert np.array_equal(oracle.e4m3_encode(x.double().numpy()),
                          x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert oracle.e4m3_encode(np.array([np.inf, np.nan])).tolist() == [0x7F, 0x7F]


def test_scale_exponent_is_the_least():
    for a in [448.0, 448.0000001, 449.0, 1.0, 1.75, 1.7500001, 3.5, 1e-30, 3e38, 2.0 ** -133]:
        e = oracle.scale_exponent(a)
        assert a <= 448 * 2.0 ** e and (e == -126 or a > 448 * 2.0 ** (e - 1))
    assert oracle.scale_exponent(0.0) == -126


def test_oracle_plan_grow_then_give_back_is_the_identity():
    tables, n_blocks, free = [[4, -1, -1], [0, 2, -1]], [1, 2], [1, 3, 5, 6]
    slots, lens, served = oracle.block_plan([10, 32], [8, 1], tables, n_blocks, free, 16, 10)
    assert served == [True, True] and lens == [18, 33] and free == [1, 3]
    assert tables == [[4, 6, -1], [0, 2, 5]]
    assert slots == [74, 75, 76, 77, 78, 79, 96, 97, 80, -1]
    oracle.block_plan([10, 32], [0, 0], tables, n_blocks, free, 16, 0)
    assert tables == [[4, -1, -1], [0, 2, -1]] and free == [1, 3, 5, 6] and n_blocks == [1, 2]


def _plan(lib, **kw):
    a = dict(lens=16, cu=32, tab=48, nb=64, fl=80, fc=96, slots=112, out=128, B=2, T=3, mb=4, N=8,
             bs=16)
    a.update(kw)
    return lib.gqa_block_plan(*(P(a[k]) for k in ("lens", "cu", "tab", "nb", "fl", "fc", "slots",
                                                  "out")),
                              a["B"], a["T"], a["mb"], a["N"], a["bs"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(mb=0), 1), (dict(N=0), 1), (dict(bs=0), 1),
    (dict(bs=24), 1), (dict(bs=256), 1), (dict(lens=None), 1), (dict(cu=None), 1),
    (dict(tab=None), 1), (dict(nb=None), 1), (dict(fl=None), 1), (dict(fc=None), 1),
    (dict(slots=None), 1), (dict(out=None), 1), (dict(tab=50), 1), (dict(out=130), 1),
    (dict(B=8193), 2), (dict(N=1 << 30, bs=128), 2), (dict(B=4096, mb=1 << 20), 2),
    (dict(mb=1 << 28), 2), (dict(T=1 << 30), 2), (dict(B=2048, mb=1 << 19), 2),
])
def test_plan_rejects_before_launch(lib, kw, code):
    assert _plan(lib, **kw) == code


def _append(lib, **kw):
    a = dict(k=16, v=32, slots=48, kp=64, vp=80, ks=96, vs=112, T=3, Hkv=2, N=8, bs=16)
    a.update(kw)
    return [f(*(P(a[n]) for n in ("k", "v", "slots", "kp", "vp", "ks", "vs")), a["T"], a["Hkv"],
              a["N"], a["bs"], None) for f in (lib.gqa_kv8_append, lib.gqa_kv8_append_f16)]


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(N=0), 1), (dict(bs=8), 1), (dict(k=None), 1),
    (dict(v=24), 1), (dict(kp=72), 1), (dict(vp=None), 1), (dict(slots=50), 1), (dict(ks=None), 1),
    (dict(vs=2), 1), (dict(N=1 << 26), 2), (dict(Hkv=70000), 2), (dict(T=1 << 30), 2),
    (dict(T=0, k=None, slots=None), 0),
])
def test_append_rejects_before_launch(lib, kw, code):
    assert _append(lib, **kw) == [code, code]


def _keep(lib, **kw):
    a = dict(kp=16, vp=32, ks=48, vs=64, tab=80, lens=96, cu=112, idx=128, ck=144, out=160,
             n=4, B=2, Hkv=2, N=8, bs=16, mb=4)
    a.update(kw)
    return lib.gqa_kv8_keep(*(P(a[n]) for n in ("kp", "vp", "ks", "vs", "tab", "lens", "cu", "idx",
                                                "ck", "out")),
                            a["n"], a["B"], a["Hkv"], a["N"], a["bs"], a["mb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(n=-1), 1), (dict(mb=0), 1), (dict(bs=48), 1), (dict(kp=None), 1),
    (dict(vp=40), 1), (dict(ks=None), 1), (dict(vs=66), 1), (dict(tab=None), 1),
    (dict(lens=None), 1), (dict(cu=None), 1), (dict(idx=None), 1), (dict(ck=None), 1),
    (dict(out=96), 1), (dict(out=98), 1), (dict(N=1 << 27), 2), (dict(mb=1 << 27), 2),
])
def test_keep_rejects_before_launch(lib, kw, code):
    assert _keep(lib, **kw) == code


def _decode(lib, **kw):
    a = dict(q=16, kp=32, vp=48, ks=64, vs=80, g=96, tab=112, lens=128, cu=144, tm=None, out=160,
             lse=None, B=2, T=3, Hq=8, Hkv=2, N=8, bs=16, mb=4, mr=2, mk=64, ws=176, wsb=1 << 30)
    a.update(kw)
    return [f(*(P(a[n]) for n in ("q", "kp", "vp", "ks", "vs", "g", "tab", "lens", "cu", "tm", "out",
                                  "lse")),
              *(a[n] for n in ("B", "T", "Hq", "Hkv", "N", "bs", "mb", "mr", "mk")), P(a["ws"]),
              a["wsb"], None) for f in (lib.gqa_kv8_decode, lib.gqa_kv8_decode_f16)]


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(mr=0), 1),
    (dict(mk=0), 1), (dict(mk=65), 1), (dict(mr=65, mk=64), 1), (dict(mb=0), 1), (dict(bs=20), 1),
    (dict(cu=None), 1), (dict(cu=None, T=2), 1), (dict(cu=None, T=2, mr=1, tm=192), 1),
    (dict(tm=196), 1), (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=56), 1), (dict(ks=None), 1),
    (dict(vs=82), 1), (dict(g=100), 1), (dict(tab=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(out=168), 1), (dict(lse=2), 1), (dict(ws=None), 5),
    (dict(wsb=64), 5), (dict(ws=184), 1), (dict(N=1 << 27), 2), (dict(T=1 << 28, Hq=8), 2),
    (dict(tm=192, mr=65, mk=128, mb=8), 2), (dict(T=0, q=None), 0),
    (dict(mk=1 << 30, mb=1 << 27), 2), (dict(Hkv=1 << 16, Hq=1 << 16, N=1, mk=1 << 23, mb=1 << 20), 2),
])
def test_decode_rejects_before_launch(lib, kw, code):
    assert _decode(lib, **kw) == [code, code]


def test_workspace_size(lib):
    assert G.kv8_workspace_size(0, 1, 8, 2, 1, 64) == 0
    one = G.kv8_workspace_size(1, 1, 24, 4, 1, 512)
    assert one >= 24 * 257 * 4
    assert G.kv8_workspace_size(16, 16, 24, 4, 1, 32768) >= 16 * one // 16
    # the size does not go by the sequences' lengths on the device, and never shrinks with T
    assert G.kv8_workspace_size(2, 9, 16, 2, 8, 4096) <= G.kv8_workspace_size(2, 10, 16, 2, 8, 4096)


def test_binding_refuses_wrong_tensors():
    q = torch.zeros(1, 8, 256, dtype=torch.bfloat16)
    pool = torch.zeros(2, 2, 16, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.zeros(2, 2)
    with pytest.raises(TypeError):
        G.kv8_decode(q.float(), pool, pool, sc, sc, None, None, None)
    with pytest.raises((TypeError, ValueError)):          # CPU tensors
        G.kv8_decode(q, pool, pool, sc, sc, None, None, None)
    with pytest.raises((TypeError, ValueError)):
        G.kv8_append(q, q, None, pool.view(torch.uint8), pool, sc, sc)
    with pytest.raises((TypeError, ValueError)):
        G.kv8_keep(pool, pool, sc, sc, None, None, None, None, None)
    with pytest.raises((TypeError, ValueError)):
        G.block_plan(torch.zeros(1, dtype=torch.int64), None, None, None, None, None, 16, 1)


def test_oracle_append_and_keep_by_hand():
    pool = np.zeros((3, 1, 16, 256), dtype=np.uint8)
    scale = np.ones((3, 1))
    x = np.ones((3, 1, 256)) * np.array([1.0, 2.0, 512.0])[:, None, None]
    oracle.kv8_append(pool, scale, x, [46, 47, 0], 16)
    # rows 14 and 15 of block 2 behind a scale of 1 (rows that were there stay), block 0 is new
    assert scale[:, 0].tolist() == [2.0, 1.0, 1.0]
    assert oracle.E4M3[pool[2, 0, 14:, 0]].tolist() == [1.0, 2.0]
    assert oracle.E4M3[pool[0, 0, 0, 0]] * 2 == 512.0
    # draft rows at positions 15, 16 (blocks 2, 0); keeping the second moves it to position 15
    oracle.kv8_keep(pool, scale, [[2, 0]], [17], [2], [[1]], 16)
    assert scale[2, 0] == 2.0 and oracle.E4M3[pool[2, 0, 15, 0]] * 2 == 512.0
    assert oracle.E4M3[pool[2, 0, 14, 0]] * 2 == 1.0
