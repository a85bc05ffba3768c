"""Host side of the K8/V8 calls and of positions with several axes: arguments
that are refused without a GPU, and which axis turns which pair."""
import ctypes

import pytest

from fp8_paged_kv_append_gb300 import build as libbuild
from fp8_paged_kv_append_gb300 import rope


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    from fp8_paged_kv_append_gb300 import k16v8
    return k16v8.load_library()


def test_pair_axes():
    assert rope.rope_pair_axes(128, [64]) == bytes(64)
    assert rope.rope_pair_axes(128, [16, 24, 24]) == bytes([0] * 16 + [1] * 24 + [2] * 24)
    assert rope.rope_pair_axes(32, [8, 4, 4]) == bytes([0] * 8 + [1] * 4 + [2] * 4)
    assert rope.rope_pair_axes(32, [8, 4, 4], True) == bytes([0, 1, 2] * 4 + [0] * 4)
    assert rope.rope_pair_axes(16, [4, 4], True) == bytes([0, 1] * 4)
    assert rope.rope_pair_axes(16, [8, 0, 0], True) == bytes(8)
    for bad in ([16, 24], [65], [], [13, 13, 13, 13, 12], [-1, 65]):
        with pytest.raises(ValueError):
            rope.rope_pair_axes(128, bad)
    with pytest.raises(ValueError):
        rope.rope_pair_axes(128, [0, 40, 24], True)
    with pytest.raises(ValueError):
        rope.rope_pair_axes(24, [12])


AXES = (ctypes.c_int8 * 64)(*([0] * 16 + [1] * 24 + [2] * 24))
BAD_AXES = (ctypes.c_int8 * 64)(*([0] * 63 + [3]))
NEG_AXES = (ctypes.c_int8 * 64)(*([0] * 63 + [-1]))
X = 1 << 20  # stands for an aligned address


def rope_axes(lib, **kw):
    a = dict(q=X, qs=0, k=X, ks=0, v=X, vs=0, dt=0, pos=X, axes=3, pair=AXES, freq=X, rot=128, il=0, f=1.0,
             slots=X, T=8, vsc=X, qo=X, kc=X, vc=X, P=4, hq=8, hkv=2, d=128, err=None, stream=None)
    a.update(kw)
    return lib.k16v8_rope_axes_kv_append(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(axes=0), 1), (dict(axes=5), 1), (dict(pair=None), 1), (dict(pair=BAD_AXES), 1),
    (dict(pair=NEG_AXES), 1), (dict(axes=2), 1), (dict(rot=0), 2), (dict(rot=24), 2), (dict(d=64), 2),
    (dict(dt=3), 1), (dict(il=2), 1), (dict(f=float("nan")), 1), (dict(pos=None), 1), (dict(k=X + 8), 1),
    (dict(T=-1), 1), (dict(T=0), 0), (dict(qs=1020), 1), (dict(qs=1028), 1), (dict(hq=-1), 1)])
def test_rope_axes_refusals(lib, kw, status):
    assert rope_axes(lib, **kw) == status


def append(lib, **kw):
    a = dict(q=X, qs=0, k=X, ks=0, v=X, vs=0, dt=0, indptr=X, T=8, pos=X, axes=3, pair=AXES, freq=X, rot=128,
             il=0, f=1.0, table=X, maxp=4, lens=X, B=2, qo=X, kc=X, vc=X, sc=X, P=4, hq=8, hkv=2, d=128,
             err=None, stream=None)
    a.update(kw)
    return lib.k16v8_rope_kv_append_k8v8(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(axes=0), 1), (dict(axes=5), 1), (dict(pair=None), 1), (dict(pair=BAD_AXES), 1), (dict(rot=8), 2),
    (dict(rot=144), 2), (dict(d=64), 2), (dict(dt=3), 1), (dict(il=2), 1), (dict(f=float("inf")), 1),
    (dict(indptr=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(sc=None), 1),
    (dict(sc=X + 4), 1), (dict(kc=X + 8), 1), (dict(pos=None), 1), (dict(freq=None), 1), (dict(q=None), 1),
    (dict(qo=None), 1), (dict(B=-1), 1), (dict(B=65536), 1), (dict(maxp=1 << 27), 1), (dict(P=0), 1),
    (dict(hkv=0), 1), (dict(ks=128), 1), (dict(vs=260), 1), (dict(T=0), 0), (dict(B=0), 0), (dict(T=-1), 1)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


def decode(lib, **kw):
    a = dict(q=X, kc=X, vc=X, sc=X, table=X, maxp=4, lens=X, B=2, hq=8, hkv=2, d=128, P=4, scale=0.1, ws=X,
             wb=1 << 30, out=X, lse=X, err=None, stream=None)
    a.update(kw)
    return lib.k16v8_paged_decode_attention_k8v8(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(d=64), 2), (dict(hq=6), 2), (dict(hq=16), 2), (dict(hq=0), 1), (dict(hkv=0), 1), (dict(B=-1), 1),
    (dict(B=8193), 1), (dict(P=0), 1), (dict(P=1 << 27), 1), (dict(maxp=1 << 27), 1), (dict(scale=-0.1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(ws=None), 1),
    (dict(ws=X + 128), 1), (dict(out=X + 8), 1), (dict(sc=X + 4), 1), (dict(lse=X + 2), 1), (dict(B=0), 0)])
def test_decode_refusals(lib, kw, status):
    assert decode(lib, **kw) == status


def attention(lib, name, **kw):
    a = dict(q=X, indptr=X, T=8, max_q=8, kc=X, vc=X, sc=X, table=X, maxp=4, lens=X, max_len=64, B=2, hq=8,
             hkv=2, d=128, P=4, scale=0.1, ws=X, wb=1 << 30, out=X, lse=X, err=None, stream=None)
    a.update(kw)
    return getattr(lib, name)(*a.values())


@pytest.mark.parametrize("name", ["k16v8_paged_prefill_attention_k8v8", "k16v8_paged_cross_attention_k8v8"])
@pytest.mark.parametrize("kw,status", [
    (dict(d=64), 2), (dict(hq=6), 2), (dict(hq=16), 2), (dict(hq=0), 1), (dict(hkv=0), 1),
    (dict(hq=16384, hkv=4096), 1), (dict(max_q=-1), 1), (dict(T=-1), 1), (dict(B=-1), 1), (dict(B=8193), 1),
    (dict(P=0), 1), (dict(P=1 << 26), 1), (dict(maxp=-1), 1), (dict(max_len=-1), 1), (dict(max_len=65), 1),
    (dict(max_len=(1 << 30) + 1, maxp=1 << 27), 1), (dict(scale=-0.1), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(indptr=None), 1), (dict(kc=None), 1),
    (dict(vc=None), 1), (dict(sc=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(ws=None), 1),
    (dict(out=None), 1), (dict(ws=X + 128), 1), (dict(q=X + 8), 1), (dict(kc=X + 8), 1), (dict(vc=X + 8), 1),
    (dict(out=X + 8), 1), (dict(sc=X + 4), 1), (dict(lse=X + 2), 1), (dict(indptr=X + 2), 1),
    (dict(lens=X + 2), 1), (dict(table=X + 2), 1), (dict(B=0), 0), (dict(T=0), 0), (dict(max_q=0), 0)])
def test_attention_refusals(lib, name, kw, status):
    assert attention(lib, name, **kw) == status


def test_workspace_sizes_of_refused_calls(lib):
    assert lib.k16v8_attention_workspace_size_k8v8(-1, 8, 2, 128) == 0
    assert lib.k16v8_attention_workspace_size_k8v8(8, 8, 2, 64) == 0
    assert lib.k16v8_attention_workspace_size_k8v8(8, 9, 2, 128) == 0
    assert lib.k16v8_decode_workspace_size_k8v8(-1, 8, 128) == 0
    assert lib.k16v8_decode_workspace_size_k8v8(8193, 8, 128) == 0
    assert lib.k16v8_decode_workspace_size_k8v8(1, 8, 64) == 0
