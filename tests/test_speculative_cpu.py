"""The speculative calls' refusals, and the host parts of the step (tree
masks, rotary frequencies), without a GPU."""
import math

import numpy as np
import pytest
import torch

from fp8_paged_kv_append_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    from fp8_paged_kv_append_gb300 import k16v8
    return k16v8.load_library()


A = 0x1000  # an address that is aligned to everything; refused calls never follow it

ROPE = dict(q=A, q_ts=0, k=A, k_ts=0, v=A, v_ts=0, x_dtype=0, positions=A, inv_freq=A, rotary=128,
            inter=0, factor=1.0, slots=A, tokens=4, v_scale=A, q_out=A, kc=A, vc=A, pages=8, hq=8,
            hkv=2, d=128, err=None, stream=None)
TREE = dict(q=A, indptr=A, total_q=8, max_nodes=8, mask=A, kc=A, vc=A, v_scale=A, table=A, maxp=8,
            lens=A, max_len=128, batch=1, hq=8, hkv=2, d=128, pages=8, scale=0.1, ws=A,
            ws_bytes=1 << 30, out=A, lse=None, err=None, stream=None)
VERIFY = dict(target=A, ts=0, draft=A, ds=0, tokens=A, parents=A, indptr=A, total_q=8, max_nodes=8,
              u=A, vocab=100, batch=1, path=A, path_len=A, nxt=A, err=None, stream=None)
COMPACT = dict(kp=A, vp=A, layers=2, table=A, maxp=8, lens=A, indptr=A, path=A, max_nodes=8,
               path_len=A, batch=1, hkv=2, d=128, pages=8, new=None, err=None, stream=None)


def call(lib, name, args, **change):
    a = dict(args)
    assert set(change) <= set(a)
    a.update(change)
    return getattr(lib, name)(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(hq=-1), 1), (dict(hkv=0), 1), (dict(pages=0), 1),
    (dict(hq=70000), 1), (dict(d=64), 2), (dict(rotary=0), 2), (dict(rotary=136), 2),
    (dict(rotary=24), 2), (dict(x_dtype=3), 1), (dict(inter=2), 1),
    (dict(factor=math.inf), 1), (dict(factor=math.nan), 1),
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(positions=None), 1), (dict(inv_freq=None), 1), (dict(slots=None), 1),
    (dict(v_scale=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(q_ts=1023), 1), (dict(k_ts=128), 1), (dict(v_ts=260), 1), (dict(x_dtype=1, v_ts=258), 1),
    (dict(q=A + 8), 1), (dict(k=A + 8), 1), (dict(v=A + 8), 1), (dict(q_out=A + 8), 1),
    (dict(kc=A + 8), 1), (dict(vc=A + 8), 1), (dict(slots=A + 4), 1), (dict(positions=A + 2), 1),
    (dict(inv_freq=A + 2), 1), (dict(v_scale=A + 2), 1), (dict(tokens=0, q=None, k=None), 0)])
def test_rope_refusals(lib, change, status):
    assert call(lib, "k16v8_rope_kv_append", ROPE, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(total_q=-1), 1), (dict(batch=-1), 1), (dict(max_nodes=-1), 1), (dict(hkv=0), 1),
    (dict(max_len=-1), 1), (dict(d=64), 2), (dict(hq=10), 2), (dict(max_nodes=65), 2),
    (dict(batch=8193), 1), (dict(hq=4 * 4096, hkv=4096), 1), (dict(pages=0), 1),
    (dict(maxp=-1), 1), (dict(maxp=7), 1), (dict(maxp=1 << 27, max_len=(1 << 30) + 1), 1),
    (dict(scale=-0.1), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(pages=1 << 26, ws_bytes=1 << 40), 1),
    (dict(q=None), 1), (dict(indptr=None), 1), (dict(mask=None), 1), (dict(kc=None), 1),
    (dict(vc=None), 1), (dict(v_scale=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(q=A + 8), 1), (dict(kc=A + 8), 1), (dict(vc=A + 8), 1),
    (dict(out=A + 8), 1), (dict(mask=A + 4), 1), (dict(indptr=A + 2), 1), (dict(lens=A + 2), 1),
    (dict(table=A + 2), 1), (dict(v_scale=A + 2), 1), (dict(lse=A + 2), 1),
    (dict(batch=0), 0), (dict(total_q=0), 0), (dict(max_nodes=0), 0)])
def test_tree_attention_refusals(lib, change, status):
    assert call(lib, "k16v8_paged_tree_attention", TREE, **change) == status


def test_tree_workspace_size_is_zero_for_refused_shapes(lib):
    good = [8, 1, 8, 8, 2, 128, 128]
    for i, v in ((0, -1), (1, -1), (2, 65), (3, 10), (4, 0), (5, 64), (6, -1)):
        bad = list(good)
        bad[i] = v
        assert lib.k16v8_tree_workspace_size(*bad) == 0


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), 1), (dict(total_q=-1), 1), (dict(max_nodes=-1), 1), (dict(vocab=0), 1),
    (dict(max_nodes=65), 2), (dict(vocab=(1 << 19) + 1), 2), (dict(ts=99), 1), (dict(ds=99), 1),
    (dict(target=None), 1), (dict(tokens=None), 1), (dict(parents=None), 1),
    (dict(indptr=None), 1), (dict(u=None), 1), (dict(path=None), 1), (dict(path_len=None), 1),
    (dict(nxt=None), 1), (dict(target=A + 2), 1), (dict(draft=A + 2), 1), (dict(tokens=A + 2), 1),
    (dict(parents=A + 2), 1), (dict(indptr=A + 2), 1), (dict(u=A + 2), 1), (dict(path=A + 2), 1),
    (dict(path_len=A + 2), 1), (dict(nxt=A + 2), 1), (dict(batch=0), 0)])
def test_tree_verify_refusals(lib, change, status):
    assert call(lib, "k16v8_tree_verify", VERIFY, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(layers=-1), 1), (dict(batch=-1), 1), (dict(max_nodes=-1), 1), (dict(maxp=-1), 1),
    (dict(maxp=1 << 28), 1), (dict(hkv=0), 1), (dict(pages=0), 1), (dict(d=64), 2),
    (dict(max_nodes=65), 2), (dict(kp=None), 1), (dict(vp=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(indptr=None), 1), (dict(path=None), 1), (dict(path_len=None), 1),
    (dict(kp=A + 4), 1), (dict(vp=A + 4), 1), (dict(table=A + 2), 1), (dict(lens=A + 2), 1),
    (dict(indptr=A + 2), 1), (dict(path=A + 2), 1), (dict(path_len=A + 2), 1),
    (dict(new=A + 2), 1), (dict(new=A), 1), (dict(batch=3, new=A + 8), 1),
    (dict(batch=0), 0), (dict(layers=0), 0)])
def test_kv_compact_refusals(lib, change, status):
    assert call(lib, "k16v8_kv_compact", COMPACT, **change) == status


def test_binding_refuses_tensors_that_are_not_on_the_device(lib):
    from fp8_paged_kv_append_gb300 import k16v8 as K
    x = torch.zeros(2, 2, 128, dtype=torch.float16)
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    f32 = torch.zeros(64)
    kc, vc = torch.zeros(1, 2, 16, 128, dtype=torch.float16), torch.zeros(1, 2, 16, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="current CUDA device"):
        K.k16v8_rope_kv_append(x, x, x, i32, f32, i64, f32, x, kc, vc)
    with pytest.raises(ValueError, match="current CUDA device"):
        K.k16v8_paged_tree_attention(x, i32, 1, i64, kc, vc, f32, i32[None], i32[:1], 16, 0.1, None, x)
    with pytest.raises(ValueError, match="current CUDA device"):
        K.k16v8_tree_verify(f32[None], None, i32, i32, i32, 1, f32, i32[None], i32, i32)
    with pytest.raises(ValueError, match="current CUDA device"):
        K.k16v8_kv_compact(i64, i64, 1, 2, 128, i32[None], i32, i32, i32[None], i32)


def test_tree_masks_and_depths():
    from fp8_paged_kv_append_gb300.tree_step import tree_depths, tree_masks
    parents = [-1, 0, 0, 1, 2, 4]
    assert tree_masks(parents).tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b110101]
    assert tree_depths(parents).tolist() == [0, 1, 1, 2, 2, 3]
    chain = tree_masks([i - 1 for i in range(64)])
    assert chain[63] == -1 and chain[62] == (1 << 63) - 1
    assert tree_masks([]).shape == (0,)
    with pytest.raises(ValueError):
        tree_masks([-1, 1])
    with pytest.raises(ValueError):
        tree_masks([-1, -1])
    with pytest.raises(ValueError):
        tree_masks([i - 1 for i in range(65)])


def test_rope_frequencies():
    from fp8_paged_kv_append_gb300.rope import rope_inv_freq
    f, a = rope_inv_freq(64, 10000.0)
    want = 10000.0 ** (-np.arange(32) / 32.0)
    assert a == 1.0 and f.dtype == torch.float32
    assert np.array_equal(f.numpy(), want.astype(np.float32))
    f2, a2 = rope_inv_freq(64, scaling="linear", factor=4.0)
    assert a2 == 1.0 and np.array_equal(f2.numpy(), (want / 4).astype(np.float32))
    # ntk: the fastest pair is kept, the slowest slowed by the factor
    f3, _ = rope_inv_freq(64, scaling="ntk", factor=8.0)
    assert f3[0] == 1.0 and abs(float(f3[-1]) * 8.0 / want[-1] - 1) < 1e-6
    # yarn: kept above beta_fast turns, divided below beta_slow, between the two in the middle
    f4, a4 = rope_inv_freq(128, scaling="yarn", factor=16.0, original_max_position=4096)
    base = 10000.0 ** (-np.arange(64) / 64.0)
    turns = 4096 * base / (2 * math.pi)
    assert a4 == pytest.approx(0.1 * math.log(16.0) + 1)
    r = f4.numpy() / base
    assert np.allclose(r[turns > 36], 1, atol=1e-6) and np.allclose(r[turns < 0.8], 1 / 16, atol=1e-6)
    assert np.all(np.diff(r) <= 1e-6)
    for bad in (dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=64, base=1.0),
                dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=64, scaling="yarn", factor=2.0),
                dict(rotary_dim=64, scaling="yarn", factor=2.0, original_max_position=64,
                     beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            rope_inv_freq(**bad)
