"""Decode attention over the K8/V8 cache against softmax attention in 64 bits
(bounds derived in k8v8_ref.check_attention)."""
import math

import numpy as np
import pytest
import torch

import k8v8_ref as R
from cases import dev, to_dev

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def workspace(K, B, hq):
    return torch.full((K.k16v8_decode_workspace_size_k8v8(B, hq, 128),), 0xFF, dtype=torch.uint8, device=dev())


def run(K, q, table, kc, vc, sc, lens, scale=SCALE, flags=0):
    B, hq = q.shape[:2]
    out = torch.full((B, hq, 128), 9.0, dtype=torch.float16, device=dev())
    lse = torch.full((B, hq), 9.0, dtype=torch.float32, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_paged_decode_attention_k8v8(to_dev(q), to_dev(kc), to_dev(vc), to_dev(sc), to_dev(table),
                                        to_dev(np.asarray(lens, np.int32)), scale, workspace(K, B, hq), out,
                                        lse, dev_error=err)
    assert K.k16v8_read_device_error(err) == flags
    return out.cpu().numpy(), lse.cpu().numpy()


def check(K, seed, lens, hkv, exps=(-9, -5), qscale=1.0, scale=SCALE):
    rng = np.random.default_rng(seed)
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv, exps)
    q = (rng.standard_normal((len(lens), 4 * hkv, 128)) * qscale).astype(np.float16)
    out, lse = run(K, q, table, kc, vc, sc, lens, scale)
    R.check_attention(out, lse, R.attention(q.astype(np.float64), kc, vc, sc, table, lens, [1] * len(lens),
                                            scale, False))


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [0, 1, 0], [1000], [4097, 33],
                                  [511, 512, 513, 0, 16, 1, 47]])
@pytest.mark.parametrize("hkv", [1, 2, 10])
def test_lengths(K, lens, hkv):
    check(K, sum(lens) + hkv, lens, hkv)


def test_batch_of_many(K):
    rng = np.random.default_rng(0)
    check(K, 1, [int(x) for x in rng.integers(0, 70, 300)], 1)


def test_one_long_sequence(K):
    check(K, 2, [40000], 1)  # more than 32 tiles per warp


@pytest.mark.parametrize("exps", [(-15, -15), (-15, 7), (7, 7), (0, 3)])
def test_scales(K, exps):
    """Over the whole range, and pages of very unlike scales side by side."""
    check(K, 3, [300, 65, 16], 2, exps, qscale=2.0 ** -6 if exps[1] > 0 else 1.0)


def test_peaked_rows(K):
    """Scores that differ by hundreds, so the maximum moves often."""
    check(K, 4, [700, 90], 2, qscale=40.0)


def test_a_score_far_above_a_flat_tail(K):
    """What the many small weights add up to survives under one large one."""
    L, hkv = 3000, 1
    rng = np.random.default_rng(5)
    table, P = R.pages_of(rng, [L])
    kc, vc = np.zeros((P, hkv, 16, 128), np.uint8), R.codes(rng, P, hkv, 16, 128)
    vc[:] = R.encode(np.abs(R.TABLE[vc]))
    sc = np.full((P, hkv, 2), 2.0 ** -6, np.float32)
    kc[table[0, 0], 0, 3] = R.encode(np.full(128, 104.0))  # 15 above the others
    q = np.full((1, 4, 128), 0.8125, np.float16)
    out, lse = run(K, q, table, kc, vc, sc, [L])
    R.check_attention(out, lse, R.attention(q.astype(np.float64), kc, vc, sc, table, [L], [1], SCALE, False))


def test_zero_and_equal_scores(K):
    check(K, 6, [100, 16], 2, scale=0.0)


def test_nan_and_inf(K):
    """A NaN at a position that is seen reaches the rows that see it (a value's
    only its own dim), and no other sequence."""
    rng = np.random.default_rng(7)
    lens, hkv = [50, 50, 50, 40], 2
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    vc[table[0, 2], 1, 9, 77] = 0x7F
    kc[table[1, 0], 0, 3, 5] = 0xFF
    q = rng.standard_normal((4, 8, 128)).astype(np.float16)
    q[2, 3, 100] = np.nan
    out, lse = run(K, q, table, kc, vc, sc, lens)
    want = R.attention(q.astype(np.float64), kc, vc, sc, table, lens, [1] * 4, SCALE, False)
    assert np.isnan(want["out"]).sum() == 4 + 4 * 128 + 128
    R.check_attention(out, lse, want)


def test_rejected_pages_and_lengths(K):
    rng = np.random.default_rng(8)
    lens, hkv = [100, 64, 40], 2
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    q = rng.standard_normal((3, 8, 128)).astype(np.float16)
    bad = table.copy()
    bad[0, 2], bad[1, 0], bad[2, :3] = len(kc), -7, -1  # the last sequence has no page left
    out, lse = run(K, q, bad, kc, vc, sc, lens, flags=K.DEVERR_PAGE)
    R.check_attention(out, lse, R.attention(q.astype(np.float64), kc, vc, sc, bad, lens, [1] * 3, SCALE, False))
    assert np.all(out[2] == 0) and np.all(lse[2] == -np.inf)
    out, lse = run(K, q, table, kc, vc, sc, [100, -3, 40], flags=K.DEVERR_SEQLEN)
    R.check_attention(out, lse, R.attention(q.astype(np.float64), kc, vc, sc, table, [100, 0, 40], [1] * 3,
                                            SCALE, False))


def test_streams_and_graph(K):
    """Two calls on two streams at once, and captured ones with new lengths and
    queries at each replay."""
    rng = np.random.default_rng(9)
    lens, hkv = [130, 700, 33], 2
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    g = [to_dev(x) for x in (kc, vc, sc, table)]
    q = [rng.standard_normal((3, 8, 128)).astype(np.float16) for _ in range(3)]
    n = to_dev(np.array(lens, np.int32))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    bufs = [(to_dev(q[i]), torch.empty((3, 8, 128), dtype=torch.float16, device=dev()),
             torch.empty((3, 8), dtype=torch.float32, device=dev()), workspace(K, 3, 8)) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (qi, out, lse, ws) in zip(streams, bufs):
            K.k16v8_paged_decode_attention_k8v8(qi, g[0], g[1], g[2], g[3], n, SCALE, ws, out, lse, stream=s)
    torch.cuda.synchronize()
    for i, (_, out, lse, _) in enumerate(bufs):
        want = R.attention(q[i].astype(np.float64), kc, vc, sc, table, lens, [1] * 3, SCALE, False)
        R.check_attention(out.cpu().numpy(), lse.cpu().numpy(), want)
    qi, out, lse, ws = bufs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.k16v8_paged_decode_attention_k8v8(qi, g[0], g[1], g[2], g[3], n, SCALE, ws, out, lse)
    for now in ([130, 700, 33], [1, 0, 16], [17, 699, 2]):
        n.copy_(to_dev(np.array(now, np.int32)))
        qi.copy_(to_dev(q[2]))
        graph.replay()
        torch.cuda.synchronize()
        want = R.attention(q[2].astype(np.float64), kc, vc, sc, table, now, [1] * 3, SCALE, False)
        R.check_attention(out.cpu().numpy(), lse.cpu().numpy(), want)


def test_same_result_every_time(K):
    rng = np.random.default_rng(10)
    lens, hkv = [2000, 5, 300], 5
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    q = rng.standard_normal((3, 20, 128)).astype(np.float16)
    first = run(K, q, table, kc, vc, sc, lens)
    for _ in range(3):
        again = run(K, q, table, kc, vc, sc, lens)
        assert all(np.array_equal(a, b) for a, b in zip(first, again))
