"""Prefill and cross attention over the K8/V8 cache against softmax attention in
64 bits (bounds derived in k8v8_ref.check_attention)."""
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


def workspace(K, max_q, hkv):
    return torch.full((K.k16v8_attention_workspace_size_k8v8(max_q, 4 * hkv, hkv, 128),), 0xFF,
                      dtype=torch.uint8, device=dev())


def call(K, causal):
    return K.k16v8_paged_prefill_attention_k8v8 if causal else K.k16v8_paged_cross_attention_k8v8


def run(K, causal, q, counts, table, kc, vc, sc, lens, scale=SCALE, flags=0, max_q=None, max_len=None,
        indptr=None):
    T, hq = q.shape[:2]
    out = torch.full((T, hq, 128), 9.0, dtype=torch.float16, device=dev())
    lse = torch.full((T, hq), 9.0, dtype=torch.float32, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    if indptr is None:
        indptr = np.concatenate([[0], np.cumsum(counts)])
    max_q = max(counts) if max_q is None else max_q
    call(K, causal)(to_dev(q), to_dev(np.asarray(indptr, np.int32)), max_q, to_dev(kc), to_dev(vc), to_dev(sc),
                    to_dev(table), to_dev(np.asarray(lens, np.int32)), max(lens) if max_len is None else max_len,
                    scale, workspace(K, max_q, hq // 4), out, lse, dev_error=err)
    assert K.k16v8_read_device_error(err) == flags
    return out.cpu().numpy(), lse.cpu().numpy()


def check(K, causal, seed, counts, lens, hkv, exps=(-9, -5), qscale=1.0, scale=SCALE, pad=0, **kw):
    rng = np.random.default_rng(seed)
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv, exps)
    T = sum(counts)
    q = (rng.standard_normal((T + pad, 4 * hkv, 128)) * qscale).astype(np.float16)
    out, lse = run(K, causal, q, counts, table, kc, vc, sc, lens, scale, **kw)
    assert np.all(out[T:] == 9.0) and np.all(lse[T:] == 9.0)
    R.check_attention(out[:T], lse[:T], R.attention(q[:T].astype(np.float64), kc, vc, sc, table, lens, counts,
                                                    scale, causal))


@pytest.mark.parametrize("counts,lens", [
    ([1], [1]), ([1], [200]), ([5], [5]), ([32], [32]), ([33], [40]), ([64], [64]), ([65], [300]),
    ([31, 1, 7], [31, 129, 128]), ([200], [200]), ([130, 1, 64, 33], [700, 1, 64, 161]), ([0, 40, 0], [9, 40, 0]),
    ([97, 128], [97, 1000])])
@pytest.mark.parametrize("hkv", [1, 3])
def test_prefill(K, counts, lens, hkv):
    check(K, True, sum(counts) + hkv, counts, lens, hkv, pad=2)


@pytest.mark.parametrize("counts,lens", [
    ([1], [1]), ([1], [1500]), ([5], [1500]), ([40], [3]), ([64], [128]), ([65], [129]), ([7, 0, 33], [0, 100, 257]),
    ([3, 3, 3], [0, 0, 0]), ([200, 1, 90], [17, 640, 0]), ([128], [2000]), ([20, 30], [5, 1000])])
@pytest.mark.parametrize("hkv", [1, 3])
def test_cross(K, counts, lens, hkv):
    check(K, False, sum(counts) + hkv, counts, lens, hkv, pad=1)


@pytest.mark.parametrize("causal", [True, False])
def test_ten_heads(K, causal):
    check(K, causal, 1, [70, 20], [170, 250], 10)


@pytest.mark.parametrize("causal", [True, False])
def test_long(K, causal):
    """Every CTA holds a part of each segment."""
    check(K, causal, 2, [3], [60000], 1)
    check(K, causal, 3, [50], [20000], 1)


@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences(K, causal):
    rng = np.random.default_rng(4)
    counts = [int(x) for x in rng.integers(0, 6, 400)]
    check(K, causal, 5, counts, [c + int(x) for c, x in zip(counts, rng.integers(0, 60, 400))], 1)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("most", [20, 120])
def test_many_pieces_per_cta(K, causal, most):
    """Every CTA goes through many segments, with one and with two row tiles in turn,
    of one tile and of several, ending in either half of a tile."""
    rng = np.random.default_rng(most)
    B, hkv = 48, 4
    counts = [int(x) for x in rng.integers(0, most + 1, B)]
    if most > 32:
        counts[::3] = [int(x) for x in rng.integers(1, 33, len(counts[::3]))]
    lens = [c + int(x) for c, x in zip(counts, rng.integers(0, 700, B))]
    lens[5], lens[17], lens[30] = counts[5], counts[17], counts[30]
    check(K, causal, most, counts, lens, hkv, pad=3)


@pytest.mark.parametrize("exps", [(-15, -15), (-15, 7), (7, 7)])
@pytest.mark.parametrize("counts", [[20], [60, 5]])
def test_scales(K, exps, counts):
    check(K, True, 6, counts, [300, 30][:len(counts)], 2, exps, qscale=2.0 ** -6 if exps[1] > 0 else 1.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("counts", [[30], [64, 10]])
def test_peaked_rows(K, causal, counts):
    check(K, causal, 7, counts, [700, 90][:len(counts)], 2, qscale=40.0)


def test_equal_scores(K):
    check(K, True, 8, [64, 20], [500, 20], 1, scale=0.0)
    check(K, False, 8, [64, 20], [500, 20], 1, scale=0.0)


def test_hints_above_the_sizes(K):
    check(K, True, 9, [20, 5], [100, 6], 2, max_q=300, max_len=112)


def test_no_lse(K):
    rng = np.random.default_rng(10)
    table, kc, vc, sc = R.poisoned_pool(rng, [90], 1)
    q = to_dev(rng.standard_normal((40, 4, 128)).astype(np.float16))
    ip, n = to_dev(np.array([0, 40], np.int32)), to_dev(np.array([90], np.int32))
    g = [to_dev(x) for x in (kc, vc, sc, table)]
    res = []
    for lse in (None, torch.empty((40, 4), device=dev())):
        out = torch.empty_like(q)
        K.k16v8_paged_cross_attention_k8v8(q, ip, 40, *g, n, 90, SCALE, workspace(K, 40, 1), out, lse)
        res.append(out)
    assert torch.equal(*res)


@pytest.mark.parametrize("causal", [True, False])
def test_nan(K, causal):
    """NaN at a position reaches the rows that see it (a value's only its dim)."""
    rng = np.random.default_rng(11)
    counts, lens, hkv = [70, 40, 40, 10], [200, 140, 130, 64], 2
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    vc[table[0, 160 // 16], 1, 0, 77] = 0x7F   # a new token's value
    vc[table[0, 2], 0, 5, 7] = 0xFF            # an earlier one's
    kc[table[1, 120 // 16], 0, 8, 5] = 0xFF    # a new token's key
    q = rng.standard_normal((160, 8, 128)).astype(np.float16)
    q[115, 3, 100] = np.nan
    out, lse = run(K, causal, q, counts, table, kc, vc, sc, lens)
    want = R.attention(q.astype(np.float64), kc, vc, sc, table, lens, counts, SCALE, causal)
    assert 0 < np.isnan(want["out"]).sum() < want["out"].size // 2
    R.check_attention(out, lse, want)


@pytest.mark.parametrize("causal", [True, False])
def test_rejected_pages(K, causal):
    rng = np.random.default_rng(12)
    counts, lens, hkv = [40, 5, 33], [300, 64, 40], 2
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    q = rng.standard_normal((78, 8, 128)).astype(np.float16)
    bad = table.copy()
    bad[0, 2], bad[0, 18], bad[1, 0], bad[2, :3] = len(kc), -7, -1, -1
    out, lse = run(K, causal, q, counts, bad, kc, vc, sc, lens, flags=K.DEVERR_PAGE)
    R.check_attention(out, lse, R.attention(q.astype(np.float64), kc, vc, sc, bad, lens, counts, SCALE, causal))
    assert np.all(out[45:] == 0) and np.all(lse[45:] == -np.inf)


@pytest.mark.parametrize("causal", [True, False])
def test_bad_sequences_are_skipped(K, causal):
    rng = np.random.default_rng(13)
    lens, hkv = [50, 60, 40], 1
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    q = rng.standard_normal((30, 4, 128)).astype(np.float16)

    def expect(indptr, now, skipped, **kw):
        out, lse = run(K, causal, q, [10] * 3, table, kc, vc, sc, now, flags=K.DEVERR_SEQLEN, indptr=indptr,
                       max_len=64, **kw)
        for b in range(3):
            a, e = indptr[b], indptr[b + 1]
            if b in skipped:
                continue
            want = R.attention(q[a:e].astype(np.float64), kc, vc, sc, table[b:b + 1], [now[b]], [e - a], SCALE,
                               causal)
            R.check_attention(out[a:e], lse[a:e], want)
        return out

    out = expect([0, 10, 20, 30], [50, 65, 40], {1})
    assert np.all(out[10:20] == 9.0)
    assert np.all(expect([0, 10, 20, 30], [50, 60, -1], {2})[20:] == 9.0)
    assert np.all(expect([0, 10, 20, 31], [50, 60, 40], {2})[20:] == 9.0)
    assert np.all(expect([0, 2, 14, 20], [50, 60, 40], {1}, max_q=10)[2:14] == 9.0)
    if causal:
        assert np.all(expect([0, 10, 20, 30], [50, 60, 9], {2})[20:] == 9.0)


def test_streams_and_graph(K):
    rng = np.random.default_rng(14)
    lens, counts, hkv = [330, 700, 90], [100, 40, 64], 2
    T = sum(counts)
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    g = [to_dev(x) for x in (kc, vc, sc, table)]
    q = rng.standard_normal((T, 8, 128)).astype(np.float16)
    ip, n = to_dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)), to_dev(np.array(lens, np.int32))
    want = {c: R.attention(q.astype(np.float64), kc, vc, sc, table, lens, counts, SCALE, c) for c in (True, False)}
    qd = to_dev(q)
    bufs = [(torch.empty_like(qd), torch.empty((T, 8), device=dev()), workspace(K, 100, hkv)) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for causal, s, (out, lse, ws) in zip((True, False), streams, bufs):
            call(K, causal)(qd, ip, 100, *g, n, 700, SCALE, ws, out, lse, stream=s)
    torch.cuda.synchronize()
    for causal, (out, lse, _) in zip((True, False), bufs):
        R.check_attention(out.cpu().numpy(), lse.cpu().numpy(), want[causal])
    out, lse, ws = bufs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(K, True)(qd, ip, 100, *g, n, 700, SCALE, ws, out, lse)
    for now, cnt in ((lens, counts), ([330, 80, 64], [1, 2, 64]), ([100, 40, 64], [100, 40, 64])):
        n.copy_(to_dev(np.array(now, np.int32)))
        ip.copy_(to_dev(np.concatenate([[0], np.cumsum(cnt)]).astype(np.int32)))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        m = sum(cnt)
        ref = R.attention(q[:m].astype(np.float64), kc, vc, sc, table, now, cnt, SCALE, True)
        R.check_attention(out.cpu().numpy()[:m], lse.cpu().numpy()[:m], ref)
        assert torch.all(out[m:] == 9.0)


def test_same_result_every_time(K):
    rng = np.random.default_rng(15)
    counts, lens, hkv = [70, 3], [900, 333], 5
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    q = rng.standard_normal((73, 20, 128)).astype(np.float16)
    for causal in (True, False):
        first = run(K, causal, q, counts, table, kc, vc, sc, lens)
        for _ in range(3):
            again = run(K, causal, q, counts, table, kc, vc, sc, lens)
            assert all(np.array_equal(a, b) for a, b in zip(first, again))


def test_refusals(K):
    q = torch.zeros((4, 4, 128), dtype=torch.float16, device=dev())
    kc = torch.zeros((2, 1, 16, 128), dtype=torch.uint8, device=dev())
    sc = torch.ones((2, 1, 2), dtype=torch.float32, device=dev())
    ip, n = to_dev(np.array([0, 4], np.int32)), to_dev(np.array([20], np.int32))
    table, ws = to_dev(np.array([[0, 1]], np.int32)), workspace(K, 4, 1)

    def go(**kw):
        a = dict(q=q, qo_indptr=ip, max_qlen=4, k_cache=kc, v_cache=kc, kv_scale=sc, block_table=table, seq_lens=n,
                 max_seq_len=32, sm_scale=SCALE, workspace=ws, out=torch.empty_like(q))
        a.update(kw)
        K.k16v8_paged_cross_attention_k8v8(**a)

    go()
    for bad in (dict(q=q.float()), dict(kv_scale=sc[0]), dict(k_cache=kc.view(torch.int8)), dict(seq_lens=n.long()),
                dict(out=torch.empty_like(q)[:3]), dict(lse=torch.empty((4, 4), device=dev()).half()),
                dict(qo_indptr=ip[:1])):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(max_seq_len=33), dict(sm_scale=-1.0), dict(sm_scale=float("nan")), dict(workspace=ws[:-256]),
                dict(workspace=None), dict(max_qlen=-1)):
        with pytest.raises(K.K16V8Error):
            go(**bad)


# ---- a wait that runs out (a copy that is never issued) ------------------------------

@pytest.mark.parametrize("counts", [[20], [64]])
def test_wait_expiry(K, counts):
    """The first CTA's keys are withheld: the error word says so, other segments
    are right, and the next call is."""
    rng = np.random.default_rng(16)
    hkv, lens = 2, [700]
    table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
    q = rng.standard_normal((counts[0], 8, 128)).astype(np.float16)
    g = [to_dev(x) for x in (kc, vc, sc, table)]
    ip, n = to_dev(np.array([0, counts[0]], np.int32)), to_dev(np.array(lens, np.int32))
    out, lse = to_dev(np.zeros_like(q)), torch.zeros((counts[0], 8), device=dev())
    err, ws = torch.zeros(1, dtype=torch.int32, device=dev()), workspace(K, counts[0], hkv)
    K.k16v8_paged_prefill_attention_k8v8_wait_test(to_dev(q), ip, counts[0], *g, n, lens[0], SCALE, ws, out, lse,
                                                   dev_error=err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_TIMEOUT
    want = R.attention(q.astype(np.float64), kc, vc, sc, table, lens, counts, SCALE, True)
    second = {k: v[:, 4:] for k, v in want.items()}  # the other KV head is another CTA's
    R.check_attention(out.cpu().numpy()[:, 4:], lse.cpu().numpy()[:, 4:], second)
    got = run(K, True, q, counts, table, kc, vc, sc, lens)
    R.check_attention(*got, want)
