"""Verification of drafted trees against the definition in exact arithmetic
(fractions of the fp32 inputs), so accepted paths and next tokens have to be
equal: the kernel counts weights in units of 2^-44, and a drawn number that
falls between two running sums closer than that is not met by these seeds."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from cases import dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def walk(p, q, tokens, parents, u):
    """One tree: p [n, V], q [n, V] or None; accepted nodes and next token."""
    n, V = p.shape
    cur, path = 0, [0]
    frac = lambda row: [Fraction(float(x)) for x in row]
    r, Z = frac(p[0]), Fraction(1)
    for i in range(1, n):
        if parents[i] != cur:
            continue
        x = int(tokens[i])
        qx = Fraction(1) if q is None else Fraction(float(q[cur, x]))
        if Fraction(float(u[i])) * qx * Z < r[x]:
            cur = i
            path.append(i)
            r, Z = frac(p[i]), Fraction(1)
            continue
        if q is None:
            r[x] = Fraction(0)
        else:
            r = [max(a - Z * b, 0) for a, b in zip(r, frac(q[cur]))]
        Z = sum(r)
    total = sum(r)
    if total == 0:
        r = frac(p[cur])
        total = sum(r)
    if total == 0:
        return path, -1
    target, run = Fraction(float(u[0])) * total, Fraction(0)
    for j, w in enumerate(r):
        run += w
        if run > target:
            return path, j
    raise AssertionError


def rows(rng, n, V, sharp=2.0):
    x = np.exp(sharp * rng.standard_normal((n, V)))
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def make(seed, nodes, V, branch, draft=True, sharp=2.0, near=0.5):
    rng = np.random.default_rng(seed)
    total = int(sum(nodes))
    p = rows(rng, total, V, sharp)
    x = p * np.exp(near * rng.standard_normal((total, V)))
    q = (x / x.sum(-1, keepdims=True)).astype(np.float32)
    parents = np.concatenate([np.concatenate([[-1], np.maximum(np.arange(1, n) - rng.integers(
        1, branch + 1, n - 1), 0)]) if n else np.zeros(0) for n in nodes]).astype(np.int32)
    indptr = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    tokens = np.zeros(total, np.int32)
    for b, n in enumerate(nodes):
        for i in range(1, n):
            row = q[indptr[b] + parents[indptr[b] + i]].astype(np.float64)
            tokens[indptr[b] + i] = rng.choice(V, p=row / row.sum())
    u = rng.random(total).astype(np.float32)
    return p, (q if draft else None), tokens, parents, indptr, u


def run(K, p, q, tokens, parents, indptr, u, max_nodes, err=None, stride=0, stream=None):
    B = len(indptr) - 1
    V = p.shape[1]

    def put(a):
        if a is None:
            return None
        wide = torch.full((a.shape[0], V + stride), 0.5, device=dev())
        wide[:, :V] = to_dev(a)
        return wide[:, :V]

    path = torch.full((B, max_nodes), 77, dtype=torch.int32, device=dev())
    plen = torch.full((B,), 77, dtype=torch.int32, device=dev())
    nxt = torch.full((B,), 77, dtype=torch.int32, device=dev())
    K.k16v8_tree_verify(put(p), put(q), to_dev(tokens), to_dev(parents), to_dev(indptr), max_nodes,
                        to_dev(u), path, plen, nxt, err, stream)
    return path.cpu().numpy(), plen.cpu().numpy(), nxt.cpu().numpy()


def compare(K, p, q, tokens, parents, indptr, u, max_nodes=None, stride=0):
    max_nodes = max_nodes or int(np.diff(indptr).max())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    path, plen, nxt = run(K, p, q, tokens, parents, indptr, u, max_nodes, err, stride)
    assert K.k16v8_read_device_error(err) == 0
    lens = []
    for b in range(len(indptr) - 1):
        a, z = int(indptr[b]), int(indptr[b + 1])
        if z == a:
            assert plen[b] == 0 and nxt[b] == -1 and np.all(path[b] == -1)
            continue
        want, tok = walk(p[a:z], None if q is None else q[a:z], tokens[a:z], parents[a:z], u[a:z])
        assert plen[b] == len(want) and path[b, :len(want)].tolist() == want
        assert np.all(path[b, len(want):] == -1) and nxt[b] == tok
        lens.append(len(want))
    return lens


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("branch", [1, 3, 8])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 100, 1000, 4099])
def test_trees(K, V, branch, draft):
    lens = compare(K, *make(V + branch, [9, 1, 16, 5, 12], V, branch, draft))
    assert len(lens) == 5


@pytest.mark.parametrize("draft", [True, False])
def test_accepted_and_rejected_paths_both_occur(K, draft):
    lens = compare(K, *make(7, [8] * 40, 50, 2, draft, near=0.3))
    # without a draft row a candidate is taken with its target probability alone
    assert min(lens) == 1 and max(lens) >= (4 if draft else 2)


@pytest.mark.parametrize("draft", [True, False])
def test_widest_trees(K, draft):
    compare(K, *make(8, [64, 64, 63], 200, 5, draft, near=1.5))
    star = make(9, [64, 64], 64, 64, draft, near=3.0)  # every node hangs on node 0, tokens repeat
    star[3][:] = np.where(star[3] < 0, -1, 0)
    compare(K, *star)


def test_idle_sequences_padding_and_strides(K):
    c = make(10, [4, 0, 6, 0], 77, 2)
    compare(K, *c, max_nodes=9, stride=5)


def test_large_vocabulary(K):
    """Too large for fractions: the walk with integers of 2^-80 units."""
    V = 131071
    p, q, tokens, parents, indptr, u = make(11, [3, 5, 2, 4], V, 1, sharp=3.0)
    path, plen, nxt = run(K, p, q, tokens, parents, indptr, u, 5)
    unit = lambda row: [int(Fraction(float(x)) * 2 ** 80) for x in row]
    for b in range(4):
        a, z = indptr[b], indptr[b + 1]
        cur = int(path[b, plen[b] - 1])
        r = unit(p[a + cur])
        if cur + 1 < z - a:  # the next node of the chain was rejected
            r = [max(x - y, 0) for x, y in zip(r, unit(q[a + cur]))]
        t, run_, j = Fraction(float(u[a])) * sum(r), 0, -1
        while run_ <= t:
            j += 1
            run_ += r[j]
        assert nxt[b] == j
        for i in range(1, z - a):
            x = tokens[a + i]
            ok = float(u[a + i]) * float(q[a + i - 1, x]) < float(p[a + i - 1, x])
            assert ok == (i <= cur)
            if not ok:
                break


def test_edges_of_the_random_numbers(K):
    p, q, tokens, parents, indptr, u = make(12, [3] * 6, 40, 1)
    p[:, :5] = 0  # weight starts behind zeros: u = 0 takes the first token with any
    p[:, 35:] = 0  # and ends before zeros
    u[0::3] = [0.0, 0.0, 0.0] + [float(np.nextafter(np.float32(1), np.float32(0)))] * 3
    u[1::3] = [0.0, 1 - 2.0 ** -24] * 3
    compare(K, p, q, tokens, parents, indptr, u)
    compare(K, p, None, tokens, parents, indptr, u)


def test_draft_equal_to_the_target_accepts_everything(K):
    p, q, tokens, parents, indptr, u = make(13, [6, 6], 90, 1)
    assert compare(K, p, p.copy(), tokens, parents, indptr, u) == [6, 6]


def test_weightless_rows(K):
    """A row of zeros gives -1; a residual without weight falls back to the row."""
    p, q, tokens, parents, indptr, u = make(14, [1, 2, 2], 33, 1)
    p[0] = 0
    p[3] = 0
    p[3, 7] = 0.25       # all of the target's weight below the draft's
    q[3] = 0
    q[3, 7] = 1.0
    tokens[4] = 7
    u[4] = 0.9           # 0.9 * 1 >= 0.25: rejected, and nothing is left
    compare(K, p, q, tokens, parents, indptr, u)
    path, plen, nxt = run(K, p, q, tokens, parents, indptr, u, 2)
    assert nxt[0] == -1 and nxt[2] == 7 and plen[2] == 1


def test_values_outside_the_unit_interval_are_clamped(K):
    p, q, tokens, parents, indptr, u = make(15, [4, 4], 50, 1)
    bad_p, bad_q = p.copy(), q.copy()
    bad_p[0, 3], bad_p[1, 4], bad_q[2, 5] = np.nan, -1.0, np.nan
    p[0, 3] = p[1, 4] = q[2, 5] = 0
    a = run(K, bad_p, bad_q, tokens, parents, indptr, u, 4)
    b = run(K, p, q, tokens, parents, indptr, u, 4)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    inf = np.full((8, 50), np.inf, np.float32)
    path, plen, nxt = run(K, inf, None, tokens, parents, indptr, u, 4)
    assert np.all((nxt >= -1) & (nxt < 50))


def test_bad_parents_and_tokens_are_flagged_and_never_reached(K):
    for what, value in (("parents", 1), ("parents", 5), ("parents", -1), ("tokens", -1),
                        ("tokens", 60), ("tokens", 1 << 30)):
        p, q, tokens, parents, indptr, u = make(16, [4, 4], 60, 1)
        u[:] = 0.0  # everything possible is accepted
        arr = tokens if what == "tokens" else parents
        arr[1] = value
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        path, plen, nxt = run(K, p, q, tokens, parents, indptr, u, 4, err)
        assert K.k16v8_read_device_error(err) == K.DEVERR_TREE
        assert plen[0] == 1 and path[0].tolist() == [0, -1, -1, -1]
        assert plen[1] == 4


def test_bad_row_ranges_are_flagged(K):
    p, q, tokens, parents, indptr, u = make(17, [4, 4], 60, 1)
    for ip, bad in (([0, 4, 9], 1), ([-1, 4, 8], 0), ([0, 8, 4], 1), ([0, 8, 8], 0)):
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        path, plen, nxt = run(K, p, q, tokens, parents, np.asarray(ip, np.int32), u, 4, err)
        assert K.k16v8_read_device_error(err) == K.DEVERR_SEQLEN
        assert plen[bad] == 0 and nxt[bad] == -1 and np.all(path[bad] == -1)


def test_same_results_on_another_stream_and_in_a_graph(K):
    c = make(18, [8] * 20, 3001, 3)
    want = run(K, *c, 8)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run(K, *c, 8, stream=s)
    assert all(np.array_equal(x, y) for x, y in zip(want, got))
    p, q, tokens, parents, indptr, u = (to_dev(x) for x in c)
    path = torch.zeros((20, 8), dtype=torch.int32, device=dev())
    plen, nxt = (torch.zeros(20, dtype=torch.int32, device=dev()) for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.k16v8_tree_verify(p, q, tokens, parents, indptr, 8, u, path, plen, nxt)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(path.cpu().numpy(), want[0]) and np.array_equal(nxt.cpu().numpy(), want[2])


def test_binding_refuses_wrong_tensors(K):
    p, q, tokens, parents, indptr, u = (to_dev(x) for x in make(19, [4, 4], 60, 1))
    path = torch.zeros((2, 4), dtype=torch.int32, device=dev())
    plen, nxt = (torch.zeros(2, dtype=torch.int32, device=dev()) for _ in range(2))
    good = dict(target_probs=p, draft_probs=q, tokens=tokens, parents=parents, qo_indptr=indptr,
                max_nodes=4, uniforms=u, path=path, path_len=plen, next_token=nxt)
    K.k16v8_tree_verify(**good)
    for name, t in (("target_probs", p.half()), ("draft_probs", q[:, :59]), ("draft_probs", q.half()),
                    ("draft_probs", q[:1].expand(8, 60)), ("target_probs", p.t().contiguous().t()),
                    ("tokens", tokens.long()), ("parents", parents[:7]), ("qo_indptr", indptr[:2]),
                    ("uniforms", u.double()), ("path", path[:, :3]), ("path_len", plen.long()),
                    ("next_token", nxt[:1])):
        with pytest.raises(ValueError):
            K.k16v8_tree_verify(**{**good, name: t})


@pytest.mark.parametrize("V", [3, 129, 1023, 20001])
def test_rows_off_the_16_byte_grid(K, V):
    """Strides and starts that put the rows of p and q on different boundaries."""
    p, q, tokens, parents, indptr, u = make(V, [6, 3, 5], V, 3, near=0.8)
    want = run(K, p, q, tokens, parents, indptr, u, 6)
    for sp, op, sq, oq in ((1, 0, 2, 0), (0, 1, 0, 1), (3, 2, 1, 3), (0, 0, 0, 2)):
        def put(a, stride, off):
            flat = torch.full((a.shape[0] * (V + stride) + off + 8,), 0.5, device=dev())
            view = flat[off:off + a.shape[0] * (V + stride)].view(a.shape[0], V + stride)[:, :V]
            view.copy_(to_dev(a))
            return view
        path = torch.zeros((3, 6), dtype=torch.int32, device=dev())
        plen, nxt = (torch.zeros(3, dtype=torch.int32, device=dev()) for _ in range(2))
        K.k16v8_tree_verify(put(p, sp, op), put(q, sq, oq), to_dev(tokens), to_dev(parents),
                            to_dev(indptr), 6, to_dev(u), path, plen, nxt)
        for x, y in zip((path, plen, nxt), want):
            assert np.array_equal(x.cpu().numpy(), y)
