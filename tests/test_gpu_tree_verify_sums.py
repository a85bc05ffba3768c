"""Verification of rows that do not sum to 1: by the formulas while the sums
fit, with an error and no result where they do not."""
import numpy as np
import pytest
import torch

from cases import dev, to_dev
from test_gpu_tree_verify import compare, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


@pytest.mark.parametrize("draft", [True, False])
def test_rows_that_sum_to_3(K, draft):
    p, q, tokens, parents, indptr, u = make(1, [9, 6, 12, 1], 60, 3, draft, sharp=0.5, near=1.0)
    p, q = np.minimum(p * np.float32(3), 1), None if q is None else np.minimum(q * np.float32(1.5), 1)
    compare(K, p, q, tokens, parents, indptr, u)


def star(children, V, p_each, q_each, seed=0):
    """Node 0 with children whose token has no weight (so each is rejected) and all of the draft's
    row; the other tokens have p_each and q_each of the two rows."""
    rng = np.random.default_rng(seed)
    n = children + 1
    p = np.full((n, V), p_each, np.float32)
    q = np.full((n, V), q_each, np.float32)
    p[:, V - 1], q[:, V - 1] = 0, 1
    return (p, q, np.full(n, V - 1, np.int32), np.array([-1] + [0] * children, np.int32),
            rng.random(n).astype(np.float32))


def join(trees):
    p, q, tokens, parents, u = (np.concatenate(x) for x in zip(*trees))
    return p, q, tokens, parents, np.concatenate([[0], np.cumsum([len(t[2]) for t in trees])]).astype(
        np.int32), u


def test_masses_that_add_up_to_64(K):
    """Rows that sum to 8: the Z of 8 rejected children are 1 + 7 * 8 = 57, of 9 they are 65."""
    good, bad = star(8, 17, 0.5, 0.0), star(9, 17, 0.5, 0.0)
    compare(K, *join([good]))
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    c = join([good, bad, good])
    path, plen, nxt = run(K, *c, 10, err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_PROBS
    assert plen.tolist() == [1, 0, 1] and nxt[1] == -1 and np.all(path[1] == -1)
    assert nxt[0] == nxt[2] and 0 <= nxt[0] < 16


def test_masses_beyond_the_integers_high_part(K):
    """Rows that sum to 500 and 40 rejected children: 19,501, where every token's weight would be
    0.78 less."""
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    path, plen, nxt = run(K, *join([star(40, 501, 1.0, 4e-5)]), 41, err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_PROBS
    assert plen[0] == 0 and nxt[0] == -1 and np.all(path == -1)


@pytest.mark.parametrize("trees", [1, 160])
def test_largest_vocabulary_of_ones(K, trees):
    """2^19 weights of 1 add up to 2^63 units; one fewer fits."""
    V = 1 << 19
    p = torch.ones(1, V, device=dev())
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev())
    indptr = torch.arange(trees + 1, dtype=torch.int32, device=dev()).clamp_(max=1)  # the rest are idle
    path = torch.zeros((trees, 1), dtype=torch.int32, device=dev())
    plen, nxt = torch.zeros(trees, dtype=torch.int32, device=dev()), torch.zeros(
        trees, dtype=torch.int32, device=dev())
    for zero, want, flags in ((False, -1, K.DEVERR_PROBS), (True, 262143, 0)):
        if zero:
            p[0, -1] = 0
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        K.k16v8_tree_verify(p, None, i32(0), i32(-1), indptr, 1, torch.full((1,), 0.5, device=dev()),
                            path, plen, nxt, err)
        assert K.k16v8_read_device_error(err) == flags
        assert int(nxt[0]) == want and int(plen[0]) == (0 if flags else 1)
