"""The error path of tree attention's bounded waits, reached without any
fault, as for the decode split and the prefill kernel: the test hook withholds
the keys of CTA 0's first tile (nothing issued, no arrival), so the wait for
them expires after a short limit.  The call must report K16V8_DEVERR_TIMEOUT,
let what is in flight land and return; rows of segments that CTA 0 has no part
of are complete, and the next call on the same stream and workspace is right."""
import time

import numpy as np
import pytest
import torch

from cases import dev, to_dev
from test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def parts_of_cta0(c):
    """Sequences with a tile in CTA 0's range (tiles of 128 positions, two units each for trees of
    more than 32 nodes; one range per SM)."""
    cost = [-(-int(L) // 128) * (2 if n > 32 else 1) * c.hkv if n else 0
            for L, n in zip(c.lens, c.nodes)]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    width = max(-(-sum(cost) // sms), 2 if c.max_nodes > 32 else 1)
    start = np.concatenate([[0], np.cumsum(cost)])
    return tuple(b for b in range(c.B) if start[b] < width)


@pytest.mark.parametrize("n", [6, 40])
@pytest.mark.parametrize("shape", ["one tile", "many tiles", "many pieces"])
def test_wait_expiry_reports_and_recovers(K, n, shape):
    if shape == "one tile":
        c = Case(1, [700, 300], [n, n], hkv=1)
    elif shape == "many tiles":
        c = Case(2, [6000, 2500, n], [n, 3, n], hkv=5)
    else:
        c = Case(3, [n + 20] * 90, [n] * 90, hkv=4)
    skip = parts_of_cta0(c)
    assert 0 in skip and len(skip) < c.B
    ws = torch.full((K.k16v8_tree_workspace_size(c.rows, c.B, c.max_nodes, c.hq, c.hkv, 128,
                                                 int(c.lens.max())),), 0, dtype=torch.uint8,
                    device=dev())
    out = torch.full((c.rows, c.hq, 128), 9.0, dtype=torch.float16, device=dev())
    lse = torch.full((c.rows, c.hq), 9.0, dtype=torch.float32, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    args = [to_dev(c.q), to_dev(c.indptr), c.max_nodes] + [
        to_dev(x) for x in (c.mask, c.kc, c.vc, c.vs, c.bt, c.lens)] + [
        int(c.lens.max()), c.scale, ws, out, lse, err]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    K.k16v8_paged_tree_attention_wait_test(*args)
    assert K.k16v8_read_device_error(err) == K.DEVERR_TIMEOUT  # the expired wait, and nothing else
    assert time.perf_counter() - t0 < 30.0
    c.check(out.cpu().numpy().astype(np.float64), lse.cpu().numpy(), skip=skip)
    err.zero_()
    out.fill_(9.0)
    lse.fill_(9.0)
    K.k16v8_paged_tree_attention(*args)
    assert K.k16v8_read_device_error(err) == 0
    c.check(out.cpu().numpy().astype(np.float64), lse.cpu().numpy())
