"""The speculative calls where a size changes how they work: batches that
leave a sequence of tree_verify two CTAs or one, vocabularies whose runs need
several rounds, the rotary write's wider units in every layout, and a plan of
tree attention that takes its sequences in several rounds."""
import numpy as np
import pytest
import torch

import test_gpu_rope_append
import test_gpu_tree_attention
import test_gpu_tree_verify
from cases import dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("batch", [39, 77, 100, 153, 200])
def test_verify_with_fewer_ctas_per_sequence(K, batch, draft):
    rng = np.random.default_rng(batch)
    nodes = [int(n) for n in rng.integers(0, 8, batch)]
    lens = test_gpu_tree_verify.compare(
        K, *test_gpu_tree_verify.make(batch, nodes, 45, 3, draft, near=0.9), max_nodes=8)
    assert min(lens) == 1 and max(lens) > 1


@pytest.mark.parametrize("V", [70001, 1 << 19])
@pytest.mark.parametrize("wide", [False, True])
def test_verify_large_vocabularies(K, V, wide):
    """A rejected child (a token without weight) leaves max(p - q, 0); u falls in the middle of a
    given token's share of it.  That share is 2^-21 of the sum at least, while the kernel's weights
    (2^-45 each), the sums here (64 bits) and u (2^-25) are off by less than 2^-23 of it together.
    `wide`: more sequences than two per SM, so each has one CTA; the rest are idle."""
    gen = torch.Generator(device=dev()).manual_seed(V)
    p = torch.softmax(torch.randn(8, V, generator=gen, device=dev()), -1)
    q = torch.softmax(p.log() + 0.7 * torch.randn(8, V, generator=gen, device=dev()), -1)
    p[:, 5], q[:, 5] = 0, 0.25
    nodes = [2, 1, 2, 2, 1]
    batch = 2 * sms() + 1 if wide else len(nodes)
    indptr = np.minimum(np.concatenate([[0], np.cumsum(nodes), np.full(batch - len(nodes), 8)]), 8)
    rng = np.random.default_rng(V)
    u, want = np.full(8, 0.5, np.float32), []
    for b, n in enumerate(nodes):
        r0 = int(indptr[b])
        r = p[r0].double().cpu().numpy()
        if n == 2:
            r = np.maximum(r - q[r0].double().cpu().numpy(), 0)
        run = np.cumsum(r)
        big = np.flatnonzero(r >= 2.0 ** -21 * run[-1])
        j = int(big[[0, -1, len(big) // 2, -2, int(rng.integers(len(big)))][b]])
        u[r0] = (run[j] - r[j] / 2) / run[-1]
        want.append(j)
    path = torch.zeros((batch, 2), dtype=torch.int32, device=dev())
    plen, nxt = (torch.zeros(batch, dtype=torch.int32, device=dev()) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_tree_verify(p, q, torch.full((8,), 5, dtype=torch.int32, device=dev()),
                        torch.zeros(8, dtype=torch.int32, device=dev()),
                        to_dev(indptr.astype(np.int32)), 2, to_dev(u), path, plen, nxt, err)
    assert K.k16v8_read_device_error(err) == 0
    assert plen.tolist() == [1] * len(nodes) + [0] * (batch - len(nodes))
    assert nxt.tolist() == want + [-1] * (batch - len(nodes))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,hq,hkv,rotary", [(1000, 40, 10, 128), (1003, 40, 10, 80), (2500, 8, 3, 112)])
def test_rope_on_full_grids(K, T, hq, hkv, rotary, dtype, interleaved):
    test_gpu_rope_append.run_and_check(K, T, T, hq, hkv, rotary, interleaved, dtype, 40000, pad=7)


@pytest.mark.parametrize("batch,hint", [(512, 32), (513, 32), (1500, 33), (8192, 32)])
def test_tree_attention_over_many_sequences(K, batch, hint):
    """Most are idle; trees stand at the ends and at the scan's borders."""
    rng = np.random.default_rng(batch)
    nodes = np.where(rng.random(batch) < 0.2, rng.integers(1, 4, batch), 0)
    nodes[[0, 1, 511, batch - 2, batch - 1]] = 3, hint, 4, 1, 5
    nodes[512:514] = 7
    lens = nodes + rng.integers(0, 140, batch) * (rng.random(batch) < 0.5)
    test_gpu_tree_attention.compare(
        K, test_gpu_tree_attention.Case(batch, lens, nodes, hkv=1, branch=3, max_nodes=hint))
