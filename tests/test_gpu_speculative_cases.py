"""Keys that are infinite in hidden places, full-width trees on two streams at
once, and steps in which the target rejects drafted tokens."""
import numpy as np
import pytest
import torch

from cases import dev, to_dev
from test_gpu_tree_attention import Case, compare
from test_gpu_tree_step import B, D, HKV, LAYERS, V, Model, attend
from test_gpu_tree_verify import walk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("n", [4, 8, 24, 50])
def test_hidden_keys_do_not_reach_other_rows(K, n, value):
    """Children of node 0 do not see each other: an infinite or NaN key of one leaves every bit of
    the others' rows as it was."""
    masks = np.array([1] + [1 | 1 << i for i in range(1, n)], np.int64)
    for prefix in (37, 150):
        c = Case(n, [n + prefix], [n], hkv=1, masks=masks)
        want, want_l = compare(K, c)
        for node in (2, n - 1):
            pos = prefix + node
            c.kc[c.bt[0, pos // 16], 0, pos % 16, 7] = value
            c.kc[c.bt[0, pos // 16], 0, pos % 16, 8] = value
        out, lse = c.run(K)
        others = [i for i in range(n) if i not in (2, n - 1)]
        assert np.array_equal(out[others], want[others])
        assert np.array_equal(lse[others], want_l[others])


def test_full_width_trees_on_two_streams_at_once(K):
    cases = [Case(90, [900, 30, 2400], [20, 4, 7], hkv=3),
             Case(91, [80, 2100, 333, 64], [64, 9, 40, 64], hkv=3)]
    streams = [torch.cuda.Stream() for _ in cases]
    held = []
    for c in cases:
        t = [to_dev(x) for x in (c.q, c.indptr, c.mask, c.kc, c.vc, c.vs, c.bt, c.lens)]
        size = K.k16v8_tree_workspace_size(c.rows, c.B, c.max_nodes, c.hq, c.hkv, 128,
                                           int(c.lens.max()))
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=dev())
        outs = [torch.zeros((c.rows, c.hq, 128), dtype=torch.float16, device=dev())
                for _ in range(20)]
        lse = torch.zeros((c.rows, c.hq), dtype=torch.float32, device=dev())
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        held.append((c, t, ws, outs, lse, err))
    torch.cuda.synchronize()
    for i in range(20):
        for s, (c, t, ws, outs, lse, err) in zip(streams, held):
            K.k16v8_paged_tree_attention(t[0], t[1], c.max_nodes, *t[2:8], int(c.lens.max()), c.scale,
                                         ws, outs[i], lse, err, s)
    torch.cuda.synchronize()
    for c, t, ws, outs, lse, err in held:
        assert K.k16v8_read_device_error(err) == 0
        c.check(outs[0].cpu().numpy().astype(np.float64), lse.cpu().numpy())
        for o in outs[1:]:
            assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))


@pytest.mark.parametrize("draft", [True, False])
def test_steps_with_rejected_tokens(K, draft):
    """Draft rows that differ from the target's: paths and next tokens are those of the exact walk,
    the accepted rows move, and the next step attends over what they leave."""
    m = Model(2 + draft)
    s, rng = m.step, m.rng
    n = s.rows
    q_rot = torch.zeros((n, 4 * HKV, D), dtype=torch.float16, device=dev())
    outs = [torch.zeros((n, 4 * HKV, D), dtype=torch.float16, device=dev()) for _ in range(LAYERS)]
    lens, kinds = [0, 0, 0, 0], set()
    for turn in range(6):
        par = [[-1] + [max(0, i - int(rng.integers(1, 4))) for i in range(1, int(k))]
               for k in rng.integers(3, 12, B)]
        if turn == 2:
            par[1] = []
        s.set_trees(par, lens)
        qs, ks, vs = m.inputs()
        s.step(qs, ks, vs, q_rot, outs)
        assert s.check() == 0
        for b in range(B):
            if par[b]:  # (q_rot holds the last layer's queries)
                attend(m, LAYERS - 1, b, q_rot, outs[-1], par[b], lens[b])
        used = sum(len(p) for p in par)
        soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)
        target = soft(2 * rng.standard_normal((n, V)))
        drafted = soft(np.log(target) + rng.standard_normal((n, V)))
        indptr = s.qo_indptr.cpu().numpy()
        tokens = np.zeros(n, np.int32)
        for b, p in enumerate(par):
            for i in range(1, len(p)):
                row = drafted[indptr[b] + p[i]].astype(np.float64)
                tokens[indptr[b] + i] = rng.choice(V, p=row / row.sum())
        u = rng.random(n).astype(np.float32)
        s.verify(to_dev(target), to_dev(drafted) if draft else None, to_dev(tokens), to_dev(u))
        path, plen, nxt = (x.cpu().numpy() for x in (s.path, s.path_len, s.next_token))
        before = [[m.rows(li, b, lens[b] + len(par[b])) for b in range(B)] for li in range(LAYERS)]
        s.compact()
        assert s.check() == 0
        new = s.new_seq_lens.cpu().numpy()
        for b, p in enumerate(par):
            if not p:
                assert plen[b] == 0 and nxt[b] == -1 and new[b] == lens[b]
                continue
            r = slice(indptr[b], indptr[b] + len(p))
            want, tok = walk(target[r], drafted[r] if draft else None, tokens[r], np.array(p), u[r])
            assert path[b, :plen[b]].tolist() == want and nxt[b] == tok
            assert new[b] == lens[b] + len(want)
            kinds.add((len(want) > 1, len(want) < len(p), want != list(range(len(want)))))
            keep = list(range(lens[b])) + [lens[b] + i for i in want]
            for li in range(LAYERS):
                for x, y in zip(m.rows(li, b, int(new[b])), before[li][b]):
                    assert np.array_equal(x, y[keep])
        assert used == indptr[-1]
        lens = [int(x) for x in new]
    # accepted and rejected ones, and paths whose rows moved
    assert (False, True, False) in kinds and (True, True, True) in kinds
