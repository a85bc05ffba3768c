"""The speculative step as it is used: several layers, the trees written,
attended, verified and compacted, and the next step over the result."""
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


LAYERS, HKV, D, B, NODES, MAX_LEN, V = 3, 2, 128, 4, 12, 200, 301


class Model:
    """Caches of LAYERS layers and an unpaged float64 copy of every row."""

    def __init__(self, seed=0):
        from fp8_paged_kv_append_gb300.rope import rope_inv_freq
        from fp8_paged_kv_append_gb300.tree_step import MultiLayerTreeDecode
        from fp8_paged_kv_append_gb300.workloads import assign_pages
        self.rng = np.random.default_rng(seed)
        bt, P = assign_pages(np.random.Generator(np.random.PCG64(seed)), [MAX_LEN] * B)
        self.kc = [torch.zeros((P, HKV, 16, D), dtype=torch.float16, device=dev()) for _ in range(LAYERS)]
        self.vc = [torch.zeros((P, HKV, 16, D), dtype=torch.uint8, device=dev()) for _ in range(LAYERS)]
        self.vs = [to_dev((self.rng.uniform(3, 5, HKV) / 448).astype(np.float32)) for _ in range(LAYERS)]
        self.freq, self.factor = rope_inv_freq(96, scaling="yarn", factor=4.0, original_max_position=64)
        self.step = MultiLayerTreeDecode(self.kc, self.vc, self.vs, bt, B, NODES, MAX_LEN, 4 * HKV,
                                         self.freq, self.factor)
        self.bt = bt

    def rows(self, li, b, length):
        """K and V rows of a sequence as the cache holds them, float64."""
        pages = torch.from_numpy(self.bt[b, :-(-length // 16)].astype(np.int64)).to(dev())
        k = self.kc[li][pages].transpose(1, 2).reshape(-1, HKV, D)[:length].double().cpu().numpy()
        v = self.vc[li][pages].transpose(1, 2).reshape(-1, HKV, D)[:length].cpu()
        v = v.view(torch.float8_e4m3fn).to(torch.float64).numpy() * self.vs[li].double().cpu().numpy()[:, None]
        return k, v

    def inputs(self):
        n = self.step.rows
        t = lambda h: [to_dev(self.rng.standard_normal((n, h, D)).astype(np.float16)) for _ in range(LAYERS)]
        return t(4 * HKV), t(HKV), t(HKV)


def trees(rng):
    out = []
    for n in rng.integers(2, NODES + 1, B):
        out.append([-1] + [max(0, i - int(rng.integers(1, 4))) for i in range(1, n)])
    out[2] = []  # an idle sequence
    return out


def attend(model, li, b, q_rot, out, parents, base):
    """Every row of one sequence against float64 attention over the cache."""
    n = len(parents)
    k, v = model.rows(li, b, base + n)
    r0 = int(model.step.qo_indptr[b])
    for i in range(n):
        see = list(range(base))
        j = i
        while j >= 0:
            see.append(base + j)
            j = parents[j]
        for h in range(4 * HKV):
            q = q_rot[r0 + i, h].double().cpu().numpy()
            s = (k[see, h // 4] @ q) / np.sqrt(D)
            p = np.exp(s - s.max())
            ref = (p / p.sum()) @ v[see, h // 4]
            got = out[r0 + i, h].double().cpu().numpy()
            assert np.abs(got - ref).max() <= 4e-3 + 4e-3 * np.abs(ref).max()


def test_two_steps_with_a_captured_graph(K):
    m = Model()
    s, rng = m.step, m.rng
    n = s.rows
    qs, ks, vs = m.inputs()
    q_rot = torch.zeros((n, 4 * HKV, D), dtype=torch.float16, device=dev())
    outs = [torch.full((n, 4 * HKV, D), 9.0, dtype=torch.float16, device=dev()) for _ in range(LAYERS)]
    lens = [0, 17, 0, 100]
    # what the sequences hold before the first step
    for b, L in enumerate(lens):
        if L:
            pos = np.arange(L)
            slots = m.bt[b, pos // 16].astype(np.int64) * 16 + pos % 16
            for li in range(LAYERS):
                x = to_dev(rng.standard_normal((L, HKV, D)).astype(np.float16))
                K.k16v8_rope_kv_append(None, x, x, to_dev(pos.astype(np.int32)), s.inv_freq,
                                       to_dev(slots), m.vs[li], None, m.kc[li], m.vc[li],
                                       attn_factor=m.factor)
    for turn in range(2):
        par = trees(rng)
        s.set_trees(par, lens)
        if turn == 0:
            s.capture(qs, ks, vs, q_rot, outs)
        else:  # new inputs in the captured buffers
            for dst, src in zip((qs, ks, vs), m.inputs()):
                for d, x in zip(dst, src):
                    d.copy_(x)
        for o in outs:
            o.fill_(9.0)
        s.replay()
        assert s.check() == 0
        used = sum(len(p) for p in par)
        for li in range(LAYERS):
            assert torch.all(outs[li][used:] == 9.0)
            # the rotation is the same for every layer's buffer; redo the last one's query
            K.k16v8_rope_kv_append(qs[li], ks[li], vs[li], s.positions, s.inv_freq, s.slots, m.vs[li],
                                   q_rot, m.kc[li], m.vc[li], attn_factor=m.factor)
            for b in range(B):
                if par[b]:
                    attend(m, li, b, q_rot, outs[li], par[b], lens[b])
        # verify
        probs = torch.softmax(2 * torch.from_numpy(rng.standard_normal((n, V))).float(), -1).to(dev())
        tokens = torch.zeros(n, dtype=torch.int32, device=dev())
        flat = np.concatenate([np.maximum(p, 0) + int(s.qo_indptr[b]) for b, p in enumerate(par) if p])
        tokens[:used] = torch.multinomial(probs[to_dev(flat.astype(np.int64))], 1)[:, 0].to(torch.int32)
        u = torch.from_numpy(rng.random(n).astype(np.float32)).to(dev()) * 0.6
        s.verify(probs, probs, tokens, u)  # the draft is the target: first children are accepted
        path, plen = s.path.cpu().numpy(), s.path_len.cpu().numpy()
        for b in range(B):
            assert (plen[b] == 0) == (not par[b])
            for a, c in zip(path[b, :plen[b]], path[b, 1:plen[b]]):
                assert par[b][c] == a and c == par[b].index(a)
        # compact
        before = [[m.rows(li, b, lens[b] + len(par[b])) for b in range(B)] for li in range(LAYERS)]
        s.compact()
        assert s.check() == 0
        new = s.new_seq_lens.cpu().numpy()
        for b in range(B):
            assert new[b] == lens[b] + plen[b]
            for li in range(LAYERS):
                want = list(range(lens[b])) + [lens[b] + int(x) for x in path[b, :plen[b]]]
                got = m.rows(li, b, int(new[b]))
                for x, y in zip(got, before[li][b]):
                    assert np.array_equal(x, y[want])
        lens = [int(x) for x in new]


def test_host_checks(K):
    m = Model(1)
    s = m.step
    with pytest.raises(ValueError):
        s.set_trees([[-1]] * (B - 1), [0] * B)
    with pytest.raises(ValueError):
        s.set_trees([[-1] + [0] * NODES] + [[]] * (B - 1), [0] * B)
    with pytest.raises(ValueError):
        s.set_trees([[-1, 0]] + [[]] * (B - 1), [MAX_LEN - 1] + [0] * (B - 1))
    with pytest.raises(RuntimeError):
        s.replay()
    from fp8_paged_kv_append_gb300.tree_step import MultiLayerTreeDecode
    with pytest.raises(ValueError):
        MultiLayerTreeDecode(m.kc, m.vc, m.vs, m.bt, B, 65, MAX_LEN, 4 * HKV, m.freq)
