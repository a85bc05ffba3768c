"""Attention of drafted trees over the paged cache, against softmax attention
in 64 bits over the cached rows.

Tolerance, per output row.  ds bounds a score's error: 128 fp32 additions of
exact products, 2^-17 sm_scale sum|q||k|, and two fp32 roundings of the scaled
score, 2^-22 |s|.  A weight exp(s - lse) is then off by a relative
2 ds (score and sum) + 2^-18 (exponential, fp32 sums, the join), and its fp16
rounding adds 2^-11, or 2^-25 absolute where it is subnormal (weights are at
least 2^-25 of a sum of at least 1).  With A = sum p|v| (64 bits):
    |out - ref| <= (2 ds + 2^-18 + 2^-11) A + L 2^-25 max|v| + 2^-11 |ref| + 2^-25
    |lse - ref| <= ds + 2^-20 |ref| + 2^-18"""
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


def e4m3(codes):
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy()


class Case:
    def __init__(self, seed, lens, nodes, hkv=2, branch=2, spare_rows=0, k_boost=1.0, masks=None,
                 max_nodes=None):
        from fp8_paged_kv_append_gb300.tree_step import tree_masks
        from fp8_paged_kv_append_gb300.workloads import assign_pages
        rng = np.random.default_rng(seed)
        self.lens, self.nodes = np.asarray(lens, np.int32), np.asarray(nodes, np.int32)
        self.hkv, self.hq, self.B = hkv, 4 * hkv, len(lens)
        self.bt, self.P = assign_pages(np.random.Generator(np.random.PCG64(seed)), self.lens)
        self.indptr = np.concatenate([[0], np.cumsum(self.nodes)]).astype(np.int32)
        self.rows = int(self.indptr[-1]) + spare_rows
        self.q = rng.standard_normal((self.rows, self.hq, 128)).astype(np.float16)
        self.kc = (k_boost * rng.standard_normal((self.P, hkv, 16, 128))).astype(np.float16)
        v = torch.from_numpy(rng.standard_normal((self.P, hkv, 16, 128)) * 90)
        self.vc = v.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        self.vs = (rng.uniform(2, 5, hkv) / 448).astype(np.float32)
        self.scale = float(np.float32(1 / np.sqrt(128)))
        if masks is None:
            masks = np.concatenate([tree_masks([-1] + [max(0, i - int(rng.integers(1, branch + 1)))
                                                       for i in range(1, n)]) if n else
                                    np.zeros(0, np.int64) for n in self.nodes])
        self.mask = np.concatenate([masks, np.full(spare_rows, -1, np.int64)]).astype(np.int64)
        self.max_nodes = int(self.nodes.max()) if max_nodes is None else max_nodes

    def run(self, K, err=None, bt=None, lens=None, max_len=None, ws_fill=0xA5, lse=True, stream=None):
        max_len = int(self.lens.max()) if max_len is None else max_len
        n = K.k16v8_tree_workspace_size(self.rows, self.B, self.max_nodes, self.hq, self.hkv, 128,
                                        max_len)
        ws = torch.full((n,), ws_fill, dtype=torch.uint8, device=dev()) if n else None
        out = torch.full((self.rows, self.hq, 128), 9.0, dtype=torch.float16, device=dev())
        l = torch.full((self.rows, self.hq), 9.0, dtype=torch.float32, device=dev()) if lse else None
        K.k16v8_paged_tree_attention(
            to_dev(self.q), to_dev(self.indptr), self.max_nodes, to_dev(self.mask), to_dev(self.kc),
            to_dev(self.vc), to_dev(self.vs), to_dev(self.bt if bt is None else bt),
            to_dev(self.lens if lens is None else lens), max_len, self.scale, ws, out, l, err, stream)
        return out.cpu().numpy().astype(np.float64), None if l is None else l.cpu().numpy()

    def check(self, out, lse, skip=(), hidden=()):
        """hidden: positions (b, pos) that no row sees."""
        for b in range(self.B):
            n, L, r0 = int(self.nodes[b]), int(self.lens[b]), int(self.indptr[b])
            if n == 0 or b in skip:
                continue
            pages = self.bt[b, :-(-L // 16)]
            see = np.ones((n, L), bool)
            for i in range(n):
                w = int(self.mask[r0 + i]) & (1 << 64) - 1
                see[i, L - n:] = [(w >> j) & 1 for j in range(n)]
            for bb, pos in hidden:
                if bb == b:
                    see[:, pos] = False
            for h in range(self.hq):
                g = h // 4
                k = self.kc[pages, g].reshape(-1, 128)[:L].astype(np.float64)
                v = e4m3(self.vc[pages, g].reshape(-1, 128)[:L]) * float(self.vs[g])
                q = self.q[r0:r0 + n, h].astype(np.float64)
                for i in range(n):
                    m = see[i]
                    o, e = out[r0 + i, h], lse[r0 + i, h]
                    if not m.any():
                        assert np.all(o == 0) and e == -np.inf
                        continue
                    s = self.scale * (k[m] @ q[i])
                    ref_l = s.max() + np.log(np.exp(s - s.max()).sum())
                    p = np.exp(s - ref_l)
                    ref = p @ v[m]
                    A = p @ np.abs(v[m])
                    ds = (2.0 ** -17 * self.scale * (np.abs(k[m]) @ np.abs(q[i])).max()
                          + 2.0 ** -22 * np.abs(s).max())
                    vmax = np.nanmax(np.abs(v[m])) if np.isfinite(v[m]).any() else 0
                    bound = ((2 * ds + 2.0 ** -18 + 2.0 ** -11) * A + L * 2.0 ** -25 * vmax
                             + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25)
                    bad = np.isnan(ref)
                    assert np.array_equal(np.isnan(o), bad), (b, h, i)
                    err = np.abs(o - ref)
                    assert np.all(err[~bad] <= bound[~bad]), (b, h, i, err[~bad].max())
                    assert abs(e - ref_l) <= ds + 2.0 ** -20 * abs(ref_l) + 2.0 ** -18, (b, h, i)


def compare(K, case, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    out, lse = case.run(K, err, **kw)
    assert K.k16v8_read_device_error(err) == 0
    case.check(out, lse)
    return out, lse


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 31, 32, 33, 63, 64])
def test_node_counts(K, n):
    compare(K, Case(10 + n, [n, n + 1, n + 15, 200 + n], [n] * 4, branch=3))


@pytest.mark.parametrize("L", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 2049])
def test_lengths(K, L):
    n = min(L, 6)
    compare(K, Case(40 + L, [L], [n], hkv=1))
    compare(K, Case(41 + L, [L], [min(L, 40)], hkv=1, branch=5))


def test_ragged_batch_with_idle_sequences_and_spare_rows(K):
    c = Case(3, [300, 5, 17, 0, 900, 64, 33], [20, 5, 1, 0, 33, 0, 9], hkv=2, spare_rows=4, branch=4)
    out, lse = compare(K, c)
    end = int(c.indptr[-1])
    assert np.all(out[end:] == 9.0) and np.all(lse[end:] == 9.0)


@pytest.mark.parametrize("hint", [32, 64])
def test_many_short_sequences(K, hint):
    """Several sequences per SM, most within one KV tile."""
    rng = np.random.default_rng(60 + hint)
    nodes = rng.integers(0, 6, 150)
    nodes[::40] = (hint, 9, 0, hint - 3)
    lens = nodes + rng.integers(0, 160, 150)
    compare(K, Case(61, lens, nodes, hkv=10, max_nodes=hint))


@pytest.mark.parametrize("n", [1, 5, 16, 32])
def test_wide_hint_over_narrow_trees(K, n):
    compare(K, Case(62 + n, [n, 40 + n, 500, 1300], [n] * 4, branch=3, max_nodes=64))


def test_wide_and_narrow_trees_in_turn(K):
    compare(K, Case(67, [700, 90, 260, 1500, 129, 64], [40, 3, 64, 32, 0, 33], hkv=3, max_nodes=64))


@pytest.mark.parametrize("n", [20, 60])
def test_replayed_graphs_that_share_a_workspace(K, n):
    """Two captured calls of different batches, replayed in turn over new queries."""
    cases = [Case(70, [900, 30, 400], [n, 4, n], hkv=3), Case(71, [60, 2100], [n, 9], hkv=3)]
    size = max(K.k16v8_tree_workspace_size(c.rows, c.B, c.max_nodes, c.hq, c.hkv, 128,
                                           int(c.lens.max())) for c in cases)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    held = []
    for c in cases:
        t = [to_dev(x) for x in (c.q, c.indptr, c.mask, c.kc, c.vc, c.vs, c.bt, c.lens)]
        out = torch.zeros((c.rows, c.hq, 128), dtype=torch.float16, device=dev())
        lse = torch.zeros((c.rows, c.hq), dtype=torch.float32, device=dev())

        def call(c=c, t=t, out=out, lse=lse):
            K.k16v8_paged_tree_attention(t[0], t[1], c.max_nodes, *t[2:8], int(c.lens.max()), c.scale,
                                         ws, out, lse, err)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        held.append((c, t, out, lse, g))
    for turn in range(2):
        for c, t, out, lse, g in held:
            c.q = np.random.default_rng(72 + turn).standard_normal(c.q.shape).astype(np.float16)
            t[0].copy_(to_dev(c.q))
            out.fill_(9.0)
        for h in held:
            h[4].replay()
        assert K.k16v8_read_device_error(err) == 0
        for c, t, out, lse, g in held:
            c.check(out.cpu().numpy().astype(np.float64), lse.cpu().numpy())


def test_calls_on_two_streams_at_once(K):
    """Narrow and wide calls in flight together, a workspace each; every round the same bits.
    (The wide one's first sequence is shorter than its tree: flagged and skipped.)"""
    cases = [Case(80, [900, 30, 2400], [20, 4, 7], hkv=3), Case(81, [60, 2100, 333], [64, 9, 40], hkv=3)]
    streams = [torch.cuda.Stream() for _ in cases]
    held = []
    for c in cases:
        t = [to_dev(x) for x in (c.q, c.indptr, c.mask, c.kc, c.vc, c.vs, c.bt, c.lens)]
        size = K.k16v8_tree_workspace_size(c.rows, c.B, c.max_nodes, c.hq, c.hkv, 128, int(c.lens.max()))
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=dev())
        outs = [torch.zeros((c.rows, c.hq, 128), dtype=torch.float16, device=dev()) for _ in range(20)]
        lse = torch.zeros((c.rows, c.hq), dtype=torch.float32, device=dev())
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        held.append((c, t, ws, outs, lse, err))
    torch.cuda.synchronize()
    for i in range(20):
        for s, (c, t, ws, outs, lse, err) in zip(streams, held):
            K.k16v8_paged_tree_attention(t[0], t[1], c.max_nodes, *t[2:8], int(c.lens.max()), c.scale, ws,
                                         outs[i], lse, err, s)
    torch.cuda.synchronize()
    for (c, t, ws, outs, lse, err), flags, skip in zip(held, (0, K.DEVERR_SEQLEN), ((), (0,))):
        assert K.k16v8_read_device_error(err) == flags
        c.check(outs[0].cpu().numpy().astype(np.float64), lse.cpu().numpy(), skip=skip)
        for o in outs[1:]:
            assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))


@pytest.mark.parametrize("hkv", [1, 3, 10])
def test_heads(K, hkv):
    compare(K, Case(4, [100, 777], [11, 5], hkv=hkv))


def test_rows_that_see_nothing(K):
    """No prefix and empty masks; some rows see one node only."""
    masks = np.array([0, 1, 0, 4, 8, 0], np.int64)
    compare(K, Case(5, [6], [6], masks=masks))
    masks = np.zeros(40, np.int64)
    masks[5] = 1 << 39
    compare(K, Case(6, [40], [40], masks=masks))


def test_bits_beyond_the_tree_are_ignored(K):
    compare(K, Case(7, [50, 20], [3, 20], masks=np.full(23, -1, np.int64)))


def test_long_context_is_split(K):
    c = Case(8, [9001], [8], hkv=1, branch=3)
    assert K.k16v8_tree_workspace_size(8, 1, 8, 4, 1, 128, 9001) > 0
    compare(K, c)
    compare(K, Case(9, [6000, 4100], [64, 33], hkv=1, branch=3))


def test_length_hint_may_be_larger(K):
    c = Case(11, [130, 70], [6, 6])
    c.bt = np.pad(c.bt, ((0, 0), (0, 600)), constant_values=-1)
    compare(K, c, max_len=9000)


def test_stretched_scores(K):
    """Keys x8: scores to several hundred, the running max moves often."""
    compare(K, Case(12, [700, 90], [16, 40], k_boost=8.0))
    compare(K, Case(13, [700, 90], [4, 6], k_boost=8.0))


@pytest.mark.parametrize("n", [4, 8, 24, 50])
def test_nan_and_inf_stay_with_the_rows_that_see_them(K, n):
    """Children of node 0 do not see each other: a NaN key or value of one stays with it."""
    masks = np.array([1] + [1 | 1 << i for i in range(1, n)], np.int64)
    c = Case(14, [n + 37], [n], hkv=1, masks=masks)
    base = 37

    def put(cache, node, value):
        pos = base + node
        cache[c.bt[0, pos // 16], 0, pos % 16, 3] = value

    put(c.vc, 2, 0x7F)
    put(c.vc, n - 1, 0xFF)
    out, lse = compare(K, c)
    clean = [i for i in range(n) if i not in (2, n - 1)]
    assert np.isfinite(out[clean]).all() and np.isnan(out[2, :, 3]).all()
    put(c.kc, 1, np.nan)
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    out, lse = c.run(K, err)
    keep = [i for i in clean if i != 1]
    assert np.isfinite(out[keep]).all() and np.isnan(out[1]).all()


def test_poison_behind_the_last_position(K):
    for n in (6, 40):
        c = Case(15, [n + 5], [n], hkv=1)
        L = n + 5
        c.kc[c.bt[0, L // 16], 0, L % 16:] = np.nan
        c.vc[c.bt[0, L // 16], 0, L % 16:] = 0x7F
        out, _ = compare(K, c)
        assert np.isfinite(out).all()


def test_bad_page_ids_are_flagged_and_seen_by_no_row(K):
    for n in (6, 40):
        c = Case(16, [n + 100, 80], [n, 3])
        for bad in (-1, c.P, 1 << 30):
            bt = c.bt.copy()
            bt[0, 2] = bad
            err = torch.zeros(1, dtype=torch.int32, device=dev())
            out, lse = c.run(K, err, bt=bt)
            assert K.k16v8_read_device_error(err) == K.DEVERR_PAGE
            c.check(out, lse, hidden=[(0, p) for p in range(32, 48)])


def test_bad_lengths_are_flagged_and_skipped(K):
    c = Case(17, [100, 80, 60], [6, 6, 6])
    for bad in (5, -1, 101):  # fewer positions than nodes, negative, beyond the hint
        lens = c.lens.copy()
        lens[1] = bad
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        out, lse = c.run(K, err, lens=lens)
        assert K.k16v8_read_device_error(err) == K.DEVERR_SEQLEN
        assert np.all(out[6:12] == 9.0) and np.all(lse[6:12] == 9.0)
        c.check(out, lse, skip=(1,))
    d = Case(18, [100, 80], [6, 9], max_nodes=6)  # a tree beyond the hint
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    out, lse = d.run(K, err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_SEQLEN
    assert np.all(out[6:] == 9.0)
    d.check(out, lse, skip=(1,))


def test_row_ranges_outside_the_batch_are_flagged(K):
    c = Case(19, [100, 80], [6, 6])
    for indptr in ([0, 6, 13], [-1, 6, 12], [0, 12, 6]):
        good = c.indptr
        c.indptr = np.asarray(indptr, np.int32)
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        c.run(K, err)
        c.indptr = good
        assert K.k16v8_read_device_error(err) & K.DEVERR_SEQLEN


def test_without_lse_and_on_another_stream(K):
    c = Case(20, [500, 90], [12, 40])
    want, _ = c.run(K)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got, _ = c.run(K, lse=False, stream=s)
    assert np.array_equal(got, want)


def test_chain_agrees_with_prefill(K):
    """A chain is causal attention of the last n tokens."""
    for n in (5, 33, 64):
        c = Case(21, [n + 400], [n], branch=1)
        out, lse = c.run(K)
        o = torch.empty((n, c.hq, 128), dtype=torch.float16, device=dev())
        K.k16v8_paged_prefill_attention(to_dev(c.q), to_dev(c.indptr), n, to_dev(c.kc), to_dev(c.vc),
                                        to_dev(c.vs), to_dev(c.bt), to_dev(c.lens), c.scale, o)
        assert np.abs(out - o.cpu().numpy()).max() <= 4e-3


def test_binding_refuses_wrong_tensors(K):
    c = Case(22, [40], [4])
    good = dict(q=to_dev(c.q), qo_indptr=to_dev(c.indptr), max_nodes=4, tree_mask=to_dev(c.mask),
                k_cache=to_dev(c.kc), v_cache=to_dev(c.vc), v_scale=to_dev(c.vs),
                block_table=to_dev(c.bt), seq_lens=to_dev(c.lens), max_seq_len=40, sm_scale=0.1,
                workspace=torch.empty(K.k16v8_tree_workspace_size(4, 1, 4, 8, 2, 128, 40),
                                      dtype=torch.uint8, device=dev()),
                out=torch.empty((4, 8, 128), dtype=torch.float16, device=dev()))
    K.k16v8_paged_tree_attention(**good)
    for name in ("q", "qo_indptr", "tree_mask", "k_cache", "v_cache", "v_scale", "block_table",
                 "seq_lens", "out"):
        t = good[name]
        for bad in (t.double() if t.dtype != torch.float64 else t.float(), t.cpu(), t[..., None]):
            with pytest.raises((ValueError, IndexError)):
                K.k16v8_paged_tree_attention(**{**good, name: bad})
    for ws in (None, good["workspace"][:-1]):
        with pytest.raises(K.K16V8Error):
            K.k16v8_paged_tree_attention(**{**good, "workspace": ws})
    with pytest.raises(K.K16V8Error):
        K.k16v8_paged_tree_attention(**{**good, "max_nodes": 65})
    with pytest.raises(K.K16V8Error):
        K.k16v8_paged_tree_attention(**{**good, "max_seq_len": 49})
