"""The move of accepted rows: every byte of every layer's cache against a
plain copy of the rows (read all, then write)."""
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


def make(seed, lens, nodes, paths, layers, hkv, max_nodes=None, spare=2):
    from fp8_paged_kv_append_gb300.workloads import assign_pages
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    need = int(sum(-(-int(x) // 16) for x in lens))
    bt, P = assign_pages(np.random.Generator(np.random.PCG64(seed)), lens, need + spare)
    ks = [rng.integers(0, 1 << 16, (P, hkv, 16, 128)).astype(np.uint16) for _ in range(layers)]
    vs = [rng.integers(0, 256, (P, hkv, 16, 128)).astype(np.uint8) for _ in range(layers)]
    indptr = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    max_nodes = max_nodes or max(max(nodes), 1)
    path = np.full((len(lens), max_nodes), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    plen = np.array([len(p) for p in paths], np.int32)
    return dict(lens=lens, bt=bt, P=P, ks=ks, vs=vs, indptr=indptr, path=path, plen=plen)


def moved(c, skip=()):
    ks, vs, new = [x.copy() for x in c["ks"]], [x.copy() for x in c["vs"]], c["lens"].copy()
    for b in range(len(c["lens"])):
        if b in skip:
            continue
        base = int(c["lens"][b]) - int(c["indptr"][b + 1] - c["indptr"][b])
        m = int(c["plen"][b])
        for j in range(m):
            s, d = base + int(c["path"][b, j]), base + j
            ps, pd = c["bt"][b, s // 16], c["bt"][b, d // 16]
            for new_c, old in ((ks, c["ks"]), (vs, c["vs"])):
                for x, y in zip(new_c, old):
                    x[pd, :, d % 16] = y[ps, :, s % 16]
        new[b] = base + m
    return ks, vs, new


def run(K, c, err=None, bt=None, want_lens=True, stream=None):
    ks = [to_dev(x.view(np.int16)).view(torch.float16) for x in c["ks"]]
    vs = [to_dev(x) for x in c["vs"]]
    new = torch.full((len(c["lens"]),), 777, dtype=torch.int32, device=dev()) if want_lens else None
    K.k16v8_kv_compact(K.layer_pointers(ks), K.layer_pointers(vs), c["P"], ks[0].shape[1], 128,
                       to_dev(c["bt"] if bt is None else bt), to_dev(c["lens"]), to_dev(c["indptr"]),
                       to_dev(c["path"]), to_dev(c["plen"]), new, err, stream)
    torch.cuda.synchronize()
    return ([x.view(torch.int16).cpu().numpy().view(np.uint16) for x in ks],
            [x.cpu().numpy() for x in vs], None if new is None else new.cpu().numpy())


def same(got, want):
    for g, w in zip(got[0] + got[1], want[0] + want[1]):
        assert np.array_equal(g, w)
    if got[2] is not None:
        assert np.array_equal(got[2], want[2])


@pytest.mark.parametrize("layers,hkv", [(1, 1), (3, 2), (7, 10)])
def test_paths_of_every_kind(K, layers, hkv):
    rng = np.random.default_rng(layers)
    nodes = [1, 5, 64, 64, 33, 16, 8, 0, 20]
    paths = [[0], [0, 1, 2, 3, 4], list(range(64)), [0] + list(range(32, 64)), [0, 3, 17, 32],
             [15], [], [], sorted(rng.permutation(20)[:9].tolist())]
    lens = [1, 100, 64, 203, 40, 16, 8, 31, 45]
    c = make(layers, lens, nodes, paths, layers, hkv)
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    got = run(K, c, err)
    assert K.k16v8_read_device_error(err) == 0
    same(got, moved(c))


@pytest.mark.parametrize("seed", range(4))
def test_random_paths(K, seed):
    rng = np.random.default_rng(seed)
    B = 30
    nodes = rng.integers(1, 65, B)
    paths = [sorted(rng.permutation(int(n))[:int(rng.integers(0, n + 1))].tolist()) for n in nodes]
    lens = nodes + rng.integers(0, 60, B)
    c = make(seed, lens, nodes, paths, 2, 3, max_nodes=64)
    same(run(K, c), moved(c))
    same(run(K, c, want_lens=False), moved(c))


def test_bad_paths_and_lengths_are_flagged_and_left_alone(K):
    for path, plen in (([0, 2, 2], 3), ([3, 1], 2), ([0, 9], 2), ([-1, 0], 2), ([0], 99), ([0], -1)):
        c = make(5, [50, 40], [9, 9], [[0, 2], [0, 3, 5]], 2, 2)
        c["path"][0, :len(path)] = path
        c["plen"][0] = plen
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        got = run(K, c, err)
        assert K.k16v8_read_device_error(err) == K.DEVERR_TREE
        same(got, moved(c, skip=(0,)))
    for lens0 in (8, 10 ** 6, -3):  # fewer positions than nodes, beyond the table, negative
        c = make(6, [50, 40], [9, 9], [[0, 2], [0, 3, 5]], 2, 2)
        c["lens"][0] = lens0
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        got = run(K, c, err)
        assert K.k16v8_read_device_error(err) == K.DEVERR_SEQLEN
        same(got, moved(c, skip=(0,)))
    c = make(7, [50, 40], [9, 9], [[0, 2], [0, 3, 5]], 2, 2)
    c["indptr"][:] = [0, 9, 40]  # more nodes than a path holds
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    got = run(K, c, err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_SEQLEN
    same(got, moved(c, skip=(1,)))


def test_bad_page_ids_are_flagged_and_not_followed(K):
    c = make(8, [48, 40], [32, 9], [[0, 20], [0, 3, 5]], 2, 2)
    for bad in (-1, c["P"], 1 << 30):
        bt = c["bt"].copy()
        bt[0, 2] = bad  # holds node 20
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        got = run(K, c, err, bt=bt)
        assert K.k16v8_read_device_error(err) == K.DEVERR_PAGE
        d = dict(c, plen=np.array([1, 3], np.int32))
        ks, vs, new = moved(d)
        new[0] = 16 + 2
        same(got, (ks, vs, new))


def test_another_stream_and_a_graph(K):
    c = make(9, [50, 40], [9, 9], [[0, 2, 7], [0, 3, 5]], 4, 2)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        same(run(K, c, stream=s), moved(c))
    # captured once, replayed over other paths in the same buffers
    start = [to_dev(x.view(np.int16)).view(torch.float16) for x in c["ks"]], [to_dev(x) for x in c["vs"]]
    ks, vs = [[x.clone() for x in xs] for xs in start]
    ptrs = K.layer_pointers(ks), K.layer_pointers(vs)
    bt, lens, indptr, path, plen = (to_dev(c[x]) for x in ("bt", "lens", "indptr", "path", "plen"))
    new = torch.zeros(2, dtype=torch.int32, device=dev())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.k16v8_kv_compact(*ptrs, c["P"], 2, 128, bt, lens, indptr, path, plen, new)
    for paths in ([[0, 2, 7], [0, 3, 5]], [[0, 1], [0, 8]], [[4], [0, 1, 2, 3, 6, 7, 8]]):
        for dst, src in zip(ks + vs, start[0] + start[1]):
            dst.copy_(src)
        d = make(9, [50, 40], [9, 9], paths, 4, 2)
        path.copy_(to_dev(d["path"]))
        plen.copy_(to_dev(d["plen"]))
        g.replay()
        torch.cuda.synchronize()
        same(([x.view(torch.int16).cpu().numpy().view(np.uint16) for x in ks],
              [x.cpu().numpy() for x in vs], new.cpu().numpy()), moved(d))


def test_bad_layer_addresses_are_flagged_and_not_followed(K):
    c = make(11, [50, 40], [9, 9], [[0, 2, 7], [0, 3, 5]], 3, 2)
    ks = [to_dev(x.view(np.int16)).view(torch.float16) for x in c["ks"]]
    vs = [to_dev(x) for x in c["vs"]]
    kp, vp = K.layer_pointers(ks), K.layer_pointers(vs)
    kp[0] = 0
    vp[2] += 8
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_kv_compact(kp, vp, c["P"], 2, 128, to_dev(c["bt"]), to_dev(c["lens"]), to_dev(c["indptr"]),
                       to_dev(c["path"]), to_dev(c["plen"]), None, err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_PAGE
    want = moved(c)
    for li in range(3):
        k, v = (want[0][li], want[1][li]) if li == 1 else (c["ks"][li], c["vs"][li])
        assert np.array_equal(ks[li].view(torch.int16).cpu().numpy().view(np.uint16), k)
        assert np.array_equal(vs[li].cpu().numpy(), v)


def test_binding_refuses_wrong_tensors(K):
    c = make(10, [50], [9], [[0, 2]], 1, 2)
    kp = torch.zeros(1, dtype=torch.int64, device=dev())
    good = dict(k_ptrs=kp, v_ptrs=kp, num_pages=c["P"], num_kv_heads=2, head_dim=128,
                block_table=to_dev(c["bt"]), seq_lens=to_dev(c["lens"]), qo_indptr=to_dev(c["indptr"]),
                path=to_dev(c["path"]), path_len=to_dev(c["plen"]))
    for name, t in (("k_ptrs", kp.int()), ("v_ptrs", kp.repeat(2)), ("block_table", to_dev(c["bt"]).long()),
                    ("seq_lens", to_dev(c["lens"]).long()), ("qo_indptr", to_dev(c["indptr"][:1])),
                    ("path", to_dev(c["path"])[:, ::2]), ("path_len", to_dev(c["plen"]).long())):
        with pytest.raises(ValueError):
            K.k16v8_kv_compact(**{**good, name: t})
    with pytest.raises(K.K16V8Error):
        K.k16v8_kv_compact(**good, new_seq_lens=good["seq_lens"])
