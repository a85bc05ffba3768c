"""Tree attention over long pieces: one CTA sums a whole context, so whatever
a weight loses by its fp16 form adds up over all of it.

Tolerance, per output row, as in test_gpu_tree_attention with the absolute
error of a small weight as the kernel holds it: weights are 2^7 times as large
as against the row's maximum, so one that is subnormal in fp16 is off by 2^-25
of 2^7 times a sum of at least 1, 2^-32 absolute; and with what long sums in
fp32 add: a row's sum takes L / 128 additions, off by 2^-24 each, its output
one accumulation per 16 positions, off by 2^-23 each (not rounded to nearest):
    |out - ref| <= (2 ds + 2^-18 + 2^-11 + L (2^-31 + 2^-27)) A + L 2^-32 max|v| + 2^-11 |ref| + 2^-25
    |lse - ref| <= ds + 2^-20 |ref| + 2^-18 + L 2^-31
(ds = 2^-17 sm_scale sum|q||k| + 2^-22 |s|, A = sum p|v|, both in 64 bits.)"""
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


def reference(q, k, v, scale):
    """q [rows, 128], k, v [L, 128] float64 on the GPU: out, lse and their bounds."""
    s = scale * (q @ k.t())
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    out, A = p @ v, p @ v.abs()
    ds = 2.0 ** -17 * scale * (q.abs() @ k.abs().t()).amax(-1) + 2.0 ** -22 * s.abs().amax(-1)
    L = len(k)
    rel = 2 * ds + 2.0 ** -18 + 2.0 ** -11 + L * (2.0 ** -31 + 2.0 ** -27)
    vmax = v.abs().nan_to_num(0.0).max()
    bound = rel[:, None] * A + L * 2.0 ** -32 * vmax + 2.0 ** -11 * out.abs() + 2.0 ** -25
    return out, lse, bound, ds + 2.0 ** -20 * lse.abs() + 2.0 ** -18 + L * 2.0 ** -31


@pytest.mark.parametrize("n", [5, 40])
@pytest.mark.parametrize("far", [0, 70000])
def test_dominant_scores_over_a_flat_tail(K, n, far):
    """Scores of a few keys 10 to 22 above a tail of 131,072 equal ones, whose share of the output
    would be lost or rounded by a third in weights of at most 1.  Every SM has a
    sequence of its own; all share the context's pages."""
    B = torch.cuda.get_device_properties(0).multi_processor_count
    L = 131072 + n
    pages = -(-L // 16)
    rng = np.random.default_rng(n)
    scale = float(np.float32(1 / np.sqrt(128)))
    gaps = np.linspace(10, 22, 4 * n).reshape(n, 4)
    q = np.zeros((n, 4, 128), np.float16)
    q[:, :, 0] = gaps
    k = torch.zeros((pages, 1, 16, 128), dtype=torch.float16)
    for pos in (far, far + 128):  # one for either slot of a narrow tree's tiles
        k[pos // 16, 0, pos % 16, 0] = 1 / scale
    v = torch.from_numpy(rng.uniform(100, 440, (pages, 1, 16, 128)).astype(np.float32))
    for pos in (far, far + 128):
        v[pos // 16, 0, pos % 16] = 0
    codes = v.to(torch.float8_e4m3fn)
    vs = np.array([3.5 / 448], np.float32)
    mask = np.full(B * n, (1 << n) - 1, np.int64)  # every node sees all of them
    indptr = np.arange(B + 1, dtype=np.int32) * n
    table = np.broadcast_to(np.arange(pages, dtype=np.int32), (B, pages))
    lens = np.full(B, L, np.int32)
    ws = torch.empty(K.k16v8_tree_workspace_size(B * n, B, n, 4, 1, 128, L), dtype=torch.uint8,
                     device=dev())
    out = torch.zeros((B * n, 4, 128), dtype=torch.float16, device=dev())
    lse = torch.zeros((B * n, 4), dtype=torch.float32, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_paged_tree_attention(to_dev(np.tile(q, (B, 1, 1))), to_dev(indptr), n, to_dev(mask),
                                 k.to(dev()), codes.view(torch.uint8).to(dev()), to_dev(vs),
                                 to_dev(table), to_dev(lens), L, scale, ws, out, lse, err)
    assert K.k16v8_read_device_error(err) == 0
    ref, ref_l, bound, bound_l = reference(
        to_dev(q.reshape(-1, 128)).double(), k.to(dev()).reshape(-1, 128)[:L].double(),
        codes.to(dev()).double().reshape(-1, 128)[:L] * float(vs[0]), scale)
    e = (out.double().view(B, 4 * n, 128) - ref).abs()
    assert torch.all(e <= bound), (float((e / ref.abs()).max()), float((e / bound).max()))
    assert torch.all((lse.double().view(B, 4 * n) - ref_l).abs() <= bound_l)


@pytest.mark.parametrize("n", [7, 50])
def test_one_long_context_in_pieces(K, n):
    """100,003 positions over all SMs, joined.  (A few of the random values lie beyond 464 and are
    NaN codes: every row sees them, and those dims are NaN in all.)"""
    hkv, L = 2, 100003
    pages = -(-L // 16)
    gen = torch.Generator(device=dev()).manual_seed(n)
    randn = lambda *s: torch.randn(s, generator=gen, device=dev())
    q, k = randn(n, 4 * hkv, 128).half(), randn(pages + 3, hkv, 16, 128).half()
    codes = (90 * randn(pages + 3, hkv, 16, 128)).to(torch.float8_e4m3fn)
    vs = torch.tensor([3.0 / 448, 4.0 / 448], device=dev())
    table = torch.randperm(pages + 3, generator=gen, device=dev())[:pages].to(torch.int32)[None]
    scale = float(np.float32(1 / np.sqrt(128)))
    mask = torch.tensor([(1 << i + 1) - 1 for i in range(n)], dtype=torch.int64, device=dev())
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev())
    ws = torch.empty(K.k16v8_tree_workspace_size(n, 1, n, 4 * hkv, hkv, 128, L), dtype=torch.uint8,
                     device=dev())
    out = torch.zeros((n, 4 * hkv, 128), dtype=torch.float16, device=dev())
    lse = torch.zeros((n, 4 * hkv), device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_paged_tree_attention(q, i32(0, n), n, mask, k, codes.view(torch.uint8), vs, table, i32(L),
                                 L, scale, ws, out, lse, err)
    assert K.k16v8_read_device_error(err) == 0
    rows = table[0].long()
    for g in range(hkv):
        kg = k[rows, g].reshape(-1, 128)[:L].double()
        vg = codes.float()[rows, g].reshape(-1, 128)[:L].double() * vs[g].double()
        for i in range(n):  # a chain: node i sees all before it
            end = L - n + i + 1
            ref, ref_l, bound, bound_l = reference(q[i, 4 * g:4 * g + 4].double(), kg[:end], vg[:end],
                                                   scale)
            got = out[i, 4 * g:4 * g + 4].double()
            assert torch.equal(got.isnan(), ref.isnan()) and not got.isnan().all()
            assert torch.all(((got - ref).abs() <= bound) | ref.isnan())
            assert torch.all((lse[i, 4 * g:4 * g + 4].double() - ref_l).abs() <= bound_l)
