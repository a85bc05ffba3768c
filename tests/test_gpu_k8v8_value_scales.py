"""Attention over the K8/V8 cache where pages of unlike value scales share a row:
a page of large scale must not cost the others' weights their bits.  Held to a
bound per dim, in which a position counts with its own value (unlike
k8v8_ref.check_attention, which takes the row's largest for all)."""
import math

import numpy as np
import pytest
import torch

import k8v8_ref as R
from cases import dev, to_dev

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)
L, PAGES, HKV = 8000, 500, 2
BIG, SMALL = 2.0 ** 7, 2.0 ** -15  # the ends of the scales' range


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def cache_of(kind, big, large, small):
    """One sequence: position 2,003 scores 7.07 above a flat tail, so each position of
    the tail has 2^-10.2 of its weight and all together seven times it.  The pages
    `big` have the larger value scale and either a weight of e^-39.6 of the tail's, or
    the tail's and no value in the upper dims."""
    rng = np.random.default_rng(len(big))
    table = rng.permutation(PAGES + 3)[:PAGES].astype(np.int32)[None]
    kc = np.zeros((PAGES + 3, HKV, 16, 128), np.uint8)
    vc = R.encode(np.abs(R.TABLE[R.codes(rng, PAGES + 3, HKV, 16, 128)]))
    sc = np.full((PAGES + 3, HKV, 2), 2.0 ** -6, np.float32)
    sc[..., 1] = small
    kc[table[0, 2003 // 16], :, 2003 % 16] = R.encode(np.full(128, 40.0))
    at = table[0, big]
    sc[at, :, 1] = large
    if kind == "no weight":
        kc[at] = R.encode(np.full(128, -224.0))
    else:
        vc[at, :, :, 64:] = 0
    return table, kc, vc, sc


def reference(n, causal, kc, vc, sc, table):
    """(out, its bound, lse, its bound) of n rows of queries 1.0, which differ in what
    they see."""
    pg = table[0]
    k, v = (R.TABLE[c[pg]].transpose(0, 2, 1, 3).reshape(-1, HKV, 128) *
            np.repeat(sc[pg][..., i].astype(np.float64), 16, 0)[..., None] for i, c in enumerate((kc, vc)))
    out, bound = np.zeros((2, n, HKV, 128))
    lse = np.zeros((n, HKV))
    # scores, exponentials and the output as in k8v8_ref.check_attention; a weight in
    # fp16 is off by 2^-11 of it, or where that is more by 2^-32 of the row's largest,
    # and never by more than itself; times its own value
    dots = np.abs(k).sum(-1).max() * SCALE
    score = 2.0 ** -19 * dots + 2.0 ** -23 * (10 + 2 * dots + 16)  # (an LSE below 10)
    w = np.expm1(2 * score) + 2.0 ** -20
    for r in range(n):
        seen = L - n + r + 1 if causal else L
        s = k[:seen].sum(-1) * float(np.float32(SCALE))
        p = np.exp(s - s.max(0))
        lse[r] = s.max(0) + np.log(p.sum(0))
        p /= p.sum(0)
        out[r] = np.einsum("jh,jhd->hd", p, v[:seen])
        size = np.einsum("jh,jhd->hd", p, np.abs(v[:seen]))
        lost = np.minimum(p, 2.0 ** -32 * p.max(0))
        bound[r] = ((2.0 ** -11 + w) * size + 2.0 ** -11 * np.abs(out[r]) + 2.0 ** -25 +
                    np.einsum("jh,jhd->hd", lost, np.abs(v[:seen])))
    assert np.all(np.abs(lse) < 10)
    return out, bound, lse, score + 2.0 ** -20 + 10 * 2.0 ** -22


BIG_PAGES = {"every 16th": np.arange(0, PAGES, 16), "first": np.array([0]), "last": np.array([PAGES - 1]),
             "ends of runs": np.arange(15, PAGES, 16)}


@pytest.mark.parametrize("call", ["decode", "prefill", "cross"])
@pytest.mark.parametrize("kind", ["no weight", "other dims"])
@pytest.mark.parametrize("scales", [(BIG, SMALL), (2.0 ** -3, SMALL), (BIG, 2.0 ** -9)])
@pytest.mark.parametrize("where", list(BIG_PAGES))
def test_a_large_value_scale_costs_the_other_pages_nothing(K, call, kind, scales, where):
    # decode: 64 rows over the same pages, some 26 of them to a warp
    n, causal = (1, False) if call == "decode" else (5, call == "prefill")
    table, kc, vc, sc = cache_of(kind, BIG_PAGES[where], *scales)
    want, bound, lse, lse_bound = reference(n, causal, kc, vc, sc, table)
    assert np.all(bound[..., 64:] < 2.0 ** -8 * np.abs(want[..., 64:]))  # it tells something
    rows = 64 if call == "decode" else n
    q = torch.ones((rows, 4 * HKV, 128), dtype=torch.float16, device=dev())
    out, got_lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    cache = [to_dev(x) for x in (kc, vc, sc)]
    if call == "decode":
        ws = torch.empty(K.k16v8_decode_workspace_size_k8v8(rows, 4 * HKV, 128), dtype=torch.uint8, device=dev())
        K.k16v8_paged_decode_attention_k8v8(q, *cache, to_dev(np.repeat(table, rows, 0)),
                                            to_dev(np.full(rows, L, np.int32)), SCALE, ws, out, got_lse,
                                            dev_error=err)
    else:
        ws = torch.empty(K.k16v8_attention_workspace_size_k8v8(n, 4 * HKV, HKV, 128), dtype=torch.uint8,
                         device=dev())
        attend = K.k16v8_paged_prefill_attention_k8v8 if causal else K.k16v8_paged_cross_attention_k8v8
        attend(q, to_dev(np.array([0, n], np.int32)), n, *cache, to_dev(table),
               to_dev(np.array([L], np.int32)), L, SCALE, ws, out, got_lse, dev_error=err)
    assert K.k16v8_read_device_error(err) == 0
    e = np.abs(out.cpu().numpy().astype(np.float64).reshape(rows, HKV, 4, 128) - want[:, :, None])
    assert np.all(e <= bound[:, :, None]), (e / bound[:, :, None]).max()
    assert np.abs(got_lse.cpu().numpy().reshape(rows, HKV, 4) - lse[..., None]).max() <= lse_bound
