"""The K8/V8 calls at the ends of their ranges: no pages at all, the largest
batch, pages whose addresses pass 32 bits, and calls that overlap on two streams."""
import math

import numpy as np
import pytest
import torch

import k8v8_ref as R
from cases import dev, to_dev

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def empty(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device=dev())


def i32(values):
    return to_dev(np.asarray(values, np.int32))


def attend(K, name, q, cache, table, lens, max_q=None, indptr=None, ws=None, stream=None):
    """(out, lse) of the decode call (indptr None) or of prefill or cross attention."""
    hq = q.shape[1]
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    if indptr is None:
        ws = empty(K.k16v8_decode_workspace_size_k8v8(len(lens), hq, 128)) if ws is None else ws
        K.k16v8_paged_decode_attention_k8v8(q, *cache, table, lens, SCALE, ws, out, lse, dev_error=err,
                                            stream=stream)
    else:
        ws = empty(K.k16v8_attention_workspace_size_k8v8(max_q, hq, hq // 4, 128)) if ws is None else ws
        getattr(K, name)(q, indptr, max_q, *cache, table, lens, table.shape[1] * 16, SCALE, ws, out, lse,
                         dev_error=err, stream=stream)
    return out, lse, err


def test_no_pages(K):
    """Tables without a column: nothing is cached, nothing may be written."""
    B, hkv = 3, 2
    table = empty(B, 0, dtype=torch.int32)
    cache = [torch.full((2, hkv, 16, 128), 0x7F, dtype=torch.uint8, device=dev()) for _ in range(2)]
    cache.append(torch.ones((2, hkv, 2), device=dev()))
    q = torch.randn((B, 8, 128), device=dev()).half()
    for indptr in (None, i32([0, 2, 2, 3])):
        out, lse, err = attend(K, "k16v8_paged_cross_attention_k8v8", q, cache, table, i32([0] * B), 2, indptr)
        assert K.k16v8_read_device_error(err) == 0
        assert torch.all(out == 0) and torch.all(lse == -math.inf)
    kv = torch.randn((4, hkv, 128), device=dev()).half()
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    qo = torch.full((4, 8, 128), 9.0, dtype=torch.float16, device=dev())
    for indptr, flags in (([0, 0, 0, 0], 0), ([0, 0, 2, 2], K.DEVERR_SEQLEN)):
        K.k16v8_rope_kv_append_k8v8(torch.randn((4, 8, 128), device=dev()).half(), kv, kv, i32(indptr), None,
                                    None, None, table, i32([0] * B), qo, *cache, dev_error=err)
        assert K.k16v8_read_device_error(err) == flags
    assert torch.all(qo == 9.0) and torch.all(cache[0] == 0x7F) and torch.all(cache[2] == 1)


def test_largest_batch(K):
    rng = np.random.default_rng(0)
    B = 8192
    lens = rng.integers(0, 20, B)
    table, kc, vc, sc = R.poisoned_pool(rng, lens, 1)
    q = rng.standard_normal((B, 4, 128)).astype(np.float16)
    cache = [to_dev(x) for x in (kc, vc, sc)]
    want = R.attention(q.astype(np.float64), kc, vc, sc, table, lens, [1] * B, SCALE, False)
    for indptr in (None, i32(np.arange(B + 1))):
        out, lse, err = attend(K, "k16v8_paged_cross_attention_k8v8", to_dev(q), cache, to_dev(table), i32(lens),
                               1, indptr)
        assert K.k16v8_read_device_error(err) == 0
        R.check_attention(out.cpu().numpy(), lse.cpu().numpy(), want)


def test_pages_beyond_32_bits(K):
    """A pool of 4.5 GB on either side: the last pages are written and read like the
    first ones."""
    hkv, P, n = 2, (9 << 29) // (2 * 2048), 70
    kc, vc = empty(P, hkv, 16, 128), empty(P, hkv, 16, 128)
    sc = torch.full((P, hkv, 2), math.nan, device=dev())
    rng = np.random.default_rng(1)
    pages = np.concatenate([P - 1 - rng.permutation(4), [0]]).astype(np.int32)
    for x in (kc, vc):
        x[to_dev(pages.astype(np.int64))] = 0x7F
    x = torch.from_numpy(rng.standard_normal((n, 8 + 2 * hkv, 128)).astype(np.float16)).to(dev())
    q = empty(n, 8, 128, dtype=torch.float16)
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    table, lens, indptr = to_dev(pages[None]), i32([n]), i32([0, n])
    K.k16v8_rope_kv_append_k8v8(x[:, :8], x[:, 8:8 + hkv], x[:, 8 + hkv:], indptr, None, None, None, table, lens,
                                q, kc, vc, sc, dev_error=err)
    assert K.k16v8_read_device_error(err) == 0
    assert torch.equal(q, x[:, :8])
    # the same few pages as a pool of their own
    at = to_dev(pages.astype(np.int64))
    hk, hv, hs = kc[at].cpu().numpy(), vc[at].cpu().numpy(), sc[at].cpu().numpy()
    ht = np.arange(len(pages), dtype=np.int32)[None]
    for i, (codes, rows) in enumerate(((hk, x[:, 8:8 + hkv]), (hv, x[:, 8 + hkv:]))):
        rows = rows.double().cpu().numpy()
        held = (R.TABLE[codes] * hs[:, :, i, None, None]).transpose(0, 2, 1, 3).reshape(-1, hkv, 128)[:n]
        assert np.all(np.abs(held - rows) <= 2.0 ** -4 * np.abs(rows) + 2.0 ** -10 * hs[:, :, i].max())
    for name, ip, rows, counts in (("", None, q[-1:], [1]), ("k16v8_paged_prefill_attention_k8v8", indptr, q, [n]),
                                   ("k16v8_paged_cross_attention_k8v8", indptr, q, [n])):
        out, lse, err = attend(K, name, rows.contiguous(), (kc, vc, sc), table, lens, n, ip)
        assert K.k16v8_read_device_error(err) == 0
        R.check_attention(out.cpu().numpy(), lse.cpu().numpy(),
                          R.attention(rows.double().cpu().numpy(), hk, hv, hs, ht, [n], counts, SCALE,
                                      "prefill" in name))


def test_overlapping_calls(K):
    """Two streams, a workspace each, calls of every kind at once: the results are
    those of the calls one after another."""
    rng = np.random.default_rng(2)
    hkv, lens = 2, [700, 33, 1500]
    sets = []
    for i in range(2):
        table, kc, vc, sc = R.poisoned_pool(rng, lens, hkv)
        cache = [to_dev(x) for x in (kc, vc, sc)]
        q = to_dev(rng.standard_normal((99, 4 * hkv, 128)).astype(np.float16))
        ws = [empty(max(K.k16v8_attention_workspace_size_k8v8(70, 4 * hkv, hkv, 128),
                        K.k16v8_decode_workspace_size_k8v8(3, 4 * hkv, 128))) for _ in range(2)]
        sets.append((q, cache, to_dev(table), i32(lens), ws))

    def calls(i, stream):
        q, cache, table, dlens, ws = sets[i]
        return (attend(K, "", q[:3], cache, table, dlens, ws=ws[0], stream=stream)[:2] +
                attend(K, "k16v8_paged_prefill_attention_k8v8", q, cache, table, dlens, 70, i32([0, 70, 71, 99]),
                       ws[1], stream)[:2] +
                attend(K, "k16v8_paged_cross_attention_k8v8", q[:40], cache, table, dlens, 32,
                       i32([0, 5, 8, 40]), ws[0], stream)[:2])

    want = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, calls(i, None)))
    torch.cuda.synchronize()
    for i, outs in got:
        for a, b in zip(outs, want[i]):
            assert torch.equal(a, b)


def test_outputs_over_the_queries(K):
    """Rows may be written over the queries they were read from: whole and cut
    segments, many and few rows."""
    rng = np.random.default_rng(3)
    lens = [900, 64, 2500]
    table, kc, vc, sc = R.poisoned_pool(rng, lens, 2)
    cache, dtable, dlens = [to_dev(x) for x in (kc, vc, sc)], to_dev(table), i32(lens)
    q = to_dev(rng.standard_normal((180, 8, 128)).astype(np.float16))
    ws = empty(max(K.k16v8_attention_workspace_size_k8v8(100, 8, 2, 128), K.k16v8_decode_workspace_size_k8v8(3, 8, 128)))
    for name, rows, most, indptr in (("decode", 3, 1, None), ("prefill", 180, 100, i32([0, 100, 120, 180])),
                                     ("cross", 180, 100, i32([0, 100, 120, 180])), ("cross", 9, 4, i32([0, 3, 5, 9]))):
        got = q[:rows].clone()
        want = torch.empty_like(got)
        for src, out in ((got, want), (got, got)):
            if name == "decode":
                K.k16v8_paged_decode_attention_k8v8(src, *cache, dtable, dlens, SCALE, ws, out)
            else:
                getattr(K, f"k16v8_paged_{name}_attention_k8v8")(src, indptr, most, *cache, dtable, dlens, max(lens),
                                                                 SCALE, ws, out)
        assert torch.equal(got, want)
