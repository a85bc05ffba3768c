"""Rotary positions fused with the cache write, against the formula in 64
bits.

Tolerance.  A rotated value r = f (a c - b s) is rounded once to fp16: half a
step, 2^-11 |r| (2^-25 among the subnormals).  Before that the fp32 arithmetic
is off by at most pert = 2^-20 f (|a| + |b|): the angle by 2^-25 of a
revolution (2^-22.3 rad), cosine and sine by 2 ulp (2^-23), each times the
factor, the products and the sum by 2^-24 each.  Value codes are the oracle's,
bit for bit: the division and the rounding are exact operations."""
import numpy as np
import pytest
import torch

import oracle
from cases import dev, to_dev

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def rotated(x, positions, freq, factor, interleaved):
    """x float64 [T, H, D] -> (rotated, |a| + |b| per element)."""
    half = len(freq)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    ang = positions.astype(np.float64)[:, None] * freq.astype(np.float64)
    c, s = factor * np.cos(ang)[:, None], factor * np.sin(ang)[:, None]
    y, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = factor * (np.abs(a) + np.abs(b))
    return y, mag


def check(got, want, mag):
    pert = 2.0 ** -20 * mag
    bound = 2.0 ** -11 * (np.abs(want) + pert) + 2.0 ** -25 + pert
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(err <= bound), (err.max(), np.argmax(err - bound))


def make(seed, T, hq, hkv, rotary, dtype, max_pos, pad=0, fused=True):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, 128)).astype(np.float32)).to(DT[dtype])
    qkv = x.to(dev())
    if fused:
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = (t.contiguous() for t in (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]))
    pages = -(-T // 16) + 2
    slots = rng.permutation(pages * 16)[:T].astype(np.int64)
    slots[rng.permutation(T)[:pad]] = -1
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    if T > 1:
        pos[0], pos[1] = 0, max_pos - 1
    freq = (10000.0 ** (-np.arange(rotary // 2) / (rotary // 2))).astype(np.float32)
    vs = (rng.uniform(2.0, 5.0, hkv) / 448).astype(np.float32)
    return x, q, k, v, slots, pos, freq, vs, pages


def run_and_check(K, seed, T, hq, hkv, rotary, interleaved, dtype, max_pos, factor=1.0, pad=0,
                  fused=True):
    x, q, k, v, slots, pos, freq, vs, pages = make(seed, T, hq, hkv, rotary, dtype, max_pos, pad,
                                                   fused)
    q_out = torch.full((T, hq, 128), 7.5, dtype=torch.float16, device=dev())
    kc = torch.full((pages, hkv, 16, 128), -3.25, dtype=torch.float16, device=dev())
    vc = torch.full((pages, hkv, 16, 128), 0x35, dtype=torch.uint8, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_rope_kv_append(q if hq else None, k, v, to_dev(pos), to_dev(freq), to_dev(slots),
                           to_dev(vs), q_out if hq else None, kc, vc, interleaved=interleaved,
                           attn_factor=factor, dev_error=err)
    assert K.k16v8_read_device_error(err) == 0
    xs = x.to(torch.float64).numpy()
    live = slots >= 0
    if hq:
        want, mag = rotated(xs[:, :hq], pos, freq, factor, interleaved)
        got = q_out.cpu().numpy()
        check(got[live], want[live], mag[live])
        assert np.all(got[~live] == 7.5)
    # the cache as token rows: slot s is row s
    rows = kc.cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * 16, hkv, 128)
    want, mag = rotated(xs[:, hq:hq + hkv], pos, freq, factor, interleaved)
    check(rows[slots[live]], want[live], mag[live])
    other = np.ones(pages * 16, bool)
    other[slots[live]] = False
    assert np.all(rows[other] == -3.25)
    codes = np.full((pages, hkv, 16, 128), 0x35, np.uint8)
    v32 = x[:, hq + hkv:].to(torch.float32).numpy()
    oracle.kv_append(np.zeros((T, hkv, 128), np.float16), v32, slots, vs,
                     np.zeros((pages, hkv, 16, 128), np.float16), codes)
    assert np.array_equal(vc.cpu().numpy(), codes)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rotary", [16, 48, 128])
def test_layouts_types_and_partial_widths(K, rotary, dtype, interleaved):
    run_and_check(K, 1, 37, 8, 2, rotary, interleaved, dtype, 4096)


@pytest.mark.parametrize("T,hq,hkv,pad", [(1, 40, 10, 0), (2, 4, 1, 1), (33, 0, 3, 5), (257, 12, 3, 40),
                                          (1000, 40, 10, 0), (1500, 4, 1, 13), (5, 5, 7, 0)])
def test_sizes_and_padding(K, T, hq, hkv, pad):
    run_and_check(K, 2, T, hq, hkv, 96, False, "fp16", 20000, pad=pad)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_and_attention_factor(K, interleaved):
    run_and_check(K, 3, 64, 8, 2, 128, interleaved, "fp32", 1 << 24, factor=1.2079)


def test_dense_rows(K):
    run_and_check(K, 4, 50, 8, 2, 64, True, "bf16", 1000, fused=False)


def test_in_place_query(K):
    x, q, k, v, slots, pos, freq, vs, pages = make(5, 40, 8, 2, 128, "fp16", 5000, fused=False)
    kc = torch.zeros((pages, 2, 16, 128), dtype=torch.float16, device=dev())
    vc = torch.zeros((pages, 2, 16, 128), dtype=torch.uint8, device=dev())
    out = torch.zeros_like(q)
    args = (k, v, to_dev(pos), to_dev(freq), to_dev(slots), to_dev(vs))
    K.k16v8_rope_kv_append(q, *args, out, kc, vc)
    K.k16v8_rope_kv_append(q, *args, q, kc, vc)
    assert torch.equal(q, out)


def test_special_values(K):
    """fp32 values beyond fp16 become inf, NaN stays NaN, and neither reaches another pair or row."""
    x, q, k, v, slots, pos, freq, vs, pages = make(6, 3, 4, 1, 128, "fp32", 10, fused=False)
    pos[:] = 0  # angle 0: a' = a, b' = b
    k[0, 0, 5], k[1, 0, 6], v[0, 0, 3], v[1, 0, 4] = 1e6, float("nan"), float("inf"), float("nan")
    kc = torch.zeros((pages, 1, 16, 128), dtype=torch.float16, device=dev())
    vc = torch.zeros((pages, 1, 16, 128), dtype=torch.uint8, device=dev())
    K.k16v8_rope_kv_append(None, k, v, to_dev(pos), to_dev(freq), to_dev(slots), to_dev(vs), None,
                           kc, vc)
    rows = kc.transpose(1, 2).reshape(-1, 128)[to_dev(slots)].float()
    assert torch.isposinf(rows[0, 5]) and torch.isfinite(rows[0, :5]).all()
    assert torch.isnan(rows[1, 6]) and torch.isnan(rows[1, 70])
    keep = [i for i in range(128) if i not in (6, 70)]
    assert torch.isfinite(rows[1, keep]).all() and torch.isfinite(rows[2]).all()
    codes = vc.transpose(1, 2).reshape(-1, 128)[to_dev(slots)]
    assert codes[0, 3] == 0x7E and (codes[1, 4] & 0x7F) == 0x7F


def test_bad_slots_and_positions_are_flagged_and_skipped(K):
    x, q, k, v, slots, pos, freq, vs, pages = make(7, 6, 4, 1, 64, "fp16", 100, fused=False)
    for bad, bit in ((dict(slot=pages * 16), K.DEVERR_SLOT), (dict(slot=1 << 40), K.DEVERR_SLOT),
                     (dict(pos=-1), K.DEVERR_POSITION), (dict(pos=1 << 24), K.DEVERR_POSITION)):
        s, p = slots.copy(), pos.copy()
        s[2] = bad.get("slot", s[2])
        p[2] = bad.get("pos", p[2])
        q_out = torch.full((6, 4, 128), 7.5, dtype=torch.float16, device=dev())
        kc = torch.zeros((pages, 1, 16, 128), dtype=torch.float16, device=dev())
        vc = torch.zeros((pages, 1, 16, 128), dtype=torch.uint8, device=dev())
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        K.k16v8_rope_kv_append(q, k, v, to_dev(p), to_dev(freq), to_dev(s), to_dev(vs), q_out, kc,
                               vc, dev_error=err)
        assert K.k16v8_read_device_error(err) == bit
        assert torch.all(q_out[2] == 7.5) and not torch.any(q_out[[0, 1, 3, 4, 5]] == 7.5)
        used = (kc != 0).any(-1).any(1).sum()
        assert int(used) == 5


def test_binding_refuses_wrong_tensors(K):
    x, q, k, v, slots, pos, freq, vs, pages = make(8, 4, 4, 1, 64, "fp16", 100)
    q_out = torch.zeros((4, 4, 128), dtype=torch.float16, device=dev())
    kc = torch.zeros((pages, 1, 16, 128), dtype=torch.float16, device=dev())
    vc = torch.zeros((pages, 1, 16, 128), dtype=torch.uint8, device=dev())
    good = dict(q=q, k=k, v=v, positions=to_dev(pos), inv_freq=to_dev(freq),
                slot_mapping=to_dev(slots), v_scale=to_dev(vs), q_out=q_out, k_cache=kc, v_cache=vc)
    K.k16v8_rope_kv_append(**good)
    for name, t in (("q", q.float()), ("v", v.float()), ("positions", to_dev(pos).long()),
                    ("positions", to_dev(pos[:3])), ("slot_mapping", to_dev(slots).int()),
                    ("inv_freq", to_dev(freq).double()), ("v_scale", to_dev(vs).half()),
                    ("q_out", q_out.float()), ("q_out", q_out[:, :, ::2]), ("k_cache", kc[:, :, :8]),
                    ("v_cache", vc.float()), ("k", k.double()), ("k", k.cpu()),
                    ("k", k[:1].expand(4, 1, 128)), ("q", q.transpose(0, 1))):
        with pytest.raises((ValueError, RuntimeError)):
            K.k16v8_rope_kv_append(**{**good, name: t})
    with pytest.raises(K.K16V8Error):
        K.k16v8_rope_kv_append(**{**good, "inv_freq": to_dev(freq[:12])})
