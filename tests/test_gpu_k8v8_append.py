"""The K8/V8 cache write and positions with several axes, against the formulas
in 64 bits.

Tolerance.  A turned value r = f (a c - b s) is off by at most pert = 2^-20 f
(|a| + |b|) before it is rounded (the angle by 2^-25 of a revolution, cosine and
sine by 2 ulp, products and sum by 2^-24 each).  Rounded to fp16: half a step,
2^-11 |r| or 2^-25.  Rounded to a code at scale s: half a step, 2^-4 |r| or 2^-10
s.  Rows that are not turned (values, rotary width 0, dims behind it) are exact
up to their one rounding: their codes are compared bit for bit, and so are the
scales wherever no maximum lies within pert of a border."""
import numpy as np
import pytest
import torch

import k8v8_ref as R
from cases import dev, to_dev
from fp8_paged_kv_append_gb300 import rope

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def grid_positions(rng, axes, T, limit):
    pos = rng.integers(0, limit, (axes, T)).astype(np.int32)
    pos[:, 0] = 0
    if T > 1:
        pos[:, 1] = limit - 1
    return pos


def pairs(axes, rotary, turns):
    half = rotary // 2
    each = half // (axes if turns else axes + 1)
    return rope.rope_pair_axes(rotary, [half - each * (axes - 1)] + [each] * (axes - 1), turns)


# ---- several axes, K16/V8 cache -------------------------------------------------

@pytest.mark.parametrize("axes,mixed,interleaved,rotary,dtype,T,hkv", [
    (3, False, False, 128, "fp16", 33, 2), (3, True, True, 96, "bf16", 40, 1),
    (2, True, False, 64, "fp32", 17, 3), (4, False, True, 128, "bf16", 300, 5),
    (1, False, False, 32, "fp16", 1, 1), (3, True, False, 128, "fp32", 700, 2)])
def test_rope_axes(K, axes, mixed, interleaved, rotary, dtype, T, hkv):
    rng = np.random.default_rng(axes * 1000 + rotary + T)
    hq = 4 * hkv
    x = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, 128)).astype(np.float32)).to(DT[dtype])
    g = x.to(dev())
    pair = pairs(axes, rotary, mixed)
    pos = grid_positions(rng, axes, T, 1 << 20)
    freq, _ = rope.rope_inv_freq(rotary)
    slots = rng.permutation(-(-T // 16) * 16 + 16)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1
    P = -(-T // 16) + 1
    kc = torch.full((P, hkv, 16, 128), 3.5, dtype=torch.float16, device=dev())
    vc = torch.full((P, hkv, 16, 128), 0x31, dtype=torch.uint8, device=dev())
    q_out = torch.full((T, hq, 128), 7.5, dtype=torch.float16, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    vs = (rng.uniform(2, 5, hkv) / 448).astype(np.float32)
    K.k16v8_rope_axes_kv_append(g[:, :hq], g[:, hq:hq + hkv], g[:, hq + hkv:], to_dev(pos), pair,
                                to_dev(freq.numpy()), to_dev(slots), to_dev(vs), q_out, kc, vc,
                                interleaved=interleaved, attn_factor=1.25, dev_error=err)
    assert K.k16v8_read_device_error(err) == 0
    xs = x.to(torch.float64).numpy()
    live = slots >= 0
    for got, src in ((q_out.cpu().numpy().astype(np.float64), xs[:, :hq]),
                     (None, xs[:, hq:hq + hkv])):
        if got is None:
            rows = kc.cpu().numpy().astype(np.float64).transpose(0, 2, 1, 3).reshape(-1, hkv, 128)
            got = np.full((T, hkv, 128), 7.5)
            got[live] = rows[slots[live]]
            rest = np.ones(len(rows), bool)
            rest[slots[live]] = False
            assert np.all(rows[rest] == 3.5)
        want, mag = R.turned(src, pos, pair, freq.numpy(), 1.25, interleaved)
        pert = 2.0 ** -20 * mag
        bound = 2.0 ** -11 * (np.abs(want) + pert) + 2.0 ** -25 + pert
        assert np.all(np.abs(got - want)[live] <= bound[live])
        assert np.all(got[~live] == 7.5)


def test_one_axis_is_the_plain_call(K):
    """With the same positions on every axis the result is the one-axis call's,
    bit for bit."""
    rng = np.random.default_rng(5)
    T, hkv, hq = 50, 2, 8
    g = to_dev(rng.standard_normal((T, hq + 2 * hkv, 128)).astype(np.float16))
    freq = to_dev(rope.rope_inv_freq(128)[0].numpy())
    pos = rng.integers(0, 100000, T).astype(np.int32)
    slots, vs = to_dev(np.arange(T, dtype=np.int64)), to_dev(np.full(hkv, 0.01, np.float32))
    res = []
    for several in (False, True):
        kc = torch.zeros((4, hkv, 16, 128), dtype=torch.float16, device=dev())
        vc = torch.zeros((4, hkv, 16, 128), dtype=torch.uint8, device=dev())
        qo = torch.zeros((T, hq, 128), dtype=torch.float16, device=dev())
        q, k, v = g[:, :hq], g[:, hq:hq + hkv], g[:, hq + hkv:]
        if several:
            K.k16v8_rope_axes_kv_append(q, k, v, to_dev(np.stack([pos] * 3)),
                                        rope.rope_pair_axes(128, [16, 24, 24]), freq, slots, vs, qo, kc,
                                        vc)
        else:
            K.k16v8_rope_kv_append(q, k, v, to_dev(pos), freq, slots, vs, qo, kc, vc)
        res.append((qo.cpu(), kc.cpu(), vc.cpu()))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_rope_axes_position_out_of_range_on_one_axis(K):
    g = torch.ones((3, 6, 128), dtype=torch.float16, device=dev())
    pos = np.array([[1, 1, 1], [2, 1 << 24, 2], [3, 3, -1]], np.int32)
    kc = torch.full((1, 1, 16, 128), 3.5, dtype=torch.float16, device=dev())
    vc = torch.full((1, 1, 16, 128), 0x31, dtype=torch.uint8, device=dev())
    qo = torch.full((3, 4, 128), 7.5, dtype=torch.float16, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_rope_axes_kv_append(g[:, :4], g[:, 4:5], g[:, 5:], to_dev(pos), bytes([0, 1, 2, 0] * 16),
                                to_dev(rope.rope_inv_freq(128)[0].numpy()),
                                to_dev(np.arange(3, dtype=np.int64)), to_dev(np.ones(1, np.float32)), qo,
                                kc, vc, dev_error=err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_POSITION
    assert torch.all(qo[1:] == 7.5) and torch.all(kc[0, 0, 1:] == 3.5) and not torch.all(qo[0] == 7.5)


# ---- the K8/V8 write ----------------------------------------------------------------

def run_append(K, rng, counts, olds, hkv, rotary, axes, interleaved, dtype, pad=0, factor=1.0, hq=None,
               mutate=None):
    """One call on a pool that holds rows of earlier calls; everything compared."""
    hq = 4 * hkv if hq is None else hq
    counts, olds = np.asarray(counts), np.asarray(olds)
    lens = olds + counts
    T = int(counts.sum()) + pad
    x = rng.standard_normal((T, hq + 2 * hkv, 128)) * 2.0 ** rng.integers(-3, 4, (T, 1, 1))
    x = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    if mutate:
        mutate(x[:, hq:])
    table, P = R.pages_of(rng, lens, maxp=int(max(lens.max(), 1) + 15) // 16 + 1)
    kc0, vc0 = R.codes(rng, P, hkv, 16, 128), R.codes(rng, P, hkv, 16, 128)
    sc0 = (2.0 ** rng.integers(-10, -4, (P, hkv, 2))).astype(np.float32)
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    freq = pos = pair = None
    if rotary:
        freq = rope.rope_inv_freq(rotary)[0].numpy()
        pair = pairs(axes, rotary, axes == 3)
        pos = grid_positions(rng, axes, T, 1 << 17)
    g = x.to(dev())
    kc, vc, sc = to_dev(kc0), to_dev(vc0), to_dev(sc0)
    qo = torch.full((T, hq, 128), 7.5, dtype=torch.float16, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.k16v8_rope_kv_append_k8v8(
        g[:, :hq] if hq else None, g[:, hq:hq + hkv], g[:, hq + hkv:], to_dev(indptr),
        to_dev(pos) if rotary else None, pair, to_dev(freq) if rotary else None, to_dev(table),
        to_dev(lens.astype(np.int32)), qo if hq else None, kc, vc, sc, interleaved=interleaved,
        attn_factor=factor, dev_error=err)
    assert K.k16v8_read_device_error(err) == 0
    xs = x.to(torch.float64).numpy()
    q, k, v = xs[:, :hq], xs[:, hq:hq + hkv], xs[:, hq + hkv:]
    if rotary:
        q, qm = R.turned(q, pos, pair, freq, factor, interleaved)
        k, km = R.turned(k, pos, pair, freq, factor, interleaved)
    else:
        qm, km = np.zeros_like(q), np.zeros_like(k)
    if hq:
        got = qo.cpu().numpy().astype(np.float64)
        n = int(indptr[-1])
        pert = 2.0 ** -20 * qm
        bound = 2.0 ** -11 * (np.abs(q) + pert) + 2.0 ** -25 + pert
        assert np.all(np.abs(got - q)[:n] <= bound[:n])
        assert np.all(got[n:] == 7.5)
    got = [kc.cpu().numpy(), vc.cpu().numpy()]
    gsc = sc.cpu().numpy()
    want, wsc = [kc0.copy(), vc0.copy()], sc0.copy()
    o = 0
    for b, (n, L) in enumerate(zip(counts, lens)):
        at = L - n
        while at < L:
            end = min((at // 16 + 1) * 16, L)
            p, lo, m = table[b, at // 16], at % 16, end - at
            for i, (src, mag) in enumerate(((k, km), (v, np.zeros_like(v)))):
                rows, pert = src[o:o + m], 2.0 ** -20 * mag[o:o + m]
                a = np.where(np.isfinite(rows), np.abs(rows), 0.0)
                for h in range(hkv):
                    floor = sc0[p, h, i] if lo else 0.0
                    s = max(R.scale_of(a[:, h].max()), floor)
                    near = {max(R.scale_of(np.max(a[:, h] + sg * pert[:, h]).clip(0)), floor) for sg in (-1, 1)}
                    assert gsc[p, h, i] in near | {s}
                    s = float(gsc[p, h, i])
                    wsc[p, h, i] = s
                    want[i][p, h, :lo] = R.encode(R.TABLE[want[i][p, h, :lo]] * (sc0[p, h, i] / s))
                    exact = R.encode(rows[:, h] / s) if not mag[o:o + m, h].any() else None
                    out = got[i][p, h, lo:lo + m]
                    if exact is not None:
                        assert np.array_equal(out & np.where((out & 0x7F) == 0x7F, 0x7F, 0xFF),
                                              exact & np.where((exact & 0x7F) == 0x7F, 0x7F, 0xFF))
                    else:
                        r = np.clip(rows[:, h], -448 * s, 448 * s)
                        bound = 2.0 ** -4 * (np.abs(r) + pert[:, h]) + 2.0 ** -10 * s + pert[:, h]
                        assert np.all(np.abs(R.TABLE[out] * s - r) <= bound)
                    want[i][p, h, lo:lo + m] = out
            o, at = o + m, end
    for i in range(2):  # everything else is as it was, and held rows are in the page's scale
        assert np.array_equal(got[i], want[i])
    assert np.array_equal(gsc, wsc)
    return got, gsc


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,axes", [(0, 1), (16, 1), (64, 3), (128, 1), (128, 3)])
def test_append(K, dtype, interleaved, rotary, axes):
    rng = np.random.default_rng(rotary + axes)
    run_append(K, rng, [5, 0, 1, 33, 16, 47], [0, 9, 15, 16, 1000, 30], 2, rotary, axes, interleaved,
               dtype, pad=3, factor=1.5 if rotary == 64 else 1.0)


@pytest.mark.parametrize("hkv,hq", [(1, 4), (5, 20), (10, 40), (3, 0), (2, 3)])
def test_append_heads(K, hkv, hq):
    run_append(K, np.random.default_rng(hkv), [20, 1], [7, 31], hkv, 128, 3, False, "fp16", hq=hq)


@pytest.mark.parametrize("batch", [1, 64, 300])
def test_append_steps(K, batch):
    """One token for each of many sequences, at every offset of a page."""
    rng = np.random.default_rng(batch)
    run_append(K, rng, [1] * batch, [int(x) for x in rng.integers(0, 100, batch)], 2, 64, 1, False, "fp16")


def many_counts(kind, rng):
    counts = rng.integers(0, 2, 300) if kind != "few each" else rng.integers(0, 6, 300)
    if kind == "a long one":
        counts[170], counts[171] = 40, 2
    if kind == "empty ends":
        counts[:140] = counts[250:] = 0
    return [int(n) for n in counts]


@pytest.mark.parametrize("kind", ["at most one", "a long one", "empty ends", "few each"])
@pytest.mark.parametrize("dtype,interleaved,hkv,hq", [("fp16", False, 1, 4), ("fp32", True, 2, 3),
                                                      ("bf16", False, 20, 30)])
def test_append_many_sequences(K, kind, dtype, interleaved, hkv, hq):
    """More sequences than a CTA has threads, of no, one or a few new tokens."""
    rng = np.random.default_rng(hkv)
    counts = many_counts(kind, rng)
    run_append(K, rng, counts, [int(x) for x in rng.integers(0, 40, 300)], hkv, 64, 3, interleaved, dtype,
               pad=7, hq=hq)


def test_append_bad_sequences_among_many(K):
    """Lengths below their new tokens: flagged and skipped, the others written."""
    B = 700
    g = torch.ones((B, 3, 128), dtype=torch.float16, device=dev())
    kc = torch.full((B, 1, 16, 128), 0x31, dtype=torch.uint8, device=dev())
    vc, sc = kc.clone(), torch.ones((B, 1, 2), dtype=torch.float32, device=dev())
    qo = torch.full((B, 1, 128), 7.5, dtype=torch.float16, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    lens = np.full(B, 5, np.int32)
    bad = [0, 3, 127, 128, 400, 699]
    lens[bad] = [0, 17, -1, 0, 2 ** 31 - 1, 0]
    K.k16v8_rope_kv_append_k8v8(g[:, :1], g[:, 1:2], g[:, 2:], to_dev(np.arange(B + 1, dtype=np.int32)), None, None,
                                None, to_dev(np.arange(B, dtype=np.int32)[:, None]), to_dev(lens), qo, kc, vc, sc,
                                dev_error=err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_SEQLEN
    want = np.ones(B, bool)
    want[bad] = False
    touched = (kc.cpu() != 0x31).any(-1).any(1).numpy()
    assert np.array_equal(touched[:, 4], want) and not touched[:, [0, 1, 2, 3, 5, 15]].any()
    assert np.array_equal((qo.cpu() == 1).all(-1).all(-1).numpy(), want)


def test_append_long(K):
    run_append(K, np.random.default_rng(1), [2000], [3], 10, 96, 3, False, "bf16", pad=1)


def test_append_not_finite(K):
    """Infinities and NaN keep their rows from setting the scale."""
    def mutate(kv):
        kv[0, :, 5] = float("inf")
        kv[1, :, 6] = float("-inf")
        kv[2, :, 7] = float("nan")
        kv[20:22] = float("inf")
        kv[22] = 0.0
    run_append(K, np.random.default_rng(2), [10, 30], [4, 0], 2, 0, 1, False, "fp32", mutate=mutate)


def test_append_extremes(K):
    """Values beyond the largest scale saturate, tiny ones take the smallest."""
    def mutate(kv):
        kv[:16] *= 1e6
        kv[16:32] *= 1e-9
        kv[32:] = 0.0
    got, sc = run_append(K, np.random.default_rng(3), [48], [0], 1, 0, 1, False, "fp32", mutate=mutate)
    assert set(np.unique(sc)) >= {2.0 ** 7, 2.0 ** -15}


def test_append_token_by_token(K):
    """A prompt written token by token holds every row within a code step of the
    page's final scale (a row is rounded again when the scale grows)."""
    rng = np.random.default_rng(4)
    hkv, T = 2, 40
    x = (rng.standard_normal((T, 2, hkv, 128)) * 2.0 ** rng.integers(-4, 3, (T, 1, 1, 1))).astype(np.float32)
    kc = torch.zeros((3, hkv, 16, 128), dtype=torch.uint8, device=dev())
    vc, sc = torch.zeros_like(kc), torch.full((3, hkv, 2), 64.0, dtype=torch.float32, device=dev())
    table, g = to_dev(np.array([[2, 0, 1]], np.int32)), to_dev(x)
    one = to_dev(np.array([0, 1], np.int32))
    for t in range(T):
        K.k16v8_rope_kv_append_k8v8(None, g[t:t + 1, 0], g[t:t + 1, 1], one, None, None, None, table,
                                    to_dev(np.array([t + 1], np.int32)), None, kc, vc, sc)
    s = sc.cpu().numpy()[[2, 0, 1]]
    for i, c in enumerate((kc, vc)):
        rows = R.TABLE[c.cpu().numpy()[[2, 0, 1]]].transpose(0, 2, 1, 3).reshape(48, hkv, 128)[:T]
        step = np.repeat(s[:, :, i], 16, 0)[:T, :, None]
        for p in range(3):
            top = np.abs(x[16 * p:16 * p + 16, i]).max((0, 2))
            assert np.array_equal(s[p, :, i], [R.scale_of(float(v)) for v in top])
        # normal codes keep their bits under a power of two: one rounding of 2^-4; subnormal
        # ones are rounded to 2^-9 of the scale each time it doubles, 2^-10 + 2^-11 + ...
        assert np.all(np.abs(rows * step - x[:, i]) <= 2.0 ** -4 * np.abs(x[:, i]) + 2.0 ** -9 * step)


def test_append_in_place_and_strided(K):
    """q_out may be q; k and v may be slices of a wider row."""
    rng = np.random.default_rng(6)
    T, hkv = 19, 2
    qkv = to_dev(rng.standard_normal((T, 24, 128)).astype(np.float16))
    freq = to_dev(rope.rope_inv_freq(128)[0].numpy())
    pos, indptr = to_dev(np.arange(T, dtype=np.int32)[None]), to_dev(np.array([0, T], np.int32))
    table, lens = to_dev(np.array([[1, 0]], np.int32)), to_dev(np.array([T], np.int32))
    res = []
    for same in (False, True):
        q = qkv[:, :8].contiguous()
        k, v = qkv[:, 10:12], qkv[:, 20:22]
        qo = q if same else torch.empty_like(q)
        kc = torch.zeros((2, hkv, 16, 128), dtype=torch.uint8, device=dev())
        vc, sc = torch.zeros_like(kc), torch.zeros((2, hkv, 2), dtype=torch.float32, device=dev())
        if same:
            k, v = k.contiguous(), v.contiguous()
        K.k16v8_rope_kv_append_k8v8(q, k, v, indptr, pos, bytes(64), freq, table, lens, qo, kc, vc, sc)
        res.append([t.cpu() for t in (qo, kc, vc, sc)])
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_append_device_errors(K):
    """Sequences, pages and positions out of range are flagged and skipped; the
    others are written."""
    hkv, T = 1, 12
    g = torch.ones((T, 6, 128), dtype=torch.float16, device=dev())
    freq = to_dev(rope.rope_inv_freq(128)[0].numpy())

    def call(indptr, lens, table, pos=None):
        kc = torch.full((4, hkv, 16, 128), 0x31, dtype=torch.uint8, device=dev())
        vc, sc = kc.clone(), torch.full((4, hkv, 2), 4.0, dtype=torch.float32, device=dev())
        qo = torch.full((T, 4, 128), 7.5, dtype=torch.float16, device=dev())
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        K.k16v8_rope_kv_append_k8v8(
            g[:, :4], g[:, 4:5], g[:, 5:], to_dev(np.array(indptr, np.int32)),
            None if pos is None else to_dev(np.array(pos, np.int32)), None if pos is None else bytes(64),
            None if pos is None else freq, to_dev(np.array(table, np.int32)),
            to_dev(np.array(lens, np.int32)), qo, kc, vc, sc, dev_error=err)
        touched = (kc.cpu() != 0x31).any(-1).any(1).numpy()  # [page][offset]
        return K.k16v8_read_device_error(err), touched, (qo.cpu() != 7.5).any(-1).any(-1).numpy(), sc.cpu()

    table = [[0, 1], [2, 3]]
    e, touched, rows, sc = call([0, 4, 12], [3, 20], table)  # more rows than positions
    assert e == K.DEVERR_SEQLEN and not touched[:2].any() and touched[2, 12:].all() and touched[3, :4].all()
    assert not rows[:4].any() and rows[4:].all()
    assert call([0, 4, 12], [4, 33], table)[0] == K.DEVERR_SEQLEN  # beyond the table
    assert call([0, 4, 13], [4, 20], table)[0] == K.DEVERR_SEQLEN  # rows beyond the tokens
    assert call([0, 6, 4], [6, 20], table)[0] == K.DEVERR_SEQLEN   # a negative count
    assert call([-5, 4, 12], [9, 20], table)[0] == K.DEVERR_SEQLEN
    e, touched, rows, sc = call([0, 4, 12], [4, 20], [[0, -1], [2, 4]])
    assert e == K.DEVERR_PAGE and touched[0, :4].all() and touched[2, 12:].all() and not touched[3].any()
    assert rows[:8].all() and not rows[8:].any()
    pos = [[1] * T]
    pos[0][2], pos[0][7] = -1, 1 << 24
    e, touched, rows, sc = call([0, 4, 12], [4, 20], table, pos)
    assert e == K.DEVERR_POSITION
    assert rows.tolist() == [i not in (2, 7) for i in range(T)]
    assert touched[0, :4].tolist() == [True, True, False, True] and touched[2, 12:].tolist() == [True] * 3 + [False]
    # a page whose rows are all skipped keeps its scale
    e, touched, rows, sc = call([0, 4, 12], [4, 20], table, [[1 << 24] * 4 + [1] * 8])
    assert e == K.DEVERR_POSITION and not touched[0].any() and torch.all(sc[0] == 4.0)


def test_append_refusals(K):
    T, hkv = 4, 1
    q = torch.zeros((T, 4, 128), dtype=torch.float16, device=dev())
    k, v = q[:, :1].contiguous(), q[:, 1:2].contiguous()
    indptr, lens = to_dev(np.array([0, T], np.int32)), to_dev(np.array([T], np.int32))
    table, pos = to_dev(np.array([[0]], np.int32)), to_dev(np.zeros((3, T), np.int32))
    freq = to_dev(rope.rope_inv_freq(128)[0].numpy())
    kc = torch.zeros((1, hkv, 16, 128), dtype=torch.uint8, device=dev())
    sc = torch.zeros((1, hkv, 2), dtype=torch.float32, device=dev())
    pair = rope.rope_pair_axes(128, [16, 24, 24])

    def call(**kw):
        a = dict(q=q, k=k, v=v, qo_indptr=indptr, positions=pos, pair_axis=pair, inv_freq=freq,
                 block_table=table, seq_lens=lens, q_out=torch.empty_like(q), k_cache=kc, v_cache=kc.clone(),
                 kv_scale=sc)
        a.update(kw)
        K.k16v8_rope_kv_append_k8v8(**a)

    call()
    for bad in (dict(kv_scale=sc[:, :, :1].contiguous()), dict(kv_scale=sc.double()), dict(k_cache=kc.half()),
                dict(pair_axis=pair[:-1]), dict(qo_indptr=indptr.long()), dict(v=v.float()),
                dict(positions=pos[:, :-1]), dict(positions=pos[0:1, :2]), dict(k=k[:, :, :64]),
                dict(inv_freq=None), dict(q_out=torch.empty_like(q).float()),
                dict(block_table=torch.zeros((1, 4), dtype=torch.int32, device=dev())[:, ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(pair_axis=bytes([3] * 64)), dict(attn_factor=float("inf")),
                dict(positions=to_dev(np.zeros((5, T), np.int32))),
                dict(inv_freq=freq[:4].contiguous(), pair_axis=bytes(4))):
        with pytest.raises(K.K16V8Error):
            call(**bad)


def test_append_garbage_offsets_spare_the_others(K):
    """Offsets out of range before and behind a sequence do not lose it."""
    g = torch.ones((12, 6, 128), dtype=torch.float16, device=dev())
    kc = torch.full((4, 1, 16, 128), 0x31, dtype=torch.uint8, device=dev())
    vc, sc = kc.clone(), torch.full((4, 1, 2), 4.0, dtype=torch.float32, device=dev())
    qo = torch.full((12, 4, 128), 7.5, dtype=torch.float16, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    indptr = np.array([0, 1000000, 8, 12, -2 ** 31, 2 ** 31 - 1], np.int32)
    K.k16v8_rope_kv_append_k8v8(g[:, :4], g[:, 4:5], g[:, 5:], to_dev(indptr), None, None, None,
                                to_dev(np.array([[0], [1], [2], [3], [3]], np.int32)),
                                to_dev(np.full(5, 9, np.int32)), qo, kc, vc, sc, dev_error=err)
    assert K.k16v8_read_device_error(err) == K.DEVERR_SEQLEN
    touched = (kc.cpu() != 0x31).any(-1).any(1).numpy()
    assert touched[2, 5:9].all() and touched.sum() == 4
    assert (qo.cpu() != 7.5).any(-1).any(-1).tolist() == [False] * 8 + [True] * 4
