"""The K8/V8 cache in 64 bits: what its write, its attention and positions with
several axes have to give.  Plain numpy, written from the definitions."""
import math

import numpy as np
import torch

PAGE, D, GROUP, E4M3_MAX = 16, 128, 4, 448.0
TABLE = (torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy())


def encode(x):
    """E4M3 codes of float64 values that fp32 holds: nearest even, saturating."""
    x = np.asarray(x, np.float64)
    sat = np.where(np.isnan(x), x, np.clip(x, -E4M3_MAX, E4M3_MAX))
    assert np.array_equal(sat.astype(np.float32).astype(np.float64), sat, equal_nan=True)
    return torch.from_numpy(sat.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def scale_of(top):
    """The smallest power of two in [2^-15, 2^7] with top <= 448 scale."""
    for e in range(-15, 8):
        if top <= E4M3_MAX * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 7


def turned(x, positions, pair_axis, freq, factor, interleaved):
    """x float64 [T,H,D], positions [axes,T] -> (turned, factor (|a| + |b|) per
    element, zero where it passes through)."""
    half = len(freq)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    ang = positions.astype(np.float64)[np.asarray(list(pair_axis)), :].T * freq.astype(np.float64)
    c, s = factor * np.cos(ang)[:, None], factor * np.sin(ang)[:, None]
    y, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = factor * (np.abs(a) + np.abs(b))
    return y, mag


def attention(q, k_codes, v_codes, kv_scale, table, lens, counts, sm_scale, causal):
    """q float64 [T,Hq,D] ragged by counts -> dict of out, lse, and what the
    error bound needs: weight = sum p |v|, dots = the largest sum |q||k|, top
    |v|, length."""
    hkv = k_codes.shape[1]
    T = int(sum(counts))
    res = {n: np.zeros((T, GROUP * hkv) + s) for n, s in
           (("out", (D,)), ("lse", ()), ("weight", (D,)), ("dots", ()), ("vmax", ()), ("len", ()))}
    row = 0
    for b, (n, L) in enumerate(zip(counts, lens)):
        pages = table[b, :-(-L // PAGE)]
        live = np.repeat((pages >= 0) & (pages < len(k_codes)), PAGE)[:L]
        pg = np.where((pages >= 0) & (pages < len(k_codes)), pages, 0)
        for h in range(hkv):
            k, v = (TABLE[c[pg, h]].reshape(-1, D)[:L] *
                    np.repeat(kv_scale[pg, h, i].astype(np.float64), PAGE)[:L, None]
                    for i, c in enumerate((k_codes, v_codes)))
            for r in range(n):
                see = live & ((np.arange(L) <= L - n + r) if causal else np.ones(L, bool))
                kk, vv = k[see], v[see]
                for j in range(GROUP):
                    at = (row + r, GROUP * h + j)
                    if not see.any():
                        res["lse"][at] = -math.inf
                        continue
                    x = q[at]
                    with np.errstate(invalid="ignore"):
                        s = kk @ x * float(np.float32(sm_scale))
                        m = s.max()
                        p = np.exp(s - m)
                        res["lse"][at] = m + math.log(p.sum()) if np.isfinite(m) else math.nan
                        p /= p.sum()
                        res["out"][at] = p @ vv
                        res["weight"][at] = p @ np.abs(vv)
                        res["dots"][at] = (np.abs(kk) @ np.abs(x)).max() * sm_scale
                        res["vmax"][at] = np.abs(vv).max()
                        res["len"][at] = len(kk)
        row += n
    return res


def check_attention(out, lse, want):
    """The kernels round as follows; everything else is fp32.
      * a score: 128 exact products summed in fp32, 8 steps of 16 -- off by at most
        2^-19 of sum |q||k| (16 roundings of 2^-23), so a weight by e^(2 * that)
      * 2^x of the scaled score: the argument (up to 2^9) to 2^-15, ex2 to 2^-22
      * a weight to fp16: 2^-11 of it, or 2^-32 of the row's largest
      * the output to fp16: 2^-11 of it, 2^-25 among the subnormals"""
    finite = np.isfinite(want["lse"])
    assert np.array_equal(lse == -np.inf, want["lse"] == -np.inf)
    nan = np.isnan(want["out"])
    assert np.array_equal(np.isnan(out), nan)
    ds = 2.0 ** -19 * want["dots"]
    arg = 2.0 ** -23 * (np.abs(np.where(finite, want["lse"], 0)) + 2 * want["dots"] + 16)
    w = np.expm1(2 * (ds + arg)) + 2.0 ** -20
    bound = ((2.0 ** -11 + w)[..., None] * want["weight"] + 2.0 ** -11 * np.abs(want["out"]) +
             2.0 ** -25 + (want["len"] * 2.0 ** -32 * want["vmax"])[..., None])
    err = np.abs(out.astype(np.float64) - want["out"])
    bad = (err > bound) & ~nan
    assert not bad.any(), (bad.sum(), bad.size, (err / bound)[~nan].max())
    e = np.abs(lse[finite].astype(np.float64) - want["lse"][finite])
    lse_bound = (ds + arg + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(finite, want["lse"], 0)))[finite]
    assert np.all(e <= lse_bound), (e / lse_bound).max()


def codes(rng, *shape, spread=90.0):
    """Random finite codes of about normal values."""
    return encode(np.clip(np.rint(rng.standard_normal(shape) * spread * 8) / 8, -448, 448))


def pages_of(rng, lens, spare=3, maxp=None):
    """Block table over a shuffled pool, -1 behind every sequence's pages."""
    need = [-(-int(n) // PAGE) for n in lens]
    total = sum(need) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), maxp or max(max(need), 1)), -1, np.int32)
    o = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[o:o + n]
        o += n
    return table, total


def poisoned_pool(rng, lens, hkv, exps=(-9, -5), nan_tail=True):
    """A pool whose pages hold random rows up to each length and NaN codes behind
    it; unused pages hold NaN codes and NaN scales."""
    table, P = pages_of(rng, lens)
    kc = np.full((P, hkv, PAGE, D), 0x7F, np.uint8)
    vc = np.full((P, hkv, PAGE, D), 0xFF, np.uint8)
    sc = np.full((P, hkv, 2), np.nan, np.float32)
    for b, L in enumerate(lens):
        for i in range(-(-int(L) // PAGE)):
            n = min(PAGE, int(L) - i * PAGE)
            p = table[b, i]
            kc[p, :, :n], vc[p, :, :n] = codes(rng, hkv, n, D), codes(rng, hkv, n, D)
            sc[p] = 2.0 ** rng.integers(exps[0], exps[1] + 1, (hkv, 2))
    return table, kc, vc, sc
