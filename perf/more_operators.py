"""Operators for models that look at images and hear sound, over a cache held in 8 bits, as cases that can
be timed and checked: rotary positions with several axes and the cache write, the write into a K8/V8 cache
(E4M3 keys and values with a power-of-two scale for each page and KV head), and attention over that cache --
single tokens, causal prompt chunks, and tokens over an encoder's states.

``run`` computes a case in its plain form (elementary torch operations) or, where ``own`` is true,
through the library's calls.  ``exact`` restates each operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 128
PAGE = 16
GROUP = 4  # query heads per KV head
E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = 2.0 ** -15, 2.0 ** 7  # of a page of the K8/V8 cache
AXES = 3  # time, height, width
IN_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # One decode step of 32 sequences of a model with image positions: the latency of one small launch.
        dict(name="axes step 32 tokens", op="axes", tokens=32, kv_heads=10, rotary=128, interleaved=False,
             mixed=False, dtype="fp16", max_pos=1152, pad=0),
        # The cache write of eight 1,024-token prompts with images, axes taking turns over the frequencies.
        dict(name="axes prefill 8x1024 bf16", op="axes", tokens=8192, kv_heads=10, rotary=128, interleaved=False,
             mixed=True, dtype="bf16", max_pos=8192, pad=0),
        # One token for each of 32 sequences into half-filled pages: latency, and pages whose scale grows.
        dict(name="append8 step b32", op="append8", batch=32, new=1, ragged=False, start=1024, kv_heads=10, rotary=128,
             axes=1, interleaved=False, dtype="fp16", pad=0),
        # Odd chunks of five long contexts, fp32 projections, padded rows behind the last sequence.
        dict(name="append8 5x311 fp32", op="append8", batch=5, new=311, ragged=True, start=70001, kv_heads=2, rotary=64,
             axes=3, interleaved=True, dtype="fp32", pad=29),
        # Eight 1,024-token prompts with images: the most bytes.
        dict(name="append8 prefill 8x1024 bf16", op="append8", batch=8, new=1024, ragged=False, start=0, kv_heads=10,
             rotary=128, axes=3, interleaved=False, dtype="bf16", pad=0),
        # One user at 1K: latency.
        dict(name="decode8 b1 1K", op="decode8", batch=1, length=1100, ragged=False, kv_heads=10),
        # The 1K/batch-32 workload, ragged.
        dict(name="decode8 b32 1K", op="decode8", batch=32, length=1151, ragged=True, kv_heads=10),
        # The 8K/batch-16 workload: the most bytes.
        dict(name="decode8 b16 8K", op="decode8", batch=16, length=8319, ragged=False, kv_heads=10),
        # Eight prompts of 1,024 tokens, all new.
        dict(name="prefill8 8x1024", op="prefill8", batch=8, new=1024, length=1024, ragged=False, kv_heads=10),
        # The last chunk of an 8,192-token prompt.
        dict(name="prefill8 1024 of 8192", op="prefill8", batch=1, new=1024, length=8192, ragged=False, kv_heads=10),
        # Five tokens of one user over 1,500 encoder states (30 seconds of sound): latency.
        dict(name="cross8 5 over 1500", op="cross8", batch=1, new=5, length=1500, ragged=False, kv_heads=10),
        # Sixteen ragged texts over the states of their recordings.
        dict(name="cross8 16x448 over 1500", op="cross8", batch=16, new=448, length=1500, ragged=True, kv_heads=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["axes", "append8", "decode8", "prefill8", "cross8"])
    heads = rng.choice([1, 2, 5, 8, 10])
    if op == "axes":
        tokens = _log_int(rng, 1, 8192)
        return dict(op=op, tokens=tokens, kv_heads=heads, rotary=rng.choice([32, 64, 96, 128]),
                    interleaved=rng.random() < 0.5, mixed=rng.random() < 0.5,
                    dtype=rng.choice(["fp16", "bf16", "fp32"] if tokens <= 4096 else ["fp16", "bf16"]),
                    max_pos=_log_int(rng, 2048, 1000000), pad=rng.randint(0, tokens // 8))
    if op == "append8":
        batch = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, 8192 // batch))
        return dict(op=op, batch=batch, new=new, ragged=rng.random() < 0.6, start=rng.choice([0, _log_int(rng, 1, 100000)]),
                    kv_heads=heads, rotary=rng.choice([0, 32, 64, 96, 128]), axes=rng.choice([1, 3]),
                    interleaved=rng.random() < 0.5, pad=rng.randint(0, 40),
                    dtype=rng.choice(["fp16", "bf16", "fp32"] if batch * new <= 4096 else ["fp16", "bf16"]))
    if op == "decode8":
        batch = _log_int(rng, 1, 256)
        return dict(op=op, batch=batch, length=_log_int(rng, 1, max(64, 131072 // batch)), ragged=rng.random() < 0.6,
                    kv_heads=heads)
    batch = _log_int(rng, 1, 32)
    new = _log_int(rng, 1, 3800 // batch)
    longest = min(7500000 // (new * batch), 120000 // batch)
    if op == "prefill8":
        length = new + rng.choice([0, _log_int(rng, 1, max(1, longest - new))])
    else:
        length = _log_int(rng, 1, longest)
    return dict(op=op, batch=batch, new=new, length=length, ragged=rng.random() < 0.6, kv_heads=heads)


# ---- inputs --------------------------------------------------------------------------------------

def _randn(g, *shape, dtype=torch.float16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _spread(batch, largest, smallest, stride):
    """A size for each sequence between `largest` (the first's) and `smallest`, the same for every seed: outputs of
    one case have one shape."""
    return (largest - np.arange(batch) * stride % (largest - smallest + 1)).astype(np.int32)


def _pages(rng, lens, spare=3):
    """A block table over a shuffled pool, as it is after a while of serving."""
    need = [-(-int(n) // PAGE) for n in lens]
    total = sum(need) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    o = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[o:o + n]
        o += n
    return table, total


def _codes(g, *shape):
    """E4M3 bytes of normal values whose page maximum lies below 448."""
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) * 90
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(g, pages, hkv):
    """Scales of keys and of values: 2^-8 to 2^-6, the pages of real activations differ by about so much."""
    e = torch.randint(-8, -5, (pages, hkv, 2), generator=g, device="cuda")
    return torch.exp2(e.float())


def _pair_axis(rotary, mixed):
    """The axis (0 time, 1 height, 2 width) that turns each pair: a quarter of the pairs are the time's, the others
    are shared by height and width.  In blocks, or taking turns with the time's last pairs at the end."""
    half = rotary // 2
    space = (half - half // 4) // 2
    if not mixed:
        return [0] * (half - 2 * space) + [1] * space + [2] * space
    out = [0] * half
    for axis in (1, 2):
        for i in range(min(space, half // 3)):
            out[axis + 3 * i] = axis
    return out


def _image_positions(rng, tokens, first, limit):
    """Positions of a prompt with images: text advances all axes, an image stands at one time and runs over rows
    and columns."""
    pos = np.zeros((AXES, tokens), np.int64)
    at, i = first, 0
    while i < tokens:
        n = min(int(rng.integers(1, 60)), tokens - i)  # text
        pos[:, i:i + n] = at + np.arange(n)
        at, i = at + n, i + n
        h, w = int(rng.integers(4, 20)), int(rng.integers(4, 20))
        n = min(h * w, tokens - i)
        j = np.arange(n)
        pos[:, i:i + n] = np.stack([np.full(n, at), at + j // w, at + j % w])
        at, i = at + max(h, w), i + n
    return np.minimum(pos, limit - 1).astype(np.int32)


def _freq(rotary):
    half = rotary // 2
    return (10000.0 ** (-np.arange(half) / half)).astype(np.float32)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(case), "op": case["op"], "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "axes":
        return _prepare_axes(case, rng, g, s)
    if case["op"] == "append8":
        return _prepare_append8(case, rng, g, s)
    return _prepare_attention(case, rng, g, s)


def _projections(case, tokens, g, s):
    """The fused projection's output: q, k and v are slices of one row."""
    hkv = case["kv_heads"]
    hq = GROUP * hkv
    qkv = _randn(g, tokens, hq + 2 * hkv, HEAD_DIM, dtype=IN_TYPES[case["dtype"]])
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["q_out"] = torch.zeros((tokens, hq, HEAD_DIM), dtype=torch.float16, device="cuda")


def _prepare_axes(case, rng, g, s):
    t, hkv = case["tokens"], case["kv_heads"]
    _projections(case, t, g, s)
    s["freq"] = _up(_freq(case["rotary"]))
    s["pair_axis"] = _pair_axis(case["rotary"], case["mixed"])
    first = int(rng.integers(0, max(1, case["max_pos"] - t)))
    s["positions"] = _up(_image_positions(rng, t, first, case["max_pos"]))
    pages = -(-t // PAGE) + 4
    slots = rng.permutation(pages * PAGE)[:t].astype(np.int64)
    if case["pad"]:
        slots[rng.permutation(t)[:case["pad"]]] = -1
    s["slots"] = _up(slots)
    s["v_scale"] = _up((rng.uniform(3.5, 5.0, hkv) / E4M3_MAX).astype(np.float32))
    s["k_cache"] = torch.zeros((pages, hkv, PAGE, HEAD_DIM), dtype=torch.float16, device="cuda")
    s["v_cache"] = torch.zeros((pages, hkv, PAGE, HEAD_DIM), dtype=torch.uint8, device="cuda")
    return s


def _prepare_append8(case, rng, g, s):
    b, n, hkv = case["batch"], case["new"], case["kv_heads"]
    counts = _spread(b, n, max(1, n // 2) if case["ragged"] else n, 7)
    olds = _spread(b, case["start"] + min(15, case["start"]), case["start"], 5)
    lens = olds + counts
    tokens = int(counts.sum()) + case["pad"]
    _projections(case, tokens, g, s)
    # page maxima of real projections differ by a few powers of two
    for x in (s["k"], s["v"]):
        x *= torch.exp2(torch.randint(-2, 2, (tokens, hkv, 1), generator=g, device="cuda").float()).to(x.dtype)
    table, pages = _pages(rng, lens - olds // PAGE * PAGE)  # the pages that the call does not touch are not needed
    wide = np.full((b, int(lens.max() - 1) // PAGE + 1), -1, np.int32)
    for i in range(b):
        got = table[i][table[i] >= 0]
        wide[i, olds[i] // PAGE:olds[i] // PAGE + len(got)] = got
    s["counts"], s["lens"], s["table"] = counts, lens, _up(wide)
    s["indptr"] = _up(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    s["seq_lens"] = _up(lens.astype(np.int32))
    s["freq"] = s["positions"] = s["pair_axis"] = None
    if case["rotary"]:
        s["freq"] = _up(_freq(case["rotary"]))
        pos = np.zeros((case["axes"], tokens), np.int32)
        o = 0
        for i in range(b):
            c = int(counts[i])
            pos[:, o:o + c] = (_image_positions(rng, c, int(olds[i]), 1 << 20) if case["axes"] == AXES
                               else olds[i] + np.arange(c))
            o += c
        s["positions"] = _up(pos)
        s["pair_axis"] = _pair_axis(case["rotary"], False) if case["axes"] == AXES else [0] * (case["rotary"] // 2)
    s["k_cache"], s["v_cache"] = _codes(g, pages, hkv, PAGE, HEAD_DIM), _codes(g, pages, hkv, PAGE, HEAD_DIM)
    s["kv_scale"] = _scales(g, pages, hkv)
    return s


def _prepare_attention(case, rng, g, s):
    b, hkv, op = case["batch"], case["kv_heads"], case["op"]
    longest = case["length"]
    new = case["new"] if op != "decode8" else 1
    counts = _spread(b, new, max(1, new // 2) if case["ragged"] else new, 11)
    lens = _spread(b, longest, max(1, longest // 2) if case["ragged"] else longest, 37)
    if op == "prefill8":
        lens = np.maximum(lens, counts)
    table, pages = _pages(rng, lens)
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    s["counts"], s["lens"] = counts, lens
    s["q"] = _randn(g, int(indptr[-1]), GROUP * hkv, HEAD_DIM)
    s["indptr"], s["seq_lens"], s["table"] = _up(indptr), _up(lens), _up(table)
    s["k_cache"], s["v_cache"] = _codes(g, pages, hkv, PAGE, HEAD_DIM), _codes(g, pages, hkv, PAGE, HEAD_DIM)
    s["kv_scale"] = _scales(g, pages, hkv)
    s["scale"] = 1.0 / math.sqrt(HEAD_DIM)
    s["max_new"], s["max_len"] = int(counts.max()), int(lens.max())
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "axes":
        return _plain_axes(state)
    if state["op"] == "append8":
        return _plain_append8(state)
    return _plain_attention(state)


def _run_own(s):
    from fp8_paged_kv_append_gb300 import k16v8 as K
    c = s["case"]
    if s["op"] == "axes":
        K.k16v8_rope_axes_kv_append(s["q"], s["k"], s["v"], s["positions"], s["pair_axis"], s["freq"], s["slots"],
                                    s["v_scale"], s["q_out"], s["k_cache"], s["v_cache"],
                                    interleaved=c["interleaved"], dev_error=s["err"])
        return s["q_out"], s["k_cache"], s["v_cache"].view(torch.float8_e4m3fn)
    if s["op"] == "append8":
        K.k16v8_rope_kv_append_k8v8(s["q"], s["k"], s["v"], s["indptr"], s["positions"], s["pair_axis"], s["freq"],
                                    s["table"], s["seq_lens"], s["q_out"], s["k_cache"], s["v_cache"], s["kv_scale"],
                                    interleaved=c["interleaved"], dev_error=s["err"])
        return _cache8(s)
    if s["op"] == "decode8":
        K.k16v8_paged_decode_attention_k8v8(s["q"], s["k_cache"], s["v_cache"], s["kv_scale"], s["table"],
                                            s["seq_lens"], s["scale"], s["workspace"], s["out"], s["lse"],
                                            dev_error=s["err"])
    else:
        call = K.k16v8_paged_prefill_attention_k8v8 if s["op"] == "prefill8" else K.k16v8_paged_cross_attention_k8v8
        call(s["q"], s["indptr"], s["max_new"], s["k_cache"], s["v_cache"], s["kv_scale"], s["table"], s["seq_lens"],
             s["max_len"], s["scale"], s["workspace"], s["out"], s["lse"], dev_error=s["err"])
    return s["out"], s["lse"]


def _cache8(s):
    return (s["q_out"], s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn),
            s["kv_scale"])


def _cos_sin(s, rows):
    """Cosines and sines [rows, 1, pairs]; angles of far positions need 64 bits."""
    axis = torch.tensor(s["pair_axis"], device="cuda")
    angle = s["positions"][:, rows].double()[axis].T * s["freq"].double()
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotate(x, cos, sin, rotary, interleaved):
    x = x.float()
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rotary // 2], r[..., rotary // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([r, x[..., rotary:]], -1)


def _plain_axes(s):
    c = s["case"]
    live = (s["slots"] >= 0).nonzero().flatten()
    slot = s["slots"][live]
    cos, sin = _cos_sin(s, live)
    s["q_out"][live] = _rotate(s["q"][live], cos, sin, c["rotary"], c["interleaved"]).half()
    page, off = slot // PAGE, slot % PAGE
    s["k_cache"][page, :, off] = _rotate(s["k"][live], cos, sin, c["rotary"], c["interleaved"]).half()
    v = (s["v"][live].float() / s["v_scale"][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    s["v_cache"][page, :, off] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return s["q_out"], s["k_cache"], s["v_cache"].view(torch.float8_e4m3fn)


def _power_of_two_above(x):
    """The smallest power of two that is not below x."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.ones_like(x), torch.where(m == 0.5, e - 1, e))


def _token_places(s):
    """Rows of the call's tokens, and the sequence and position of each."""
    first = s["indptr"].long()
    counts = first[1:] - first[:-1]
    seq = torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts)
    row = torch.arange(int(seq.numel()), device="cuda")
    return row, seq, s["seq_lens"].long()[seq] - counts[seq] + row - first[seq]


def _plain_append8(s):
    c = s["case"]
    row, seq, pos = _token_places(s)
    page, off = s["table"].long()[seq, pos // PAGE], pos % PAGE
    q, k, v = s["q"][row].float(), s["k"][row].float(), s["v"][row].float()
    if c["rotary"]:
        cos, sin = _cos_sin(s, row)
        q, k = (_rotate(x, cos, sin, c["rotary"], c["interleaved"]) for x in (q, k))
    s["q_out"][row] = q.half()
    # the pages that are written, and the rows that they held before
    pages, which = torch.unique(page, return_inverse=True)
    held = torch.full((pages.numel(),), PAGE, device="cuda").scatter_reduce(0, which, off, "amin")
    old = torch.arange(PAGE, device="cuda")[None] < held[:, None]
    for i, (cache, x) in enumerate(((s["k_cache"], k), (s["v_cache"], v))):
        top = torch.zeros((pages.numel(), c["kv_heads"]), device="cuda")
        top = top.scatter_reduce(0, which[:, None].expand(-1, c["kv_heads"]), x.abs().amax(-1), "amax")
        scale = _power_of_two_above(top / E4M3_MAX).clamp(SCALE_MIN, SCALE_MAX)
        before = s["kv_scale"][pages, :, i]
        scale = torch.where((held > 0)[:, None], torch.maximum(scale, before), scale)
        # rows that were there are held in the new scale
        value = cache[pages].view(torch.float8_e4m3fn).float() * (before / scale)[..., None, None]
        again = value.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[pages] = torch.where(old[:, None, :, None], again, cache[pages])
        code = (x / scale[which][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[page, :, off] = code
        s["kv_scale"][pages, :, i] = scale
    return _cache8(s)


def _plain_attention(s):
    c = s["case"]
    hkv, b, n, length = c["kv_heads"], c["batch"], s["max_new"], s["max_len"]
    lens, first = s["seq_lens"].long(), s["indptr"].long()
    counts = first[1:] - first[:-1]
    pos = torch.arange(length, device="cuda")
    # the sequences' rows, gathered from their pages
    table = s["table"].long().clamp(min=0)

    def rows(cache, i):
        x = cache.view(torch.float8_e4m3fn)[table].float() * s["kv_scale"][table][..., i, None, None]
        return x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :length]

    k, v = rows(s["k_cache"], 0), rows(s["v_cache"], 1)
    # the queries of a sequence, padded to the longest
    token = torch.arange(n, device="cuda")
    row = (first[:-1, None] + token).clamp(max=int(s["q"].shape[0]) - 1)
    q = s["q"][row].float().view(b, n, hkv, GROUP, HEAD_DIM).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * GROUP, HEAD_DIM)
    see = (pos[None] < lens[:, None])[:, None]
    if s["op"] == "prefill8":
        see = see & (pos <= ((lens - counts)[:, None] + token)[..., None])
        see = see.repeat_interleave(GROUP, 1)
    score = torch.where(see[:, None], (q @ k.transpose(-1, -2)) * s["scale"], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    del score
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total
    lse = (top + torch.log(total))[..., 0]
    out = out.view(b, hkv, n, GROUP, HEAD_DIM).permute(0, 2, 1, 3, 4).reshape(b, n, GROUP * hkv, HEAD_DIM)
    lse = lse.view(b, hkv, n, GROUP).permute(0, 2, 1, 3).reshape(b, n, GROUP * hkv)
    live = token[None] < counts[:, None]
    s["out"], s["lse"] = out[live].half(), lse[live].float()
    return s["out"], s["lse"]


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    hkv = case["kv_heads"]
    if case["op"] == "axes":
        size = 4 if case["dtype"] == "fp32" else 2
        live = case["tokens"] - case["pad"]
        row = 6 * hkv * HEAD_DIM * size + 4 * hkv * HEAD_DIM * 2 + hkv * HEAD_DIM * 3
        return {"bytes": live * (row + 4 * AXES) + case["tokens"] * 8, "flops": live * 5 * hkv * case["rotary"] * 3}
    b = case["batch"]
    share = 0.75 if case["ragged"] else 1.0  # sizes are spread over the upper half
    if case["op"] == "append8":
        size = 4 if case["dtype"] == "fp32" else 2
        tokens = b * max(1.0, case["new"] * share)
        row = 6 * hkv * HEAD_DIM * size + 4 * hkv * HEAD_DIM * 2 + hkv * HEAD_DIM * 2
        return {"bytes": tokens * (row + 4 * case["axes"]) + tokens / PAGE * hkv * 8,
                "flops": tokens * hkv * (15 * case["rotary"] + 4 * HEAD_DIM)}
    new, length = 1, case["length"] * share
    if case["op"] != "decode8":
        new = max(1.0, case["new"] * share)
    seen = length - (new - 1) / 2 if case["op"] == "prefill8" else length
    return {"bytes": b * hkv * (length * (2 * HEAD_DIM + 0.5) + new * GROUP * (HEAD_DIM * 4 + 4)),
            "flops": b * new * max(seen, 1.0) * GROUP * hkv * HEAD_DIM * 4}


# ---- the definitions, in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "axes":
        return _exact_axes(s)
    if case["op"] == "append8":
        return _exact_append8(s)
    return _exact_attention(s)


def _turned(s, x):
    """Pair i of a head is (x[i], x[i + half]) or (x[2i], x[2i + 1]), a complex number that is turned."""
    half = s["case"]["rotary"] // 2
    i = torch.arange(half, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + half)
    angle = torch.stack([s["positions"][a].double() * f for a, f in zip(s["pair_axis"], s["freq"].double())], 1)
    y = x.double().clone()
    z = torch.complex(y[..., ia], y[..., ib]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _exact_axes(s):
    q, k = _turned(s, s["q"]), _turned(s, s["k"])
    v = s["v"].double() / s["v_scale"].double()[:, None]
    q_out, k_cache = s["q_out"].double(), s["k_cache"].double()
    v_cache = s["v_cache"].view(torch.float8_e4m3fn).to(torch.float32).double()
    live = s["slots"] >= 0
    q_out[live] = q[live]
    where = s["slots"][live]
    k_cache.transpose(1, 2)[where // PAGE, where % PAGE] = k[live]
    v_cache.transpose(1, 2)[where // PAGE, where % PAGE] = v[live].clamp(-E4M3_MAX, E4M3_MAX)
    return q_out, k_cache, v_cache


def _exact_append8(s):
    turn = s["case"]["rotary"] > 0
    q, k = (_turned(s, s[n]) if turn else s[n].double() for n in ("q", "k"))
    rows = int(s["indptr"][-1])
    q_out = s["q_out"].double()
    q_out[:rows] = q[:rows]
    caches = [s[n].view(torch.float8_e4m3fn).to(torch.float32).double() for n in ("k_cache", "v_cache")]
    scales = s["kv_scale"].double().cpu().numpy()
    table, o = s["table"].cpu().numpy(), 0
    for b, (n, length) in enumerate(zip(s["counts"].tolist(), s["lens"].tolist())):
        at = length - n
        while at < length:  # page by page
            end = min((at // PAGE + 1) * PAGE, length)
            page, lo = int(table[b, at // PAGE]), at % PAGE
            for i, x in enumerate((k, s["v"].double())):
                new = x[o:o + end - at]
                top = new.abs().amax((0, 2)).cpu().numpy()
                factors = []
                for h in range(top.size):
                    m, e = math.frexp(float(top[h]) / E4M3_MAX)
                    scale = min(max(math.ldexp(1.0, e - 1 if m == 0.5 else e) if m else 0.0, SCALE_MIN), SCALE_MAX)
                    if lo:
                        scale = max(scale, float(scales[page, h, i]))
                    factors.append(float(scales[page, h, i]) / scale)
                    scales[page, h, i] = scale
                caches[i][page, :, :lo] *= _up(np.array(factors))[:, None, None]
                code = new / _up(scales[page, :, i])[:, None]
                caches[i][page, :, lo:lo + end - at] = code.clamp(-E4M3_MAX, E4M3_MAX).transpose(0, 1)
            o, at = o + end - at, end
    return q_out, caches[0], caches[1], _up(scales)


def _exact_attention(s):
    hkv, causal = s["case"]["kv_heads"], s["op"] == "prefill8"
    outs, lses, row = [], [], 0
    for b, (n, length) in enumerate(zip(s["counts"].tolist(), s["lens"].tolist())):
        pages = s["table"][b, :-(-length // PAGE)].long()
        hide = None
        if causal:
            hide = torch.ones((n, length), dtype=torch.bool, device="cuda").triu(length - n + 1)
        o = torch.empty((n, GROUP * hkv, HEAD_DIM), dtype=torch.float64, device="cuda")
        e = torch.empty((n, GROUP * hkv), dtype=torch.float64, device="cuda")
        for h in range(hkv):
            k, v = (s[name][pages, h].view(torch.float8_e4m3fn).to(torch.float32).double() *
                    s["kv_scale"][pages, h, i].double()[:, None, None] for i, name in enumerate(("k_cache", "v_cache")))
            k, v = k.reshape(-1, HEAD_DIM)[:length], v.reshape(-1, HEAD_DIM)[:length]
            q = s["q"][row:row + n, GROUP * h:GROUP * (h + 1)].double()
            score = torch.einsum("nhd,ld->hnl", q, k) * float(np.float32(s["scale"]))
            if causal:
                score.masked_fill_(hide, -math.inf)
            o[:, GROUP * h:GROUP * (h + 1)] = torch.einsum("hnl,ld->nhd", torch.softmax(score, -1), v)
            e[:, GROUP * h:GROUP * (h + 1)] = torch.logsumexp(score, -1).T
        outs.append(o)
        lses.append(e)
        row += n
    return torch.cat(outs), torch.cat(lses)
