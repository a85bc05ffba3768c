"""The operators of a speculative serving step over the paged K16/V8 cache, as cases that can be timed
and checked: rotary positions with the cache write, attention of drafted token trees, verification of
the drafted tokens, and the move of the accepted rows.

``run`` computes a case in its plain form (elementary torch operations) or, where ``own`` is true,
through the library's calls.  ``exact`` restates each operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 128
PAGE = 16
E4M3_MAX = 448.0
IN_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # One decode step of 32 sequences (the 1K/batch-32 workload): the latency of one small launch.
        dict(name="rope step 32 tokens", op="rope", tokens=32, kv_heads=10, rotary=128, interleaved=False,
             dtype="fp16", max_pos=1152, pad=0, scaled=False),
        # A mid-sized chunk of a long context: interleaved pairs, fp32 projections, padded rows, far positions.
        dict(name="rope 1531 interleaved fp32", op="rope", tokens=1531, kv_heads=2, rotary=64, interleaved=True,
             dtype="fp32", max_pos=131072, pad=37, scaled=True),
        # The cache write of eight 1,024-token prompts, three quarters of the head rotated, bf16 projections.
        dict(name="rope prefill 8x1024 bf16", op="rope", tokens=8192, kv_heads=10, rotary=96, interleaved=False,
             dtype="bf16", max_pos=8192, pad=0, scaled=True),
        # One user, a chain of four drafted tokens after the last one, 1K of context: latency.
        dict(name="tree chain 5 b1 1K", op="tree", batch=1, nodes=5, branch=1, length=1024, ragged=False, kv_heads=10),
        # A batch of small ragged drafts at 1K context.
        dict(name="tree 16 b32 1K", op="tree", batch=32, nodes=16, branch=3, length=1100, ragged=True, kv_heads=10),
        # The widest trees over 8K contexts: the most arithmetic.
        dict(name="tree 64 b16 8K", op="tree", batch=16, nodes=64, branch=4, length=8192, ragged=False, kv_heads=10),
        # One document-long context: the work is split along one axis.
        dict(name="tree 8 b1 128K", op="tree", batch=1, nodes=8, branch=2, length=131071, ragged=False, kv_heads=10),
        # One user, five drafted tokens, a small vocabulary: latency.
        dict(name="verify chain 6 b1 32K", op="verify", batch=1, nodes=6, branch=1, vocab=32000, draft=True, ragged=False),
        # Trees whose tokens were picked without sampling (no draft probabilities), an odd vocabulary.
        dict(name="verify tree 16 b32 50257", op="verify", batch=32, nodes=16, branch=3, vocab=50257, draft=False,
             ragged=True),
        # A full batch of short drafts over a large vocabulary: the most bytes.
        dict(name="verify 8 b64 128K", op="verify", batch=64, nodes=8, branch=2, vocab=128000, draft=True, ragged=False),
        # One user's tree over a 40-layer cache: latency.
        dict(name="compact 16 b1 40 layers", op="compact", batch=1, nodes=16, accepted=4, layers=40, length=200, kv_heads=10),
        # A full batch of wide trees, several accepted tokens each, over 40 layers.
        dict(name="compact 64 b64 40 layers", op="compact", batch=64, nodes=64, accepted=9, layers=40, length=100, kv_heads=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "tree", "verify", "compact"])
    if op == "rope":
        tokens = _log_int(rng, 1, 8192)
        return dict(op=op, tokens=tokens, kv_heads=rng.choice([1, 2, 5, 8, 10]), rotary=rng.choice([32, 64, 96, 128]),
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["fp16", "bf16", "fp32"] if tokens <= 4096 else ["fp16", "bf16"]),
                    max_pos=_log_int(rng, 2048, 1000000), pad=rng.randint(0, tokens // 8), scaled=rng.random() < 0.5)
    if op == "tree":
        nodes = rng.randint(1, 64)
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, nodes=nodes, branch=rng.randint(1, 5),
                    length=max(nodes, _log_int(rng, 16, max(64, 131000 // max(batch, nodes // 4 + 1)))),
                    ragged=rng.random() < 0.6, kv_heads=rng.choice([1, 2, 5, 8, 10]))
    if op == "verify":
        nodes = rng.randint(1, 64)
        return dict(op=op, batch=min(64, _log_int(rng, 1, max(1, 512 // nodes))), nodes=nodes, branch=rng.randint(1, 5),
                    vocab=_log_int(rng, 1000, 128000), draft=rng.random() < 0.7, ragged=rng.random() < 0.5)
    nodes = rng.randint(2, 64)
    return dict(op=op, batch=_log_int(rng, 1, 64), nodes=nodes, accepted=rng.randint(1, min(nodes, 9)),
                layers=rng.choice([1, 8, 24, 40]), length=max(nodes, rng.randint(64, 100)), kv_heads=rng.choice([2, 8, 10]))


# ---- inputs --------------------------------------------------------------------------------------

def _randn(g, *shape, dtype=torch.float16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _spread(case, largest, smallest, stride):
    """A size for each sequence between `largest` (the first's) and `smallest`, the same for every seed: outputs of
    one case have one shape."""
    return (largest - np.arange(case["batch"]) * stride % (largest - smallest + 1)).astype(np.int32)


def _node_counts(case):
    n = case["nodes"]
    return _spread(case, n, max(1, n // 2) if case["ragged"] else n, 5)


def _trees(rng, counts, branch):
    """Parents of every node: node 0 is the last token of the sequence, node i hangs on one of the `branch`
    nodes before it (a chain for 1)."""
    rows = []
    for n in counts:
        i = np.arange(1, n)
        back = rng.integers(1, branch + 1, max(0, n - 1))
        rows.append(np.concatenate([[-1], np.maximum(i - back, 0)]).astype(np.int32))
    return rows


def _masks(parents):
    """Bit j of a node's mask: node j is the node itself or one of its ancestors."""
    out = []
    for par in parents:
        m = []
        for i, p in enumerate(par):
            m.append((m[p] if p >= 0 else 0) | (1 << i))
        out += m
    return np.array(out, np.uint64).view(np.int64)


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
    """E4M3 bytes of calibrated normal values (the largest a little below 448)."""
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) * 90
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(case), "op": case["op"], "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    return {"rope": _prepare_rope, "tree": _prepare_tree, "verify": _prepare_verify,
            "compact": _prepare_compact}[case["op"]](case, rng, g, s)


def _prepare_rope(case, rng, g, s):
    t, hkv = case["tokens"], case["kv_heads"]
    hq = 4 * hkv
    # the fused projection's output: q, k and v are slices of one row
    qkv = _randn(g, t, (hq + 2 * hkv), HEAD_DIM, dtype=IN_TYPES[case["dtype"]])
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    half = case["rotary"] // 2
    freq = 10000.0 ** (-np.arange(half) / half)
    s["factor"] = 1.0
    if case["scaled"]:  # interpolated by parts for a context 8 times as long
        low, high = half * 0.3, half * 0.7
        keep = 1.0 - np.clip((np.arange(half) - low) / (high - low), 0, 1)
        freq = freq / 8.0 * (1 - keep) + freq * keep
        s["factor"] = 0.1 * math.log(8.0) + 1.0
    s["freq"] = _up(freq.astype(np.float32))
    s["positions"] = _up(rng.integers(0, case["max_pos"], t).astype(np.int32))
    pages = -(-t // PAGE) + 4
    slots = rng.permutation(pages * PAGE)[:t].astype(np.int64)
    if case["pad"]:
        slots[rng.permutation(t)[:case["pad"]]] = -1
    s["slots"] = _up(slots)
    s["v_scale"] = _up((rng.uniform(3.5, 5.0, hkv) / E4M3_MAX).astype(np.float32))
    s["q_out"] = torch.zeros((t, hq, HEAD_DIM), dtype=torch.float16, device="cuda")
    s["k_cache"] = torch.zeros((pages, hkv, PAGE, HEAD_DIM), dtype=torch.float16, device="cuda")
    s["v_cache"] = torch.zeros((pages, hkv, PAGE, HEAD_DIM), dtype=torch.uint8, device="cuda")
    return s


def _prepare_tree(case, rng, g, s):
    hkv = case["kv_heads"]
    counts = _node_counts(case)
    longest = case["length"]
    lens = np.maximum(_spread(case, longest, max(1, longest // 2) if case["ragged"] else longest, 37), counts)
    table, pages = _pages(rng, lens)
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    s["counts"], s["lens"] = counts, lens
    s["q"] = _randn(g, int(indptr[-1]), 4 * hkv, HEAD_DIM)
    s["mask"] = _up(_masks(_trees(rng, counts, case["branch"])))
    s["indptr"], s["seq_lens"], s["table"] = _up(indptr), _up(lens), _up(table)
    s["k_cache"] = torch.randn((pages, hkv, PAGE, HEAD_DIM), generator=g, device="cuda", dtype=torch.float16)
    s["v_cache"] = _codes(g, pages, hkv, PAGE, HEAD_DIM)
    s["v_scale"] = _up((rng.uniform(3.5, 5.0, hkv) / E4M3_MAX).astype(np.float32))
    s["scale"] = 1.0 / math.sqrt(HEAD_DIM)
    s["max_nodes"], s["max_len"] = int(counts.max()), int(lens.max())
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    s["workspace"] = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    return s


def _prepare_verify(case, rng, g, s):
    counts = _node_counts(case)
    parents = _trees(rng, counts, case["branch"])
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total, v = int(indptr[-1]), case["vocab"]
    # peaked rows, as a language model gives them, and a draft that is near the target
    logits = torch.randn((total, v), generator=g, device="cuda") * 3.0
    s["target"] = torch.softmax(logits, -1)
    draft = torch.softmax(logits + 0.7 * torch.randn((total, v), generator=g, device="cuda"), -1)
    del logits
    flat = np.concatenate([np.where(p < 0, 0, p) + o for p, o in zip(parents, indptr[:-1])])
    tokens = torch.multinomial(draft[_up(flat)], 1, generator=g).flatten().to(torch.int32)
    s["tokens"] = tokens
    s["draft"] = draft if case["draft"] else None
    s["parents"], s["indptr"] = _up(np.concatenate(parents)), _up(indptr)
    s["counts"] = counts
    s["uniforms"] = torch.rand(total, generator=g, device="cuda")
    s["max_nodes"] = int(counts.max())
    b = case["batch"]
    s["path"] = torch.zeros((b, s["max_nodes"]), dtype=torch.int32, device="cuda")
    s["path_len"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    s["next"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    return s


def _prepare_compact(case, rng, g, s):
    b, n, layers, hkv = case["batch"], case["nodes"], case["layers"], case["kv_heads"]
    lens = np.maximum(_spread(case, case["length"], case["length"] // 2, 7), n)
    table, pages = _pages(rng, lens)
    s["path_len"] = _up(np.full(b, case["accepted"], np.int32))
    path = np.full((b, n), -1, np.int32)
    for i in range(b):
        path[i, 1:case["accepted"]] = np.sort(rng.permutation(n - 1)[:case["accepted"] - 1] + 1)
        path[i, 0] = 0
    s["path"] = _up(path)
    s["indptr"] = _up((np.arange(b + 1) * n).astype(np.int32))
    s["seq_lens"], s["table"], s["pages"] = _up(lens), _up(table), pages
    s["k_cache"] = torch.randn((layers, pages, hkv, PAGE, HEAD_DIM), generator=g, device="cuda", dtype=torch.float16)
    s["v_cache"] = _codes(g, layers, pages, hkv, PAGE, HEAD_DIM)
    # every layer has a cache of its own: what a program keeps is their addresses
    s["k_ptrs"] = torch.tensor([c.data_ptr() for c in s["k_cache"]], dtype=torch.int64, device="cuda")
    s["v_ptrs"] = torch.tensor([c.data_ptr() for c in s["v_cache"]], dtype=torch.int64, device="cuda")
    s["new_lens"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "tree": _plain_tree, "verify": _plain_verify,
            "compact": _plain_compact}[state["op"]](state)


def _run_own(s):
    from fp8_paged_kv_append_gb300 import k16v8 as K
    if s["op"] == "rope":
        K.k16v8_rope_kv_append(s["q"], s["k"], s["v"], s["positions"], s["freq"], s["slots"], s["v_scale"],
                               s["q_out"], s["k_cache"], s["v_cache"], interleaved=s["case"]["interleaved"],
                               attn_factor=s["factor"], dev_error=s["err"])
        return s["q_out"], s["k_cache"], s["v_cache"].view(torch.float8_e4m3fn)
    if s["op"] == "tree":
        K.k16v8_paged_tree_attention(s["q"], s["indptr"], s["max_nodes"], s["mask"], s["k_cache"], s["v_cache"],
                                     s["v_scale"], s["table"], s["seq_lens"], s["max_len"], s["scale"], s["workspace"],
                                     s["out"], s["lse"], dev_error=s["err"])
        return s["out"], s["lse"]
    if s["op"] == "verify":
        K.k16v8_tree_verify(s["target"], s["draft"], s["tokens"], s["parents"], s["indptr"], s["max_nodes"],
                            s["uniforms"], s["path"], s["path_len"], s["next"], dev_error=s["err"])
        return s["path"], s["path_len"], s["next"]
    c = s["case"]
    K.k16v8_kv_compact(s["k_ptrs"], s["v_ptrs"], s["pages"], c["kv_heads"], HEAD_DIM, s["table"], s["seq_lens"],
                       s["indptr"], s["path"], s["path_len"], s["new_lens"], dev_error=s["err"])
    return s["k_cache"], s["v_cache"].view(torch.float8_e4m3fn), s["new_lens"]


def _rotate(x, cos, sin, rotary, interleaved):
    x = x.float()
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rotary // 2], r[..., rotary // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([r, x[..., rotary:]], -1).half()


def _plain_rope(s):
    c = s["case"]
    live = (s["slots"] >= 0).nonzero().flatten()
    slot = s["slots"][live]
    angle = s["positions"][live].double()[:, None] * s["freq"].double()[None]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    s["q_out"][live] = _rotate(s["q"][live], cos, sin, c["rotary"], c["interleaved"])
    page, off = slot // PAGE, slot % PAGE
    s["k_cache"][page, :, off] = _rotate(s["k"][live], cos, sin, c["rotary"], c["interleaved"])
    v = (s["v"][live].float() / s["v_scale"][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    s["v_cache"][page, :, off] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return s["q_out"], s["k_cache"], s["v_cache"].view(torch.float8_e4m3fn)


def _plain_tree(s):
    hkv = s["case"]["kv_heads"]
    b, n, length = s["case"]["batch"], s["max_nodes"], s["max_len"]
    lens, first = s["seq_lens"].long(), s["indptr"].long()
    counts = first[1:] - first[:-1]
    pos = torch.arange(length, device="cuda")
    # the sequences' rows, gathered from their pages
    table = s["table"].long().clamp(min=0)
    k = s["k_cache"][table].permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :length].float()
    v = s["v_cache"].view(torch.float8_e4m3fn)[table].permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :length].float()
    v = v * s["v_scale"][None, :, None, None]
    # the queries of a sequence, padded to the widest tree
    node = torch.arange(n, device="cuda")
    row = (first[:-1, None] + node).clamp(max=int(s["q"].shape[0]) - 1)
    q = s["q"][row].float().view(b, n, hkv, 4, HEAD_DIM).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * 4, HEAD_DIM)
    rel = pos[None] - (lens - counts)[:, None]
    bit = (s["mask"][row][:, :, None] >> rel.clamp(0, 63)[:, None, :]) & 1
    see = ((rel < 0)[:, None] | (bit == 1)) & (pos[None] < lens[:, None])[:, None]
    see = see.repeat_interleave(4, 1)[:, None]
    score = torch.where(see, (q @ k.transpose(-1, -2)) * s["scale"], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.clamp(min=1e-38)
    lse = (top + torch.log(total))[..., 0]
    out = out.view(b, hkv, n, 4, HEAD_DIM).permute(0, 2, 1, 3, 4).reshape(b, n, 4 * hkv, HEAD_DIM)
    lse = lse.view(b, hkv, n, 4).permute(0, 2, 1, 3).reshape(b, n, 4 * hkv)
    live = node[None] < counts[:, None]
    s["out"], s["lse"] = out[live].half(), lse[live].float()
    return s["out"], s["lse"]


def _plain_verify(s):
    """One step for each node, every sequence at once: the nodes come in an order in which parents stand before
    their children, so each is tested when its parent is the last accepted one.  Sums are in 64 bits."""
    first = s["indptr"].long()
    b, n = s["case"]["batch"], s["max_nodes"]
    counts = first[1:] - first[:-1]
    at = torch.zeros(b, dtype=torch.int64, device="cuda")  # the last accepted node
    length = torch.ones_like(at)
    path = torch.full((b, n), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    weight = s["target"][first[:-1]].double()  # what the next token of each sequence is drawn from
    mass = torch.ones(b, dtype=torch.float64, device="cuda")
    for i in range(1, n):
        row = (first[:-1] + i).clamp(max=s["tokens"].numel() - 1)
        tok = s["tokens"][row].long()[:, None]
        mine = (i < counts) & (s["parents"][row] == at)
        w = weight.gather(1, tok)[:, 0]
        q = 1.0 if s["draft"] is None else s["draft"][first[:-1] + at].gather(1, tok)[:, 0].double()
        good = mine & (s["uniforms"][row].double() * q * mass < w)
        # a rejected token takes the draft's share out of the weights
        if s["draft"] is None:
            left = weight.scatter(1, tok, 0.0)
        else:
            left = (weight - mass[:, None] * s["draft"][first[:-1] + at].double()).clamp(min=0)
        bad = (mine & ~good)[:, None]
        weight = torch.where(good[:, None], s["target"][row].double(), torch.where(bad, left, weight))
        mass = torch.where(good, 1.0, torch.where(bad[:, 0], left.sum(1), mass))
        path.scatter_(1, torch.where(good, length, 0)[:, None],
                      torch.where(good, i, path[:, 0]).to(torch.int32)[:, None])
        at, length = torch.where(good, i, at), length + good
    u = s["uniforms"][first[:-1]].double()[:, None]
    above = weight.cumsum(1)
    s["next"] = torch.searchsorted(above, u * above[:, -1:], right=True)[:, 0].clamp(max=weight.shape[1] - 1).to(torch.int32)
    s["path"], s["path_len"] = path, length.to(torch.int32)
    return s["path"], s["path_len"], s["next"]


def _plain_compact(s):
    counts = s["indptr"][1:] - s["indptr"][:-1]
    base = (s["seq_lens"] - counts).long()
    j = torch.arange(s["path"].shape[1], device="cuda")
    live = j[None] < s["path_len"][:, None]
    seq, to = live.nonzero(as_tuple=True)
    src, dst = base[seq] + s["path"][seq, to], base[seq] + to
    table = s["table"].long()
    ps, pd = table[seq, src // PAGE], table[seq, dst // PAGE]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, pd, :, dst % PAGE] = cache[:, ps, :, src % PAGE]
    s["new_lens"] = (base + s["path_len"]).to(torch.int32)
    return s["k_cache"], s["v_cache"].view(torch.float8_e4m3fn), s["new_lens"]


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        live, hkv = case["tokens"] - case["pad"], case["kv_heads"]
        row = 6 * hkv * HEAD_DIM * size + 4 * hkv * HEAD_DIM * 2 + hkv * HEAD_DIM * 3
        return {"bytes": live * (row + 4) + case["tokens"] * 8, "flops": live * 5 * hkv * case["rotary"] * 3}
    if case["op"] == "tree":
        b, n, hkv = case["batch"], case["nodes"], case["kv_heads"]
        mean = case["length"] * (0.75 if case["ragged"] else 1.0)
        nodes = n * (0.75 if case["ragged"] else 1.0)
        return {"bytes": b * (mean * hkv * HEAD_DIM * 3 + nodes * (4 * hkv * (HEAD_DIM * 4 + 4) + 8)),
                "flops": b * mean * nodes * 4 * hkv * HEAD_DIM * 4}
    if case["op"] == "verify":
        rows = 2 if case["draft"] else 1
        return {"bytes": case["batch"] * case["vocab"] * 4 * rows, "flops": case["batch"] * case["vocab"] * 2 * rows}
    moved = case["batch"] * max(case["accepted"] - 1, 1) * case["layers"] * case["kv_heads"]
    return {"bytes": moved * HEAD_DIM * 3 * 2, "flops": 0}


# ---- the definitions, in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "verify": _exact_verify,
            "compact": _exact_compact}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    r, half = c["rotary"], c["rotary"] // 2
    # pair i of a head is (x[i], x[i + half]) or (x[2i], x[2i + 1]), a complex number that is turned
    i = torch.arange(half, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device="cuda").expand(c["tokens"], half).contiguous(),
                       torch.outer(s["positions"].double(), s["freq"].double()))[:, None]

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., ia], y[..., ib]) * turn
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    q, k = turned(s["q"]), turned(s["k"])
    v = s["v"].double() / s["v_scale"].double()[:, None]
    q_out, k_cache = s["q_out"].double(), s["k_cache"].double()
    v_cache = s["v_cache"].view(torch.float8_e4m3fn).to(torch.float32).double()
    live = s["slots"] >= 0
    q_out[live] = q[live]
    where = s["slots"][live]
    k_cache.transpose(1, 2)[where // PAGE, where % PAGE] = k[live]
    v_cache.transpose(1, 2)[where // PAGE, where % PAGE] = v[live].clamp(-E4M3_MAX, E4M3_MAX)
    return q_out, k_cache, v_cache


def _exact_tree(s):
    hkv = s["case"]["kv_heads"]
    outs, lses, row = [], [], 0
    mask = s["mask"].cpu().numpy().view(np.uint64)
    for b, (n, length) in enumerate(zip(s["counts"].tolist(), s["lens"].tolist())):
        pages = s["table"][b, :-(-length // PAGE)].long()
        see = np.ones((n, length), bool)
        for i in range(n):
            see[i, length - n:] = [(int(mask[row + i]) >> j) & 1 for j in range(n)]
        hide = _up(~see)
        o = torch.empty((n, 4 * hkv, HEAD_DIM), dtype=torch.float64, device="cuda")
        e = torch.empty((n, 4 * hkv), dtype=torch.float64, device="cuda")
        for h in range(hkv):
            k = s["k_cache"][pages, h].reshape(-1, HEAD_DIM)[:length].double()
            v = s["v_cache"][pages, h].reshape(-1, HEAD_DIM)[:length].view(torch.float8_e4m3fn).to(torch.float32).double()
            v = v * s["v_scale"][h].double()
            q = s["q"][row:row + n, 4 * h:4 * h + 4].double()
            score = torch.einsum("nhd,ld->hnl", q, k) * float(np.float32(s["scale"]))
            score.masked_fill_(hide, -math.inf)
            o[:, 4 * h:4 * h + 4] = torch.einsum("hnl,ld->nhd", torch.softmax(score, -1), v)
            e[:, 4 * h:4 * h + 4] = torch.logsumexp(score, -1).T
        outs.append(o)
        lses.append(e)
        row += n
    return torch.cat(outs), torch.cat(lses)


def _exact_verify(s):
    first = s["indptr"].tolist()
    tokens, parents, u = (s[n].cpu().numpy() for n in ("tokens", "parents", "uniforms"))
    b, n = s["case"]["batch"], s["max_nodes"]
    path, length, nxt = np.full((b, n), -1, np.int32), np.zeros(b, np.int32), np.zeros(b, np.int32)

    def row(name, r):
        return s[name][r].double().cpu().numpy()

    for i in range(b):
        o, taken, left = first[i], [0], None
        while left is None:
            p, node = row("target", o + taken[-1]), taken[-1]
            q = None if s["draft"] is None else row("draft", o + node)
            norm = 1.0  # the weights left, as shares of their sum
            left = p
            for c in range(node + 1, first[i + 1] - o):
                if parents[o + c] != node:
                    continue
                x = tokens[o + c]
                if float(u[o + c]) * (1.0 if q is None else q[x]) < left[x] / norm:
                    taken.append(c)
                    left = None
                    break
                if q is None:
                    left = left.copy()
                    left[x] = 0
                else:
                    left = np.maximum(left / norm - q, 0)
                norm = math.fsum(left)
        path[i, :len(taken)], length[i] = taken, len(taken)
        share = np.cumsum(left)
        nxt[i] = min(int(np.searchsorted(share, float(u[o]) * share[-1], side="right")), len(share) - 1)
    return torch.from_numpy(path), torch.from_numpy(length), torch.from_numpy(nxt)


def _exact_compact(s):
    k, v = s["k_cache"].double(), s["v_cache"].view(torch.float8_e4m3fn).to(torch.float32)
    old_k, old_v = s["k_cache"], s["v_cache"].view(torch.float8_e4m3fn)
    lens, first, path = s["seq_lens"].tolist(), s["indptr"].tolist(), s["path"].tolist()
    table, new = s["table"].tolist(), []
    for b, count in enumerate(s["path_len"].tolist()):
        start = lens[b] - (first[b + 1] - first[b])
        for j in range(count):
            a, c = start + path[b][j], start + j
            pa, pc = table[b][a // PAGE], table[b][c // PAGE]
            k[:, pc, :, c % PAGE] = old_k[:, pa, :, a % PAGE].double()
            v[:, pc, :, c % PAGE] = old_v[:, pa, :, a % PAGE].to(torch.float32)
        new.append(start + count)
    return k, v.double(), torch.tensor(new, dtype=torch.int32)
