"""The K8/V8 calls as a model that reads images and an encoder's states uses
them: prompts in chunks (cache write with positions of three axes, causal
attention, cross attention), then single tokens, eager and as one captured
graph.  Every attention is compared with 64-bit attention over what the cache
holds at that moment, and what it holds with what was written."""
import math

import numpy as np
import pytest
import torch

import k8v8_ref as R
from cases import dev, to_dev
from fp8_paged_kv_append_gb300 import rope

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)
HKV, HQ = 2, 8


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


class Cache:
    def __init__(self, rng, lens):
        self.table, pages = R.pages_of(rng, lens)
        self.k = torch.full((pages, HKV, 16, 128), 0x7F, dtype=torch.uint8, device=dev())
        self.v = self.k.clone()
        self.scale = torch.full((pages, HKV, 2), float("nan"), dtype=torch.float32, device=dev())
        self.dtable = to_dev(self.table)

    def host(self):
        return self.k.cpu().numpy(), self.v.cpu().numpy(), self.scale.cpu().numpy()

    def want(self, q, lens, counts, causal):
        k, v, s = self.host()
        return R.attention(q.astype(np.float64), k, v, s, self.table, lens, counts, SCALE, causal)

    def rows(self, b, length):
        """(keys, values) [length, HKV, 128] that the cache stands for."""
        k, v, s = self.host()
        pages = self.table[b, :-(-length // 16)]
        return [(R.TABLE[c[pages]] * s[pages][:, :, i, None, None].astype(np.float64))
                .transpose(0, 2, 1, 3).reshape(-1, HKV, 128)[:length] for i, c in enumerate((k, v))]


def test_chunks_then_steps(K):
    rng = np.random.default_rng(0)
    B, final, enc_len = 3, [75, 150, 30], [40, 0, 129]
    text, enc = Cache(rng, final), Cache(rng, enc_len)
    pair = rope.rope_pair_axes(128, [16, 24, 24], interleaved=False)
    freq = to_dev(rope.rope_inv_freq(128)[0].numpy())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    ws = torch.empty(max(K.k16v8_attention_workspace_size_k8v8(64, HQ, HKV, 128),
                         K.k16v8_decode_workspace_size_k8v8(B, HQ, 128)), dtype=torch.uint8, device=dev())

    # the encoder's states: no queries, no positions
    ip = to_dev(np.concatenate([[0], np.cumsum(enc_len)]).astype(np.int32))
    kv = to_dev(rng.standard_normal((sum(enc_len), 2, HKV, 128)).astype(np.float32))
    enc_lens = to_dev(np.array(enc_len, np.int32))
    K.k16v8_rope_kv_append_k8v8(None, kv[:, 0], kv[:, 1], ip, None, None, None, enc.dtable, enc_lens, None, enc.k,
                                enc.v, enc.scale, dev_error=err)
    written = {b: [] for b in range(B)}  # turned keys and values, as they were given

    def forward(counts, lens):
        T = sum(counts)
        x = to_dev(rng.standard_normal((T, HQ + 2 * HKV, 128)).astype(np.float16))
        pos = rng.integers(0, 5000, (3, T)).astype(np.int32)
        ip = to_dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        n = to_dev(np.array(lens, np.int32))
        q = torch.empty((T, HQ, 128), dtype=torch.float16, device=dev())
        K.k16v8_rope_kv_append_k8v8(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], ip, to_dev(pos), pair, freq,
                                    text.dtable, n, q, text.k, text.v, text.scale, dev_error=err)
        xs = x.cpu().numpy().astype(np.float64)
        turned = R.turned(xs[:, HQ:HQ + HKV], pos, pair, freq.cpu().numpy(), 1.0, False)[0]
        o = 0
        for b, c in enumerate(counts):
            written[b].append((turned[o:o + c], xs[o:o + c, HQ + HKV:]))
            o += c
        out = [torch.full_like(q, 9.0) for _ in range(2)]
        lse = [torch.full((T, HQ), 9.0, device=dev()) for _ in range(2)]
        if max(counts) == 1 and min(counts) == 1:  # single tokens
            K.k16v8_paged_decode_attention_k8v8(q, text.k, text.v, text.scale, text.dtable, n, SCALE, ws, out[0],
                                                lse[0], dev_error=err)
        else:
            K.k16v8_paged_prefill_attention_k8v8(q, ip, max(counts), text.k, text.v, text.scale, text.dtable, n,
                                                 max(lens), SCALE, ws, out[0], lse[0], dev_error=err)
        K.k16v8_paged_cross_attention_k8v8(q, ip, max(counts), enc.k, enc.v, enc.scale, enc.dtable, enc_lens,
                                           max(enc_len), SCALE, ws, out[1], lse[1], dev_error=err)
        assert K.k16v8_read_device_error(err) == 0
        qh = q.cpu().numpy()
        R.check_attention(out[0].cpu().numpy(), lse[0].cpu().numpy(), text.want(qh, lens, counts, True))
        R.check_attention(out[1].cpu().numpy(), lse[1].cpu().numpy(), enc.want(qh, enc_len, counts, False))

    done = [0, 0, 0]
    for counts in ([64, 64, 5], [0, 37, 20], [7, 45, 1]):
        done = [d + c for d, c in zip(done, counts)]
        forward(counts, done)
    for _ in range(4):
        done = [d + 1 for d in done]
        forward([1, 1, 1], done)
    assert done == final
    for b in range(B):
        for i, got in enumerate(text.rows(b, final[b])):
            given = np.concatenate([w[i] for w in written[b]])
            step = np.repeat(text.host()[2][text.table[b, :-(-final[b] // 16)]][:, :, i], 16, 0)[:final[b], :, None]
            # one rounding of 2^-4, and of 2^-9 of the scale for small values each time it grows
            assert np.all(np.abs(got - given) <= 2.0 ** -4 * np.abs(given) + 2.0 ** -9 * step + 1e-5)


def test_captured_step(K):
    """A decode step -- write, attend, cross -- captured once and replayed with new
    rows, positions and lengths."""
    rng = np.random.default_rng(1)
    B, start, enc_len, steps = 4, [15, 16, 47, 100], [20, 300, 1, 64], 5
    text, enc = Cache(rng, [s + steps for s in start]), Cache(rng, enc_len)
    ip_e = to_dev(np.concatenate([[0], np.cumsum(enc_len)]).astype(np.int32))
    enc_lens = to_dev(np.array(enc_len, np.int32))
    kv = to_dev(rng.standard_normal((sum(enc_len), 2, HKV, 128)).astype(np.float16))
    K.k16v8_rope_kv_append_k8v8(None, kv[:, 0], kv[:, 1], ip_e, None, None, None, enc.dtable, enc_lens, None, enc.k,
                                enc.v, enc.scale)
    ip_t = to_dev(np.concatenate([[0], np.cumsum(start)]).astype(np.int32))
    kv = to_dev(rng.standard_normal((sum(start), 2, HKV, 128)).astype(np.float16))
    n = to_dev(np.array(start, np.int32))
    K.k16v8_rope_kv_append_k8v8(None, kv[:, 0], kv[:, 1], ip_t, None, None, None, text.dtable, n, None, text.k,
                                text.v, text.scale)
    x = torch.zeros((B, HQ + 2 * HKV, 128), dtype=torch.bfloat16, device=dev())
    pos = torch.zeros((3, B), dtype=torch.int32, device=dev())
    ip = to_dev(np.arange(B + 1, dtype=np.int32))
    freq, pair = to_dev(rope.rope_inv_freq(64)[0].numpy()), rope.rope_pair_axes(64, [12, 10, 10], True)
    q = torch.empty((B, HQ, 128), dtype=torch.float16, device=dev())
    out = [torch.empty_like(q) for _ in range(2)]
    lse = [torch.empty((B, HQ), device=dev()) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    ws = [torch.empty(K.k16v8_decode_workspace_size_k8v8(B, HQ, 128), dtype=torch.uint8, device=dev())
          for _ in range(2)]

    def step():
        K.k16v8_rope_kv_append_k8v8(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], ip, pos, pair, freq, text.dtable,
                                    n, q, text.k, text.v, text.scale, interleaved=True, dev_error=err)
        for c, o, l, lens, w in ((text, out[0], lse[0], n, ws[0]), (enc, out[1], lse[1], enc_lens, ws[1])):
            K.k16v8_paged_decode_attention_k8v8(q, c.k, c.v, c.scale, c.dtable, lens, SCALE, w, o, l, dev_error=err)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        x.copy_(to_dev(rng.standard_normal((B, HQ + 2 * HKV, 128)).astype(np.float32) * 2.0 ** (i - 2)))
        pos.copy_(to_dev(rng.integers(0, 1 << 20, (3, B)).astype(np.int32)))
        lens = [s + i + 1 for s in start]
        n.copy_(to_dev(np.array(lens, np.int32)))
        graph.replay()
        assert K.k16v8_read_device_error(err) == 0
        qh = q.cpu().numpy()
        want = R.turned(x[:, :HQ].double().cpu().numpy(), pos.cpu().numpy(), pair, freq.cpu().numpy(), 1.0, True)[0]
        assert np.all(np.abs(qh - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -18 * 2.0 ** (i - 2) * 8)
        R.check_attention(out[0].cpu().numpy(), lse[0].cpu().numpy(), text.want(qh, lens, [1] * B, True))
        R.check_attention(out[1].cpu().numpy(), lse[1].cpu().numpy(), enc.want(qh, enc_len, [1] * B, False))


def test_decode_is_prefill_is_cross_of_one_token(K):
    """The three calls agree where they say the same."""
    rng = np.random.default_rng(2)
    lens = [300, 17, 1, 64]
    table, kc, vc, sc = R.poisoned_pool(rng, lens, HKV)
    g = [to_dev(v) for v in (kc, vc, sc, table)]
    q = to_dev(rng.standard_normal((4, HQ, 128)).astype(np.float16))
    n, ip = to_dev(np.array(lens, np.int32)), to_dev(np.arange(5, dtype=np.int32))
    ws = torch.empty(max(K.k16v8_attention_workspace_size_k8v8(1, HQ, HKV, 128),
                         K.k16v8_decode_workspace_size_k8v8(4, HQ, 128)), dtype=torch.uint8, device=dev())
    want = R.attention(q.cpu().numpy().astype(np.float64), kc, vc, sc, table, lens, [1] * 4, SCALE, False)
    for call in ("decode", "prefill", "cross"):
        out, lse = torch.empty_like(q), torch.empty((4, HQ), device=dev())
        if call == "decode":
            K.k16v8_paged_decode_attention_k8v8(q, *g, n, SCALE, ws, out, lse)
        else:
            getattr(K, f"k16v8_paged_{call}_attention_k8v8")(q, ip, 1, *g, n, 300, SCALE, ws, out, lse)
        R.check_attention(out.cpu().numpy(), lse.cpu().numpy(), want)
