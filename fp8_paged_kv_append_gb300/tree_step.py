"""A whole-model speculative step: rotary positions with the cache write and
tree attention for every layer as one CUDA graph, then the verification of
the drafted tokens and the move of the accepted rows.

The buffers that describe the trees are fixed, so a captured step serves new
trees: set_trees() fills them from the host.  All computation runs in
libk16v8's kernels; this module sequences the calls ("Phi-4: quality transfer
and interrupted throughput studies", intro: the cache format and geometry).
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import k16v8 as K
from .decode_step import validate_scales


def _checked_parents(parents):
    """(node, its parent) for every node; a parent but the first node's has to
    be an earlier node."""
    if len(parents) > K.MAX_TREE_NODES:
        raise ValueError(f"a tree has at most {K.MAX_TREE_NODES} nodes, got {len(parents)}")
    for i, p in enumerate(parents):
        if i and not 0 <= p < i:
            raise ValueError(f"parent of node {i} must be an earlier node, got {p}")
        yield i, p


def tree_masks(parents) -> np.ndarray:
    """int64 [n]: bit j of word i is set where node j is node i or one of its
    ancestors.  parents[0] is not read; parents[i] < i."""
    words: list[int] = []
    for i, p in _checked_parents(parents):
        words.append((words[p] if i else 0) | 1 << i)
    return np.array(words, np.uint64).view(np.int64)


def tree_depths(parents) -> np.ndarray:
    """int32 [n]: edges between node 0 and each node.  parents as for
    tree_masks."""
    depth: list[int] = []
    for i, p in _checked_parents(parents):
        depth.append(depth[p] + 1 if i else 0)
    return np.array(depth, np.int32)


class MultiLayerTreeDecode:
    """Speculative step over `len(k_caches)` layers that share one page table.

    k_caches[l] fp16 [P,Hkv,16,D], v_caches[l] uint8, v_scales[l] fp32 [Hkv];
    block_table int32 [B, max_pages] on the host (numpy) covering every
    position up to max_seq_len; inv_freq / attn_factor from
    rope.rope_inv_freq.  Row buffers hold batch * max_nodes rows; rows behind
    the last tree are padding (slot -1) and stay as they are.  The workspace and
    the tree buffers serve one step at a time: steps and replays that overlap
    need an object each."""

    def __init__(self, k_caches, v_caches, v_scales, block_table, batch, max_nodes, max_seq_len,
                 num_qo_heads, inv_freq, attn_factor=1.0, interleaved=False, sm_scale=None,
                 validate=True):
        if validate:
            validate_scales(v_scales)
        dev = k_caches[0].device
        self.k_caches, self.v_caches, self.v_scales = k_caches, v_caches, v_scales
        self.layers = len(k_caches)
        self.num_pages, self.hkv, _, self.d = k_caches[0].shape
        self.hq, self.batch = int(num_qo_heads), int(batch)
        self.max_nodes, self.max_seq_len = int(max_nodes), int(max_seq_len)
        self.rows = self.batch * self.max_nodes
        self.interleaved, self.attn_factor = bool(interleaved), float(attn_factor)
        self.sm_scale = float(sm_scale if sm_scale is not None else 1.0 / math.sqrt(self.d))
        self.inv_freq = inv_freq.to(dev)
        self.table_host = np.ascontiguousarray(block_table, np.int32)
        self.block_table = torch.from_numpy(self.table_host).to(dev)

        def ints(n, dtype=torch.int32):
            return torch.zeros(n, dtype=dtype, device=dev)

        self.qo_indptr, self.seq_lens = ints(self.batch + 1), ints(self.batch)
        self.new_seq_lens = ints(self.batch)
        self.tree_mask, self.slots = ints(self.rows, torch.int64), ints(self.rows, torch.int64)
        self.slots.fill_(-1)
        self.positions, self.parents = ints(self.rows), ints(self.rows)
        self.path, self.path_len = ints((self.batch, self.max_nodes)), ints(self.batch)
        self.next_token = ints(self.batch)
        self.dev_error = ints(1)
        self.k_ptrs, self.v_ptrs = K.layer_pointers(k_caches), K.layer_pointers(v_caches)
        n = K.k16v8_tree_workspace_size(self.rows, self.batch, self.max_nodes, self.hq, self.hkv,
                                        self.d, self.max_seq_len)
        if n == 0:
            raise ValueError(f"no tree attention for {self.batch} sequences of up to "
                             f"{self.max_nodes} nodes and {self.max_seq_len} positions, "
                             f"{self.hq} over {self.hkv} heads of {self.d}")
        self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        self.graph = None

    def set_trees(self, parents, prefix_lens) -> None:
        """The trees of the next step: parents[b] of sequence b's nodes (at
        most max_nodes; none for an idle sequence), which take the positions
        prefix_lens[b] ..  of its cache."""
        if len(parents) != self.batch or len(prefix_lens) != self.batch:
            raise ValueError(f"{self.batch} sequences expected")
        indptr = np.zeros(self.batch + 1, np.int32)
        lens = np.zeros(self.batch, np.int32)
        mask, slots = np.zeros(self.rows, np.int64), np.full(self.rows, -1, np.int64)
        positions, par = np.zeros(self.rows, np.int32), np.full(self.rows, -1, np.int32)
        o = 0
        for b, (p, base) in enumerate(zip(parents, prefix_lens)):
            n, base = len(p), int(base)
            if n > self.max_nodes:
                raise ValueError(f"sequence {b}: {n} nodes, at most {self.max_nodes}")
            if base < 0 or base + n > min(self.max_seq_len, self.table_host.shape[1] * K.PAGE_SIZE):
                raise ValueError(f"sequence {b}: positions {base}..{base + n} beyond its cache")
            mask[o:o + n] = tree_masks(p)
            positions[o:o + n] = base + tree_depths(p)
            par[o:o + n] = p
            at = base + np.arange(n, dtype=np.int64)
            slots[o:o + n] = (self.table_host[b, at // K.PAGE_SIZE].astype(np.int64) * K.PAGE_SIZE
                              + at % K.PAGE_SIZE)
            o += n
            indptr[b + 1], lens[b] = o, base + n
        for dst, src in ((self.qo_indptr, indptr), (self.seq_lens, lens), (self.tree_mask, mask),
                         (self.slots, slots), (self.positions, positions), (self.parents, par)):
            dst.copy_(torch.from_numpy(src))

    def layer(self, li, q, k, v, q_rot, out, lse=None):
        """Layer li: q, k, v [rows, heads, D] of the nodes before rotation;
        q_rot fp16 scratch [rows, Hq, D]; out fp16 [rows, Hq, D]."""
        K.k16v8_rope_kv_append(q, k, v, self.positions, self.inv_freq, self.slots,
                               self.v_scales[li], q_rot, self.k_caches[li], self.v_caches[li],
                               self.interleaved, self.attn_factor, self.dev_error)
        K.k16v8_paged_tree_attention(q_rot, self.qo_indptr, self.max_nodes, self.tree_mask,
                                     self.k_caches[li], self.v_caches[li], self.v_scales[li],
                                     self.block_table, self.seq_lens, self.max_seq_len,
                                     self.sm_scale, self.workspace, out, lse, self.dev_error)

    def step(self, qs, ks, vs, q_rot, outs, lses=None):
        for li in range(self.layers):
            self.layer(li, qs[li], ks[li], vs[li], q_rot, outs[li],
                       None if lses is None else lses[li])

    def verify(self, target_probs, draft_probs, tokens, uniforms):
        """Accepted paths and next tokens into path, path_len, next_token."""
        K.k16v8_tree_verify(target_probs, draft_probs, tokens, self.parents, self.qo_indptr,
                            self.max_nodes, uniforms, self.path, self.path_len, self.next_token,
                            self.dev_error)

    def compact(self):
        """The accepted rows to the front of their trees, in every layer; the
        lengths after the step into new_seq_lens."""
        K.k16v8_kv_compact(self.k_ptrs, self.v_ptrs, self.num_pages, self.hkv, self.d,
                           self.block_table, self.seq_lens, self.qo_indptr, self.path,
                           self.path_len, self.new_seq_lens, self.dev_error)

    def capture(self, qs, ks, vs, q_rot, outs, lses=None):
        """Capture the layers' step into a CUDA graph over these buffers."""
        self.step(qs, ks, vs, q_rot, outs, lses)  # eager run configures the kernels
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="thread_local"):
            self.step(qs, ks, vs, q_rot, outs, lses)
        self.graph = g
        return g

    def replay(self):
        if self.graph is None:
            raise RuntimeError("capture() first")
        self.graph.replay()

    def check(self) -> int:
        """Synchronise and return the device error word (0 = clean)."""
        return K.k16v8_read_device_error(self.dev_error)
