"""Paged forms of a step's dense caches, for the paged tables' tests."""

import numpy as np
import torch

from stream_speculative_decode_gb300.inputs import NKV, D, to_torch_bf16


def page_lists(keys, page, seed, spare=3, extra_ids=()):
    """Scattered page lists of streams with ``keys`` keys: (lists, n_pages)."""
    need = [-(-k // page) for k in keys]
    n_pages = sum(need) + spare
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    lists, at = [], 0
    for n in need:
        lists.append(ids[at:at + n])
        at += n
    return lists, n_pages


def to_pool(caches, keys, lists, page, n_pages, fill=float("nan")):
    """A pool [n_pages][NKV][page][D] holding each cache's first keys in its
    pages, and ``fill`` (NaN by default) everywhere else."""
    pool = torch.full((n_pages, NKV, page, D), fill, dtype=torch.bfloat16, device="cuda")
    for c, k, ids in zip(caches, keys, lists):
        c = c if isinstance(c, torch.Tensor) else to_torch_bf16(c)
        for i, p in enumerate(ids):
            n = min(page, k - i * page)
            pool[int(p), :, :n] = c[:, i * page:i * page + n]
    return pool


class PagedAttn:
    """A step's attention inputs in pages: the table and its buffers."""

    def __init__(self, tf, inp, page, seed=0, fill=float("nan"), prompt=False):
        self.tf, self.inp = tf, inp
        keys = [k for _, _, k in inp.streams]
        self.lists, self.n_pages = page_lists(keys, page, seed)
        n_attn = len(inp.q)
        self.K = [to_pool(inp.K[l], keys, self.lists, page, self.n_pages, fill) for l in range(n_attn)]
        self.V = [to_pool(inp.V[l], keys, self.lists, page, self.n_pages, fill) for l in range(n_attn)]
        self.q = [x.cuda() if isinstance(x, torch.Tensor) else to_torch_bf16(x) for x in inp.q]
        table = [(r, o, k, len(ids) * page) for (r, o, k), ids in zip(inp.streams, self.lists)]
        ids = np.concatenate(self.lists)
        if prompt:
            r, _, k, cap = table[0]
            self.seg = tf.tf_paged_prompt_build(r, k, cap, None, ids, page, self.n_pages, self.K, self.V, 0, n_attn)
        else:
            self.seg = tf.tf_paged_build(table, None, None, ids, page, self.n_pages, self.K, self.V, 0, n_attn)
        self.partials = torch.full((max(self.seg.partials_bytes // 4, 4),), float("nan"), device="cuda")
        self.out = [torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for q in self.q]

    def run(self, full=False, stream=None):
        for l, (q, out) in enumerate(zip(self.q, self.out)):
            self.tf.tf_attn_paged(self.seg, l, q, self.partials, out, full, stream)
        return self.out
