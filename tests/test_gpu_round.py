"""The serving operators together, as a round over a paged cache runs them: a
prompt's rows normed, rotated and appended, its attention; a verify round of
several streams (append, attention, sampled picks, accept) queued without a
host wait; a fork of a stream by a copied last page; the round after it.

Each operator's result is checked against its float64 oracle on what it read
(the tolerances are those of the operators' own tests), so the chain is held
link by link.
"""

import numpy as np
import pytest

from oracle import sample as OS
from oracle import step as O

pytestmark = pytest.mark.gpu

LAYERS, PAGE, POOL, VOCAB = 2, 16, 160, 2000


@pytest.fixture(scope="module")
def mods():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf, inputs
    torch.cuda.set_device(0)
    return tf, inputs, torch


class Model:
    """Pools of two attention layers and the projections' stand-ins of a call."""

    def __init__(self, mods, seed):
        self.tf, self.inputs, self.torch = mods
        torch = self.torch
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        nan = float("nan")
        self.K, self.V = ([torch.full((POOL, 8, PAGE, 64), nan, dtype=torch.bfloat16, device="cuda")
                           for _ in range(LAYERS)] for _ in range(2))
        self.qw, self.kw = 1 + self.normal(64, std=0.2), 1 + self.normal(64, std=0.2)
        self.free = [int(x) for x in np.random.default_rng(seed).permutation(POOL)]

    def normal(self, *shape, std=1.0):
        return (self.torch.randn(shape, generator=self.g, device="cuda") * std).to(self.torch.bfloat16)

    def grow(self, pages, keys):
        while len(pages) * PAGE < keys:
            pages.append(self.free.pop())
        return pages

    def projections(self, rows):
        return [(self.normal(rows, 2048), self.normal(rows, 512), self.normal(rows, 512)) for _ in range(LAYERS)]

    def layers(self, seg, proj, rows, full=False):
        """Every layer's append and attention; the rotated queries and outputs."""
        tf, torch = self.tf, self.torch
        partials = torch.empty(max(16, seg.partials_bytes), dtype=torch.uint8, device="cuda")
        qs, outs = [], []
        for l, (q, k, v) in enumerate(proj):
            qo, out = (torch.empty((rows, 32, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            tf.tf_qk_rows(seg, l, q, 2048, k, 512, v, 512, self.qw, self.kw, 1e-5, 1e6, qo)
            tf.tf_attn_paged(seg, l, qo, partials, out, full)
            qs.append(qo)
            outs.append(out)
        return qs, outs

    def cache(self, pool, pages, keys):
        """bf16 bits [8][keys][64] of a stream's keys."""
        c = pool[self.torch.tensor(pages, device="cuda")].permute(1, 0, 2, 3).reshape(8, -1, 64)[:, :keys]
        return self.inputs.to_numpy_bits(c)

    def check_attention(self, streams, qs, outs, full=False):
        """streams: [(rows, offset, keys, pages)]"""
        for l in range(LAYERS):
            q, out = self.inputs.to_numpy_bits(qs[l]), O.bf16_to_f64(self.inputs.to_numpy_bits(outs[l]))
            for r, o, k, pages in streams:
                K, V = self.cache(self.K[l], pages, k), self.cache(self.V[l], pages, k)
                ref = O.attention_stream(q[o:o + r], K, V, k, r, full=full)
                err = np.abs(out[o:o + r] - ref)
                assert (err <= 2e-3 + 2.0 ** -8 * (np.abs(ref) + 2e-3)).all()

    def check_append(self, streams, proj, qs):
        from test_gpu_qk import check
        torch = self.torch
        for l, (q, k, v) in enumerate(proj):
            for r, o, n, pages in streams:
                pos = np.arange(n - r, n)
                check(qs[l][o:o + r], q[o:o + r].view(r, 32, 64), self.qw, pos, "q")
                at = torch.tensor([pages[p // PAGE] for p in pos], device="cuda"), torch.from_numpy(pos % PAGE).cuda()
                check(self.K[l][at[0], :, at[1]], k[o:o + r].view(r, 8, 64), self.kw, pos, "k")
                assert torch.equal(self.V[l][at[0], :, at[1]].view(torch.int16), v[o:o + r].view(r, 8, 64).view(torch.int16))


def table(m, streams):
    """A verify table of [(rows, keys, pages)]; the same with row offsets."""
    off, rows, full = 0, [], []
    for r, k, pages in streams:
        rows.append((r, off, k, len(pages) * PAGE))
        full.append((r, off, k, pages))
        off += r
    seg = m.tf.tf_paged_build(rows, None, None, [p for _, _, pages in streams for p in pages], PAGE, POOL, m.K, m.V, 0, LAYERS)
    return seg, full


def test_prompt_round_fork_round(mods):
    tf, inputs, torch = mods
    m = Model(mods, 3)

    # a prompt of 70 rows in two calls, then one of 5
    long, short = [], []
    done = 0
    for rows in (37, 33):
        m.grow(long, done + rows)
        seg = tf.tf_paged_prompt_build(rows, done + rows, len(long) * PAGE, None, long, PAGE, POOL, m.K, m.V, 0, LAYERS)
        proj = m.projections(rows)
        qs, outs = m.layers(seg, proj, rows)
        torch.cuda.synchronize()
        done += rows
        at = [(rows, 0, done, long)]
        m.check_append(at, proj, qs)
        m.check_attention(at, qs, outs)
        seg.free()
    m.grow(short, 5)
    seg = tf.tf_paged_prompt_build(5, 5, PAGE, None, short, PAGE, POOL, m.K, m.V, 0, LAYERS)
    qs, outs = m.layers(seg, m.projections(5), 5)
    torch.cuda.synchronize()
    m.check_attention([(5, 0, 5, short)], qs, outs)
    seg.free()

    # a verify round: windows of 10 rows (tensor cores) and 3; append, attention,
    # sampled picks and accept queued with no host wait between
    R = 13
    seg, streams = table(m, [(10, 80, m.grow(long, 80)), (3, 8, short)])
    proj = m.projections(R)
    logits = m.normal(R, VOCAB, std=3.0)
    logits[4, 7] = float("nan")
    u = torch.rand(R, generator=m.g, device="cuda") * 0.999
    t, p = torch.full((R,), 0.9, device="cuda"), torch.full((R,), 0.8, device="cuda")
    k = torch.full((R,), 60, dtype=torch.int32, device="cuda")
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    pick, prob, flag = i32(R), torch.empty(R, device="cuda"), torch.empty(R, dtype=torch.uint8, device="cuda")
    picks, _, flags = OS.sample_rows(inputs.to_numpy_bits(logits), u.cpu().numpy(), temperature=t.cpu().numpy(),
                                     top_k=k.cpu().numpy(), top_p=p.cpu().numpy())
    ids = np.zeros(R, np.int32)
    ids[1:4] = picks[:3]                        # three drafts that the target draws too, then row 4's NaN
    ids[11] = (picks[10] + 1) % VOCAB
    ids_dev = torch.from_numpy(ids).cuda()
    acc, nxt, keys, sflag = i32(2), i32(2), i32(2), torch.empty(2, dtype=torch.uint8, device="cuda")
    qs, outs = m.layers(seg, proj, R)
    tf.tf_sample_rows(logits, R, VOCAB, VOCAB, t, k, p, None, u, pick, prob, flag)
    tf.tf_accept(seg, ids_dev, pick, flag, VOCAB, acc, nxt, keys, sflag, rewind_conv=False)
    torch.cuda.synchronize()
    m.check_append(streams, proj, qs)
    m.check_attention(streams, qs, outs)
    assert np.array_equal(pick.cpu().numpy(), picks) and np.array_equal(flag.cpu().numpy(), flags)
    want = O.accept_all([(r, o, n) for r, o, n, _ in streams], ids, picks, flags, VOCAB)
    for a, b in zip((acc, nxt, keys, sflag), want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert acc.tolist() == [3, 0] and keys.tolist() == [74, 6]
    seg.free()

    # both streams fork at their accepted keys: whole pages are shared, the last
    # one is copied in every layer's pools
    grown = []
    src, dst, n = [], [], []
    for (r, o, _, pages), length in zip(streams, keys.tolist()):
        pages = pages[:-(-length // PAGE)]
        child = pages[:-1] + [m.free.pop()]
        if length % PAGE == 0:
            child = list(pages)
        else:
            src.append(pages[-1])
            dst.append(child[-1])
            n.append(length % PAGE)
        grown += [(pages, length), (child, length)]
    tf.tf_pages_copy(m.K + m.V, PAGE, POOL, src, dst, n)

    # the next round: parent and child take the same rows, then see the same keys
    windows = []
    for pages, length in grown:
        windows.append((2, length + 2, m.grow(list(pages), length + 2)))
    seg, streams = table(m, windows)
    proj = m.projections(8)
    for q, k_, v in proj:
        for x in (q, k_, v):
            x[2:4], x[6:8] = x[0:2].clone(), x[4:6].clone()
    qs, outs = m.layers(seg, proj, 8)
    torch.cuda.synchronize()
    m.check_append(streams, proj, qs)
    m.check_attention(streams, qs, outs)
    for l in range(LAYERS):
        b = outs[l].view(torch.int16)
        assert torch.equal(b[0:2], b[2:4]) and torch.equal(b[4:6], b[6:8])
    qs, outs = m.layers(seg, proj, 8, full=True)      # the drafter's block form on the same table
    torch.cuda.synchronize()
    m.check_attention(streams, qs, outs, full=True)
    seg.free()


def test_round_in_a_graph(mods):
    """A round captured once and replayed on new projections, logits and numbers."""
    tf, inputs, torch = mods
    m = Model(mods, 5)
    R = 14
    a, b = m.grow([], 300), m.grow([], 41)
    for pool in m.K + m.V:
        pool.copy_(m.normal(*pool.shape))
    seg, streams = table(m, [(12, 300, a), (2, 41, b)])
    proj = m.projections(R)
    logits, u = m.normal(R, VOCAB, std=3.0), torch.rand(R, generator=m.g, device="cuda")
    qo, out = ([torch.empty((R, 32, 64), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)] for _ in range(2))
    partials = torch.empty(max(16, seg.partials_bytes), dtype=torch.uint8, device="cuda")
    pick, flag = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.uint8, device="cuda")

    def round_():
        for l, (q, k, v) in enumerate(proj):
            tf.tf_qk_rows(seg, l, q, 2048, k, 512, v, 512, m.qw, m.kw, 1e-5, 1e6, qo[l])
            tf.tf_attn_paged(seg, l, qo[l], partials, out[l])
        tf.tf_sample_rows(logits, R, VOCAB, VOCAB, None, None, None, None, u, pick, None, flag)
        tf.tf_pages_copy(m.K + m.V, PAGE, POOL, [a[0]], [m.free[0]])

    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        round_()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for x in [y for layer in proj for y in layer]:
            x.copy_(m.normal(*x.shape))
        logits.copy_(m.normal(R, VOCAB, std=3.0))
        u.uniform_(0, 0.999)
        g.replay()
        torch.cuda.synchronize()
        m.check_append(streams, proj, qo)
        m.check_attention(streams, qo, out)
        picks, _, flags = OS.sample_rows(inputs.to_numpy_bits(logits), u.cpu().numpy())
        assert np.array_equal(pick.cpu().numpy(), picks) and np.array_equal(flag.cpu().numpy(), flags)
        for pool in m.K + m.V:
            assert torch.equal(pool[m.free[0]].view(torch.int16), pool[a[0]].view(torch.int16))
        bits = [o.view(torch.int16).clone() for o in out]
        round_()                                       # the same calls outside the graph
        torch.cuda.synchronize()
        assert all(torch.equal(x, o.view(torch.int16)) for x, o in zip(bits, out))
    seg.free()
