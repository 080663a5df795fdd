"""The low-precision operators together, as a round's layers run them: norm of the
residual stream into 8-bit rows, the projections by 4-bit weights, the append to an
8-bit paged cache, its attention, the output projection, the next norm; a prompt, a
verify round, a fork by a copied last page, the round after it, and the logits. All
of it is queued without a host wait, then each operator's result is held to its own
float64 reference on what it read (the operators' own bounds)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

LAYERS, PAGE, POOL, H, VOCAB = 2, 16, 120, 2048, 1000
EPS, THETA = 1e-5, 1e6


@pytest.fixture(scope="module")
def tf():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf


class Model:
    def __init__(self, tf, seed):
        from test_gpu_linear import weights
        self.tf = tf
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        pool = lambda *s: torch.full((POOL, 8) + s, 0x7F, dtype=torch.uint8, device="cuda")
        self.K, self.V = ([pool(PAGE, 64) for _ in range(LAYERS)] for _ in range(2))
        self.ks, self.vs = ([pool(PAGE // 16) for _ in range(LAYERS)] for _ in range(2))
        self.free = [int(x) for x in np.random.default_rng(seed).permutation(POOL)]
        unit = lambda w: (w[0], torch.full_like(w[1], 0x38), w[2] / (w[0].shape[1] * 2 * 21.5) ** 0.5)
        self.w = [{n: unit(weights(N, H, 10 * l + i)) for i, (n, N) in
                   enumerate((("q", 2048), ("k", 512), ("v", 512), ("o", H)))} for l in range(LAYERS)]
        self.head = unit(weights(VOCAB, H, 99))
        self.norm = [(1 + self.normal(H, std=0.2)) for _ in range(LAYERS + 1)]
        self.qw, self.kw = 1 + self.normal(64, std=0.2), 1 + self.normal(64, std=0.2)

    def normal(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * std).to(torch.bfloat16)

    def grow(self, pages, keys):
        while len(pages) * PAGE < keys:
            pages.append(self.free.pop())
        return pages

    def linear(self, x, scales, w, log, what):
        y = torch.empty((len(x), len(w[0])), dtype=torch.bfloat16, device="cuda")
        self.tf.tf_linear_rows(x, x.shape[1], scales, len(x), x.shape[1], *w, len(w[0]), y, len(w[0]))
        log.append((what, "linear", (x.clone(), None if scales is None else scales.clone(), w, y)))
        return y

    def forward(self, seg, streams, x, log):
        """The layers over the rows x; streams [(rows, offset, keys, pages)]."""
        tf, R = self.tf, len(x)
        partials = torch.empty(max(16, seg.partials_bytes), dtype=torch.uint8, device="cuda")
        res = torch.zeros_like(x)
        for l in range(LAYERS + 1):
            total = torch.empty_like(x)
            codes = torch.empty((R, H), dtype=torch.uint8, device="cuda")
            scales = torch.empty((R, H // 32), dtype=torch.uint8, device="cuda")
            tf.tf_norm_rows(x, H, res, H, self.norm[l], EPS, R, H, total, H, codes, scales)
            log.append((l, "norm", (x, res, self.norm[l], total, codes, scales)))
            res = total
            if l == LAYERS:
                return self.linear(codes, scales, self.head, log, "head")
            q, k, v = (self.linear(codes, scales, self.w[l][n], log, (l, n)) for n in "qkv")
            qo, out = (torch.empty((R, 32, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            pools = [c[l] for c in (self.K, self.V, self.ks, self.vs)]
            before = [c.clone() for c in pools]
            tf.tf_qk_rows(seg, l, q, 2048, k, 512, v, 512, self.qw, self.kw, EPS, THETA, qo)
            after = [c.clone() for c in pools]
            log.append((l, "append", (streams, q, k, v, qo, before, after)))
            tf.tf_attn_paged(seg, l, qo, partials, out)
            log.append((l, "attention", (streams, qo, after, out)))
            x = self.linear(out.view(R, 2048), None, self.w[l]["o"], log, (l, "o"))

    def check(self, log):
        import test_gpu_linear
        import test_gpu_norm
        from scaled import ScaledAttn, check_attention, value
        from test_gpu_qk import check as check_qk
        from test_gpu_qk import reference
        for what, kind, a in log:
            if kind == "norm":
                test_gpu_norm.check(H, *a, what=what)
            elif kind == "linear":
                x, xs, w, y = a
                v = x.double() if xs is None else value(x, xs.repeat_interleave(32, 1))
                test_gpu_linear.check(y, v, *w, what=what)
            elif kind == "attention":
                streams, q, (K, V, ks, vs), out = a
                for r, o, n, pages in streams:
                    kv, _ = ScaledAttn.cache(None, K, ks, pages, n)
                    vv, vb = ScaledAttn.cache(None, V, vs, pages, n)
                    check_attention(q[o:o + r], kv, vv, vb, n, out[o:o + r], what=what)
            else:
                streams, q, k, v, qo, before, after = a
                for r, o, n, pages in streams:
                    pos = np.arange(n - r, n)
                    check_qk(qo[o:o + r], q[o:o + r].view(r, 32, 64), self.qw, pos, what)
                    for c, x in ((0, torch.from_numpy(reference(k[o:o + r].view(r, 8, 64), self.kw, pos)[0]).cuda()),
                                 (1, v[o:o + r].view(r, 8, 64).double())):
                        new, s = ScaledAttn.cache(None, after[c], after[2 + c], pages, n)
                        x = x.transpose(0, 1)
                        step = torch.ldexp(torch.full_like(x, 2.0 ** -10), s[:, n - r:, None].int() - 127)
                        err = (new[:, n - r:] - x).abs()
                        # half a step, and (K) the fp32 rotation's 2^-19 of both partners, at most 2^-19 * 2 * 464 scales
                        assert (err <= torch.maximum(2.0 ** -4 * x.abs(), step) * (1 + 2.0 ** -10) + step * 2).all(), what
                        old, _ = ScaledAttn.cache(None, before[c], before[2 + c], pages, n - r)
                        kept = new[:, :n - r]
                        low = torch.ldexp(torch.ones_like(kept), s[:, :n - r, None].int() - 127 - 6)
                        assert (torch.where(old.abs() >= low, old == kept, (old - kept).abs() <= low / 8)).all(), what


def table(m, streams):
    off, rows, full = 0, [], []
    for r, k, pages in streams:
        rows.append((r, off, k, len(pages) * PAGE))
        full.append((r, off, k, pages))
        off += r
    seg = m.tf.tf_paged_scaled_build(rows, None, None, [p for _, _, x in streams for p in x], PAGE, POOL, m.K, m.V, m.ks,
                                     m.vs, 0, LAYERS)
    return seg, full


def test_prompt_round_fork_round(tf):
    m, log, segs = Model(tf, 3), [], []
    long, short, done = [], [], 0
    for rows in (37, 33):
        m.grow(long, done + rows)
        seg = tf.tf_paged_scaled_prompt_build(rows, done + rows, len(long) * PAGE, None, long, PAGE, POOL, m.K, m.V, m.ks,
                                              m.vs, 0, LAYERS)
        done += rows
        m.forward(seg, [(rows, 0, done, list(long))], m.normal(rows, H), log)
        segs.append(seg)
    m.grow(short, 5)
    seg = tf.tf_paged_scaled_prompt_build(5, 5, len(short) * PAGE, None, short, PAGE, POOL, m.K, m.V, m.ks, m.vs, 0, LAYERS)
    m.forward(seg, [(5, 0, 5, list(short))], m.normal(5, H), log)
    segs.append(seg)

    # a verify round; half of the long stream's window is rejected
    m.grow(long, 70 + 9)
    m.grow(short, 5 + 2)
    seg, full = table(m, [(9, 79, list(long)), (2, 7, list(short))])
    logits = m.forward(seg, full, m.normal(11, H), log)
    segs.append(seg)
    pick = torch.empty(11, dtype=torch.int32, device="cuda")
    flag = torch.empty(11, dtype=torch.uint8, device="cuda")
    tf.tf_argmax_rows(logits, 11, VOCAB, VOCAB, pick, flag)

    # the long stream forks at 74 keys: a copied last page, then both go on
    child = long[:74 // PAGE] + [m.free.pop()]
    tf.tf_pages_copy_scaled(m.K + m.V, m.ks + m.vs, PAGE, POOL, [long[74 // PAGE]], [child[-1]], [74 % PAGE])
    parent = list(long)
    seg, full = table(m, [(3, 77, parent), (4, 78, child), (1, 7, list(short))])
    m.forward(seg, full, m.normal(8, H), log)
    segs.append(seg)

    torch.cuda.synchronize()
    assert not flag.any() and torch.equal(pick.long(), logits.float().argmax(1))
    m.check(log)
    for s in segs:
        assert tf.tf_segments_status(s) == (tf.TF_OK, 0)


def test_a_round_in_a_graph(tf):
    """The same round captured and replayed gives the same bytes."""
    m = Model(tf, 4)
    lists = [m.grow([], 40), m.grow([], 300)]
    seg = tf.tf_paged_scaled_prompt_build(292, 292, len(lists[1]) * PAGE, None, lists[1], PAGE, POOL, m.K, m.V, m.ks, m.vs,
                                          0, LAYERS)
    m.forward(seg, [(292, 0, 292, lists[1])], m.normal(292, H), [])
    seg2, full = table(m, [(16, 16, lists[0][:1]), (8, 300, lists[1])])
    x = m.normal(24, H)
    start = [[c.clone() for c in p] for p in (m.K, m.V, m.ks, m.vs)]
    want = m.forward(seg2, full, x, []).clone()
    end = [[c.clone() for c in p] for p in (m.K, m.V, m.ks, m.vs)]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        got = m.forward(seg2, full, x, [])
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        for p, q in zip((m.K, m.V, m.ks, m.vs), start):
            for c, d in zip(p, q):
                c.copy_(d)
        got.zero_()
        g.replay()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        for p, q in zip((m.K, m.V, m.ks, m.vs), end):
            assert all(torch.equal(c, d) for c, d in zip(p, q))
