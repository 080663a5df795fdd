"""tf_qk_rows against the formula in float64.

Tolerance, per element, with n the normed head in float64: the fp32 norm is off
by at most 2^-20 of n (a 64-term sum of squares in 18 additions, halved by the
root; a reciprocal square root of 2 ulp, three products), a sine or cosine by
4 * 2^-24 (2^-25 half turns of angle from its 24-bit fraction, times pi, and 2
ulp), two products and a sum by 3 * 2^-24: together below
e = 2^-19 (|n_j| + |n_{j+32}|). The store rounds to bf16: half a step, 2^-8 of
the value. V and every other slot of the caches: bit for bit.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

EPS, THETA = 1e-5, 1e6


@pytest.fixture(scope="module")
def mods():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf, torch


def reference(x, w, pos, eps=EPS, theta=THETA):
    """(y, |n_j| + |n_{j+32}|) in float64 of heads x [R][heads][64] at pos [R]."""
    x, w = x.double().cpu().numpy(), w.double().cpu().numpy()
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    a = np.asarray(pos, dtype=np.float64)[:, None] * theta ** (-np.arange(32) / 32)   # good to 2^-31 at 2^22
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    lo, hi = n[..., :32], n[..., 32:]
    size = np.abs(lo) + np.abs(hi)
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1), np.concatenate([size, size], -1)


def check(got, x, w, pos, what, **kw):
    ref, size = reference(x, w, pos, **kw)
    e = 2.0 ** -19 * size
    err = np.abs(got.double().cpu().numpy() - ref)
    over = err - (e + 2.0 ** -8 * (np.abs(ref) + e) + 2.0 ** -126)
    assert not (over > 0).any(), (what, float(over.max()))


def bits(t):
    return t.contiguous().view(t.dtype if t.dtype != _bf16() else _i16())


def _bf16():
    import torch
    return torch.bfloat16


def _i16():
    import torch
    return torch.int16


class Case:
    """Inputs of a table: caches filled with random bits to see what is left alone."""

    def __init__(self, mods, streams, page=0, n_layers=2, seed=0, prompt=False, pads=(0, 0, 0), lists=None, n_pages=None):
        tf, torch = mods
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        off, table = 0, []
        for r, k in streams:
            table.append((r, off, k, -(-k // page) * page if page else k + 5))
            off += r
        self.R, self.table, self.page = off, table, page
        if page:
            if lists is None:
                from paged import page_lists
                lists, n_pages = page_lists([k for _, k in streams], page, seed)
            self.lists = lists
            self.K, self.V = ([normal(n_pages, 8, page, 64) for _ in range(n_layers)] for _ in range(2))
            ids = np.concatenate(lists)
            if prompt:
                r, _, k, cap = table[0]
                self.seg = tf.tf_paged_prompt_build(r, k, cap, None, ids, page, n_pages, self.K, self.V, 0, n_layers)
            else:
                self.seg = tf.tf_paged_build(table, None, None, ids, page, n_pages, self.K, self.V, 0, n_layers)
        else:
            self.K, self.V = ([[normal(8, t[3], 64) for t in table] for _ in range(n_layers)] for _ in range(2))
            k, v = [c for l in self.K for c in l], [c for l in self.V for c in l]
            if prompt:
                r, _, n, cap = table[0]
                self.seg = tf.tf_prompt_build(r, n, cap, None, k, v, 0, n_layers)
            else:
                self.seg = tf.tf_segments_build(table, None, None, k, v, 0, n_layers)
        self.qb, self.kb, self.vb = normal(off, 2048 + pads[0]), normal(off, 512 + pads[1]), normal(off, 512 + pads[2])
        self.q, self.k, self.v = self.qb[:, :2048], self.kb[:, :512], self.vb[:, :512]
        self.qw, self.kw = 1 + normal(64, std=0.3), 1 + normal(64, std=0.3)
        self.pos = np.concatenate([np.arange(k - r, k) for r, k in streams])
        self.who = np.concatenate([np.full(r, s) for s, (r, _) in enumerate(streams)])
        self.out = torch.full((off, 32, 64), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, mods, layer=1, out=None, eps=EPS, theta=THETA, stream=None):
        mods[0].tf_qk_rows(self.seg, layer, self.qb, self.qb.shape[1], self.kb, self.kb.shape[1], self.vb,
                           self.vb.shape[1], self.qw, self.kw, eps, theta, self.out if out is None else out, stream)

    def copies(self):
        flat = lambda c: [x.clone() for x in c] if self.page else [[x.clone() for x in l] for l in c]
        return flat(self.K), flat(self.V)

    def rows_of(self, cache):
        """The appended rows [R][8][64] of a layer's caches, and the caches with them put back to zero."""
        import torch
        left = [cache.clone()] if self.page else [c.clone() for c in cache]
        got = []
        for s, p in zip(self.who, self.pos):
            at = (left[0][int(self.lists[s][p // self.page])], p % self.page) if self.page else (left[s], p)
            got.append(at[0][:, at[1]].clone())
            at[0][:, at[1]] = 0
        return torch.stack(got), left

    def check(self, mods, before, layer=1, q=None, out=None, **kw):
        import torch
        torch.cuda.synchronize()
        q = self.q if q is None else q
        check((self.out if out is None else out).view(self.R, 32, 64), q.reshape(self.R, 32, 64), self.qw, self.pos, "q", **kw)
        krows, kleft = self.rows_of(self.K[layer])
        vrows, vleft = self.rows_of(self.V[layer])
        check(krows, self.k.reshape(self.R, 8, 64), self.kw, self.pos, "k", **kw)
        assert torch.equal(bits(vrows), bits(self.v.reshape(self.R, 8, 64)))
        for l in range(len(self.K)):
            for now, old, left in ((self.K[l], before[0][l], kleft), (self.V[l], before[1][l], vleft)):
                if l == layer:      # every other slot as it was
                    want = self.rows_of(old)[1]
                    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(left, want))
                else:
                    now, old = ([now], [old]) if self.page else (now, old)
                    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(now, old))


STREAMS = [(1, 1), (16, 16), (3, 500), (8, 65), (1, 64), (2, 33), (5, 4097)]


@pytest.mark.parametrize("page", [0, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("layer", [0, 1])
def test_rounds(mods, page, layer):
    c = Case(mods, STREAMS, page, seed=page + layer)
    before = c.copies()
    c.run(mods, layer)
    c.check(mods, before, layer)
    c.seg.free()


@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("rows,cached", [(1, 0), (31, 0), (33, 100), (700, 5)])
def test_prompt(mods, page, rows, cached):
    c = Case(mods, [(rows, rows + cached)], page, seed=rows, prompt=True)
    before = c.copies()
    c.run(mods)
    c.check(mods, before)
    c.seg.free()


@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("streams", [64, 14, 15])
def test_many_rows(mods, page, streams):
    """1,024 rows, and rows about the 512 from which a warp takes a whole row (504 and 540)."""
    shape = [(16, 20 + 61 * s) for s in range(64)] if streams == 64 else STREAMS * streams
    c = Case(mods, shape, page, seed=streams + page, pads=(8, 0, 0))
    before = c.copies()
    c.run(mods)
    c.check(mods, before)
    c.seg.free()


def test_many_rows_in_place(mods):
    c = Case(mods, STREAMS * 20, 64, seed=30)
    before, q = c.copies(), c.q.clone()
    c.run(mods, out=c.qb)
    c.check(mods, before, q=q, out=c.qb)
    c.seg.free()


@pytest.mark.parametrize("pads", [(64, 0, 8), (8, 128, 512), (0, 8, 0)])
def test_row_strides(mods, pads):
    c = Case(mods, STREAMS, 16, seed=3, pads=pads)
    before = c.copies()
    c.run(mods)
    c.check(mods, before)
    c.seg.free()


def test_slices_of_one_projection(mods):
    """q, k and v as column ranges of one buffer's rows (1,088 more columns behind them)."""
    tf, torch = mods
    c = Case(mods, STREAMS, 0, seed=4)
    width = 2048 + 512 + 512 + 1088
    buf = torch.randn((c.R, width), device="cuda").to(torch.bfloat16)
    c.q, c.k, c.v = buf[:, :2048], buf[:, 2048:2560], buf[:, 2560:2560 + 512]
    before = c.copies()
    tf.tf_qk_rows(c.seg, 1, c.q, width, c.k, width, c.v, width, c.qw, c.kw, EPS, THETA, c.out)
    c.check(mods, before)
    c.seg.free()


def test_in_place(mods):
    c = Case(mods, STREAMS, 32, seed=5)
    before, q = c.copies(), c.q.clone()
    c.run(mods, out=c.qb)
    c.check(mods, before, q=q, out=c.qb)
    c.seg.free()


@pytest.mark.parametrize("theta,eps", [(10000.0, 1e-6), (1.0, 1e-5), (5e8, 0.5)])
def test_theta_and_eps(mods, theta, eps):
    c = Case(mods, [(2, 30000), (4, 70)], 16, seed=6)
    before = c.copies()
    c.run(mods, theta=theta, eps=float(np.float32(eps)))
    c.check(mods, before, theta=theta, eps=float(np.float32(eps)))
    c.seg.free()


def test_last_position(mods):
    """Rows that end 2^22 keys: a stream whose list repeats one page up to its window's."""
    n = (1 << 22) // 256
    lists = [np.concatenate([np.zeros(n - 1, np.int32), [1]]).astype(np.int32)]
    c = Case(mods, [(16, 1 << 22)], 256, seed=7, lists=lists, n_pages=2)
    before = c.copies()
    c.run(mods)
    c.check(mods, before)
    c.seg.free()


def test_zero_tiny_and_nonfinite_heads(mods):
    tf, torch = mods
    c = Case(mods, STREAMS, 16, seed=8)
    q = c.qb.view(c.R, 32, 64)
    q[0, 0] = 0
    q[1, 5] *= 2.0 ** -60          # eps carries the norm
    q[2, 31] *= 2.0 ** 40
    c.qb.view(c.R, 32, 64)[3, 7, 9] = float("nan")
    c.kb.view(c.R, 8, 64)[4, 2, 63] = float("inf")
    c.run(mods)
    torch.cuda.synchronize()
    ok = torch.ones((c.R, 32), dtype=torch.bool, device="cuda")
    ok[3, 7] = False
    assert torch.isnan(c.out[3, 7]).all() and torch.isfinite(c.out[ok]).all()
    assert (c.out[0, 0] == 0).all()
    keep = torch.tensor([r for r in range(c.R) if r != 3], device="cuda")
    check(c.out[keep], q[keep], c.qw, c.pos[keep.cpu().numpy()], "q")
    krows, _ = c.rows_of(c.K[1])
    assert torch.isnan(krows[4, 2]).any()
    krows[4, 2] = 0
    assert torch.isfinite(krows).all()
    c.seg.free()


def test_captured_and_replayed(mods):
    tf, torch = mods
    c = Case(mods, STREAMS, 64, seed=9)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        c.run(mods, 0, stream=torch.cuda.current_stream())
        c.run(mods, 1, stream=torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    c.qb.copy_(torch.randn(c.qb.shape, device="cuda"))
    c.kb.copy_(torch.randn(c.kb.shape, device="cuda"))
    before = c.copies()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    k0, _ = c.rows_of(c.K[0])
    k1, _ = c.rows_of(c.K[1])
    assert torch.equal(bits(k0), bits(k1))
    before[0][0] = c.K[0].clone()      # layer 0 was written too
    before[1][0] = c.V[0].clone()
    c.check(mods, before)
    c.seg.free()


def test_refusals(mods):
    tf, torch = mods
    c = Case(mods, [(2, 20)], 16, seed=10)
    base = dict(layer=0, q=c.qb, qs=2048, k=c.kb, ks=512, v=c.vb, vs=512, qw=c.qw, kw=c.kw, eps=EPS, theta=THETA, out=c.out)
    bad = [dict(layer=-1), dict(layer=2), dict(q=None), dict(k=None), dict(v=None), dict(qw=None), dict(kw=None),
           dict(out=None), dict(q=c.qb.data_ptr() + 2), dict(kw=c.kw.data_ptr() + 8), dict(qs=2047), dict(qs=2040),
           dict(qs=2052), dict(ks=511), dict(ks=516), dict(vs=0), dict(vs=-512), dict(eps=0.0), dict(eps=-1.0),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(theta=0.5), dict(theta=float("nan")),
           dict(theta=float("inf")), dict(out=c.qb.data_ptr() + 16), dict(out=c.kb), dict(out=c.vb),
           dict(q=c.qb, qs=2056, out=c.qb)]
    for change in bad:
        a = {**base, **change}
        with pytest.raises(tf.TFError) as e:
            tf.tf_qk_rows(c.seg, a["layer"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"],
                          a["eps"], a["theta"], a["out"])
        assert e.value.status == tf.TF_EINVAL, change
    with pytest.raises(tf.TFError) as e:
        tf.tf_qk_rows(c.seg, 0, c.qb, (1 << 32) + 8, c.kb, 512, c.vb, 512, c.qw, c.kw, EPS, THETA, c.out)
    assert e.value.status == tf.TF_ERANGE
    assert tf.lib().tf_qk_rows(None, 0, c.qb.data_ptr(), 2048, c.kb.data_ptr(), 512, c.vb.data_ptr(), 512,
                               c.qw.data_ptr(), c.kw.data_ptr(), EPS, THETA, c.out.data_ptr(), None) == tf.TF_EINVAL
    c.seg.free()


def test_output_over_the_norm_weights_is_refused(mods):
    """q_out must not hold an input: rows would be normed with what others wrote."""
    tf, torch = mods
    c = Case(mods, [(2, 20)], 16, seed=11)
    buf = torch.ones(2 * 2048 + 64, dtype=torch.bfloat16, device="cuda")      # q_out's rows and 64 more
    for name, at in (("q_norm", 0), ("k_norm", 0), ("q_norm", 1000), ("k_norm", 4096 - 8)):
        qw, kw = (buf[at:at + 64] if name == n else w for n, w in (("q_norm", c.qw), ("k_norm", c.kw)))
        with pytest.raises(tf.TFError) as e:
            tf.tf_qk_rows(c.seg, 0, c.qb, 2048, c.kb, 512, c.vb, 512, qw, kw, EPS, THETA, buf)
        assert e.value.status == tf.TF_EINVAL, (name, at)
    c.kw, c.qw = buf[4096:], c.kw                                            # right behind it: allowed
    before = c.copies()
    c.run(mods, out=buf)
    c.check(mods, before, out=buf[:4096])
    c.seg.free()
