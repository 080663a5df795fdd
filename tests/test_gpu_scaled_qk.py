"""tf_qk_rows over scaled pools: queries and keys against the formula in float64 (the
bounds of test_gpu_qk), the coding against scaled.py's.

V is coded from bf16 inputs, so its codes and scales are compared bit for bit. A key
element's fp32 value is off by at most e (test_gpu_qk's bound), its code by half a
step more: 2^-4 of the value, or 2^-10 of the scale. The scale of K is the expected
one, or its neighbour where the block's largest lies within 2^-18 of the border
between them.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS, THETA = 1e-5, 1e6


@pytest.fixture(scope="module")
def tf():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf


class Case:
    """Pools of random codes (each block's scale its own codes'), a call's rows, and what the pools should hold."""

    def __init__(self, tf, streams, page, seed=0, layers=2, prompt=False, pads=(0, 0, 0), v_std=1.0):
        from scaled import ScaledAttn
        self.tf = tf
        self.a = ScaledAttn(tf, streams, page, seed=seed, layers=layers, prompt=prompt)
        g = torch.Generator(device="cuda").manual_seed(seed + 1000)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        R = self.a.R
        self.qb, self.kb, self.vb = normal(R, 2048 + pads[0]), normal(R, 512 + pads[1]), normal(R, 512 + pads[2], std=v_std)
        self.q, self.k, self.v = self.qb[:, :2048], self.kb[:, :512], self.vb[:, :512]
        self.qw, self.kw = 1 + normal(64, std=0.3), 1 + normal(64, std=0.3)
        self.out = torch.full((R, 32, 64), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, layer=1, out=None, stream=None, seg=None):
        self.tf.tf_qk_rows(seg or self.a.seg, layer, self.qb, self.qb.shape[1], self.kb, self.kb.shape[1], self.vb,
                           self.vb.shape[1], self.qw, self.kw, EPS, THETA, self.out if out is None else out, stream)

    def snapshot(self):
        return [[x.clone() for x in p] for p in (self.a.K, self.a.V, self.a.ks, self.a.vs)]

    def check(self, before, layer=1, what=""):
        """The pools after a call on `layer`, given a snapshot from before it."""
        from scaled import BLOCK, code, exponent, value
        from test_gpu_qk import check, reference
        a = self.a
        pos = np.concatenate([np.arange(k - r, k) for r, _, k in a.streams])
        check(self.out, self.q.reshape(-1, 32, 64), self.qw, pos, (what, "q"))
        ref, size = reference(self.k.reshape(-1, 8, 64), self.kw, pos)
        ref, size = (torch.from_numpy(x).cuda() for x in (ref, size))
        for l in range(a.layers):
            for n, (codes, scales) in enumerate(((a.K, a.ks), (a.V, a.vs))):
                want_c, want_s = before[n][l].clone(), before[2 + n][l].clone()
                if l == layer:
                    for (r, o, k), ids in zip(a.streams, a.lists):
                        for b in range((k - r) // BLOCK, (k - 1) // BLOCK + 1):
                            page, at = int(ids[b * BLOCK // a.page]), b * BLOCK % a.page
                            lo, hi = max(b * BLOCK, k - r) - b * BLOCK, min(b * BLOCK + BLOCK, k) - b * BLOCK
                            rows = slice(o + b * BLOCK + lo - (k - r), o + b * BLOCK + hi - (k - r))
                            old = value(want_c[page, :, at:at + lo], want_s[page, :, at // BLOCK][:, None, None])
                            new = ref[rows] if n == 0 else self.v[rows].reshape(-1, 8, 64).double()
                            x = torch.cat([old, new.transpose(0, 1)], 1)              # [8][hi][64]
                            e = exponent(x.reshape(8, -1), -1)
                            got_e = scales[l][page, :, at // BLOCK].int()[:, None] - 127
                            if n == 0:
                                big = torch.where(torch.isfinite(x), x.abs(), 0.0).amax((1, 2))
                                edge = torch.ldexp(torch.full_like(big, 464), torch.minimum(e, got_e)[:, 0])
                                near = (big / edge - 1).abs() < 2.0 ** -18
                                assert ((e == got_e)[:, 0] | near).all(), (what, "scale", l, b)
                                e = got_e
                            want_s[page, :, at // BLOCK] = (e[:, 0] + 127).to(torch.uint8)
                            want_c[page, :, at:at + lo] = code(old, e[..., None])     # kept rows
                            got = codes[l][page, :, at + lo:at + hi]
                            if n == 1:
                                want_c[page, :, at + lo:at + hi] = code(x[:, lo:], e[..., None])
                            else:
                                err = (value(got, want_s[page, :, at // BLOCK][:, None, None]) - x[:, lo:]).abs()
                                d = 2.0 ** -19 * size[rows].transpose(0, 1)
                                half = torch.maximum(2.0 ** -4 * (x[:, lo:].abs() + d),
                                                     torch.ldexp(torch.full_like(d, 2.0 ** -10), e[..., None]))
                                assert (err <= d + half).all(), (what, "K", l, b, float((err - d - half).max()))
                                want_c[page, :, at + lo:at + hi] = got
                assert torch.equal(scales[l], want_s), (what, "KV"[n], "scales", l)
                assert torch.equal(codes[l], want_c), (what, "KV"[n], "codes", l)


@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("streams", [
    [(1, 1)], [(16, 16)], [(1, 16), (1, 17), (1, 32), (2, 17), (16, 31), (16, 40), (3, 1000), (7, 16 * 9 + 3)],
    [(1, 300 + 7 * i) for i in range(64)]])
def test_verify(tf, page, streams):
    c = Case(tf, streams, page, seed=len(streams) + page)
    before = c.snapshot()
    c.run()
    c.check(before)


@pytest.mark.parametrize("rows,cached", [(1, 0), (15, 0), (33, 7), (64, 16), (1000, 1701)])
def test_prompt(tf, rows, cached):
    c = Case(tf, [(rows, rows + cached)], 32, seed=rows, prompt=True)
    before = c.snapshot()
    c.run()
    c.check(before)


@pytest.mark.parametrize("v_std", [1e-38, 2.0 ** -60, 1e-3, 1e4, 1e37])
def test_v_of_any_size(tf, v_std):
    """The new rows dwarf the kept ones, or the kept ones them."""
    c = Case(tf, [(2, 30), (5, 16), (16, 48)], 16, seed=3, v_std=v_std)
    before = c.snapshot()
    c.run()
    c.check(before, what=v_std)


def test_slices_of_one_projection_in_place(tf):
    """q, k, v as slices of one tensor's rows; q_out over q where q is dense."""
    c = Case(tf, [(3, 50), (1, 64)], 64, seed=4)
    rows = torch.cat([c.q, c.k, c.v, c.q[:, :8]], 1).contiguous()
    before = c.snapshot()
    at = rows.data_ptr()
    c.tf.tf_qk_rows(c.a.seg, 1, at, rows.shape[1], at + 2 * 2048, rows.shape[1], at + 2 * 2560, rows.shape[1], c.qw, c.kw,
                    EPS, THETA, c.out)
    c.check(before)
    q = c.q.clone()
    c.tf.tf_qk_rows(c.a.seg, 0, q, 2048, c.k, 512, c.v, 512, c.qw, c.kw, EPS, THETA, q)
    assert torch.equal(q.view(-1).view(torch.int16), c.out.view(-1).view(torch.int16))


def test_strides(tf):
    c = Case(tf, [(3, 50), (1, 64)], 64, seed=5, pads=(8, 24, 512))
    before = c.snapshot()
    c.run()
    c.check(before)


def test_nonfinite_rows(tf):
    """NaN and infinities become NaN codes; the block's other rows and its scale do not notice. V's elements are alone;
    a key's head is normed as a whole: over an infinite root, zeros, and NaN where the infinity and its rotation
    partner (dimensions 5 and 37) were."""
    c = Case(tf, [(4, 39)], 16, seed=6)
    c.k[1, 64 * 3 + 5] = float("inf")
    c.v[2, 64 * 7 + 9] = float("-inf")
    c.v[0, 1] = float("nan")
    before = c.snapshot()
    c.run()
    page, at = int(c.a.lists[0][35 // 16]), 35 % 16
    K = c.a.K[1]
    head = (K[page, 3, at + 1] & 0x7F).tolist()
    assert head == [0x7F if d in (5, 37) else 0 for d in range(64)]
    c.k[1, 64 * 3:64 * 4] = 0                        # the rest as if that head had been zero
    K[page, 3, at + 1] = 0
    c.check(before)


def test_appending_again_changes_nothing(tf):
    """The scale follows from the codes' values: the same call on its own result leaves every byte."""
    c = Case(tf, [(1, 30), (9, 47), (16, 16)], 32, seed=7)
    c.run()
    once = c.snapshot()
    for _ in range(2):
        c.run()
    for x, y in zip(once, c.snapshot()):
        assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_windows_with_rejected_rows(tf):
    """Rounds whose windows are partly rejected and written again: the blocks end up as if the accepted rows had been
    appended one by one, where all lie in their scales' normal range (a drafted reply's cache is an undrafted one's)."""
    from scaled import ScaledAttn
    g = torch.Generator(device="cuda").manual_seed(8)
    n, page = 60, 16
    k, v = ((torch.rand((n, 512), generator=g, device="cuda") + 0.5).to(torch.bfloat16) for _ in range(2))
    v[20] *= 64                                     # raises its block's scale
    q, qo = torch.randn((n, 2048), generator=g, device="cuda").to(torch.bfloat16), \
        torch.empty((n, 32, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pools = []
    for widths in ([1] * n, [5, 3, 16, 9, 16, 16, 4, 16]):
        a = ScaledAttn(tf, [(1, n)], page, seed=9)
        done, i = 0, 0
        while done < n:
            rows = min(widths[i % len(widths)], n - done)
            seg = tf.tf_paged_scaled_build([(rows, 0, done + rows, 64)], None, None, a.lists[0], page, a.n_pages, a.K, a.V,
                                           a.ks, a.vs, 0, 1)
            rk, rv = k[done:done + rows].clone(), v[done:done + rows].clone()
            keep = rows if rows == 1 else (rows + 1) // 2
            rk[keep:] *= -3                          # rejected drafts
            rv[keep:] *= 1000
            tf.tf_qk_rows(seg, 0, q[done:], 2048, rk, 512, rv, 512, w, w, EPS, THETA, qo)
            done += keep if done + rows < n or rows == 1 else keep
            i += 1
        pools.append(a)
    x, y = pools
    for cx, sx, cy, sy in ((x.K, x.ks, y.K, y.ks), (x.V, x.vs, y.V, y.vs)):
        got, s0 = x.cache(cx[0], sx[0], x.lists[0], n)
        want, s1 = y.cache(cy[0], sy[0], y.lists[0], n)
        assert torch.equal(s0, s1)
        # an element that a rejected row's scale made subnormal (2^-6 of it) may have lost bits
        lost = torch.ldexp(torch.full((), 2.0 ** -9, dtype=torch.float64, device="cuda"), s0.int()[..., None] - 127 + 10)
        assert ((got - want).abs() <= torch.where(want.abs() >= lost * 8, 0.0, lost)).all()


def test_captured(tf):
    """Two layers in a graph; its replays append the current rows."""
    c = Case(tf, [(2, 30), (1, 100)], 16, seed=10)
    before = c.snapshot()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        c.run(1, stream=torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    c.kb.copy_(c.kb * 2)
    c.vb.copy_(c.vb * 5)
    g.replay()
    c.check(before)


def test_refusals(tf):
    c = Case(tf, [(2, 30)], 16, seed=11)
    for args in ((2, c.out), (-1, c.out), (0, c.kb), (0, None)):
        with pytest.raises(tf.TFError) as e:
            c.run(args[0], out=args[1] if args[1] is not None else c.out.data_ptr() + 2)
        assert e.value.status == tf.TF_EINVAL
