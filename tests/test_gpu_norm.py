"""tf_norm_rows against the formula in float64 and scaled.py's coding.

The sum is fp32 rounded to bf16: bit for bit torch's. The fp32 norm n is off by at
most d = 2^-18 |n|: a sum of squares in at most 8 * 8 + 5 + 8 additions of 2^-24,
halved by the root, a division and two products of 2^-24, rsqrtf's 2 ulp. A code is
off by half a step more (2^-4 of the value, 2^-10 of the scale). The scale is the
expected one, or its neighbour where the group's largest is within 2^-17 of the
border between them.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def tf():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf


def inputs(R, W, seed, residual, pads=(0, 0, 0), std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r, s = (torch.randn((R, W + p), generator=g, device="cuda").mul_(std).to(torch.bfloat16) for p in pads)
    w = (1 + 0.3 * torch.randn(W, generator=g, device="cuda")).to(torch.bfloat16)
    x[:, 5::61] *= 30
    codes = torch.full((R, W), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, W // 32), 0xAA, dtype=torch.uint8, device="cuda")
    return x, r if residual else None, w, s if residual else None, codes, scales


def call(tf, W, x, r, w, s, codes, scales, eps=EPS, stream=None):
    n = lambda t: W if t is None else t.stride(0)
    tf.tf_norm_rows(x, n(x), r, n(r), w, eps, x.shape[0], W, s, n(s), codes, scales, stream)


def check(W, x, r, w, s, codes, scales, eps=EPS, what=""):
    from scaled import exponent, value
    h = x[:, :W]
    if r is not None:
        h = (x[:, :W].float() + r[:, :W].float()).to(torch.bfloat16)
        assert torch.equal(s[:, :W].view(torch.int16), h.view(torch.int16)), what
    h = h.double()
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()
    n = n.view(len(h), W // 32, 32)
    got_e = scales.int()[..., None] - 127
    e = exponent(n, -1)
    edge = torch.ldexp(torch.full_like(n[..., :1], 464), torch.minimum(e, got_e))
    near = (n.abs().amax(-1, keepdim=True) / edge - 1).abs() < 2.0 ** -17
    assert ((e == got_e) | near).all(), what
    d = 2.0 ** -18 * n.abs()
    half = torch.maximum(2.0 ** -4 * (n.abs() + d), torch.ldexp(torch.full_like(d, 2.0 ** -10), got_e))
    err = (value(codes, scales.repeat_interleave(32, 1)).view_as(n) - n).abs()
    assert (err <= d + half).all(), (what, float((err - d - half).max()))


@pytest.mark.parametrize("W", [32, 64, 224, 256, 288, 2016, 2048, 2080, 4096, 6144, 8224, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_widths(tf, W, residual):
    for R in (1, 5, 67):
        a = inputs(R, W, R + W, residual)
        call(tf, W, *a)
        check(W, *a, what=(W, R))


@pytest.mark.parametrize("residual", [False, True])
def test_many_rows(tf, residual):
    a = inputs(20000, 2048, 3, residual)
    call(tf, 2048, *a)
    check(2048, *a)


@pytest.mark.parametrize("W", [32, 96, 480, 992, 1024, 1056])
@pytest.mark.parametrize("residual", [False, True])
def test_many_narrow_rows(tf, W, residual):
    """Several rows a CTA, the last one's partly missing; rows behind the last stay as they are."""
    for R in (1024, 1031, 3000):
        x, r, w, s, codes, scales = inputs(R + 9, W, R, residual, pads=(8, 16, 24))
        cut = lambda t: None if t is None else t[:R]
        call(tf, W, x[:R], cut(r), w, cut(s), codes[:R], scales[:R])
        check(W, x[:R], cut(r), w, cut(s), codes[:R], scales[:R], what=(W, R))
        assert (codes[R:] == 0xAA).all() and (scales[R:] == 0xAA).all()


@pytest.mark.parametrize("R", [3, 1500])
def test_infinite_products(tf, R):
    """Infinite weights and products past fp32: NaN codes there, the others' scales as if they were not."""
    W = 256
    x, r, w, s, codes, scales = inputs(R, W, 9, False)
    x[:, 40] = 2.0
    w[40] = float("inf")
    w[70] = float("-inf")
    w[100] = 3e38
    x[:, 100] = 1e4
    call(tf, W, x, r, w, s, codes, scales)
    bad = [40, 70, 100]
    assert ((codes[:, bad] & 0x7F) == 0x7F).all()
    keep = torch.ones(W, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert ((codes[:, keep] & 0x7F) != 0x7F).all()
    from scaled import exponent
    h = x.double()
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * torch.where(keep, w.double(), 0.0)
    top = n.view(R, W // 32, 32).abs().amax(-1)
    e = exponent(n.view(R, W // 32, 32), -1)[..., 0]
    near = (top / torch.ldexp(torch.full_like(top, 464), e) - 1).abs() < 2.0 ** -16
    assert ((scales.int() - 127 == e) | near).all()


@pytest.mark.parametrize("std", [0.0, 1e-30, 1e-4, 1e15])
def test_sizes(tf, std):
    for W in (96, 2048):
        a = inputs(3, W, 4, True, std=std)
        call(tf, W, *a)
        check(W, *a, what=std)


def test_strides_and_scales_at_odd_addresses(tf):
    W = 2048
    x, r, w, s, codes, scales = inputs(9, W, 5, True, pads=(8, 72, 2048))
    odd = torch.full((9 * W // 32 + 3,), 0xAA, dtype=torch.uint8, device="cuda")
    scales = odd[3:].view(9, W // 32)
    before = s.clone()
    call(tf, W, x, r, w, s, codes, scales)
    check(W, x, r, w, s, codes, scales)
    assert torch.equal(s[:, W:].view(torch.int16), before[:, W:].view(torch.int16)) and (odd[:3] == 0xAA).all()


@pytest.mark.parametrize("which", ["x", "res"])
def test_in_place(tf, which):
    """The sum over an addend; side by side with the other in rows of one tensor."""
    W = 512
    x, r, w, s, codes, scales = inputs(7, W, 6, True)
    x0, r0 = x.clone(), r.clone()
    s = x if which == "x" else r
    call(tf, W, x, r, w, s, codes, scales)
    check(W, x0, r0, w, s, codes, scales)
    both = torch.cat([x0, r0, torch.zeros_like(x0)], 1).contiguous()
    call(tf, W, both[:, :W], both[:, W:2 * W], w, both[:, 2 * W:], codes, scales)
    check(W, x0, r0, w, both[:, 2 * W:], codes, scales)


def test_nonfinite_rows(tf):
    W = 2048
    x, r, w, s, codes, scales = inputs(6, W, 7, True)
    x[1, 77] = float("nan")
    x[4, 5] = float("inf")
    call(tf, W, x, r, w, s, codes, scales)
    assert ((codes[1] & 0x7F) == 0x7F).all()
    bad = codes[4] & 0x7F                              # everything over infinity, the infinity itself NaN
    assert bad[5] == 0x7F and (torch.cat([bad[:5], bad[6:]]) == 0).all()
    keep = [0, 2, 3, 5]
    check(W, x[keep], r[keep], w, s[keep], codes[keep], scales[keep])


def test_captured_on_another_stream(tf):
    W = 2048
    a = inputs(16, W, 8, True)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        call(tf, W, *a, stream=torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    a[0].mul_(3)
    g.replay()
    check(W, *a)


def test_empty_and_host_memory(tf):
    call(tf, 64, *inputs(0, 64, 9, True))


@pytest.mark.parametrize("R,W", [(1 << 24, 32), (3, 1 << 14)])
def test_the_largest_sizes(tf, R, W):
    x, r, w, s, codes, scales = inputs(R, W, 11, True)
    call(tf, W, x, r, w, s, codes, scales)
    for i in (0, R // 2, R - min(R, 1 << 20)):
        at = slice(i, i + (1 << 20))
        check(W, x[at], r[at], w, s[at], codes[at], scales[at], what=i)


def test_no_rows_write_nothing(tf):
    W = 64
    x, r, w, s, codes, scales = inputs(2, W, 10, True)
    before = [t.clone() for t in (s, codes, scales)]
    tf.tf_norm_rows(x, W, r, W, w, EPS, 0, W, s, W, codes, scales)
    tf.tf_norm_rows(x, W, None, W, w, EPS, 0, W, None, W, codes, scales)
    for a, b in zip((s, codes, scales), before):
        assert torch.equal(a, b)
