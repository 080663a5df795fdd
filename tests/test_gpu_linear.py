"""tf_linear_rows against float64, and exactly where the sums are exact.

The products are exact in the kernel and the sums fp32: at most K / 16 + 64 steps,
each rounding by at most 2^-23 of the partial sums, which are at most A = sum |x w|;
then a product with s (2^-24) and the bf16 store, half a step: 2^-8 of the value.
With small integers every partial sum is exact, and y is the exact sum's bf16.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tf():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf


def weights(N, K, seed, whole=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if whole:
        gs = torch.tensor([0.5, 1, 2, -1], device="cuda")[torch.randint(0, 4, (N, K // 32), generator=g, device="cuda")]
        s = torch.ones(N, device="cuda")
    else:
        gs = torch.randn((N, K // 32), generator=g, device="cuda").exp2()
        s = torch.rand(N, generator=g, device="cuda") + 0.1
    return w, gs.to(torch.float8_e4m3fn).view(torch.uint8), s


def matrix(w, gs):
    c = torch.stack([w & 15, w >> 4], -1).view(len(w), -1).double() - 8
    return c * gs.view(torch.float8_e4m3fn).double().repeat_interleave(32, 1)


def rows(R, K, seed, x8, whole=False, pad=0):
    """(x, scales or None, float64 values)"""
    from scaled import code, exponent, value
    g = torch.Generator(device="cuda").manual_seed(seed)
    if whole:
        v = torch.randint(-2, 3, (R, K + pad), generator=g, device="cuda").float()
    else:
        v = torch.randn((R, K + pad), generator=g, device="cuda") * torch.exp2(torch.rand((R, 1), generator=g, device="cuda") * 20 - 10)
    if not x8:
        x = v.to(torch.bfloat16)
        return x, None, x[:, :K].double()
    e = exponent(v[:, :K].reshape(R, K // 32, 32), -1)
    if whole:
        e = torch.zeros_like(e) + torch.randint(-1, 2, e.shape, generator=g, device="cuda", dtype=e.dtype)
        v[:, :K] = torch.ldexp(v[:, :K].reshape(R, K // 32, 32), e).view(R, K)
    x = torch.full((R, K + pad), 0x7F, dtype=torch.uint8, device="cuda")
    x[:, :K] = code(v[:, :K].reshape(R, K // 32, 32), e).view(R, K)
    scales = (e[..., 0] + 127).to(torch.uint8)
    return x, scales, value(x[:, :K], scales.repeat_interleave(32, 1))


def call(tf, x, xs, w, gs, s, N=None, y=None, K=None):
    N, K = len(w), w.shape[1] * 2
    y = torch.full((len(x), N), float("nan"), dtype=torch.bfloat16, device="cuda") if y is None else y
    tf.tf_linear_rows(x, x.stride(0), xs, len(x), K, w, gs, s, N, y, y.stride(0))
    return y


def check(y, v, w, gs, s, what=""):
    m = matrix(w, gs)
    ref, A = v @ m.T * s.double(), v.abs() @ m.abs().T * s.double().abs()
    d = ((v.shape[1] / 16 + 64) * 2.0 ** -23 + 2.0 ** -24) * A
    err = (y.double() - ref).abs()
    over = err - (d + 2.0 ** -8 * (ref.abs() + d) + 2.0 ** -133)
    assert (over <= 0).all(), (what, float(over.max()), torch.nonzero(over > 0)[:4].tolist())


SHAPES = [(1, 32), (15, 64), (16, 96), (17, 128), (40, 160), (100, 512), (512, 2048), (2048, 2048), (33, 4224),
          (2432, 256), (5000, 288), (64, 16384)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("x8", [False, True])
def test_shapes(tf, N, K, x8):
    w = weights(N, K, N + K)
    exact = weights(N, K, N + K, whole=True)
    for R in (1, 2, 8, 9, 16, 17, 33):
        x, xs, v = rows(R, K, R, x8)
        check(call(tf, x, xs, *w), v, *w, what=(N, K, R))
        x, xs, v = rows(R, K, R, x8, whole=True)
        want = (v @ matrix(*exact[:2]).T).float().to(torch.bfloat16)
        assert torch.equal(call(tf, x, xs, *exact), want), (N, K, R)


@pytest.mark.parametrize("x8", [False, True])
def test_inputs_in_slabs(tf, x8):
    """More inputs than shared memory holds at a time, for each tile of rows."""
    w = weights(70, 40960, 1, whole=True)
    for R in (3, 12, 40):
        x, xs, v = rows(R, 40960, 2, x8, whole=True)
        want = (v @ matrix(*w[:2]).T).float().to(torch.bfloat16)
        assert torch.equal(call(tf, x, xs, *w), want), R


@pytest.mark.parametrize("x8", [False, True])
def test_odd_inputs_in_slabs(tf, x8):
    """The same with a last chunk of one group, and scales at an odd address."""
    w, gs, s = weights(45, 41024, 23, whole=True)
    gs = torch.cat([gs.new_zeros(1), gs.reshape(-1)])[1:].view(gs.shape)
    for R in (2, 11, 26):
        x, xs, v = rows(R, 41024, 24, x8, whole=True)
        want = (v @ matrix(w, gs).T).float().to(torch.bfloat16)
        assert torch.equal(call(tf, x, xs, w, gs, s), want), R


def test_vocabulary(tf):
    w = weights(128000, 2048, 3)
    x, xs, v = rows(5, 2048, 4, False)
    check(call(tf, x, xs, *w), v, *w)


@pytest.mark.parametrize("N,K", [(20011, 1024), (31000, 768), (9001, 256)])
@pytest.mark.parametrize("x8", [False, True])
def test_runs_of_tiles(tf, N, K, x8):
    """Runs of several tiles a CTA, whose warps begin and end inside tiles, for each tile of rows."""
    w = weights(N, K, 15, whole=True)
    for R in (1, 12, 20, 40):
        x, xs, v = rows(R, K, R + 16, x8, whole=True)
        want = (v @ matrix(*w[:2]).T).float().to(torch.bfloat16)
        assert torch.equal(call(tf, x, xs, *w), want), R


def test_scales_far_from_one(tf):
    """Row scales from 2^-100 to 2^90: exact sums under a power of two are its multiples."""
    w = weights(300, 256, 17, whole=True)
    x, xs, v = rows(9, 256, 18, True, whole=True)
    want = v @ matrix(*w[:2]).T
    for e in (-100, 90):
        got = call(tf, x, (xs.int() + e).to(torch.uint8), *w)
        assert torch.equal(got, torch.ldexp(want, torch.tensor(e, device="cuda")).float().to(torch.bfloat16)), e


def test_two_streams_at_once(tf):
    w = [weights(5000, 2048, 19 + i) for i in range(2)]
    x = [rows(R, 2048, 21 + i, bool(i)) for i, R in enumerate((7, 16))]
    want = [call(tf, x[i][0], x[i][1], *w[i]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(call(tf, x[i][0], x[i][1], *w[i]))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("x8", [False, True])
def test_many_rows(tf, x8):
    w = weights(200, 320, 5)
    x, xs, v = rows(3001, 320, 6, x8)
    check(call(tf, x, xs, *w), v, *w)
    w = weights(48, 64, 7, whole=True)
    x, xs, v = rows(32 * 200, 64, 8, x8, whole=True)         # more tiles of rows than SMs
    assert torch.equal(call(tf, x, xs, *w), (v @ matrix(*w[:2]).T).float().to(torch.bfloat16))


@pytest.mark.parametrize("R,N,K", [(1024, 2048, 2048), (2049, 1000, 2080), (64, 20000, 2048)])
@pytest.mark.parametrize("x8", [False, True])
def test_a_layer_of_many_rows(tf, R, N, K, x8):
    """A prompt's or a drafted round's rows through a projection, exactly."""
    w = weights(N, K, 27, whole=True)
    x, xs, v = rows(R, K, 28, x8, whole=True)
    assert torch.equal(call(tf, x, xs, *w), (v @ matrix(*w[:2]).T).float().to(torch.bfloat16))


@pytest.mark.parametrize("R,N,K", [(40, 20000, 2176), (70, 300, 4224), (33, 70, 40960)])
def test_bits_do_not_depend_on_a_rows_place(tf, R, N, K):
    w = weights(N, K, 29)
    x, xs, v = rows(R, K, 30, False)
    want = call(tf, x, xs, *w)
    move = torch.randperm(R, generator=torch.Generator().manual_seed(31)).cuda()
    got = call(tf, x[move].contiguous(), None, *w)
    assert torch.equal(got.view(torch.int16), want[move].view(torch.int16))


@pytest.mark.parametrize("R,K,N", [(1 << 20, 32, 40), (1, 32, 1 << 24), (9, 1 << 20, 20)])
def test_the_largest_sizes(tf, R, K, N):
    """The documented limits, one at a time. (Products are multiples of 1/4 of either sign, some 10 in size: the sums of
    2^20 of them stay near 2^14, far below the 2^22 up to which fp32 holds them exactly.)"""
    w = weights(N, K, 34, whole=True)
    x, xs, v = rows(R, K, 35, True, whole=True)
    got = call(tf, x, xs, *w)
    for n in range(0, N, 1 << 21):
        m = matrix(w[0][n:n + (1 << 21)], w[1][n:n + (1 << 21)])
        assert torch.equal(got[:, n:n + (1 << 21)], (v @ m.T).float().to(torch.bfloat16)), n


def test_no_rows_write_nothing(tf):
    w = weights(40, 64, 32)
    x, xs, v = rows(2, 64, 33, False)
    y = torch.full((2, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    tf.tf_linear_rows(x, 64, None, 0, 64, *w, 40, y, 40)
    assert (y == 7).all()


@pytest.mark.parametrize("x8", [False, True])
def test_strides_and_odd_addresses(tf, x8):
    """Padded rows of x (NaN between them) and y (left alone between them), y and the scales at odd addresses."""
    N, K, R = 37, 256, 11
    w, gs, s = weights(N, K, 9)
    x, xs, v = rows(R, K, 10, x8, pad=48)
    if not x8:
        x[:, K:] = float("nan")
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    gs = off(gs)
    xs = None if xs is None else off(xs)
    buf = torch.full((R * 51 + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[1:].view(R, 51)[:, :N]
    call(tf, x, xs, w, gs, s, y=y)
    check(y, v, w, gs, s)
    assert (buf[:1] == 7).all() and (buf[1:].view(R, 51)[:, N:] == 7).all()


@pytest.mark.parametrize("N,K", [(20000, 2176), (12000, 896), (9500, 384), (300, 640), (70, 41088)])
@pytest.mark.parametrize("x8", [False, True])
def test_bits_do_not_depend_on_an_address(tf, N, K, x8):
    """An odd number of whole 128-input chunks, as runs of tiles and in slabs: the scales at a multiple of 4 and
    behind it give the same bits, for each tile of rows."""
    w, gs, s = weights(N, K, 25)
    for R in (1, 12, 20, 40):
        x, xs, v = rows(R, K, 26, x8)
        want = call(tf, x, xs, w, gs, s)
        for off in (1, 2):
            at = torch.cat([gs.new_zeros(off), gs.reshape(-1)])[off:].view(gs.shape)
            got = call(tf, x, xs, w, at, s)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16)), (R, off)


@pytest.mark.parametrize("x8", [False, True])
def test_nonfinite_rows(tf, x8):
    w = weights(300, 512, 11)
    x, xs, v = rows(12, 512, 12, x8)
    want = call(tf, x, xs, *w)
    if x8:
        x[3, 100] = 0x7F
    else:
        x[3, 100] = float("nan")
        x[7, 0] = float("inf")
    got = call(tf, x, xs, *w)
    assert torch.isnan(got[3]).all()
    keep = [r for r in range(12) if r != 3 and (x8 or r != 7)]
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))


def test_from_the_norms_rows(tf):
    """The norm's output as it stands is this call's input; captured together and replayed."""
    from scaled import value
    W, N, R = 2048, 640, 6
    g = torch.Generator(device="cuda").manual_seed(13)
    h, res = (torch.randn((R, W), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    nw = torch.ones(W, dtype=torch.bfloat16, device="cuda")
    total = torch.empty_like(h)
    codes = torch.empty((R, W), dtype=torch.uint8, device="cuda")
    scales = torch.empty((R, W // 32), dtype=torch.uint8, device="cuda")
    w = weights(N, W, 14)
    y = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")

    def both(stream=None):
        tf.tf_norm_rows(h, W, res, W, nw, 1e-5, R, W, total, W, codes, scales, stream)
        tf.tf_linear_rows(codes, W, scales, R, W, w[0], w[1], w[2], N, y, N, stream)

    both()
    check(y, value(codes, scales.repeat_interleave(32, 1)), *w)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        both(torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    h.mul_(-2)
    for _ in range(3):
        graph.replay()
    check(y, value(codes, scales.repeat_interleave(32, 1)), *w)
