"""tf_sample_rows against the float64 oracle: picks and flags equal, probabilities
within fp32's rounding (half a step, 2^-24, of a value whose 64-bit masses are
good to 2^-40 at these sizes: 2^-23 in all).

The kernel's masses are good to about 1e-12, so a pick could differ where u (or
a top-p border) lies that close to a border: with fewer than 2^17 borders a row
and about 3,000 rows here the chance of one is below 1e-3; it has not occurred.
"""

import math

import numpy as np
import pytest

from oracle import sample as OS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf, torch


def run(mods, logits, V, u, temperature=None, top_k=None, top_p=None, min_p=None, offset=0, want_prob=True, stream=None):
    """logits: a bf16 [R][stride] CUDA tensor whose row holds the V tokens from `offset`."""
    tf, torch = mods
    R, stride = logits.shape

    def dev(x, dt):
        return None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=dt)).cuda()

    pick = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((R,), -7.0, device="cuda") if want_prob else None
    flag = torch.full((R,), 77, dtype=torch.uint8, device="cuda")
    par = [dev(temperature, np.float32), dev(top_k, np.int32), dev(top_p, np.float32), dev(min_p, np.float32)]
    tf.tf_sample_rows(logits.data_ptr() + 2 * offset, R, V, stride, *par, dev(u, np.float32), pick, prob, flag, stream)
    torch.cuda.synchronize()
    return pick.cpu().numpy(), prob.cpu().numpy() if want_prob else None, flag.cpu().numpy()


def host_bits(logits, V, offset=0):
    import torch
    return logits.view(torch.int16).cpu().numpy().view(np.uint16)[:, offset:offset + V]


def check(mods, logits, V, u, offset=0, **kw):
    f32 = lambda x: None if x is None else np.asarray(x, np.float32)
    kw = {n: v if n == "top_k" else f32(v) for n, v in kw.items()}
    u = f32(u)
    pick, prob, flag = run(mods, logits, V, u, offset=offset, **kw)
    rp, rq, rf = OS.sample_rows(host_bits(logits, V, offset), u, **kw)
    assert np.array_equal(flag, rf), np.nonzero(flag != rf)
    assert np.array_equal(pick, rp), [(i, pick[i], rp[i]) for i in np.nonzero(pick != rp)[0][:8]]
    assert np.all(np.abs(prob - rq) <= 2.0 ** -23 * rq + 2.0 ** -149)
    return pick, prob, flag


def settings(R, seed):
    rng = np.random.default_rng(seed)
    t = rng.uniform(0.3, 2.0, R)
    t[rng.random(R) < 0.1] = 0
    return dict(temperature=t, top_k=np.where(rng.random(R) < 0.4, rng.integers(1, 300, R), 0),
                top_p=np.where(rng.random(R) < 0.5, rng.uniform(0.05, 0.999, R), 1.0),
                min_p=np.where(rng.random(R) < 0.4, rng.uniform(0.001, 0.5, R), 0.0)), rng.random(R) * (1 - 2.0 ** -20)


def normal(torch, R, V, std, seed, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((R, V), generator=g, device="cuda") * std + mean).to(torch.bfloat16)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 255, 1000, 4097, 12345, 65536])
def test_settings_mixed(mods, V):
    x = normal(mods[1], 64, V, 3.0, V)
    kw, u = settings(64, V)
    check(mods, x, V, u, **kw)


@pytest.mark.parametrize("std,mean", [(0.01, 0.0), (1e-4, 0.0), (30.0, 0.0), (3.0, 50.0), (3.0, -50.0), (1.0, -3000.0)])
def test_scales(mods, std, mean):
    """Values of one sign, near zero, of many windows' range."""
    x = normal(mods[1], 24, 5000, std, 5, mean)
    kw, u = settings(24, 6)
    check(mods, x, 5000, u, **kw)
    check(mods, x, 5000, u)


def test_every_bf16_value(mods):
    """A row holding every finite bf16 value (and -Inf) once, at several temperatures."""
    _, torch = mods
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    val = (bits.astype(np.uint32) << 16).view(np.float32)
    bits = bits[np.isfinite(val) | (val == -np.inf)]
    np.random.default_rng(1).shuffle(bits)
    t = [1.0, 1e-3, 1e30, 3.3e38, 1e38, 5.0]
    x = torch.from_numpy(np.tile(bits.view(np.int16), (len(t) * 8, 1))).cuda().view(torch.bfloat16)
    u = np.tile([0.0, 1e-6, 0.1, 0.37, 0.5, 0.77, 0.93, 0.99999], len(t))
    check(mods, x, len(bits), u, temperature=np.repeat(t, 8))
    check(mods, x, len(bits), u, temperature=np.repeat(t, 8), top_k=np.full(48, 40000), top_p=np.full(48, 0.7))


def test_vocabulary_rows(mods):
    """128,000 tokens of N(0, 3): no filter, and the settings mixed."""
    x = normal(mods[1], 96, 128000, 3.0, 7).clamp_(-19, 19)
    kw, u = settings(96, 8)
    check(mods, x, 128000, u)
    check(mods, x, 128000, u, **kw)


@pytest.mark.parametrize("R,V", [(1, 140000), (2, 131072), (5, 70001), (40, 33000), (100, 20000), (400, 9000)])
@pytest.mark.parametrize("outside", [False, True])
def test_clusters(mods, R, V, outside):
    """Rows shared by 8, 8, 4, 2, 1 and 1 CTAs, with values outside the folded window
    (large, tiny, both signs) in some rows or none."""
    x = normal(mods[1], R, V, 3.0, V)
    if outside:
        x[::2, 11:5000:7] = 300.0
        x[::2, 3] = -2.0 ** -60
        x[::3, V - 1] = 2.0 ** -40
        x[R - 1, V // 2] = -9000.0
    kw, u = settings(R, V + 1)
    kw["temperature"] = np.where(kw["temperature"] > 0, kw["temperature"] * (20 if outside else 1), 0)
    check(mods, x, V, u)
    check(mods, x, V, u, **kw)


def test_same_value_everywhere_at_a_border(mods):
    """Values at the folded window's edges: 127.5, 128, 2^-33 and its neighbours, both signs."""
    torch = mods[1]
    edge = [127.5, 128.0, 2.0 ** -33, 2.0 ** -33 * (1 + 2.0 ** -7), 2.0 ** -33 * (1 - 2.0 ** -8), 0.0, -0.0, 1.0]
    vals = torch.tensor([s * e for e in edge for s in (1, -1)], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(31)
    x = vals[torch.randint(0, len(vals), (64, 3000), generator=g, device="cuda")].to(torch.bfloat16)
    for r in range(16):                    # rows of one edge value and ones, so that they stay inside or not
        x[r] = torch.where(torch.rand(3000, generator=g, device="cuda") < 0.5, vals[r], torch.ones_like(vals[r])).to(torch.bfloat16)
    kw, u = settings(64, 32)
    kw["temperature"] = kw["temperature"] * 50
    check(mods, x, 3000, u, **kw)
    check(mods, x, 3000, u, temperature=np.full(64, 200.0))


def test_two_streams_at_once(mods):
    """Calls on two streams share nothing."""
    tf, torch = mods
    xs = [normal(torch, 300, 30000, 3.0, s) for s in (33, 34)]
    us = [torch.rand(300, device="cuda") * 0.999 for _ in xs]
    outs = [(torch.empty(300, dtype=torch.int32, device="cuda"), torch.empty(300, dtype=torch.uint8, device="cuda")) for _ in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        for x, u, o, s in zip(xs, us, outs, streams):
            tf.tf_sample_rows(x, 300, 30000, 30000, None, None, None, None, u, o[0], None, o[1], stream=s)
    torch.cuda.synchronize()
    for x, u, o in zip(xs, us, outs):
        rp, _, _ = OS.sample_rows(host_bits(x, 30000), u.cpu().numpy())
        assert np.array_equal(o[0].cpu().numpy(), rp)


def test_largest_vocabulary(mods):
    x = normal(mods[1], 3, 1 << 19, 2.0, 9)
    check(mods, x, 1 << 19, [0.2, 0.6, 0.99999], temperature=[1.0, 3.0, 0.8])


@pytest.mark.parametrize("offset,stride", [(0, 1003), (1, 1010), (3, 1016), (8, 1024), (5, 1001 + 5)])
def test_alignment_and_strides(mods, offset, stride):
    """Rows that start and end anywhere; a NaN just outside each row is not read into it."""
    tf, torch = mods
    V = 1001
    x = torch.full((40, stride), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:, offset:offset + V] = normal(torch, 40, V, 3.0, 11)[:, :min(V, stride - offset)]
    kw, u = settings(40, 12)
    check(mods, x, V, u, offset=offset, **kw)


def test_equal_logits_have_exact_borders(mods):
    """Weights of 1: u = j / V draws token j, top-p = n / V keeps n tokens."""
    tf, torch = mods
    V = 4096
    x = torch.full((V, V), -2.5, dtype=torch.bfloat16, device="cuda")
    j = np.arange(V)
    pick, prob, flag = run(mods, x, V, j / V)
    assert np.array_equal(pick, j) and not flag.any() and (prob == np.float32(1 / V)).all()
    n = np.maximum(j, 1)
    pick, prob, _ = run(mods, x, V, np.full(V, 1 - 2.0 ** -24), top_p=j / V)
    assert np.array_equal(pick, n - 1)
    assert np.array_equal(prob, (1 / n).astype(np.float32))
    pick, _, _ = run(mods, x, V, np.full(V, 1 - 2.0 ** -24), top_k=n, min_p=np.ones(V))
    assert np.array_equal(pick, n - 1)


def test_ties_and_zeros(mods):
    """Signed zeros are one value; among equals the lower ids come first."""
    tf, torch = mods
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.choice([0.0, -0.0, 1.0, -1.0, 2.0 ** -130, -2.0 ** -130], (200, 777)).astype(np.float32))
    x = x.to(torch.bfloat16).cuda()
    kw, u = settings(200, 4)
    check(mods, x, 777, u, **kw)
    check(mods, x, 777, u)


def test_masks(mods):
    """-Inf and the type's lowest value; rows with one token or none left."""
    tf, torch = mods
    x = normal(torch, 60, 3001, 3.0, 13)
    g = torch.Generator(device="cuda").manual_seed(14)
    off = torch.rand(x.shape, generator=g, device="cuda") < 0.97
    low = torch.finfo(torch.bfloat16).min
    x[:20] = torch.where(off[:20], -math.inf, x[:20].float()).to(x.dtype)
    x[20:40] = torch.where(off[20:40], low, x[20:40].float()).to(x.dtype)
    x[40] = -math.inf
    x[41] = -math.inf
    x[41, 3000] = -7.0
    x[42] = low
    x[43, :] = low
    x[43, 5] = 0.0
    kw, u = settings(60, 15)
    pick, _, flag = check(mods, x, 3001, u, **kw)
    assert flag[40] == 1 and pick[40] == -1 and pick[41] == 3000 and flag.sum() == 1
    check(mods, x, 3001, u)


@pytest.mark.parametrize("mask", [-128.0, -133.0, -500.0, -1e4, -1e9, -3.3895313892515355e38])
def test_finite_masks(mods, mask):
    """Large negative numbers in masked places, from where they still have weight to where they have none."""
    tf, torch = mods
    R, V = 96, 3001
    x = normal(torch, R, V, 3.0, 40)
    g = torch.Generator(device="cuda").manual_seed(41)
    off = torch.rand(x.shape, generator=g, device="cuda") < torch.linspace(0, 1, R, device="cuda")[:, None]
    x = torch.where(off, mask, x.float()).to(torch.bfloat16)
    x[0::8, 17] = 0.0                     # with zeros, masked ones by -Inf, tiny and large ones beside them
    x[1::8, ::3] = -math.inf
    x[2::8, 100] = 2.0 ** -60
    x[3::8, 2000] = 130.0
    kw, u = settings(R, 42)
    check(mods, x, V, u, **kw)
    for t in (1.0, 2.9, 3.1, 3.3, 50.0, 1e3, 1e8, 1e30, 3.4e38):
        check(mods, x, V, u, **(kw | dict(temperature=np.full(R, t))))


def test_nonfinite_rows_and_bad_settings(mods):
    tf, torch = mods
    R, V = 24, 2000
    x = normal(torch, R, V, 3.0, 16)
    x[0, 0], x[1, V - 1], x[2, 777] = math.nan, math.inf, -math.nan
    x[3, 5] = math.inf
    x[3, 6] = -math.inf
    kw, u = settings(R, 17)
    for name, rows, v in (("temperature", (3, 4, 5, 6), (-1.0, -1e-30, math.inf, math.nan)), ("top_p", (7,), (math.nan,)),
                          ("min_p", (8, 9), (math.nan, 1.0001))):
        kw[name][list(rows)] = v
    u[10:14] = [1.0, -1e-9, math.nan, 2.0]
    kw["top_k"][14:16] = [-2 ** 31, 2 ** 31 - 1]
    kw["top_p"][16:18] = [-math.inf, math.inf]
    kw["min_p"][18] = -math.inf
    _, _, flag = check(mods, x, V, u, **kw)
    assert flag[:14].tolist() == [1, 1, 1, 3, 2, 2, 2, 2, 2, 2, 2, 2, 2, 2] and not flag[14:].any()


def test_extreme_temperatures(mods):
    tf, torch = mods
    t = np.array([1e-45, 1e-30, 1e-3, 1e3, 1e30, 3.4e38] * 8, np.float32)
    x = normal(torch, 48, 3000, 3.0, 18)
    check(mods, x, 3000, np.random.default_rng(19).random(48), temperature=t)


def test_zero_temperature_is_the_greedy_pick(mods):
    tf, torch = mods
    x = normal(torch, 300, 5003, 3.0, 20)
    pick, prob, _ = run(mods, x, 5003, np.full(300, 0.9), temperature=np.zeros(300))
    want, wflag = (torch.empty(300, dtype=d, device="cuda") for d in (torch.int32, torch.uint8))
    tf.tf_argmax_rows(x, 300, 5003, 5003, want, wflag)
    assert np.array_equal(pick, want.cpu().numpy()) and (prob == 1).all()


def test_no_probabilities_no_rows_many_rows(mods):
    tf, torch = mods
    x = normal(torch, 70000, 40, 3.0, 21)
    u = np.random.default_rng(22).random(70000).astype(np.float32) * np.float32(1 - 2.0 ** -20)
    pick, _, flag = run(mods, x, 40, u, want_prob=False)
    rp, _, _ = OS.sample_rows(host_bits(x[-300:], 40), u[-300:])
    assert np.array_equal(pick[-300:], rp) and not flag.any() and (pick >= 0).all()
    tf.tf_sample_rows(None, 0, 40, 40, None, None, None, None, None, None, None, None)


def test_captured_and_replayed(mods):
    """A graph on another stream; the same bits every time, changed inputs seen."""
    tf, torch = mods
    R, V = 40, 20000
    x = normal(torch, R, V, 3.0, 23)
    u = torch.rand(R, device="cuda")
    t = torch.full((R,), 0.8, device="cuda")
    pick, flag = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.uint8, device="cuda")
    prob = torch.empty(R, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        tf.tf_sample_rows(x, R, V, V, t, None, None, None, u, pick, prob, flag)
    torch.cuda.current_stream().wait_stream(s)
    for k in range(3):
        u.uniform_(0, 0.999)
        g.replay()
        torch.cuda.synchronize()
        rp, _, _ = OS.sample_rows(host_bits(x, V), u.cpu().numpy(), temperature=t.cpu().numpy())
        assert np.array_equal(pick.cpu().numpy(), rp)


def test_settings_of_more_rows_than_a_launch(mods):
    """70,000 rows go in two launches: each row has its own settings and results in both."""
    tf, torch = mods
    R, V = 70000, 40
    x = normal(torch, R, V, 3.0, 43)
    kw, u = settings(R, 44)
    f32 = lambda a: np.asarray(a, np.float32)
    kw = {n: v if n == "top_k" else f32(v) for n, v in kw.items()}
    pick, prob, flag = run(mods, x, V, u, **kw)
    rows = np.r_[0:200, 65535 - 300:65535 + 300, R - 200:R]
    rp, rq, rf = OS.sample_rows(host_bits(x, V)[rows], f32(u)[rows], **{n: v[rows] for n, v in kw.items()})
    assert np.array_equal(flag[rows], rf) and np.array_equal(pick[rows], rp)
    assert np.all(np.abs(prob[rows] - rq) <= 2.0 ** -23 * rq + 2.0 ** -149)
    assert not flag.any() and ((pick >= 0) & (pick < V)).all() and ((prob > 0) & (prob <= 1)).all()
