"""The sampling oracle's pins and tf_sample_rows' host refusals, on the CPU."""

import math

import numpy as np
import pytest

from oracle import sample as OS


def bf16(*x):
    import torch
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


# logits 0, ln 2 would not be bf16: powers of two come from T = 1 / ln 2 (w = 2^(x - max))
T2 = 1 / math.log(2)
ROW = bf16(1, 3, 2, 3, -math.inf, 0)     # order 1, 3, 2, 0, 5; w 1, 1, 1/2, 1/4, 1/8: cumulative 8 16 20 22 23 of 23


@pytest.mark.parametrize("u,kw,pick,num,den", [
    (0.0, {}, 1, 8, 23), (7.9 / 23, {}, 1, 8, 23), (8.1 / 23, {}, 3, 8, 23), (16.1 / 23, {}, 2, 4, 23),
    (20.1 / 23, {}, 0, 2, 23), (22.1 / 23, {}, 5, 1, 23), (0.999999, {}, 5, 1, 23),
    (0.9, dict(top_k=1), 1, 1, 1), (0.9, dict(top_k=3), 2, 4, 20), (0.79, dict(top_k=3), 3, 8, 20),
    (0.99, dict(top_p=0.0), 1, 1, 1), (0.99, dict(top_p=-3.0), 1, 1, 1), (0.99, dict(top_p=7.9 / 23), 1, 1, 1),
    (0.99, dict(top_p=8.1 / 23), 3, 8, 16), (0.99, dict(top_p=20.1 / 23), 0, 2, 22), (0.99, dict(top_p=1.0), 5, 1, 23),
    (0.99, dict(min_p=0.2), 0, 2, 22), (0.99, dict(min_p=0.3), 2, 4, 20), (0.99, dict(min_p=1.0), 3, 8, 16),
    (0.99, dict(min_p=-1.0, top_k=-5), 5, 1, 23),
    (0.99, dict(top_k=3, top_p=0.79), 3, 8, 16),          # p of the three kept tokens' mass (15.8 of 20)
    (0.99, dict(top_k=3, top_p=0.81, min_p=0.6), 3, 8, 16),
])
def test_worked(u, kw, pick, num, den):
    got = OS.sample_row(ROW, u, temperature=T2, **kw)
    assert got[0] == pick and got[2] == 0
    assert got[1] == pytest.approx(num / den, rel=1e-12)


def test_greedy_and_ties():
    assert OS.sample_row(ROW, 0.99, temperature=0) == (1, 1.0, 0)
    assert OS.sample_row(bf16(-0.0, 0.0, -1), 0.3)[0] == 0          # -0 and +0 are one value
    assert OS.sample_row(bf16(0.0, -0.0, -1), 0.6, top_k=2)[0] == 1


@pytest.mark.parametrize("row,kw,flag", [
    (bf16(0, math.nan), {}, 1), (bf16(0, math.inf), {}, 1), (bf16(-math.inf, -math.inf), {}, 1),
    (bf16(0, 1), dict(temperature=-1.0), 2), (bf16(0, 1), dict(temperature=math.inf), 2),
    (bf16(0, 1), dict(temperature=math.nan), 2), (bf16(0, 1), dict(top_p=math.nan), 2),
    (bf16(0, 1), dict(min_p=math.nan), 2), (bf16(0, 1), dict(min_p=1.5), 2), (bf16(0, math.nan), dict(min_p=1.5), 3),
])
def test_flags(row, kw, flag):
    assert OS.sample_row(row, 0.5, **kw) == (-1, 0.0, flag)
    assert OS.sample_row(bf16(0, 1), 1.0)[2] == 2 and OS.sample_row(bf16(0, 1), math.nan)[2] == 2


def test_draws_follow_the_kept_distribution():
    """Over an even grid of u the picks come in proportion to the kept weights."""
    n = 4000
    picks = [OS.sample_row(ROW, (i + 0.5) / n, temperature=T2, top_k=4)[0] for i in range(n)]
    for token, share in ((1, 8 / 22), (3, 8 / 22), (2, 4 / 22), (0, 2 / 22), (5, 0), (4, 0)):
        assert abs(picks.count(token) / n - share) <= 1 / n


@pytest.fixture(scope="module")
def T():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    return tf


def test_refusals(T):
    P = 0x7F0000000000
    f = T.lib().tf_sample_rows
    ok = [P, 4, 100, 100, P, P, P, P, P, P, P, P, None]

    def status(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 8, 9, 11):                       # logits, u, pick, flag
        assert status(**{f"a{i}": None}) == T.TF_EINVAL
    assert status(a0=P + 1) == T.TF_EINVAL        # an odd address
    assert status(a1=-1) == T.TF_EINVAL and status(a2=0) == T.TF_EINVAL and status(a3=99) == T.TF_EINVAL
    assert status(a2=(1 << 19) + 1, a3=1 << 20) == T.TF_ERANGE
    assert status(a1=(1 << 24) + 1) == T.TF_ERANGE
    assert status(a1=0, a0=None) == T.TF_OK       # no rows: nothing to do


def test_misaligned_arrays_are_refused(T):
    """The 4-byte arrays: an address that is no multiple of 4 would fault on the device.
    (With a vocabulary beyond the limit too, so that no answer to this call is a launch.)"""
    P = 0x7F0000000000
    f = T.lib().tf_sample_rows
    call = [P, 4, (1 << 19) + 1, 1 << 20, P, P, P, P, P, P, P, P, None]
    assert f(*call) == T.TF_ERANGE
    for i in (4, 5, 6, 7, 8, 9, 10):              # temperature, top_k, top_p, min_p, u, pick, prob
        for off in (1, 2, 3):
            a = list(call)
            a[i] = P + off
            assert f(*a) == T.TF_EINVAL, (i, off)
    assert f(*call[:11], P + 1, None) == T.TF_ERANGE          # flag holds bytes
