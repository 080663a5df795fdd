"""How near to a border tf_sample_rows' picks stay right: rows of one peak and a
flat tail, whose borders have a closed form, with the uniform numbers that lie
closest to them.

Tokens of a row: one of weight 1, the other n of weight w = exp(-d / T). With u
the pick is the j-th of the tail (from 0), j = floor(x) of x = (u M - 1) / w,
M = 1 + n w, which float64 gives to about 1e-16 of u. Borders are w / M apart in u, so u is
|x - round(x)| w / M from the nearest one. The kernel answers for u that are
1e-12 or more from a border; asked are fp32 values that are twice that.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROWS = 128


@pytest.fixture(scope="module")
def mods():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf, torch


def bf16(torch, v):
    return float(torch.tensor(v, dtype=torch.float64).to(torch.bfloat16))


def closest(n, w, rows, seed):
    """(u, j): the `rows` fp32 numbers above 1/2 closest to a border (2e-12 at least), and their tail tokens."""
    k = np.random.default_rng(seed).choice(1 << 23, 1 << 21, replace=False) + (1 << 23)
    u = k / float(1 << 24)
    M = 1 + n * w
    x = (u * M - 1) / w
    away = np.abs(x - np.round(x)) * w / M
    away[(away < 2e-12) | (x < 0) | (x >= n)] = 1
    at = np.argsort(away)[:rows]
    assert away[at].max() < 1e-9          # which the test is for
    return u[at].astype(np.float32), np.floor(x[at]).astype(np.int64)


def ask(mods, V, T, peak, tail, rows=ROWS, keep=None, at=0):
    """Rows of `tail` with `peak` at token `at`; `keep`: top-k."""
    tf, torch = mods
    peak, tail, T = bf16(torch, peak), bf16(torch, tail), float(np.float32(T))
    n = V - 1 if keep is None else keep - 1
    u, j = closest(n, float(np.exp((tail - peak) / T)), rows, V + at)
    x = torch.full((rows, V), tail, dtype=torch.bfloat16, device="cuda")
    x[:, at] = peak
    pick, flag = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.uint8, device="cuda")
    temp = torch.full((rows,), T, device="cuda")
    k = None if keep is None else torch.full((rows,), keep, dtype=torch.int32, device="cuda")
    tf.tf_sample_rows(x, rows, V, V, temp, k, None, None, torch.from_numpy(u).cuda(), pick, None, flag)
    torch.cuda.synchronize()
    want = np.where(j < at, j, j + 1)
    got = pick.cpu().numpy()
    assert not flag.any().item()
    assert np.array_equal(got, want), f"{int((got != want).sum())} of {rows} picks differ"


@pytest.mark.parametrize("rows", [2, ROWS])
@pytest.mark.parametrize("V,T,peak,tail", [
    (128000, 0.7, 0.0, -12.4375), (1 << 19, 1.0, 0.0, -11.875), (1 << 19, 2.0, 30.0, 6.0), (300001, 1.0, -100.0, -112.0)])
def test_flat_tail(mods, V, T, peak, tail, rows):
    ask(mods, V, T, peak, tail, rows=rows, at=V // 3)


@pytest.mark.parametrize("rows", [3, ROWS])
@pytest.mark.parametrize("V,T,peak,tail", [
    (128000, 1.0, 130.0, 118.0), (1 << 19, 50.0, -300.0, -900.0), (300001, 3e37, 3e38, -6e37),
    (1 << 19, 7.65e-42, 2.0 ** -132, 2.0 ** -133), (1 << 19, 4e-21, 2.0 ** -64, 2.0 ** -70)])
def test_flat_tail_of_other_values(mods, V, T, peak, tail, rows):
    """Values of 128 and more, and below 2^-33, are counted in other windows."""
    ask(mods, V, T, peak, tail, rows=rows)


@pytest.mark.parametrize("V,keep", [(1 << 19, 200001), (128000, 90000)])
def test_flat_tail_cut_by_top_k(mods, V, keep):
    ask(mods, V, 1.0, 0.0, -11.875, keep=keep, at=7)


@pytest.mark.parametrize("V", [1 << 19, 400001])
def test_a_whole_row_of_one_value(mods, V):
    """The largest mass a row can have: u = j / V draws token j (V a power of two: exactly)."""
    tf, torch = mods
    rows = 64
    j = np.random.default_rng(1).integers(0, V, rows)
    u = (j / V if V == 1 << 19 else (j + 0.5) / V).astype(np.float32)
    j = j if V == 1 << 19 else np.floor(u.astype(np.float64) * V).astype(np.int64)
    x = torch.full((rows, V), 5.0, dtype=torch.bfloat16, device="cuda")
    pick, flag = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.uint8, device="cuda")
    prob = torch.empty(rows, device="cuda")
    tf.tf_sample_rows(x, rows, V, V, None, None, None, None, torch.from_numpy(u).cuda(), pick, prob, flag)
    torch.cuda.synchronize()
    assert np.array_equal(pick.cpu().numpy(), j) and (prob.cpu().numpy() == np.float32(1 / V)).all()


@pytest.mark.parametrize("T,peak,tail", [(1e-6, 1.2e-5, 0.0), (1e-8, 1.5e-7, 2.0 ** -25), (1e-9, -2.0 ** -26, -2.7e-8)])
def test_flat_tail_at_small_temperatures(mods, T, peak, tail):
    """Differences of a few T, with T far below the values' usual distances."""
    ask(mods, 1 << 19, T, peak, tail)
