"""Scaled pools, norm and product rows on the CPU: every refusal is made on the host
before a GPU is touched. (What is refused by where the memory lies needs a device.)"""

import numpy as np
import pytest

P0 = 0x7F0000000000      # made-up device addresses, 16-byte aligned, far apart
POOL = 1 << 36


@pytest.fixture(scope="module")
def T():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    return tf


KV = dict(k=[P0], v=[P0 + POOL], ks=[P0 + 2 * POOL], vs=[P0 + 3 * POOL])
GOOD = [(2, 0, 20, 32), (1, 2, 33, 48)]


def build(T, streams, pages, page=16, n_pages=64, n_attn=1, **kw):
    a = {**KV, **kw}
    rc, h = T.tf_paged_scaled_build_status(streams, None, None, pages, page, n_pages, a["k"], a["v"], a["ks"], a["vs"], 0,
                                           n_attn, stream=0)
    assert h is None
    return rc


def prompt(T, rows, keys, cap, pages, page=16, n_pages=64, **kw):
    a = {**KV, **kw}
    rc, h = T.tf_paged_scaled_prompt_build_status(rows, keys, cap, None, pages, page, n_pages, a["k"], a["v"], a["ks"],
                                                  a["vs"], 0, 1, stream=0)
    assert h is None
    return rc


@pytest.mark.parametrize("page", [0, 8, 24, 512, -16])
def test_page_size(T, page):
    assert build(T, [(1, 0, 1, 512)], np.zeros(64, np.int32), page=page) == T.TF_EINVAL
    assert prompt(T, 1, 1, 512, np.zeros(64, np.int32), page=page) == T.TF_EINVAL


@pytest.mark.parametrize("pages", [[0, 64, 2, 3, 4], [0, 1, 2, -1, 4], [0, 1, 2, 3, 1], [0, 1, 1, 3, 4]])
def test_page_lists(T, pages):
    """Ids out of the pool, window pages that stand twice."""
    assert build(T, GOOD, pages) == T.TF_EINVAL


def test_streams(T):
    for streams in ([(1, 0, 1, 24)], [(4, 0, 3, 16)], [(1, 0, 17, 16)], [(2, 0, 20, 32), (1, 3, 33, 48)]):
        assert build(T, streams, list(range(8))) == T.TF_EINVAL
    assert build(T, [(17, 0, 20, 32)], [0, 1]) == T.TF_ERANGE
    assert prompt(T, 65537, 65537, 65552, np.zeros(4097, np.int32)) == T.TF_ERANGE
    assert prompt(T, 33, 40, 48, [0, 1, 0]) == T.TF_EINVAL
    assert build(T, [(1, 0, 1, 16)], [0], n_pages=(1 << 24) + 1) == T.TF_ERANGE


def test_pools_and_scales(T):
    ok = [(1, 0, 1, 16)]
    nb, ns = 64 * 8 * 16 * 64, 64 * 8                # a pool's codes and scales
    for name in KV:
        assert build(T, ok, [0], **{name: [None]}) == T.TF_EINVAL
        assert build(T, ok, [0], **{name: None}) == T.TF_EINVAL
        assert prompt(T, 1, 1, 16, [0], **{name: None}) == T.TF_EINVAL
    assert build(T, ok, [0], v=[P0 + POOL + 8]) == T.TF_EINVAL               # codes at 8 bytes
    assert build(T, ok, [0], v=[P0 + nb - 16]) == T.TF_EINVAL                # K and V overlap
    assert build(T, ok, [0], ks=[P0 + nb - 1]) == T.TF_EINVAL                # scales in the codes
    assert build(T, ok, [0], vs=[P0 + 2 * POOL + ns - 1]) == T.TF_EINVAL     # scales of K and V overlap
    two = dict(k=[P0, P0 + 4 * POOL], v=[P0 + POOL, P0 + 5 * POOL], vs=[P0 + 3 * POOL, P0 + 7 * POOL])
    assert build(T, ok, [0], n_attn=2, ks=[P0 + 2 * POOL, P0 + 2 * POOL], **two) == T.TF_EINVAL
    assert build(T, ok, None) == T.TF_EINVAL


def test_copy(T):
    def status(pools, scales, src, dst, keys=None, page=16, n_pages=8):
        with pytest.raises(T.TFError) as e:
            T.tf_pages_copy_scaled(pools, scales, page, n_pages, src, dst, keys, stream=0)
        return e.value.status

    pools, scales = [P0, P0 + POOL], [P0 + 2 * POOL, P0 + 3 * POOL + 1]
    nb = 8 * 8 * 16 * 64
    for src, dst, keys in (([0], [8], None), ([-1], [1], None), ([0, 1], [2, 2], None), ([0, 2], [2, 3], None),
                           ([0], [1], [17]), ([0], [1], [-1])):
        assert status(pools, scales, src, dst, keys) == T.TF_EINVAL
    assert status(pools, [P0 + 2 * POOL, None], [0], [1]) == T.TF_EINVAL
    assert status([P0, P0 + 8], scales, [0], [1]) == T.TF_EINVAL
    assert status([P0, P0 + nb - 16], scales, [0], [1]) == T.TF_EINVAL
    assert status(pools, [P0 + nb - 1, P0 + 3 * POOL], [0], [1]) == T.TF_EINVAL
    assert status(pools, [P0 + 2 * POOL, P0 + 2 * POOL + 63], [0], [1]) == T.TF_EINVAL
    assert status(pools, scales, [0], [1], page=24) == T.TF_EINVAL
    assert status(pools, scales, [0], [1], n_pages=(1 << 24) + 1) == T.TF_ERANGE
    with pytest.raises(ValueError):
        T.tf_pages_copy_scaled(pools, scales[:1], 16, 8, [0], [1], stream=0)
    T.tf_pages_copy_scaled(pools, scales, 16, 8, [], [], stream=0)          # nothing to do


def test_norm(T):
    A = dict(x=P0, xs=64, res=P0 + POOL, rs=64, w=P0 + 2 * POOL, eps=1e-5, R=4, width=64, sum=P0 + 3 * POOL, ss=64,
             codes=P0 + 4 * POOL, scales=P0 + 5 * POOL)

    def status(**kw):
        a = {**A, **kw}
        with pytest.raises(T.TFError) as e:
            T.tf_norm_rows(a["x"], a["xs"], a["res"], a["rs"], a["w"], a["eps"], a["R"], a["width"], a["sum"], a["ss"],
                           a["codes"], a["scales"], stream=0)
        return e.value.status

    for name in ("x", "w", "codes", "scales"):
        assert status(**{name: None}) == T.TF_EINVAL
    for name in ("x", "res", "w", "sum", "codes"):
        assert status(**{name: A[name] + 8}) == T.TF_EINVAL
    assert status(res=None) == T.TF_EINVAL and status(sum=None) == T.TF_EINVAL
    for kw in (dict(width=0), dict(width=48), dict(xs=56), dict(rs=68), dict(ss=32), dict(R=-1), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert status(**kw) == T.TF_EINVAL, kw
    assert status(R=(1 << 24) + 1) == T.TF_ERANGE
    wide = (1 << 14) + 32
    assert status(width=wide, xs=wide, rs=wide, ss=wide) == T.TF_ERANGE
    assert status(xs=(1 << 32) + 8) == T.TF_ERANGE
    row = 128                                        # bytes of a row
    for kw in (dict(sum=P0 + 3 * row + 112), dict(sum=P0 + 16), dict(sum=P0, ss=72), dict(codes=P0 + 3 * row),
               dict(codes=A["w"] + 112), dict(scales=A["sum"] + 4 * row - 1), dict(scales=A["codes"] + 255),
               dict(sum=A["w"]), dict(codes=A["res"]), dict(x=P0, xs=128, sum=P0 + 64, ss=128)):
        assert status(**kw) == T.TF_EINVAL, kw
    T.tf_norm_rows(None, 0, None, 0, None, 1e-5, 0, 64, None, 0, None, None, stream=0)       # no rows


def test_linear(T):
    A = dict(x=P0, xs=64, sc=None, R=4, K=64, w=P0 + POOL, g=P0 + 2 * POOL, s=P0 + 3 * POOL, N=40, y=P0 + 4 * POOL, ys=40)

    def status(**kw):
        a = {**A, **kw}
        with pytest.raises(T.TFError) as e:
            T.tf_linear_rows(a["x"], a["xs"], a["sc"], a["R"], a["K"], a["w"], a["g"], a["s"], a["N"], a["y"], a["ys"],
                             stream=0)
        return e.value.status

    for name in ("x", "w", "g", "s", "y"):
        assert status(**{name: None}) == T.TF_EINVAL
    for name, off in (("x", 8), ("w", 8), ("s", 2), ("y", 1)):
        assert status(**{name: A[name] + off}) == T.TF_EINVAL
    for kw in (dict(K=0), dict(K=48), dict(N=0), dict(R=-1), dict(xs=56), dict(xs=68), dict(sc=P0 + 5 * POOL, xs=72),
               dict(ys=39)):
        assert status(**kw) == T.TF_EINVAL, kw
    for kw in (dict(R=(1 << 20) + 1), dict(K=(1 << 20) + 32, xs=1 << 21), dict(N=(1 << 24) + 1, ys=1 << 25),
               dict(xs=(1 << 32) + 8), dict(ys=(1 << 32) + 1)):
        assert status(**kw) == T.TF_ERANGE, kw
    for kw in (dict(y=P0 + 4 * 128 - 2), dict(y=A["w"] + 40 * 32 - 2), dict(y=A["g"]), dict(y=A["s"] + 158),
               dict(sc=A["y"] + 4 * 80 - 1)):
        assert status(**kw) == T.TF_EINVAL, kw
    T.tf_linear_rows(None, 64, None, 0, 64, None, None, None, 40, None, 40, stream=0)        # no rows
