"""tf_pages_copy's refusals, made on the host before a GPU is touched."""

import numpy as np
import pytest

P0, POOL = 0x7F0000000000, 1 << 36      # made-up device addresses


@pytest.fixture(scope="module")
def T():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    return tf


def status(T, pools=(P0, P0 + POOL), page=16, n_pages=8, src=(0, 1), dst=(2, 3), keys=None):
    with pytest.raises(T.TFError) as e:
        T.tf_pages_copy(list(pools), page, n_pages, list(src), list(dst), keys, stream=0)
    return e.value.status


@pytest.mark.parametrize("change", [
    dict(page=0), dict(page=8), dict(page=24), dict(page=512), dict(n_pages=0), dict(n_pages=-3),
    dict(pools=(P0, None)), dict(pools=(P0, P0 + POOL + 8)), dict(pools=(P0, P0)),
    dict(pools=(P0, P0 + 8 * 8 * 16 * 128 - 16)),                   # one pool runs into the next
    dict(src=(0, 8)), dict(src=(-1, 0)), dict(dst=(2, 8)), dict(dst=(-2, 3)),
    dict(dst=(2, 2)),                                               # written twice
    dict(dst=(2, 0)), dict(src=(0, 3)), dict(src=(2, 1)),           # written and read
    dict(keys=[16, 17]), dict(keys=[-1, 4]),
    dict(n_pages=1 << 20, dst=(1 << 19, 1 << 19)),                  # the same in a pool far larger than the lists
    dict(n_pages=1 << 20, dst=(2, 0)), dict(n_pages=1 << 20, src=(9, 1 << 19), dst=(1 << 19, 3)),
    dict(n_pages=1 << 20, src=(0, 1 << 20)),
])
def test_refused(T, change):
    assert status(T, **change) == T.TF_EINVAL


def test_limits(T):
    assert status(T, n_pages=(1 << 24) + 1) == T.TF_ERANGE
    assert status(T, pools=[P0 + i * POOL for i in range(8193)]) == T.TF_ERANGE


def test_null_lists(T):
    pools = (__import__("ctypes").c_void_p * 1)(P0)
    assert T.lib().tf_pages_copy(None, 1, 16, 8, None, None, None, 0, None) == T.TF_EINVAL
    assert T.lib().tf_pages_copy(pools, 1, 16, 8, None, None, None, 1, None) == T.TF_EINVAL
    assert T.lib().tf_pages_copy(pools, -1, 16, 8, None, None, None, 0, None) == T.TF_EINVAL
    assert T.lib().tf_pages_copy(pools, 1, 16, 8, None, None, None, -1, None) == T.TF_EINVAL


def test_nothing_to_copy(T):
    T.tf_pages_copy([P0], 16, 8, [], [], stream=0)
    T.tf_pages_copy([], 16, 8, [0], [1], stream=0)
    T.tf_pages_copy([P0], 16, 8, [0, 1], [2, 3], [0, 0], stream=0)


def test_list_lengths(T):
    with pytest.raises(ValueError):
        T.tf_pages_copy([P0], 16, 8, [0, 1], [2], stream=0)
    with pytest.raises(ValueError):
        T.tf_pages_copy([P0], 16, 8, np.array([0, 1], np.int32), np.array([2, 3], np.int32), [4], stream=0)
