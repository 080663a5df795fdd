"""Paged tables on the CPU: every refusal is made on the host before a GPU is touched."""

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


def build(T, streams, pages, page=16, n_pages=64, k=(P0,), v=(P0 + POOL,), n_attn=1):
    rc, h = T.tf_paged_build_status(streams, None, None, pages, page, n_pages, list(k), list(v), 0, n_attn, stream=0)
    assert h is None
    return rc


GOOD = [(2, 0, 20, 32), (1, 2, 33, 48)]


@pytest.mark.parametrize("page", [0, 8, 12, 24, 48, 512, -16])
def test_page_size(T, page):
    rc, h = T.tf_paged_build_status([(1, 0, 1, 512)], None, None, np.zeros(64, np.int32), page, 64, [P0], [P0 + POOL],
                                    0, 1, stream=0)
    assert rc == T.TF_EINVAL and h is None
    rc, h = T.tf_paged_prompt_build_status(1, 1, 512, None, np.zeros(64, np.int32), page, 64, [P0], [P0 + POOL], 0, 1,
                                           stream=0)
    assert rc == T.TF_EINVAL and h is None


@pytest.mark.parametrize("pages", [[0, 64, 2, 3, 4], [0, 1, 2, -1, 4], [0, 1, 2, 3, 1 << 30]])
def test_page_id_out_of_the_pool(T, pages):
    assert build(T, GOOD, pages) == T.TF_EINVAL
    assert build(T, [(1, 0, 1, 80)], pages) == T.TF_EINVAL      # past the stream's keys too
    rc, h = T.tf_paged_prompt_build_status(2, 66, 80, None, pages, 16, 64, [P0], [P0 + POOL], 0, 1, stream=0)
    assert rc == T.TF_EINVAL and h is None


@pytest.mark.parametrize("pages", [
    [0, 1, 2, 3, 1],      # stream 1's window page (list index 2) is stream 0's
    [0, 1, 1, 3, 4],      # stream 0's window page is read by stream 1
    [0, 1, 4, 3, 4],      # a window page twice in its own list
])
def test_shared_window_page(T, pages):
    assert build(T, GOOD, pages) == T.TF_EINVAL


def test_window_over_two_pages(T):
    """Rows at keys 15 and 16: both pages are the window's."""
    assert build(T, [(2, 0, 17, 32), (1, 2, 17, 32)], [0, 1, 0, 3]) == T.TF_EINVAL
    rc, h = T.tf_paged_prompt_build_status(33, 40, 48, None, [0, 1, 0], 16, 8, [P0], [P0 + POOL], 0, 1, stream=0)
    assert rc == T.TF_EINVAL and h is None


def test_spare_capacity_counts_as_a_use(T):
    """A window page that another list holds past its keys is refused as well."""
    assert build(T, [(1, 0, 1, 16), (1, 1, 1, 32)], [5, 6, 5]) == T.TF_EINVAL


@pytest.mark.parametrize("n_pages,code", [(0, 1), (-1, 1), ((1 << 24) + 1, 2)])
def test_pool_size(T, n_pages, code):
    assert build(T, [(1, 0, 1, 16)], [0], n_pages=n_pages) == code


def test_pools(T):
    ok = [(1, 0, 1, 16)]
    assert build(T, ok, [0], k=(None,)) == T.TF_EINVAL
    assert build(T, ok, [0], v=(P0 + POOL + 8,)) == T.TF_EINVAL                 # misaligned
    nb = 64 * 8 * 16 * 64 * 2
    assert build(T, ok, [0], v=(P0 + nb - 16,)) == T.TF_EINVAL                  # K and V pools overlap
    assert build(T, ok, [0], k=(P0, P0), v=(P0 + POOL, P0 + 2 * POOL), n_attn=2) == T.TF_EINVAL
    assert build(T, ok, None) == T.TF_EINVAL
    rc, h = T.tf_paged_build_status(ok, None, None, [0], 16, 64, None, [P0], 0, 1, stream=0)
    assert rc == T.TF_EINVAL and h is None


@pytest.mark.parametrize("streams", [
    [(1, 0, 1, 24)],                 # capacity is no whole number of pages
    [(4, 0, 3, 16)],                 # what tf_segments_build refuses
    [(1, 0, 17, 16)],
    [(2, 0, 20, 32), (1, 3, 33, 48)],
])
def test_streams(T, streams):
    assert build(T, streams, list(range(8))) == T.TF_EINVAL


def test_limits(T):
    n = (1 << 28) // (1 << 18) + 1           # lists of 2^18 ids each, one stream more than fit
    ids = np.zeros(n << 18, np.int32)
    streams = [(1, s, 1, 1 << 22) for s in range(n)]
    assert build(T, streams, ids) == T.TF_ERANGE
    assert T.tf_paged_prompt_build_status(65537, 65537, 65552, None, np.zeros(4097, np.int32), 16, 64, [P0],
                                          [P0 + POOL], 0, 1, stream=0)[0] == T.TF_ERANGE


def test_short_list_is_refused_by_the_binding(T):
    with pytest.raises(ValueError):
        build(T, GOOD, [0, 1, 2, 3])
    with pytest.raises(ValueError):
        T.tf_paged_prompt_build(1, 33, 48, None, [0, 1], 16, 64, [P0], [P0 + POOL], 0, 1, stream=0)


def test_attn_paged_refuses_no_table(T):
    assert T.lib().tf_attn_paged(None, 0, P0, P0, P0, 0, None) == T.TF_EINVAL


def test_host_arrays(T):
    """The binding's int32 arrays: used in place where they fit, copied where not."""
    import ctypes

    import torch

    def read(x, n):
        at, keep = T._int32_array(x, n)
        return list((ctypes.c_int32 * n).from_address(at))

    a = np.arange(6, dtype=np.int32)
    assert T._int32_array(a, 6)[0] == a.ctypes.data
    frozen = a.copy()
    frozen.setflags(write=False)
    assert read(frozen, 6) == read(a, 6) == list(range(6))
    for x in (a[::2], a[::2].astype(np.int64), [0, 2, 4], (0, 2, 4), torch.tensor([0, 2, 4]),
              torch.tensor([0, 2, 4], dtype=torch.int32)):
        assert read(x, 3) == [0, 2, 4]
    assert T._int32_array(None) == (None, None)
    T._int32_array(np.array([], np.int32), 0)
    with pytest.raises(ValueError):
        T._int32_array(a, 7)
    with pytest.raises(OverflowError):
        T._int32_array([1 << 31], 1)


def test_block_tables_and_foreign_byte_orders(T):
    """Page lists as a [streams][pages] array are read row after row, other lists have one
    dimension; other byte orders are converted."""
    import ctypes

    import torch

    def read(x, n, **kw):
        at, keep = T._int32_array(x, n, **kw)
        return list((ctypes.c_int32 * n).from_address(at))

    a = np.arange(6, dtype=np.int32)
    wide = np.arange(12, dtype=np.int32).reshape(2, 6)
    for x in (a.reshape(2, 3), a.reshape(3, 2).astype(np.int64), torch.arange(6).view(2, 3),
              torch.arange(6, dtype=torch.int32).view(3, 2), a.reshape(2, 3).astype(">i4"), a):
        assert read(x, 6, table=True) == list(range(6))
    assert read(wide[:, ::2], 6, table=True) == [0, 2, 4, 6, 8, 10]
    assert read(wide[:, 1:3], 4, table=True) == [1, 2, 7, 8]
    assert read(a.astype(">i4"), 6) == list(range(6))
    assert read([torch.tensor(5), np.int64(6)], 2) == [5, 6]
    assert T._int32_array(a.reshape(2, 3), 6, table=True)[0] == a.ctypes.data          # in place
    for x, kw in ((a.reshape(2, 3), dict()), (torch.zeros(2, 2, dtype=torch.int32), dict()),
                  (np.int32(3).reshape(()), dict(table=True)), (a.reshape(1, 2, 3), dict(table=True)),
                  (a.reshape(2, 3), dict(n=7, table=True))):
        with pytest.raises(ValueError):
            T._int32_array(x, **kw)
    # two streams' lists as a table: taken, and a bad id in the second row is seen
    for bad, streams in ((64, [(1, 0, 1, 32), (1, 1, 17, 32)]), (-1, [(1, 0, 1, 32), (1, 1, 1, 32)])):
        assert build(T, streams, np.array([[0, 1], [2, bad]], np.int32)) == T.TF_EINVAL
        assert build(T, streams, torch.tensor([[0, 1], [2, bad]])) == T.TF_EINVAL
    with pytest.raises(ValueError):
        T.tf_pages_copy([P0], 16, 8, np.array([[0, 1], [2, 3]], np.int32), [4, 5], stream=0)
