"""tf_pages_copy against a copy in plain indexing, bit for bit over whole pools."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf, torch


def pools_of(torch, n, n_pages, page, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(-32768, 32768, (n_pages, 8, page, 64), generator=g, device="cuda", dtype=torch.int32)
            .to(torch.int16).view(torch.bfloat16) for _ in range(n)]


def expect(torch, pools, src, dst, keys):
    out = []
    for p in pools:
        w = p.view(torch.int16).clone()
        for i, (a, b) in enumerate(zip(src, dst)):
            n = p.shape[2] if keys is None else int(keys[i])
            w[int(b), :, :n] = w[int(a), :, :n]
        out.append(w)
    return out


def same(torch, pools, want):
    torch.cuda.synchronize()
    return all(torch.equal(p.view(torch.int16), w) for p, w in zip(pools, want))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("n_pools,copies", [(1, 1), (3, 7), (2, 70)])
def test_copies(mods, page, whole, n_pools, copies):
    tf, torch = mods
    n_pages = 2 * copies + 3
    pools = pools_of(torch, n_pools, n_pages, page, page + copies)
    rng = np.random.default_rng(copies)
    ids = rng.permutation(n_pages)
    src, dst = ids[:copies], ids[copies:2 * copies]
    keys = None if whole else np.resize([1, page, 0, page - 1, 7], copies)
    want = expect(torch, pools, src, dst, keys)
    tf.tf_pages_copy(pools, page, n_pages, src, dst, keys)
    assert same(torch, pools, want)


def test_one_source_many_forks(mods):
    tf, torch = mods
    pools = pools_of(torch, 4, 12, 16, 1)
    src, dst, keys = [5] * 6, [0, 1, 2, 3, 4, 6], [3, 16, 1, 9, 0, 15]
    want = expect(torch, pools, src, dst, keys)
    tf.tf_pages_copy(pools, 16, 12, src, dst, keys)
    assert same(torch, pools, want)


def test_more_than_a_launch_holds(mods):
    """Several argument blocks of copies, and of pools."""
    tf, torch = mods
    n = 5000
    pools = pools_of(torch, 2, 2 * n, 16, 2)
    ids = np.random.default_rng(2).permutation(2 * n).astype(np.int32)
    src, dst = ids[:n].copy(), ids[n:].copy()
    want = [p.view(torch.int16).clone() for p in pools]
    for w in want:
        w[torch.from_numpy(dst).long()] = w[torch.from_numpy(src).long()]
    tf.tf_pages_copy(pools, 16, 2 * n, src, dst)
    assert same(torch, pools, want)
    pools = pools_of(torch, 130, 4, 16, 3)
    want = expect(torch, pools, [0, 1], [3, 2], [16, 5])
    tf.tf_pages_copy(pools, 16, 4, [0, 1], [3, 2], [16, 5])
    assert same(torch, pools, want)


def test_pages_beyond_32_bits(mods):
    tf, torch = mods
    n_pages = (1 << 15) + 8                       # 256 KB a page: 8.6 GB
    pool = torch.empty((n_pages, 8, 256, 64), dtype=torch.bfloat16, device="cuda")
    pool[n_pages - 1] = torch.randn((8, 256, 64), device="cuda")
    pool[1] = 0
    pool[n_pages - 2] = 0
    tf.tf_pages_copy([pool], 256, n_pages, [n_pages - 1, n_pages - 1], [1, n_pages - 2], [256, 100])
    torch.cuda.synchronize()
    assert torch.equal(pool[1], pool[n_pages - 1])
    assert torch.equal(pool[n_pages - 2, :, :100], pool[n_pages - 1, :, :100])
    assert (pool[n_pages - 2, :, 100:] == 0).all()


def test_captured_and_replayed(mods):
    """A graph keeps the lists it was captured with, on another stream."""
    tf, torch = mods
    pools = pools_of(torch, 2, 9, 32, 4)
    src, dst, keys = np.array([0, 1], np.int32), np.array([7, 8], np.int32), np.array([32, 5], np.int32)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        tf.tf_pages_copy(pools, 32, 9, src, dst, keys)
    torch.cuda.current_stream().wait_stream(s)
    src[:], dst[:], keys[:] = 3, 4, 1             # changed after the capture: not seen
    for _ in range(2):
        for p in pools:
            p[:7] = torch.randn(p[:7].shape, device="cuda").to(p.dtype)
        want = expect(torch, pools, [0, 1], [7, 8], [32, 5])
        g.replay()
        assert same(torch, pools, want)
