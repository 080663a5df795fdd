"""tf_pages_copy_scaled: bytes, so every comparison is exact."""

import numpy as np
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


def make(n_pools, n_pages, page, seed, odd=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pools, scales = [], []
    for _ in range(n_pools):
        pools.append(torch.randint(0, 256, (n_pages, 8, page, 64), generator=g, device="cuda", dtype=torch.uint8))
        s = torch.randint(0, 255, (n_pages * 8 * page // 16 + 1,), generator=g, device="cuda", dtype=torch.uint8)
        scales.append(s[1 if odd else 0:][:n_pages * 8 * page // 16].view(n_pages, 8, page // 16))
    return pools, scales


def expect(pools, scales, src, dst, keys, page):
    want = [p.clone() for p in pools], [s.clone() for s in scales]
    for i, (a, b) in enumerate(zip(src, dst)):
        n = page if keys is None else int(keys[i])
        for p, q in zip(want[0], pools):
            p[b, :, :n] = q[a, :, :n]
        for p, q in zip(want[1], scales):
            p[b, :, :-(-n // 16)] = q[a, :, :-(-n // 16)]
    return want


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("n,n_pools", [(1, 1), (7, 3), (65, 2)])
def test_copy(tf, page, whole, n, n_pools):
    n_pages = 2 * n + 3
    pools, scales = make(n_pools, n_pages, page, n + page, odd=n == 7)
    ids = np.random.default_rng(n).permutation(n_pages)
    src, dst = ids[:n], ids[n:2 * n]
    keys = None if whole else np.random.default_rng(2).integers(0, page + 1, n)
    if keys is not None:
        keys[0] = 0 if n > 1 else 1
    want = expect(pools, scales, src, dst, keys, page)
    tf.tf_pages_copy_scaled(pools, scales, page, n_pages, src, dst, keys)
    for x, y in zip(pools + scales, want[0] + want[1]):
        assert torch.equal(x, y)


def test_many(tf):
    """More copies than a launch holds, more pools than a launch holds, a source several times."""
    pools, scales = make(70, 40, 16, 1)
    src, dst = np.zeros(20, np.int32), np.arange(20, 40, dtype=np.int32)
    want = expect(pools, scales, src, dst, None, 16)
    tf.tf_pages_copy_scaled(pools, scales, 16, 40, src, dst)
    assert all(torch.equal(x, y) for x, y in zip(pools + scales, want[0] + want[1]))
    pools, scales = make(2, 6000, 16, 2)
    ids = np.random.default_rng(3).permutation(6000)
    src, dst = ids[:3000], ids[3000:]
    keys = np.random.default_rng(4).integers(0, 17, 3000)
    at, to = (torch.as_tensor(x, device="cuda") for x in (src, dst))
    n = torch.as_tensor(keys, device="cuda")[:, None]
    want = [p.clone() for p in pools], [s.clone() for s in scales]
    for p, q in zip(want[0], pools):
        p[to] = torch.where((torch.arange(16, device="cuda") < n)[:, None, :, None], q[at], q[to])
    for p, q in zip(want[1], scales):
        p[to] = torch.where(n[:, :, None] > 0, q[at], q[to])
    tf.tf_pages_copy_scaled(pools, scales, 16, 6000, src, dst, keys)
    assert all(torch.equal(x, y) for x, y in zip(pools + scales, want[0] + want[1]))


def test_captured(tf):
    pools, scales = make(2, 8, 32, 5)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        tf.tf_pages_copy_scaled(pools, scales, 32, 8, [1, 2], [5, 6], [20, 32], torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    pools[0][1] ^= 0x55
    want = expect(pools, scales, [1, 2], [5, 6], [20, 32], 32)
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(pools + scales, want[0] + want[1]))


def test_host_memory_is_refused_by_the_list(tf):
    with pytest.raises(ValueError):
        pools, scales = make(1, 4, 16, 6)
        tf.tf_pages_copy_scaled(pools, scales, 16, 4, torch.zeros(1, dtype=torch.int32, device="cuda"), [1])
