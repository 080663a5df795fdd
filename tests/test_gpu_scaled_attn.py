"""Attention over scaled pools against float64 on the codes' values; the bounds are
derived in scaled.check_attention. Slots past a stream's keys and spare pages hold
NaN codes and the largest scale."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGES = [16, 32, 64, 128, 256]


@pytest.fixture(scope="module")
def tf():
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf
    torch.cuda.set_device(0)
    return tf


# rows of every tile width; keys of one, around a block's, a stage's and a page's end, of several chunks
STREAMS = [(1, 1), (1, 17), (2, 64), (8, 65), (9, 31), (16, 16), (5, 1025), (12, 4700), (16, 8193), (1, 3001),
           (3, 257), (7, 2049), (6, 32)]


def bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("full", [False, True])
def test_small_rounds(tf, page, full):
    from scaled import ScaledAttn
    a = ScaledAttn(tf, STREAMS, page, seed=page)
    a.run(full)
    a.check(full)
    assert tf.tf_segments_status(a.seg) == (tf.TF_OK, 0)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16])
def test_rows_of_a_window(tf, rows):
    """Tables whose widest window has these rows (one kernel variant each)."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(rows, max(rows, k)) for k in (rows, 16, 33, 700, 2500)], 32, seed=rows)
    a.run()
    a.check(what=rows)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("rows,cached", [(1, 0), (33, 7), (300, 1700), (64, 8200)])
def test_prompt(tf, page, rows, cached):
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(rows, rows + cached)], page, seed=rows, prompt=True)
    a.run()
    a.check()


@pytest.mark.parametrize("path", ["mma", "tc"])
@pytest.mark.parametrize("page", [16, 128])
def test_forced_kernel(tf, path, page, monkeypatch):
    """Every window on either kernel, causal and FULL."""
    from scaled import ScaledAttn
    monkeypatch.setenv("TF_ATTN_PATH", path)
    a = ScaledAttn(tf, [(16, 9000), (1, 70), (10, 33), (4, 5000), (1, 1), (2, 16), (13, 8192), (7, 64)], page, seed=14)
    for full in (False, True):
        a.run(full)
        a.check(full, what=(path, full))
    assert tf.tf_segments_status(a.seg) == (tf.TF_OK, 0)


def test_many_short_units(tf):
    """Units of a tile or two, more of them than CTAs, run after one another in a CTA."""
    from scaled import ScaledAttn
    g = np.random.default_rng(5)
    a = ScaledAttn(tf, [(int(r), int(r + k)) for r, k in zip(g.integers(9, 17, 150), g.integers(0, 200, 150))], 16, seed=15)
    for _ in range(3):
        a.out[0].fill_(float("nan"))
        a.run()
        a.check()
    assert tf.tf_segments_status(a.seg) == (tf.TF_OK, 0)


@pytest.mark.parametrize("std", [1e-30, 2e-5, 300.0, 1e30])
def test_v_of_any_size(tf, std):
    """Scores and outputs far from 1: K of that size with queries of its inverse, V of that size."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(16, 2100), (1, 1500), (4, 40)], 64, seed=3, std=std, spread=6.0)
    a.q[0] = (a.q[0].float() / std).to(torch.bfloat16)
    a.run()
    a.check(what=std)


def test_zeros(tf):
    """Caches and queries of zeros (scale bytes 0), at window edges too: the mean of V, and zeros."""
    from scaled import ScaledAttn
    for keys in (9, 40, 3000):
        a = ScaledAttn(tf, [(6, keys), (1, keys), (8, keys)], 16, seed=13)
        a.K[0].zero_()
        a.ks[0].zero_()
        a.run()
        a.check(what=("K", keys))
        a.q[0].zero_()
        a.run()
        a.check(what=("q", keys))
        a.V[0].zero_()
        a.vs[0].zero_()
        assert (a.run()[0] == 0).all()


def test_blocks_of_very_different_size(tf):
    """V blocks up to 2^40 apart; the weights sit on small and on large ones."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(1, 900), (8, 1400), (16, 3000)], 16, seed=4, spread=0.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    used = a.vs[0] != 0xFE
    shift = torch.randint(-40, 1, a.vs[0].shape, generator=g, device="cuda", dtype=torch.int32)
    a.vs[0][:] = torch.where(used, (a.vs[0].int() + shift).clamp(0, 254).to(torch.uint8), a.vs[0])
    a.q[0] *= 6           # few keys carry a row
    a.run()
    a.check()


@pytest.mark.parametrize("path", ["mma", "tc"])
def test_weights_count_with_their_scales(tf, path, monkeypatch):
    """V blocks 2^45 to 2^60 below others under weights 2^34 to 2^38 above theirs. With A = sum p |v|, an output is off
    by (as in scaled.check_attention) the error of the scores, e, and of the sums, 2^-11 of a weight in fp16, and
    2^-31 of the row's largest p times its scale, where that is more, times a code of up to 448: no key may
    vanish beside a weight that its own scale makes small. The weights' exponents are sums of up to 128 in size."""
    from scaled import ScaledAttn, BLOCK, NKV
    monkeypatch.setenv("TF_ATTN_PATH", path)
    a = ScaledAttn(tf, [(16, 9000), (1, 900), (12, 70), (6, 40), (4, 3001)], 64, seed=21)
    g = torch.Generator(device="cuda").manual_seed(22)
    used = (a.K[0] & 0x7F) != 0x7F
    low = torch.rand(a.ks[0].shape, generator=g, device="cuda") < 0.5      # blocks of small weights, large V
    pick = lambda *v: torch.tensor(v, device="cuda")[torch.randint(0, len(v), a.K[0].shape[:3], generator=g, device="cuda")]
    k = torch.where(low.repeat_interleave(BLOCK, 2), pick(0.0, 0.25), pick(3.0, 3.25))    # q.k / 8 = 8 k of queries of ones
    a.K[0] = torch.where(used, k.to(torch.float8_e4m3fn).view(torch.uint8)[..., None], a.K[0])
    a.ks[0] = torch.full_like(a.ks[0], 127)
    down = torch.randint(0, 11, a.vs[0].shape, generator=g, device="cuda", dtype=torch.int32)
    a.vs[0] = (127 - torch.where(low, down, 45 + (down * 3) // 2)).to(torch.uint8)
    a.q[0] = torch.ones_like(a.q[0]) * (1 - 0.5 * (torch.rand(a.q[0].shape[:2] + (1,), generator=g, device="cuda") < 0.3)).to(torch.bfloat16)
    a.build()
    a.run()
    for (rows, o, keys), ids in zip(a.streams, a.lists):
        kv, _ = a.cache(a.K[0], a.ks[0], ids, keys)
        v, vs = a.cache(a.V[0], a.vs[0], ids, keys)
        sees = torch.arange(keys, device="cuda")[None] < keys - rows + 1 + torch.arange(rows, device="cuda")[:, None]
        q = a.q[0][o:o + rows].double().view(rows, NKV, -1, 64)
        for h in range(NKV):
            s = torch.einsum("rhd,kd->rhk", q[:, h], kv[h]) / 8
            p = torch.softmax(torch.where(sees[:, None], s, -torch.inf), -1)
            ref, A = p @ v[h], p @ v[h].abs()
            e = 70 * 2.0 ** -23 * s.abs().amax(-1) + 2.0 ** -21 + 2.0 ** -22 * 128
            top = (p * torch.exp2(vs[h].double() - 127)).amax(-1)
            bound = (2 * e + 2.0 ** -11 + 2 * (keys / 64 + 64) * 2.0 ** -23)[..., None] * A \
                + (keys * 2.0 ** -31 * 448 * top)[..., None]
            bound = bound + 2.0 ** -8 * (ref.abs() + bound)
            err = (a.out[0][o:o + rows].view(rows, NKV, -1, 64)[:, h].double() - ref).abs()
            assert (err <= bound).all(), (rows, keys, h, float((err / bound).max()), float((err / ref.abs()).max()))


@pytest.mark.parametrize("path", ["mma", "tc"])
def test_the_smallest_scale_of_k(tf, path, monkeypatch):
    """Scale byte 0 is 2^-127, which queries near 2^120 can tell from 0."""
    from scaled import ScaledAttn
    monkeypatch.setenv("TF_ATTN_PATH", path)
    a = ScaledAttn(tf, [(16, 700), (4, 90), (1, 2100), (10, 3000)], 32, seed=23)
    a.ks[0].zero_()
    a.q[0] = (a.q[0].float() * 2.0 ** 120).to(torch.bfloat16)
    a.run()
    a.check(what=path)


@pytest.mark.parametrize("factor", [0.0, 2.0 ** -120, 2.0 ** 100])
def test_queries_of_any_size(tf, factor):
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(2, 400), (1, 30)], 16, seed=5)
    a.q[0] = (a.q[0].double() * factor).to(torch.bfloat16)
    for s in a.ks:
        s[:] = torch.where(s == 0xFE, s, (s.int() - (100 if factor > 1 else 0)).clamp(min=0).to(torch.uint8))
    a.run()
    a.check(what=factor)


@pytest.mark.parametrize("path", ["mma", "tc"])
def test_nan_stays_with_the_rows_that_see_it(tf, path, monkeypatch):
    """NaN codes of K and V at the window's own keys, and deep in the cache, over one and several chunks."""
    from scaled import ScaledAttn
    monkeypatch.setenv("TF_ATTN_PATH", path)
    for keys in (40, 1500, 9000):
        clean = ScaledAttn(tf, [(16, keys), (6, keys), (1, keys)], 32, seed=6)
        clean.run()
        for pool in ("K", "V"):
            a = ScaledAttn(tf, [(16, keys), (6, keys), (1, keys)], 32, seed=6)
            seen = []
            for (r, o, k), ids, at in zip(a.streams, a.lists, (keys - 11, keys - 2, 3)):
                getattr(a, pool)[0][int(ids[at // 32]), 2, at % 32, 5] = 0x7F     # head 2, dimension 5
                seen.append(at)
            a.run()
            for (r, o, k), at in zip(a.streams, seen):
                for i in range(r):
                    hit = at < k - r + i + 1
                    got, want = a.out[0][o + i].clone(), clean.out[0][o + i].clone()
                    if hit:
                        head = got[8:12] if pool == "K" else got[8:12, 5]
                        assert torch.isnan(head).all(), (pool, keys, r, i)
                        head.zero_()
                        (want[8:12] if pool == "K" else want[8:12, 5]).zero_()
                    assert torch.equal(bits(got), bits(want)), (pool, keys, r, i)


def test_nan_queries(tf):
    """A NaN or an infinity in a query's head stays in that head's row."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(4, 3000), (16, 90)], 64, seed=7)
    want = a.run()[0].clone()
    a.q[0][1, 6, 3] = float("nan")
    a.q[0][9, 31, 63] = float("inf")
    got = a.run()[0]
    for r, h in ((1, 6), (9, 31)):
        assert torch.isnan(got[r, h]).all()
        got[r, h] = want[r, h]
    assert torch.equal(bits(got), bits(want))


def test_result_is_the_streams_own(tf):
    """A stream's bits depend neither on its pages nor on the other streams of its width's kernel."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(5, 2000), (6, 5000)], 16, seed=8)
    a.run()
    g = np.random.default_rng(1)
    move = torch.as_tensor(g.permutation(a.n_pages), device="cuda")
    b = ScaledAttn(tf, [(5, 2000), (6, 5000)], 16, seed=8)
    for x, y in ((a.K, b.K), (a.V, b.V), (a.ks, b.ks), (a.vs, b.vs)):
        y[0][move] = x[0]
    b.lists = [move[torch.as_tensor(l.astype(np.int64), device="cuda")].cpu().numpy().astype(np.int32) for l in a.lists]
    b.build()
    b.run()
    assert torch.equal(bits(a.out[0]), bits(b.out[0]))


def test_bits_alone_and_in_company(tf):
    """A stream alone and among wider windows, narrower ones and those of the other kernel: the same bits. Large
    queries move the references often."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(5, 2000), (1, 3001), (8, 1200), (3, 900), (2, 40), (16, 2100), (6, 1555), (12, 9000)], 32,
                   seed=18)
    a.q[0] *= 5
    a.run()
    a.check()
    for (r, o, k), ids in zip(a.streams, a.lists):
        seg = tf.tf_paged_scaled_build([(r, 0, k, len(ids) * 32)], None, None, ids, 32, a.n_pages, a.K, a.V, a.ks, a.vs,
                                       0, 1)
        partials = torch.empty(max(seg.partials_bytes // 4, 4), device="cuda")
        out = torch.empty_like(a.out[0][o:o + r])
        tf.tf_attn_paged(seg, 0, a.q[0][o:o + r].contiguous(), partials, out)
        assert torch.equal(bits(out), bits(a.out[0][o:o + r])), (r, k)


def test_layers_side_by_side(tf):
    """Two layers of one table on two streams at once, each with partials of its own."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(16, 8300), (2, 5000), (9, 70), (1, 900), (16, 20000)], 64, seed=19, layers=2)
    want = [x.clone() for x in a.run()]
    partials = [torch.full_like(a.partials, float("nan")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o in a.out:
            o.zero_()
        torch.cuda.synchronize()
        for l in (0, 1):
            tf.tf_attn_paged(a.seg, l, a.q[l], partials[l], a.out[l], False, streams[l])
        torch.cuda.synchronize()
        for l in (0, 1):
            assert torch.equal(bits(a.out[l]), bits(want[l])), l
    assert tf.tf_segments_status(a.seg) == (tf.TF_OK, 0)


@pytest.mark.parametrize("streams,prompt", [([(16, 2049), (9, 8192), (12, 8193), (16, 33000), (8, 4096)], False),
                                            ([(1, 20000), (4, 12000), (2, 8193), (6, 30000), (16, 9000)], False),
                                            ([(1, 9217), (3, 9216)], False),
                                            ([(20, 4100)], True), ([(65, 2600)], True), ([(300, 5001)], True)])
def test_chunks_and_their_scratch(tf, streams, prompt):
    """Windows of as many chunks as their table gives them, and nothing behind the table's scratch is written."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, streams, 256, seed=20, prompt=prompt)
    n = a.seg.partials_bytes // 4
    a.partials = torch.full((n + 4096,), 7.0, device="cuda")
    for full in (False,) if prompt else (False, True):   # (a prompt's windows end at their own last row)
        a.run(full)
        a.check(full, what=full)
    assert (a.partials[n:] == 7).all()


def test_pool_beyond_32_bits(tf):
    """Pages past 4 GB of codes."""
    from scaled import ScaledAttn
    page, n_pages = 256, (1 << 15) + 100           # 128 KB a page
    ids = [np.arange(n_pages - 3, n_pages, dtype=np.int32), np.array([5, n_pages - 9, n_pages - 20, 16390], np.int32)]
    small = ScaledAttn(tf, [(1, 600), (16, 900)], page, seed=9)
    want = small.run()[0]
    a = small
    pools = []
    for x in (a.K, a.V, a.ks, a.vs):
        big = torch.zeros((n_pages,) + x[0].shape[1:], dtype=torch.uint8, device="cuda")
        for far, near in zip(ids, a.lists):
            big[torch.as_tensor(far.astype(np.int64), device="cuda")] = x[0][torch.as_tensor(near.astype(np.int64), device="cuda")]
        pools.append([big])
    table = [(r, o, k, len(x) * page) for (r, o, k), x in zip(a.streams, ids)]
    seg = tf.tf_paged_scaled_build(table, None, None, np.concatenate(ids), page, n_pages, *pools, 0, 1)
    out = torch.empty_like(want)
    tf.tf_attn_paged(seg, 0, a.q[0], a.partials, out)
    assert torch.equal(bits(out), bits(want))


def test_captured_and_replayed(tf):
    """Two layers in a graph on a side stream, replayed on changed queries."""
    from scaled import ScaledAttn
    p = ScaledAttn(tf, [(1, 900), (9, 70), (16, 8300), (3, 2050)], 64, seed=10, layers=2)
    want = [x.clone() for x in p.run()]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        p.run(stream=torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(s)
    for o in p.out:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(p.out, want):
        assert torch.equal(bits(a), bits(b))
    p.q[0].copy_(p.q[1])
    g.replay()
    p.check()


def test_a_wait_that_runs_out(tf):
    """With a wait limit of 0 the tensor-core kernel gives up, reports it, and works again afterwards."""
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(16, 9000), (12, 300)], 64, seed=16)
    want = a.run()[0].clone()
    torch.cuda.synchronize()
    try:
        tf.tf_set_wait_limit_ns(0)
        a.run()
        rc, bits_ = tf.tf_segments_status(a.seg)
        assert rc == tf.TF_ETIMEOUT and bits_ == tf.TF_STATUS_ATTN_TIMEOUT
    finally:
        tf.tf_set_wait_limit_ns(tf.TF_WAIT_LIMIT_DEFAULT_NS)
    assert tf.tf_segments_status(a.seg) == (tf.TF_OK, 0)
    a.run()
    assert torch.equal(bits(a.out[0]), bits(want)) and tf.tf_segments_status(a.seg) == (tf.TF_OK, 0)


def test_refusals(tf):
    from scaled import ScaledAttn
    a = ScaledAttn(tf, [(2, 40)], 16, seed=11)
    out32 = torch.empty((a.R, 32, 64), device="cuda")

    def status(fn, *args):
        with pytest.raises(tf.TFError) as e:
            fn(*args)
        return e.value.status

    for fn in (tf.tf_attn, tf.tf_attn_block):
        assert status(fn, a.seg, 0, a.q[0], a.partials, out32) == tf.TF_EINVAL
    assert status(tf.tf_attn_partials, a.seg, 0, a.q[0], a.partials) == tf.TF_EINVAL
    assert status(tf.tf_attn_merge, a.seg, a.partials, out32) == tf.TF_EINVAL
    assert status(tf.tf_attn_static, a.seg, 0, a.q[0], out32) == tf.TF_EINVAL
    for layer in (-1, 1):
        assert status(tf.tf_attn_paged, a.seg, layer, a.q[0], a.partials, a.out[0]) == tf.TF_EINVAL
    assert status(tf.tf_attn_paged, a.seg, 0, a.q[0], a.partials, a.q[0]) == tf.TF_EINVAL
    assert status(tf.tf_attn_paged, a.seg, 0, a.q[0], a.partials, a.out[0].data_ptr() + 2) == tf.TF_EINVAL
    assert status(tf.tf_attn_paged, a.seg, 0, None, a.partials, a.out[0]) == tf.TF_EINVAL
