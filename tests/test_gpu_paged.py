"""Attention over paged caches against the dense kernels and the float64 oracle.

The paged kernels do the dense ones' arithmetic in the same order, so a paged
result is the dense fp32 result rounded once to bf16, bit for bit, whatever the
pages. Against the oracle the dense bar (max-abs 2e-3, relative L2 1e-3 of the
fp32 result) grows by that rounding: half a step of bf16, 2^-8 of the value.

Unused slots of the pools (past a stream's keys, spare pages) hold NaN.
"""

import numpy as np
import pytest

from oracle import step as O
from parity import check_exact

pytestmark = pytest.mark.gpu

PAGES = [16, 32, 64, 128, 256]


@pytest.fixture(scope="module")
def mods():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import tf, inputs, step
    torch.cuda.set_device(0)
    return tf, inputs, step, torch


def work(inputs, rows, keys, n_attn=1, seed=5):
    return inputs.Workload("paged", rows, keys, 0, n_attn, vocab=8, drafts="none", seed=seed)


def dense_bits(mods, inp, full=False, prompt=False):
    """The dense call's fp32 output rounded to bf16."""
    tf, inputs, step, torch = mods
    d = step.DeviceStep(inp, keep_history=False, prompt=prompt)
    outs = []
    for l in range(len(inp.q)):
        (tf.tf_attn_block if full else tf.tf_attn)(d.seg, l, d.q[l], d.partials, d.out[l])
        outs.append(inputs.to_numpy_bits(d.out[l].to(torch.bfloat16)))
    torch.cuda.synchronize()
    d.free()
    return outs


def check_oracle(mods, inp, outs, full=False, what="paged"):
    _, inputs, _, _ = mods
    for l, out in enumerate(outs):
        got = O.bf16_to_f64(out)
        for s, (r, o, k) in enumerate(inp.streams):
            ref = O.attention_stream(inp.q[l][o:o + r], inp.K[l][s], inp.V[l][s], k, r, full=full)
            err = np.abs(got[o:o + r] - ref)
            bound = 2e-3 + 2.0 ** -8 * (np.abs(ref) + 2e-3)
            assert not (err > bound).any(), (what, l, s, float((err - bound).max()))
            rel = np.linalg.norm(got[o:o + r] - ref) / np.linalg.norm(ref)
            assert rel <= 1e-3 + 2.0 ** -8, (what, l, s, rel)


def run(mods, inp, page, full=False, prompt=False, seed=1):
    from paged import PagedAttn
    tf, inputs, _, torch = mods
    p = PagedAttn(tf, inp, page, seed, prompt=prompt)
    p.run(full)
    torch.cuda.synchronize()
    outs = [inputs.to_numpy_bits(x) for x in p.out]
    assert tf.tf_segments_status(p.seg) == (tf.TF_OK, 0)
    p.seg.free()
    return outs


# rows of both kernels; keys of one, around a page's and a tile's end, of several chunks
ROWS = [1, 1, 2, 8, 9, 16, 5, 12, 16, 1, 3]
KEYS = [1, 17, 64, 65, 31, 16, 1025, 4700, 8193, 3001, 257]


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("full", [False, True])
def test_small_rounds(mods, page, full):
    _, inputs, _, _ = mods
    inp = inputs.make_inputs(work(inputs, ROWS, KEYS), backend="numpy")
    outs = run(mods, inp, page, full)
    check_exact(outs[0], dense_bits(mods, inp, full)[0], "paged against dense")
    check_oracle(mods, inp, outs, full)


@pytest.mark.parametrize("path", ["mma", "tc"])
@pytest.mark.parametrize("page", [16, 128])
def test_forced_kernel(mods, path, page, monkeypatch):
    monkeypatch.setenv("TF_ATTN_PATH", path)
    _, inputs, _, _ = mods
    inp = inputs.make_inputs(work(inputs, [16, 1, 10, 4], [9000, 70, 33, 5000]), backend="numpy")
    outs = run(mods, inp, page)
    check_exact(outs[0], dense_bits(mods, inp)[0], "paged against dense")
    check_oracle(mods, inp, outs)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("rows,cached", [(1, 0), (33, 7), (300, 1700), (64, 8200)])
def test_prompt(mods, page, rows, cached):
    _, inputs, _, _ = mods
    inp = inputs.make_inputs(inputs.prompt_workload(rows, cached, 0, 1, seed=rows + cached), backend="numpy")
    outs = run(mods, inp, page, prompt=True)
    check_exact(outs[0], dense_bits(mods, inp, prompt=True)[0], "paged prompt against dense")
    check_oracle(mods, inp, outs)


@pytest.mark.parametrize("k", [17, -20])
def test_v_beyond_fp16(mods, k):
    """V of 2^17 and 2^-20 scale: the exact recompute finds its pages again."""
    from test_gpu_vrange import scale_bits
    _, inputs, _, _ = mods
    inp = inputs.make_inputs(work(inputs, [16, 4, 1, 9], [8300, 1100, 40, 100]), backend="numpy")
    inp.V = [[scale_bits(v, k) for v in vs] for vs in inp.V]
    outs = run(mods, inp, 16)
    check_exact(outs[0], dense_bits(mods, inp)[0], "paged against dense")


def test_shared_prefix(mods):
    """Streams listing the same pages for a common prefix equal streams with copies."""
    tf, inputs, _, torch = mods
    from paged import PagedAttn
    page, shared = 32, 160
    rows, keys = [1, 16, 4], [170, 200, 161 + 3]
    inp = inputs.make_inputs(work(inputs, rows, keys), backend="numpy")
    for s in (1, 2):
        inp.K[0][s][:, :shared] = inp.K[0][0][:, :shared]
        inp.V[0][s][:, :shared] = inp.V[0][0][:, :shared]
    p = PagedAttn(tf, inp, page)
    lists = [p.lists[0]] + [np.concatenate([p.lists[0][:shared // page], x[shared // page:]]) for x in p.lists[1:]]
    table = [(r, o, k, len(x) * page) for (r, o, k), x in zip(inp.streams, lists)]
    seg = tf.tf_paged_build(table, None, None, np.concatenate(lists), page, p.n_pages, p.K, p.V, 0, 1)
    out = torch.empty_like(p.out[0])
    tf.tf_attn_paged(seg, 0, p.q[0], p.partials, out)
    want = p.run()[0]
    torch.cuda.synchronize()
    check_exact(inputs.to_numpy_bits(out), inputs.to_numpy_bits(want), "shared prefix")
    check_oracle(mods, inp, [inputs.to_numpy_bits(out)])
    seg.free()
    p.seg.free()


def test_pool_beyond_32_bits(mods):
    """Pages past 4 GB of a pool (and past 2^32 elements with both pools)."""
    tf, inputs, _, torch = mods
    page, n_pages = 256, (1 << 15) + 100            # 256 KB a page: 8.6 GB a pool
    rows, keys = [1, 16], [600, 900]
    inp = inputs.make_inputs(work(inputs, rows, keys), backend="numpy")
    ids = [np.arange(n_pages - 3, n_pages, dtype=np.int32), np.array([5, n_pages - 9, n_pages - 20, 16390], np.int32)]
    pools = []
    for c in (inp.K[0], inp.V[0]):
        pool = torch.empty((n_pages, 8, page, 64), dtype=torch.bfloat16, device="cuda")
        for cache, k, x in zip(c, keys, ids):
            t = inputs.to_torch_bf16(cache)
            for i, pg in enumerate(x):
                n = min(page, k - i * page)
                pool[int(pg), :, :n] = t[:, i * page:i * page + n]
        pools.append(pool)
    table = [(r, o, k, len(x) * page) for (r, o, k), x in zip(inp.streams, ids)]
    seg = tf.tf_paged_build(table, None, None, np.concatenate(ids), page, n_pages, [pools[0]], [pools[1]], 0, 1)
    q = inputs.to_torch_bf16(inp.q[0])
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    partials = torch.empty(max(16, seg.partials_bytes), dtype=torch.uint8, device="cuda")
    tf.tf_attn_paged(seg, 0, q, partials, out)
    torch.cuda.synchronize()
    check_exact(inputs.to_numpy_bits(out), dense_bits(mods, inp)[0], "far pages")
    seg.free()


def test_captured_and_replayed(mods):
    """Two layers in a graph on a side stream, replayed on changed inputs."""
    tf, inputs, _, torch = mods
    from paged import PagedAttn
    inp = inputs.make_inputs(work(inputs, [1, 9, 16, 3], [900, 70, 8300, 2050], n_attn=2), backend="numpy")
    p = PagedAttn(tf, inp, 64)
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
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    p.q[0].copy_(p.q[1])                       # other queries, same graph
    eager = [torch.empty_like(o) for o in p.out]
    g.replay()
    got = [o.clone() for o in p.out]
    tf.tf_attn_paged(p.seg, 0, p.q[0], p.partials, eager[0])
    torch.cuda.synchronize()
    assert torch.equal(got[0].view(torch.int16), eager[0].view(torch.int16))
    p.seg.free()


def test_refusals_of_table_kinds(mods):
    """Dense attention calls refuse a paged table, tf_attn_paged a dense one."""
    tf, inputs, step, torch = mods
    from paged import PagedAttn
    inp = inputs.make_inputs(work(inputs, [2], [40]), backend="numpy")
    p, d = PagedAttn(tf, inp, 16), step.DeviceStep(inp, keep_history=False)
    out32 = torch.empty((2, 32, 64), device="cuda")
    calls = [lambda: tf.tf_attn(p.seg, 0, p.q[0], p.partials, out32),
             lambda: tf.tf_attn_block(p.seg, 0, p.q[0], p.partials, out32),
             lambda: tf.tf_attn_partials(p.seg, 0, p.q[0], p.partials),
             lambda: tf.tf_attn_block_partials(p.seg, 0, p.q[0], p.partials),
             lambda: tf.tf_attn_merge(p.seg, p.partials, out32),
             lambda: tf.tf_attn_static(p.seg, 0, p.q[0], out32),
             lambda: tf.tf_attn_paged(d.seg, 0, d.q[0], d.partials, p.out[0]),
             lambda: tf.tf_attn_paged(p.seg, 1, p.q[0], p.partials, p.out[0]),
             lambda: tf.tf_attn_paged(p.seg, -1, p.q[0], p.partials, p.out[0]),
             lambda: tf.tf_attn_paged(p.seg, 0, p.q[0], None, p.out[0]),
             lambda: tf.tf_attn_paged(p.seg, 0, p.q[0], p.partials, p.out[0].data_ptr() + 2)]
    for call in calls:
        with pytest.raises(tf.TFError) as e:
            call()
        assert e.value.status == tf.TF_EINVAL
    empty = tf.tf_paged_build([], None, None, [], 16, 1, p.K, p.V, 0, 1)
    tf.tf_attn_paged(empty, 0, None, None, None)        # an empty round: nothing to do
    for s in (p.seg, d.seg, empty):
        s.free()


def test_whole_step_on_pages(mods):
    """Conv, accept and rewind of a paged table equal the dense table's."""
    tf, inputs, step, torch = mods
    w = inputs.Workload("paged step", [4, 1, 9], [50, 20, 100], 1, 1, vocab=500, drafts="geom=0.7", seed=8)
    inp = inputs.make_inputs(w, backend="numpy")
    d = step.DeviceStep(inp)
    d.run()
    want = d.results()
    e = step.DeviceStep(inp)
    from paged import page_lists, to_pool
    keys = [k for _, _, k in inp.streams]
    lists, n_pages = page_lists(keys, 16, 3)
    K, V = (to_pool(c[0], keys, lists, 16, n_pages) for c in (inp.K, inp.V))
    table = [(r, o, k, len(x) * 16) for (r, o, k), x in zip(inp.streams, lists)]
    e.seg.free()
    hist = [e.hist[0].data_ptr() + int(e.hist_off[s]) * 2048 * 2 for s in range(3)]
    e.seg = tf.tf_paged_build(table, [e.state[0].data_ptr() + s * 8192 for s in range(3)], hist,
                              np.concatenate(lists), 16, n_pages, [K], [V], 1, 1)
    out = torch.empty((inp.R, 32, 64), dtype=torch.bfloat16, device="cuda")
    e.conv(0)
    tf.tf_attn_paged(e.seg, 0, e.q[0], e.partials, out)
    e.head()
    got = e.results()
    for a, b in zip(got["accept"], want["accept"]):
        assert np.array_equal(a, b)
    assert np.array_equal(got["y"][0], want["y"][0])
    for a, b in zip(got["states"][0], want["states"][0]):
        assert np.array_equal(a, b)
    assert torch.equal(out.cpu(), torch.from_numpy(want["out"][0]).to(torch.bfloat16))
    d.free()
    e.free()


@pytest.mark.parametrize("page", [16, 64])
def test_wait_that_runs_out(mods, page):
    """The tensor-core kernel's bounded waits over pages: a limit of 0 gives up without
    a fault, the status word says so, and the next call is right again."""
    tf, inputs, _, torch = mods
    from paged import PagedAttn
    inp = inputs.make_inputs(work(inputs, [16, 12, 2], [9000, 700, 40]), backend="numpy")
    p = PagedAttn(tf, inp, page)
    try:
        for _ in range(5):
            tf.tf_set_wait_limit_ns(0)
            p.run()
            tf.tf_set_wait_limit_ns(tf.TF_WAIT_LIMIT_DEFAULT_NS)
            torch.cuda.synchronize()
            rc, bits = tf.tf_segments_status(p.seg)
            if rc == tf.TF_ETIMEOUT:
                break
        assert rc == tf.TF_ETIMEOUT and bits & tf.TF_STATUS_ATTN_TIMEOUT
    finally:
        tf.tf_set_wait_limit_ns(tf.TF_WAIT_LIMIT_DEFAULT_NS)
    out = [inputs.to_numpy_bits(x) for x in p.run()]
    torch.cuda.synchronize()
    assert tf.tf_segments_status(p.seg) == (tf.TF_OK, 0)
    check_exact(out[0], dense_bits(mods, inp)[0], "after a wait ran out")
    p.seg.free()


def test_two_rounds_at_once(mods):
    """Two tables over the same pools, their calls on two streams at once (scratch apart)."""
    tf, inputs, _, torch = mods
    from paged import PagedAttn
    inp = inputs.make_inputs(work(inputs, [16, 1, 8, 10], [4000, 900, 2100, 65]), backend="numpy")
    a = PagedAttn(tf, inp, 32)
    table = [(r, o, k, len(x) * 32) for (r, o, k), x in zip(inp.streams, a.lists)]
    seg = tf.tf_paged_build(table, None, None, np.concatenate(a.lists), 32, a.n_pages, a.K, a.V, 0, 1)
    out, partials = torch.empty_like(a.out[0]), torch.empty_like(a.partials)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(6):
        tf.tf_attn_paged(a.seg, 0, a.q[0], a.partials, a.out[0], stream=s[0])
        tf.tf_attn_paged(seg, 0, a.q[0], partials, out, stream=s[1])
    torch.cuda.synchronize()
    check_exact(inputs.to_numpy_bits(out), inputs.to_numpy_bits(a.out[0]), "two at once")
    check_exact(inputs.to_numpy_bits(out), dense_bits(mods, inp)[0], "two at once, dense")
    seg.free()
    a.seg.free()


def test_refuses_an_output_over_its_inputs(mods):
    """bf16 in and out have one size, but queries are read again after outputs are
    written (the exact recompute), and so are the records: all three lie apart."""
    tf, inputs, _, torch = mods
    from paged import PagedAttn
    inp = inputs.make_inputs(work(inputs, [16, 2], [9000, 40]), backend="numpy")
    p = PagedAttn(tf, inp, 16)
    n, scratch = p.q[0].numel() * 2, p.seg.partials_bytes
    buf = torch.zeros(2 * n + 32 + max(scratch, n), dtype=torch.uint8, device="cuda")
    at = buf.data_ptr()
    for q, partials, out in ((at, p.partials, at), (at, p.partials, at + 16), (at + n - 16, p.partials, at),
                             (p.q[0], at, at), (p.q[0], at, at + scratch - 16), (p.q[0], at + n - 16, at),
                             (at, at, p.out[0]), (at + scratch - 16, at, p.out[0]), (at, at + n - 16, p.out[0])):
        with pytest.raises(tf.TFError) as e:
            tf.tf_attn_paged(p.seg, 0, q, partials, out)
        assert e.value.status == tf.TF_EINVAL
    buf[:n].copy_(p.q[0].view(-1).view(torch.uint8))
    tf.tf_attn_paged(p.seg, 0, at, p.partials, at + n)          # side by side: allowed
    want = p.run()[0]
    torch.cuda.synchronize()
    assert torch.equal(buf[n:2 * n], want.view(-1).view(torch.uint8))
    p.seg.free()
