"""A decode layer in low precision on real work: what is measured, and its
plain forms.

Five operators that follow one another in a round whose caches hold 8 bits and
whose weights hold 4: the residual's addition and norm with its 8-bit rows
(``tf_norm_rows``), the products of those rows with 4-bit weights
(``tf_linear_rows``), the queries' and keys' norm and rotation with the append to an
8-bit paged cache (``tf_qk_rows`` on a table of ``tf_paged_scaled_build``), the
attention over it (``tf_attn_paged``), and the copies of its pages behind a fork
or a compaction (``tf_pages_copy_scaled``). With ``own`` false ``run`` computes them
with elementary torch operations in 32 bits (angles in 64); with ``own`` true it
makes the library's calls.

8-bit values are e4m3 codes under a power-of-two scale, held as the byte e + 127
and shared by a group of 32 columns (rows) or by 16 keys of a head (caches): the
smallest scale under which no value saturates, that is with the group's largest
magnitude at most 464 * 2^e. Codes and scales come back as float8 tensors.
"""

import math
import random

import numpy as np
import torch

own = False

NQ, NKV, D = 32, 8, 64
BLOCK, GROUP = 16, 32
THETA, EPS = 1000000.0, 1e-5
BF16, E4M3, E8M0 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # decode attention of a plain round: 16 streams of one row each, small pages
        dict(name="attn 16x1 p16", op="attn", streams=16, rows=1, keys_lo=256, keys_hi=4096, page=16, kseed=12),
        # drafted windows of 64 streams, contexts from a few keys to 32,768
        dict(name="attn 64x16 p64", op="attn", streams=64, rows=16, keys_lo=16, keys_hi=32768, page=64, kseed=15),
        # long contexts, six-row windows
        dict(name="attn 4x6 long p32", op="attn", streams=4, rows=6, keys_lo=65536, keys_hi=130816, page=32, kseed=14),
        # a chunk of a prompt behind its cached part
        dict(name="attn prompt 2048 p128", op="attn", prompt=True, streams=1, rows=2048, keys_lo=8179, keys_hi=8179,
             page=128, kseed=19),
        # one decode layer of a plain round: 16 streams append a key each
        dict(name="qk 16x1 p16", op="qk", streams=16, rows=1, keys_lo=256, keys_hi=4096, page=16, kseed=12),
        # a long prompt's chunk, its positions up to 131,000
        dict(name="qk prompt 16381 p32", op="qk", prompt=True, streams=1, rows=16381, keys_lo=131001, keys_hi=131001,
             page=32, kseed=17),
        # copy-on-write of 64 forks' partly filled last pages, ten attention layers
        dict(name="copy fork 64 p64", op="copy", pools=20, n_pages=1024, page=64, copies=64, whole=False, kseed=13),
        # compaction of a pool: a thousand whole pages of four layers
        dict(name="copy compact 1000 p128", op="copy", pools=8, n_pages=2048, page=128, copies=1000, whole=True,
             kseed=14),
        # a plain round's rows between two layers: residual, norm and the next projection's input
        dict(name="norm 16", op="norm", rows=16, width=2048, residual=True),
        # a long prompt's rows
        dict(name="norm 16381", op="norm", rows=16381, width=2048, residual=True),
        # a single stream's query projection, from the norm's 8-bit rows
        dict(name="product 1 x 2048 x 2048", op="product", rows=1, k=2048, n=2048, x8=True),
        # the logits of 16 rows over the whole vocabulary, from bf16 rows
        dict(name="product 16 x 2048 x 128000", op="product", rows=16, k=2048, n=128000, x8=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "qk", "copy", "norm", "product", "product"])
    kseed = rng.randrange(1 << 20)
    if op == "attn":
        if rng.random() < 0.3:
            rows = _log_int(rng, 17, 2000)
            keys = rows + _log_int(rng, 1, 6000)
            return dict(op="attn", prompt=True, streams=1, rows=rows, keys_lo=keys, keys_hi=keys,
                        page=rng.choice([16, 32, 64, 128, 256]), kseed=kseed)
        hi = _log_int(rng, 64, 16000)
        return dict(op="attn", streams=_log_int(rng, 1, 48), rows=rng.randint(1, 16), keys_lo=16, keys_hi=hi,
                    page=rng.choice([16, 32, 64, 128, 256]), kseed=kseed)
    if op == "qk":
        if rng.random() < 0.4:
            rows = _log_int(rng, 17, 16000)
            keys = rows + _log_int(rng, 1, 110000)
            return dict(op="qk", prompt=True, streams=1, rows=rows, keys_lo=keys, keys_hi=keys,
                        page=rng.choice([16, 32, 64, 128, 256]), kseed=kseed)
        lo = _log_int(rng, 16, 8000)
        return dict(op="qk", streams=_log_int(rng, 1, 64), rows=rng.randint(1, 16), keys_lo=lo,
                    keys_hi=lo + rng.randint(1, 900), page=rng.choice([16, 32, 64, 128, 256]), kseed=kseed)
    if op == "copy":
        page = rng.choice([16, 32, 64, 128, 256])
        n_pages = _log_int(rng, 64, 16384 // page * 8)
        return dict(op="copy", pools=rng.randint(1, 8), n_pages=n_pages, page=page,
                    copies=_log_int(rng, 1, n_pages // 2), whole=rng.random() < 0.5, kseed=kseed)
    if op == "norm":
        width = rng.choice([2048, 32 * _log_int(rng, 1, 256)])
        return dict(op="norm", rows=_log_int(rng, 1, 16000 * 2048 // max(width, 2048)), width=width,
                    residual=rng.random() < 0.7)
    k = rng.choice([2048, 32 * _log_int(rng, 2, 256)])
    return dict(op="product", rows=_log_int(rng, 1, 64), k=k, n=_log_int(rng, 16, min(128000, 2048 * 60000 // k)),
                x8=rng.random() < 0.5)


# ------------------------------------------------------------------ shapes

def _streams(case):
    """[(rows, row_offset, keys)] of a case, from its own seed."""
    rng = random.Random(case["kseed"])
    out, off = [], 0
    for _ in range(case["streams"]):
        keys = max(case["rows"], _log_int(rng, case["keys_lo"], case["keys_hi"]))
        out.append((case["rows"], off, keys))
        off += case["rows"]
    return out


def _page_lists(case, streams, seed):
    """Each stream's pages in a scattered pool, and the pool's size."""
    need = [-(-k // case["page"]) for _, _, k in streams]
    n_pages = sum(need) * 9 // 8 + 1
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    ends = np.cumsum(need)
    return [ids[e - n:e] for n, e in zip(need, ends)], n_pages


def _copy_lists(case, seed):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(case["n_pages"]).astype(np.int32)
    n = case["copies"]
    keys = None if case["whole"] else rng.integers(1, case["page"] + 1, n).astype(np.int32)
    return np.ascontiguousarray(ids[:n]), np.ascontiguousarray(ids[n:2 * n]), keys


def _touched(streams, lists, P):
    """The 16-key blocks that the windows' rows fall in: the page and the block in the page, which of the block's
    slots hold rows before the window and which hold rows at all, and each row's block and slot."""
    page, block, before, held, row_block, row_slot = [], [], [], [], [], []
    slot = np.arange(BLOCK)
    for (rows, _, keys), pages in zip(streams, lists):
        first = (keys - rows) // BLOCK
        b = np.arange(first, (keys - 1) // BLOCK + 1)
        page.append(pages[b * BLOCK // P])
        block.append(b % (P // BLOCK))
        before.append(b[:, None] * BLOCK + slot < keys - rows)
        held.append(b[:, None] * BLOCK + slot < keys)
        pos = np.arange(keys - rows, keys)
        row_block.append(pos // BLOCK - first + sum(map(len, page[:-1])))
        row_slot.append(pos % BLOCK)
    cat = [np.concatenate(x) for x in (page, block, before, held, row_block, row_slot)]
    return [torch.from_numpy(x if x.dtype == bool else x.astype(np.int64)).cuda() for x in cat]


# ------------------------------------------------------------------ 8 bits

def _exponent(amax):
    """The smallest e >= -127 with amax <= 464 * 2^e (464 = 0.90625 * 2^9)."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.90625).int(), -127).clamp(min=-127)


def _codes(x, e):
    return torch.ldexp(x, -e).to(E4M3).view(torch.uint8)


def _byte(e):
    return (e + 127).to(torch.uint8)


def _value(codes, scales):
    """Values of codes under their scale bytes, both uint8 and broadcast together."""
    return torch.ldexp(codes.view(E4M3).float(), scales.int() - 127)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)

    def pool(n_pages, P):
        """A pool of pages in 8 bits, its blocks of different sizes, and their scales."""
        x = torch.randn((n_pages, NKV, P // BLOCK, BLOCK * D), generator=g, device="cuda")
        x *= torch.exp2(torch.rand((n_pages, NKV, P // BLOCK, 1), generator=g, device="cuda") * 3 - 1.5)
        e = _exponent(x.abs().amax(-1, keepdim=True))
        return _codes(x, e).view(n_pages, NKV, P, D), _byte(e[..., 0])

    op = case["op"]
    st = dict(case=case)
    if op in ("qk", "attn"):
        streams = _streams(case)
        R, P = sum(r for r, _, _ in streams), case["page"]
        lists, n_pages = _page_lists(case, streams, seed)
        K, ks = pool(n_pages, P)
        V, vs = pool(n_pages, P)
        st.update(streams=streams, K=K, V=V, ks=ks, vs=vs, q=normal(R, NQ, D),
                  pages=[torch.from_numpy(x.astype(np.int64)).cuda() for x in lists])
        if op == "qk":
            pos = np.concatenate([np.arange(k - r, k) for r, _, k in streams])
            st.update(k=normal(R, NKV, D), v=normal(R, NKV, D), qw=1 + normal(D, std=0.25), kw=1 + normal(D, std=0.25),
                      pos=torch.from_numpy(pos).cuda(), touched=_touched(streams, lists, P))
        if own:
            from stream_speculative_decode_gb300 import tf
            table = [(r, o, k, -(-k // P) * P) for r, o, k in streams]
            if case.get("prompt"):
                r, _, k, cap = table[0]
                st["seg"] = tf.tf_paged_scaled_prompt_build(r, k, cap, None, lists[0], P, n_pages, [K], [V], [ks], [vs],
                                                            0, 1)
            else:
                st["seg"] = tf.tf_paged_scaled_build(table, None, None, np.concatenate(lists), P, n_pages, [K], [V],
                                                     [ks], [vs], 0, 1)
            st["out"] = torch.empty((R, NQ, D), dtype=BF16, device="cuda")
            if op == "attn":
                st["partials"] = torch.empty(max(16, st["seg"].partials_bytes), dtype=torch.uint8, device="cuda")
    elif op == "copy":
        src, dst, keys = _copy_lists(case, seed)
        made = [pool(case["n_pages"], case["page"]) for _ in range(case["pools"])]
        slot = torch.arange(case["page"], device="cuda")[None]
        n = None if keys is None else torch.from_numpy(keys).cuda()[:, None]
        st.update(pools=[m[0] for m in made], scales=[m[1] for m in made], src=src, dst=dst, keys=keys,
                  src_dev=torch.from_numpy(src).cuda().long(), dst_dev=torch.from_numpy(dst).cuda().long(),
                  keep=None if n is None else (slot < n)[:, None, :, None],
                  keep_scale=None if n is None else (slot[:, ::BLOCK] < n)[:, None])
    elif op == "norm":
        R, W = case["rows"], case["width"]
        x = normal(R, W)
        x[:, ::97] *= 20          # channels that stand out, as a trained model's do
        st.update(x=x, res=normal(R, W, std=2.0) if case["residual"] else None, w=1 + normal(W, std=0.25))
        if own:
            st.update(sum=torch.empty_like(x) if case["residual"] else None,
                      codes=torch.empty((R, W), dtype=torch.uint8, device="cuda"),
                      scales=torch.empty((R, W // GROUP), dtype=torch.uint8, device="cuda"))
    else:
        R, K, N = case["rows"], case["k"], case["n"]
        x = normal(R, K)
        if case["x8"]:
            e = _exponent(x.float().view(R, K // GROUP, GROUP).abs().amax(-1))
            x, xs = _codes(x.float().view(R, K // GROUP, GROUP), e[..., None]).view(R, K), _byte(e)
        else:
            xs = None
        st.update(x=x, xs=xs, w=torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                  g=(0.5 + torch.rand((N, K // GROUP), generator=g, device="cuda")).to(E4M3).view(torch.uint8),
                  s=(0.5 + torch.rand(N, generator=g, device="cuda")) / math.sqrt(21.5 * K))
        if own:
            st["y"] = torch.empty((R, N), dtype=BF16, device="cuda")
    if own:
        st["outputs"] = _outputs(st, case)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return {"qk": _qk, "attn": _attn, "copy": _copy, "norm": _norm, "product": _product}[case["op"]](st, case)


def _cache(st):
    return dict(K=st["K"].view(E4M3), V=st["V"].view(E4M3), ks=st["ks"].view(E8M0), vs=st["vs"].view(E8M0))


def _outputs(st, case):
    """What ``_run_own`` returns: the buffers that its call writes, as the values they stand for."""
    op = case["op"]
    if op == "qk":
        return dict(q=st["out"], **_cache(st))
    if op == "attn":
        return dict(out=st["out"])
    if op == "copy":
        return dict(pools=[p.view(E4M3) for p in st["pools"]], scales=[s.view(E8M0) for s in st["scales"]])
    if op == "norm":
        return dict(sum=st["sum"], codes=st["codes"].view(E4M3), scales=st["scales"].view(E8M0))
    return dict(y=st["y"])


def _run_own(st, case):
    from stream_speculative_decode_gb300 import tf
    op = case["op"]
    if op == "qk":
        tf.tf_qk_rows(st["seg"], 0, st["q"], NQ * D, st["k"], NKV * D, st["v"], NKV * D, st["qw"], st["kw"], EPS, THETA,
                      st["out"])
    elif op == "attn":
        tf.tf_attn_paged(st["seg"], 0, st["q"], st["partials"], st["out"])
    elif op == "copy":
        tf.tf_pages_copy_scaled(st["pools"], st["scales"], case["page"], case["n_pages"], st["src"], st["dst"],
                                st["keys"])
    elif op == "norm":
        W = case["width"]
        tf.tf_norm_rows(st["x"], W, st["res"], W, st["w"], EPS, case["rows"], W, st["sum"], W, st["codes"],
                        st["scales"])
    else:
        tf.tf_linear_rows(st["x"], case["k"], st["xs"], case["rows"], case["k"], st["w"], st["g"], st["s"], case["n"],
                          st["y"], case["n"])
    return st["outputs"]


def _qk(st, case):
    turn = st["pos"].double()[:, None] * THETA ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]

    def norm_rotate(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    page, block, before, held, row_block, row_slot = st["touched"]

    def append(pool, scales, rows):
        blocks = pool.view(pool.shape[0], NKV, -1, BLOCK, D)
        old = blocks[page, :, block]
        x = torch.where(before[:, None, :, None], _value(old, scales[page, :, block][..., None, None]), 0.0)
        x[row_block, :, row_slot] = rows
        e = _exponent(x.abs().amax((2, 3)))
        blocks[page, :, block] = torch.where(held[:, None, :, None], _codes(x, e[..., None, None]), old)
        scales[page, :, block] = _byte(e)

    append(st["K"], st["ks"], norm_rotate(st["k"], st["kw"]))
    append(st["V"], st["vs"], st["v"].float())
    return dict(q=norm_rotate(st["q"], st["qw"]).to(BF16), **_cache(st))


def _attn(st, case):
    def read(pool, scales, pages, keys):
        n = len(pages)
        x = _value(pool[pages].view(n, NKV, -1, BLOCK * D), scales[pages][..., None])
        return x.view(n, NKV, -1, D).transpose(0, 1).reshape(NKV, -1, D)[:, :keys]

    out = []
    for (rows, off, keys), pages in zip(st["streams"], st["pages"]):   # streams differ in length
        q = st["q"][off:off + rows].float().view(rows, NKV, NQ // NKV, D).permute(1, 2, 0, 3).reshape(NKV, -1, D)
        k, v = read(st["K"], st["ks"], pages, keys), read(st["V"], st["vs"], pages, keys)
        s = (q @ k.transpose(1, 2)).view(NKV, NQ // NKV, rows, keys) * (1 / math.sqrt(D))
        if rows > 1:
            row = torch.arange(rows, device="cuda")[:, None]
            s.masked_fill_(torch.arange(keys, device="cuda")[None] > keys - rows + row, -math.inf)
        s = torch.exp(s - s.amax(-1, keepdim=True))
        o = (s.view(NKV, -1, keys) @ v).view(NKV, NQ // NKV, rows, D) / s.sum(-1, keepdim=True)
        out.append(o.permute(2, 0, 1, 3).reshape(rows, NQ, D))
    return dict(out=torch.cat(out).to(BF16))


def _copy(st, case):
    src, dst, keep, keep_scale = st["src_dev"], st["dst_dev"], st["keep"], st["keep_scale"]
    for pool, scales in zip(st["pools"], st["scales"]):
        pool[dst] = pool[src] if keep is None else torch.where(keep, pool[src], pool[dst])
        scales[dst] = scales[src] if keep is None else torch.where(keep_scale, scales[src], scales[dst])
    return dict(pools=[p.view(E4M3) for p in st["pools"]], scales=[s.view(E8M0) for s in st["scales"]])


def _norm(st, case):
    R, W = case["rows"], case["width"]
    h = st["x"].float()
    if st["res"] is not None:
        h = (h + st["res"].float()).to(BF16)
    total, h = h, h.float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["w"].float()
    n = n.view(R, W // GROUP, GROUP)
    e = _exponent(n.abs().amax(-1))
    return dict(sum=None if st["res"] is None else total, codes=_codes(n, e[..., None]).view(R, W).view(E4M3),
                scales=_byte(e).view(E8M0))


def _product(st, case):
    R, K, N = case["rows"], case["k"], case["n"]
    x = st["x"].float() if st["xs"] is None else _value(st["x"].view(R, -1, GROUP), st["xs"][..., None]).view(R, K)
    w = torch.stack([st["w"] & 15, st["w"] >> 4], -1).view(N, K // GROUP, GROUP).float() - 8
    w = (w * st["g"].view(E4M3).float()[..., None]).view(N, K)
    return dict(y=(x @ w.T * st["s"]).to(BF16))


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(st, case["page"])
    if case["op"] == "attn":
        return dict(out=_exact_attn(st, case["page"]))
    if case["op"] == "copy":
        pools, scales = [_table(E4M3)[p.long()] for p in st["pools"]], [s.double() - 127 for s in st["scales"]]
        for i in range(case["copies"]):
            n = case["page"] if st["keys"] is None else int(st["keys"][i])
            for p, s in zip(pools, scales):
                p[int(st["dst"][i]), :, :n] = p[int(st["src"][i]), :, :n]
                s[int(st["dst"][i]), :, :-(-n // BLOCK)] = s[int(st["src"][i]), :, :-(-n // BLOCK)]
        return dict(pools=pools, scales=[2.0 ** s for s in scales])
    if case["op"] == "norm":
        x = st["x"].double()
        if st["res"] is not None:
            x = x + st["res"].double()
        h = x.to(BF16).double()
        n = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["width"] + EPS) * st["w"].double()
        n = n.unflatten(1, (-1, GROUP))
        scale = _scale64(n.abs().amax(2))
        return dict(sum=None if st["res"] is None else x, codes=(n / scale[..., None]).flatten(1), scales=scale)
    return dict(y=_exact_product(st, case))


def _table(dtype):
    """The value of each byte."""
    return torch.arange(256, dtype=torch.uint8).view(dtype).double().cuda()


def _scale64(amax):
    return 2.0 ** torch.ceil(torch.log2(amax / 464)).clamp(min=-127)


def _exact_qk(st, P):
    freq = torch.tensor([THETA ** (-2 * j / D) for j in range(D // 2)], dtype=torch.float64, device="cuda")
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), st["pos"].double().outer(freq))

    def rotated(x, w):
        x = x.double()
        y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + EPS) * w.double()
        y = torch.complex(y[..., :D // 2], y[..., D // 2:]) * z[:, None]
        return torch.cat([y.real, y.imag], -1)

    out = dict(q=rotated(st["q"], st["qw"]))
    for name, sname, new in (("K", "ks", rotated(st["k"], st["kw"])), ("V", "vs", st["v"].double())):
        codes, scales = _table(E4M3)[st[name].long()], 2.0 ** (st[sname].double() - 127)
        for (rows, off, keys), pages in zip(st["streams"], st["pages"]):
            start = (keys - rows) // BLOCK * BLOCK               # the window's blocks as one run of keys
            t = torch.arange(start, keys, device="cuda")
            x = codes[pages[t // P], :, t % P] * scales[pages[t // P], :, t % P // BLOCK][..., None]
            x[keys - rows - start:] = new[off:off + rows]
            most = torch.zeros((len(t) + BLOCK - 1) // BLOCK, NKV, dtype=torch.float64, device="cuda")
            most.index_reduce_(0, (t - start) // BLOCK, x.abs().amax(-1), "amax")
            scale = _scale64(most)
            b = torch.arange(len(most), device="cuda") * BLOCK + start
            scales[pages[b // P], :, b % P // BLOCK] = scale
            codes[pages[t // P], :, t % P] = x / scale[(t - start) // BLOCK][..., None]
        out.update({name: codes, sname: scales})
    return out


def _exact_attn(st, P):
    value, out = _table(E4M3), torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for (rows, off, keys), pages in zip(st["streams"], st["pages"]):
        t = torch.arange(keys, device="cuda")
        page, slot = pages[t // P], t % P
        sees = t[None] < (keys - rows + 1 + torch.arange(rows, device="cuda"))[:, None]
        for g in range(NKV):
            k, v = (value[c[page, g, slot].long()] * 2.0 ** (s[page, g, slot // BLOCK].double() - 127)[:, None]
                    for c, s in ((st["K"], st["ks"]), (st["V"], st["vs"])))
            for h in range(g * 4, g * 4 + 4):
                s = st["q"][off:off + rows, h].double() @ k.T / 8
                out[off:off + rows, h] = torch.softmax(torch.where(sees, s, -math.inf), 1) @ v
    return out


def _exact_product(st, case):
    """In runs of outputs, the even and the odd inputs apart."""
    x = st["x"].double() if st["xs"] is None else \
        _table(E4M3)[st["x"].long()] * (2.0 ** (st["xs"].double() - 127)).repeat_interleave(GROUP, 1)
    g = _table(E4M3)[st["g"].long()]
    y = []
    for n in range(0, case["n"], 8192):
        w, scale = st["w"][n:n + 8192].double(), g[n:n + 8192].repeat_interleave(GROUP // 2, 1)
        high = torch.floor(w / 16)
        y.append((x[:, ::2] @ ((w - 16 * high - 8) * scale).T + x[:, 1::2] @ ((high - 8) * scale).T))
    return torch.cat(y, 1) * st["s"].double()


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("qk", "attn"):
        streams = _streams(case)
        keys, rows = sum(k for _, _, k in streams), sum(r for r, _, _ in streams)
        blocks = sum((k - 1) // BLOCK - (k - r) // BLOCK + 1 for r, _, k in streams)
        if op == "qk":
            kept = sum((k - r) % BLOCK for r, _, k in streams)          # read for the scale of their block
            return dict(bytes=rows * (2 * NQ + 3 * NKV) * D * 2 + (kept * D + blocks * 3) * NKV * 2,
                        flops=rows * (NQ + NKV) * D * 8)
        seen = sum(r * k - r * (r - 1) // 2 for r, _, k in streams)
        return dict(bytes=keys * NKV * D * 2 + sum(-(-k // BLOCK) for _, _, k in streams) * NKV * 2 + rows * NQ * D * 4,
                    flops=4 * D * NQ * seen)
    if op == "copy":
        keys = case["page"] if case["whole"] else (case["page"] + 1) / 2   # on average
        return dict(bytes=2 * case["copies"] * case["pools"] * NKV * keys * (D + 1 / BLOCK), flops=0)
    if op == "norm":
        n = case["rows"] * case["width"]
        return dict(bytes=n * (7 if case["residual"] else 3) + n // GROUP + 2 * case["width"], flops=6 * n)
    R, K, N = case["rows"], case["k"], case["n"]
    x = R * K + R * K // GROUP if case["x8"] else 2 * R * K
    return dict(bytes=N * K // 2 + N * K // GROUP + 4 * N + x + 2 * R * N, flops=2 * R * K * N)
