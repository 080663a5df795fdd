"""The paged-cache serving operators on real work: what is measured, and their
plain forms.

Four operators that follow one another in a round over a paged cache: the
queries' and keys' norm and rotation with the append (``tf_qk_rows``), the
attention of the round's windows over the pages (``tf_attn_paged``), the copies
of pages behind a fork or a compaction (``tf_pages_copy``), and the sampling of
the next tokens (``tf_sample_rows``). With ``own`` false ``run`` computes them
with elementary torch operations in 32 bits (angles, sampling masses and their
sums in 64); with ``own`` true it makes the library's calls.

Widths are the library's: 32 query heads, 8 KV heads, 64 dimensions a head.
"""

import math
import random

import numpy as np
import torch

own = False

NQ, NKV, D = 32, 8, 64
THETA, EPS = 1000000.0, 1e-5
BF16 = torch.bfloat16


def listed():
    return [
        # one decode layer of a plain round: 16 streams of one row each, dense caches
        dict(name="qk 16x1 dense", op="qk", streams=16, rows=1, keys_lo=256, keys_hi=4096, page=0, shared=0, kseed=2),
        # a verify layer of 64 drafted windows behind one shared prompt, in pages
        dict(name="qk 64x16 pages", op="qk", streams=64, rows=16, keys_lo=8300, keys_hi=8700, page=64, shared=8192,
             kseed=5),
        # a long prompt's chunk, its positions up to 131,000
        dict(name="qk prompt 16381", op="qk", prompt=True, streams=1, rows=16381, keys_lo=131001, keys_hi=131001,
             page=32, shared=0, kseed=7),
        # decode attention of a plain round over small pages
        dict(name="attn 16x1 p16", op="attn", streams=16, rows=1, keys_lo=256, keys_hi=4096, page=16, kseed=2),
        # drafted windows of 64 streams
        dict(name="attn 64x16 p64", op="attn", streams=64, rows=16, keys_lo=16, keys_hi=32768, page=64, kseed=5),
        # long contexts, six-row windows
        dict(name="attn 4x6 long p32", op="attn", streams=4, rows=6, keys_lo=65536, keys_hi=130816, page=32, kseed=4),
        # a chunk of a prompt behind its cached part
        dict(name="attn prompt 2048 p128", op="attn", prompt=True, streams=1, rows=2048, keys_lo=8179, keys_hi=8179,
             page=128, kseed=9),
        # copy-on-write of 64 forks' partly filled last pages, ten attention layers
        dict(name="copy fork 64 p16", op="copy", pools=20, n_pages=1024, page=16, copies=64, whole=False, kseed=3),
        # compaction of a pool: a thousand whole pages of four layers
        dict(name="copy compact 1000 p64", op="copy", pools=8, n_pages=2048, page=64, copies=1000, whole=True,
             kseed=4),
        # a plain round's sampled rows, settings of their own a row
        dict(name="sample 16 mixed", op="sample", rows=16, vocab=128000, stride=128000, kind="mixed", masked=0.0),
        # every row of 64 drafted windows, temperature alone: the whole vocabulary counts
        dict(name="sample 1024 plain", op="sample", rows=1024, vocab=128000, stride=128000, kind="plain", masked=0.0),
        # the same rows with top-k, top-p and min-p; a quarter of the rows under a grammar's mask
        dict(name="sample 1021 mixed", op="sample", rows=1021, vocab=127997, stride=128000, kind="mixed", masked=0.9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "attn", "copy", "sample"])
    kseed = rng.randrange(1 << 20)
    if op == "qk":
        if rng.random() < 0.3:
            rows = _log_int(rng, 17, 16000)
            keys = rows + _log_int(rng, 1, 110000)
            return dict(op="qk", prompt=True, streams=1, rows=rows, keys_lo=keys, keys_hi=keys,
                        page=rng.choice([16, 32, 64, 128, 256]), shared=0, kseed=kseed)
        shared = rng.choice([0, 256 * rng.randint(1, 100)])
        lo = shared + rng.randint(16, 300)
        return dict(op="qk", streams=_log_int(rng, 1, 64), rows=rng.randint(1, 16), keys_lo=lo,
                    keys_hi=lo + rng.randint(1, 900), page=rng.choice([16, 32, 64, 128, 256] if shared else [0, 16, 64]),
                    shared=shared, kseed=kseed)
    if op == "attn":
        if rng.random() < 0.3:
            rows = _log_int(rng, 17, 2000)
            keys = rows + _log_int(rng, 1, 6000)
            return dict(op="attn", prompt=True, streams=1, rows=rows, keys_lo=keys, keys_hi=keys,
                        page=rng.choice([16, 32, 64, 128, 256]), kseed=kseed)
        hi = _log_int(rng, 64, 16000)
        return dict(op="attn", streams=_log_int(rng, 1, 48), rows=rng.randint(1, 16), keys_lo=16, keys_hi=hi,
                    page=rng.choice([16, 32, 64, 128, 256]), kseed=kseed)
    if op == "copy":
        page = rng.choice([16, 32, 64, 128, 256])
        n_pages = _log_int(rng, 64, 16384 // page * 8)
        return dict(op="copy", pools=rng.randint(1, 8), n_pages=n_pages, page=page,
                    copies=_log_int(rng, 1, n_pages // 2), whole=rng.random() < 0.5, kseed=kseed)
    vocab = rng.choice([rng.randint(1000, 128000), 128000, 65536])
    return dict(op="sample", rows=_log_int(rng, 1, 900), vocab=vocab, stride=vocab + rng.choice([0, 3, -vocab % 8]),
                kind=rng.choice(["plain", "mixed"]), masked=rng.choice([0.0, 0.5, 0.9]), kseed=kseed)


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
    """Each stream's pages in a scattered pool (the shared prefix's pages come
    first in every list) and the pool's size."""
    P, shared = case["page"], case.get("shared", 0) // case["page"]
    need = [-(-k // P) - shared for _, _, k in streams]
    n_pages = (shared + sum(need)) * 9 // 8 + 1
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    lists, at = [], shared
    for n in need:
        lists.append(np.concatenate([ids[:shared], ids[at:at + n]]))
        at += n
    return lists, n_pages


def _copy_lists(case, seed):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(case["n_pages"]).astype(np.int32)
    n = case["copies"]
    keys = None if case["whole"] else rng.integers(1, case["page"] + 1, n).astype(np.int32)
    return np.ascontiguousarray(ids[:n]), np.ascontiguousarray(ids[n:2 * n]), keys


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)

    op = case["op"]
    st = dict(case=case)
    if op in ("qk", "attn"):
        streams = _streams(case)
        S, R, P = len(streams), sum(r for r, _, _ in streams), case["page"]
        prompt = case.get("prompt", False)
        pos = np.concatenate([np.arange(k - r, k) for r, _, k in streams])
        who = np.concatenate([np.full(r, s) for s, (r, _, _) in enumerate(streams)])
        if P:
            lists, n_pages = _page_lists(case, streams, seed)
            K, V = normal(n_pages, NKV, P, D), normal(n_pages, NKV, P, D)
            page = np.array([lists[s][p // P] for s, p in zip(who, pos)])
            at = (torch.from_numpy(page.astype(np.int64)).cuda(), torch.from_numpy(pos % P).cuda())
            st["pages"] = [torch.from_numpy(x.astype(np.int64)).cuda() for x in lists]
        else:
            cap = -(-max(k for _, _, k in streams) // 64) * 64
            K, V = normal(S, NKV, cap, D), normal(S, NKV, cap, D)
            at = (torch.from_numpy(who).cuda(), torch.from_numpy(pos).cuda())
        st.update(streams=streams, K=K, V=V, at=at, pos=torch.from_numpy(pos).cuda(), q=normal(R, NQ, D))
        if op == "qk":
            st.update(k=normal(R, NKV, D), v=normal(R, NKV, D), qw=1 + normal(D, std=0.25), kw=1 + normal(D, std=0.25))
        if own:
            from stream_speculative_decode_gb300 import tf
            table = [(r, o, k, -(-k // P) * P if P else K.shape[2]) for r, o, k in streams]
            if not P:
                step = K[0].numel() * 2
                st["seg"] = tf.tf_segments_build(table, None, None, [K.data_ptr() + s * step for s in range(S)],
                                                 [V.data_ptr() + s * step for s in range(S)], 0, 1)
            elif prompt:
                r, _, k, cap = table[0]
                st["seg"] = tf.tf_paged_prompt_build(r, k, cap, None, lists[0], P, n_pages, [K], [V], 0, 1)
            else:
                st["seg"] = tf.tf_paged_build(table, None, None, np.concatenate(lists), P, n_pages, [K], [V], 0, 1)
            st["out"] = torch.empty((R, NQ, D), dtype=BF16, device="cuda")
            if op == "attn":
                st["partials"] = torch.empty(max(16, st["seg"].partials_bytes), dtype=torch.uint8, device="cuda")
    elif op == "copy":
        src, dst, keys = _copy_lists(case, seed)
        st.update(pools=[normal(case["n_pages"], NKV, case["page"], D) for _ in range(case["pools"])],
                  src=src, dst=dst, keys=keys, src_dev=torch.from_numpy(src).cuda().long(),
                  dst_dev=torch.from_numpy(dst).cuda().long(),
                  keep=None if keys is None else (torch.arange(case["page"], device="cuda")[None]
                                                  < torch.from_numpy(keys).cuda()[:, None])[:, None, :, None])
    else:
        R, V, stride = case["rows"], case["vocab"], case["stride"]
        buf = normal(R, stride, std=3.0).clamp_(-19, 19)
        rng = np.random.default_rng(seed)
        if case["masked"]:
            under = torch.from_numpy(rng.random(R) < 0.25).cuda()[:, None]
            buf[under & (torch.rand((R, stride), generator=g, device="cuda") < case["masked"])] = -math.inf
        t = rng.uniform(0.5, 1.3, R).astype(np.float32)
        k, p, m = np.zeros(R, np.int32), np.ones(R, np.float32), np.zeros(R, np.float32)
        if case["kind"] == "mixed":
            t[rng.random(R) < 0.1] = 0
            k = np.where(rng.random(R) < 0.4, rng.integers(1, 200, R), 0).astype(np.int32)
            p = np.where(rng.random(R) < 0.6, rng.uniform(0.5, 0.99, R), 1).astype(np.float32)
            m = np.where(rng.random(R) < 0.3, rng.uniform(0.01, 0.2, R), 0).astype(np.float32)
        st.update(buf=buf, logits=buf[:, :V], u=torch.from_numpy(rng.random(R).astype(np.float32) * (1 - 2 ** -20)).cuda())
        st.update({n: torch.from_numpy(x).cuda() for n, x in (("t", t), ("k", k), ("p", p), ("m", m))})
        if case["kind"] == "plain":
            st.update(k=None, p=None, m=None)
        if own:
            st.update(pick=torch.empty(R, dtype=torch.int32, device="cuda"), prob=torch.empty(R, device="cuda"),
                      flag=torch.empty(R, dtype=torch.uint8, device="cuda"))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return {"qk": _qk, "attn": _attn, "copy": _copy, "sample": _sample}[case["op"]](st, case)


def _run_own(st, case):
    from stream_speculative_decode_gb300 import tf
    op = case["op"]
    if op == "qk":
        tf.tf_qk_rows(st["seg"], 0, st["q"], NQ * D, st["k"], NKV * D, st["v"], NKV * D, st["qw"], st["kw"], EPS, THETA,
                      st["out"])
        return dict(q=st["out"], K=st["K"], V=st["V"])
    if op == "attn":
        tf.tf_attn_paged(st["seg"], 0, st["q"], st["partials"], st["out"])
        return dict(out=st["out"])
    if op == "copy":
        tf.tf_pages_copy(st["pools"], case["page"], case["n_pages"], st["src"], st["dst"], st["keys"])
        return dict(pools=st["pools"])
    tf.tf_sample_rows(st["buf"], case["rows"], case["vocab"], case["stride"], st["t"], st["k"], st["p"], st["m"],
                      st["u"], st["pick"], st["prob"], st["flag"])
    return dict(pick=st["pick"], prob=st["prob"], flag=st["flag"])


def _qk(st, case):
    turn = st["pos"].double()[:, None] * THETA ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]

    def norm_rotate(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(BF16)

    i, j = st["at"]
    st["K"][i, :, j] = norm_rotate(st["k"], st["kw"])
    st["V"][i, :, j] = st["v"]
    return dict(q=norm_rotate(st["q"], st["qw"]), K=st["K"], V=st["V"])


def _attn(st, case):
    out = []
    for (rows, off, keys), pages in zip(st["streams"], st["pages"]):   # streams differ in length
        q = st["q"][off:off + rows].float().view(rows, NKV, NQ // NKV, D).permute(1, 2, 0, 3).reshape(NKV, -1, D)
        k = st["K"][pages].permute(1, 0, 2, 3).reshape(NKV, -1, D)[:, :keys].float()
        v = st["V"][pages].permute(1, 0, 2, 3).reshape(NKV, -1, D)[:, :keys].float()
        s = (q @ k.transpose(1, 2)).view(NKV, NQ // NKV, rows, keys) * (1 / math.sqrt(D))
        if rows > 1:
            row = torch.arange(rows, device="cuda")[:, None]
            s.masked_fill_(torch.arange(keys, device="cuda")[None] > keys - rows + row, -math.inf)
        s = torch.exp(s - s.amax(-1, keepdim=True))
        o = (s.view(NKV, -1, keys) @ v).view(NKV, NQ // NKV, rows, D) / s.sum(-1, keepdim=True)
        out.append(o.permute(2, 0, 1, 3).reshape(rows, NQ, D))
    return dict(out=torch.cat(out).to(BF16))


def _copy(st, case):
    src, dst, keep = st["src_dev"], st["dst_dev"], st["keep"]
    for pool in st["pools"]:
        pool[dst] = pool[src] if keep is None else torch.where(keep, pool[src], pool[dst])
    return dict(pools=st["pools"])


def _sample(st, case):
    x = st["logits"].float()
    bad = (torch.isnan(x) | (x == math.inf)).any(1)
    x, token = torch.sort(torch.where(bad[:, None], torch.zeros_like(x), x), dim=1, descending=True, stable=True)
    bad |= x[:, 0] == -math.inf
    greedy = st["t"] == 0
    w = torch.exp((x - x[:, :1].clamp(min=-1e38)).double() / torch.where(greedy, 1.0, st["t"]).double()[:, None])
    rank = torch.arange(case["vocab"], device="cuda")
    if st["k"] is not None:
        w = torch.where((rank < torch.where(st["k"] > 0, st["k"], case["vocab"])[:, None]), w, 0.0)
    mass = w.cumsum(1)
    kept = torch.full_like(st["u"], case["vocab"], dtype=torch.int64)
    if st["p"] is not None:
        kept = torch.where(st["p"] < 1, 1 + (mass < st["p"].double()[:, None] * mass[:, -1:]).sum(1), kept)
    if st["m"] is not None:
        kept = torch.where(st["m"] > 0, torch.minimum(kept, (w >= st["m"].double()[:, None]).sum(1)), kept)
    total = mass.gather(1, kept[:, None].clamp(min=1) - 1)
    at = torch.minimum((mass <= st["u"].double()[:, None] * total).sum(1), kept - 1).clamp(min=0)
    at = torch.where(greedy, 0, at)[:, None]
    prob = torch.where(greedy, 1.0, (w.gather(1, at) / total)[:, 0])
    return dict(pick=torch.where(bad, -1, token.gather(1, at)[:, 0]).int(), prob=torch.where(bad, 0.0, prob).float(),
                flag=bad.to(torch.uint8))


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(st)
    if case["op"] == "attn":
        return dict(out=_exact_attn(st, case["page"]))
    if case["op"] == "copy":
        pools = [p.double() for p in st["pools"]]
        for i in range(case["copies"]):
            n = case["page"] if st["keys"] is None else int(st["keys"][i])
            for p in pools:
                p[int(st["dst"][i]), :, :n] = p[int(st["src"][i]), :, :n]
        return dict(pools=pools)
    return _exact_sample(st, case)


def _exact_qk(st):
    freq = torch.tensor([THETA ** (-2 * j / D) for j in range(D // 2)], dtype=torch.float64, device="cuda")
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), st["pos"].double().outer(freq))

    def rotated(x, w):
        x = x.double()
        y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + EPS) * w.double()
        y = torch.complex(y[..., :D // 2], y[..., D // 2:]) * z[:, None]
        return torch.cat([y.real, y.imag], -1)

    K, V = st["K"].double(), st["V"].double()
    heads = torch.arange(NKV, device="cuda")
    i, j = (a[:, None] for a in st["at"])
    K[i, heads[None], j] = rotated(st["k"], st["kw"])
    V[i, heads[None], j] = st["v"].double()
    return dict(q=rotated(st["q"], st["qw"]), K=K, V=V)


def _exact_attn(st, P):
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for (rows, off, keys), pages in zip(st["streams"], st["pages"]):
        t = torch.arange(keys, device="cuda")
        sees = t[None] < (keys - rows + 1 + torch.arange(rows, device="cuda"))[:, None]
        for g in range(NKV):
            k, v = (c[pages[t // P], g, t % P].double() for c in (st["K"], st["V"]))
            for h in range(g * 4, g * 4 + 4):
                s = st["q"][off:off + rows, h].double() @ k.T / 8
                p = torch.softmax(torch.where(sees, s, -math.inf), 1)
                out[off:off + rows, h] = p @ v
    return out


def _exact_sample(st, case):
    """Row by row on the host: the tokens in order of their logits' bits."""
    bits = st["logits"].contiguous().view(torch.int16).cpu().numpy()
    par = {n: None if st[n] is None else st[n].cpu().numpy().astype(np.float64) for n in "tkpmu"}
    R = case["rows"]
    pick, prob, flag = np.full(R, -1, np.int32), np.zeros(R), np.zeros(R, np.uint8)
    for r in range(R):
        b = np.where(bits[r] == -32768, 0, bits[r])            # -0 is +0
        low = np.where(b >= 0, ~b, b & 0x7FFF).astype(np.int16)    # ascending as the logits descend
        value = (b.astype(np.int32) << 16).view(np.float32).astype(np.float64)
        if np.isnan(value).any() or value.max() == np.inf or value.max() == -np.inf:
            flag[r] = 1
            continue
        if par["t"][r] == 0:
            pick[r], prob[r] = int(value.argmax()), 1.0
            continue
        order = np.argsort(low, kind="stable")
        k = int(par["k"][r]) if par["k"] is not None else 0
        order = order[:k] if 0 < k else order
        w = np.exp((value[order] - value.max()) / par["t"][r])
        mass = np.cumsum(w)
        n = len(order)
        if par["p"] is not None and par["p"][r] < 1:
            n = int(np.searchsorted(mass, par["p"][r] * mass[-1])) + 1
        if par["m"] is not None and par["m"][r] > 0:
            n = min(n, int((w >= par["m"][r]).sum()))
        at = min(int(np.searchsorted(mass[:n], par["u"][r] * mass[n - 1], side="right")), n - 1)
        pick[r], prob[r] = order[at], w[at] / mass[n - 1]
    return dict(pick=pick, prob=prob, flag=flag)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "qk":
        rows = case["streams"] * case["rows"]
        return dict(bytes=2 * rows * (NQ + 2 * NKV) * D * 2, flops=rows * (NQ + NKV) * D * 8)
    if op == "attn":
        streams = _streams(case)
        keys, rows = sum(k for _, _, k in streams), sum(r for r, _, _ in streams)
        seen = sum(r * k - r * (r - 1) // 2 for r, _, k in streams)
        return dict(bytes=keys * NKV * D * 4 + rows * NQ * D * 4, flops=4 * D * NQ * seen)
    if op == "copy":
        if case["whole"]:
            keys = case["page"] * case["copies"]
        else:
            keys = case["copies"] * (case["page"] + 1) // 2   # on average
        return dict(bytes=2 * keys * NKV * D * 2 * case["pools"], flops=0)
    return dict(bytes=case["rows"] * case["vocab"] * 2, flops=case["rows"] * case["vocab"] * 2)
