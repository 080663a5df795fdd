"""Scaled values (e4m3 codes under shared powers of two) and scaled pools, for the
tests: coding in plain torch, pools from float caches, and attention over them in
float64 with the error that the kernels' arithmetic allows.

The coding is independent of the library's: the exponent comes from frexp, the
codes from torch's own e4m3 conversion.
"""

import numpy as np
import torch

NQ, NKV, D, BLOCK, GROUP = 32, 8, 64, 16, 32
E4M3 = torch.float8_e4m3fn


def exponent(x, dim):
    """The smallest e >= -127 with the largest finite magnitude at most 464 * 2^e."""
    a = torch.where(torch.isfinite(x), x.double().abs(), 0.0)
    a = a.amax(dim, keepdim=True)
    m, p = torch.frexp(a)                       # a = m * 2^p, 464 = 0.90625 * 2^9
    return torch.where(a > 0, p - 9 + (m > 0.90625).to(p.dtype), -127).clamp(min=-127)


def code(x, e):
    """Codes (uint8) of x under 2^e; what is not finite becomes NaN."""
    y = torch.ldexp(torch.where(torch.isfinite(x), x.double(), 0.0), -e).float().to(E4M3)
    return torch.where(torch.isfinite(x), y.view(torch.uint8), 0x7F)


def value(codes, scales):
    """float64 values of codes under broadcast scale bytes."""
    return torch.ldexp(codes.contiguous().view(E4M3).double(), scales.int() - 127)


def code_blocks(x):
    """Codes and scale bytes of caches or pools [..., keys, D], keys a multiple of BLOCK."""
    y = x.reshape(*x.shape[:-2], x.shape[-2] // BLOCK, BLOCK * D)
    e = exponent(y, -1)
    return code(y, e).view(x.shape), (e[..., 0] + 127).to(torch.uint8)


def page_lists(keys, page, seed, spare=3):
    need = [-(-k // page) for k in keys]
    n_pages = sum(need) + spare
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    ends = np.cumsum(need)
    return [ids[e - n:e] for n, e in zip(need, ends)], n_pages


class ScaledAttn:
    """Streams [(rows, keys)] over scaled pools of random codes: table and buffers.
    Slots past a stream's keys and spare pages hold NaN codes and wild scales."""

    def __init__(self, tf, streams, page, seed=0, layers=1, prompt=False, spread=2.0, std=1.0, lists=None, n_pages=None):
        self.tf, self.page, self.layers, self.prompt = tf, page, layers, prompt
        g = torch.Generator(device="cuda").manual_seed(seed)
        keys = [k for _, k in streams]
        if lists is None:
            lists, n_pages = page_lists(keys, page, seed)
        self.lists, self.n_pages = lists, n_pages
        offs = np.cumsum([0] + [r for r, _ in streams])
        self.streams = [(r, int(o), k) for (r, k), o in zip(streams, offs)]
        self.R = int(offs[-1])
        self.K, self.V, self.ks, self.vs = [], [], [], []
        for _ in range(layers):
            for codes, scales in ((self.K, self.ks), (self.V, self.vs)):
                x = torch.randn((n_pages, NKV, page // BLOCK, BLOCK * D), generator=g, device="cuda") * std
                x *= torch.exp2((torch.rand((n_pages, NKV, page // BLOCK, 1), generator=g, device="cuda") - 0.5) * spread)
                c, s = code_blocks(x.view(n_pages, NKV, page, D))
                used = torch.zeros((n_pages, page), dtype=torch.bool, device="cuda")
                for ids, k in zip(lists, keys):
                    for i, p in enumerate(ids):
                        used[int(p), :max(0, min(page, k - i * page))] = True
                junk = torch.where(torch.rand(c.shape, generator=g, device="cuda") < 0.5, 0x7F, 0xFF).to(torch.uint8)
                c = torch.where(used[:, None, :, None], c, junk)
                s = torch.where(used[:, ::BLOCK][:, None], s, 0xFE)
                codes.append(c.contiguous())
                scales.append(s.contiguous())
        self.q = [torch.randn((self.R, NQ, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(layers)]
        self.build()
        self.out = [torch.full((self.R, NQ, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                    for _ in range(layers)]

    def build(self):
        tf, page = self.tf, self.page
        table = [(r, o, k, len(ids) * page) for (r, o, k), ids in zip(self.streams, self.lists)]
        pools = (self.K, self.V, self.ks, self.vs)
        if self.prompt:
            r, _, k, cap = table[0]
            self.seg = tf.tf_paged_scaled_prompt_build(r, k, cap, None, self.lists[0], page, self.n_pages, *pools, 0,
                                                       self.layers)
        else:
            self.seg = tf.tf_paged_scaled_build(table, None, None, np.concatenate(self.lists), page, self.n_pages,
                                                *pools, 0, self.layers)
        self.partials = torch.full((max(self.seg.partials_bytes // 4, 4),), float("nan"), device="cuda")

    def run(self, full=False, stream=None):
        for l in range(self.layers):
            self.tf.tf_attn_paged(self.seg, l, self.q[l], self.partials, self.out[l], full, stream)
        return self.out

    def cache(self, pool, scales, ids, keys):
        """Values, scale bytes a key, [NKV][keys][D] and [NKV][keys], of a stream."""
        ids = torch.as_tensor(np.asarray(ids).astype(np.int64), device="cuda")
        c = pool[ids].permute(1, 0, 2, 3).reshape(NKV, -1, D)[:, :keys]
        s = scales[ids].permute(1, 0, 2).reshape(NKV, -1).repeat_interleave(BLOCK, 1)[:, :keys]
        return value(c, s[..., None]), s

    def check(self, full=False, what="", rows_of=None):
        for l in range(self.layers):
            for (r, o, k), ids in zip(self.streams, self.lists):
                kv, _ = self.cache(self.K[l], self.ks[l], ids, k)
                vv, vs = self.cache(self.V[l], self.vs[l], ids, k)
                check_attention(self.q[l][o:o + r], kv, vv, vs, k, self.out[l][o:o + r], full, (what, l, r, k))


def check_attention(q, k, v, vs, keys, out, full=False, what=""):
    """A stream's outputs [rows][NQ][D] against float64, each within what the kernel's
    arithmetic allows. With p the softmax weights and A = sum p |v|:
      scores    a sum of 64 exact products in fp32 (a rounding of up to 2^-23 of the
                partial sums, which are at most S = sum |q k| / 8, each time), three
                factors, log2 units: off by e = 70 * 2^-23 * S * log2(e); a weight by
                e * ln 2 + 2^-21 (ex2 and its argument's rounding, 2^-23 |x|). Wide windows
                split a query into two e4m3 parts, which hold 8 bits down to 2^-9 of its
                largest: an element below 2^-8 of it is off by at most 2^-17 of the largest
      weights   fp16: 2^-11 of each, or 2^-31 of the chunk's largest weight where that
                is more, times a value of up to 448 of the chunk's largest V scale
      sums      P.V over n keys: (n / 64 + 64) roundings of 2^-23 of A, and as many
                for the sum of the weights; merging a few more
      store     bf16: 2^-8 of the value.
    """
    rows = q.shape[0]
    t = torch.arange(keys, device="cuda")
    sees = t[None] < (keys if full else keys - rows + 1 + torch.arange(rows, device="cuda"))[:, None] \
        if not full else torch.ones((rows, keys), dtype=torch.bool, device="cuda")
    qd = q.double().view(rows, NKV, NQ // NKV, D)
    for g in range(NKV):
        s = torch.einsum("rhd,kd->rhk", qd[:, g], k[g]) / 8
        size = torch.einsum("rhd,kd->rhk", qd[:, g].abs(), k[g].abs()) / 8
        s = torch.where(sees[:, None], s, -torch.inf)
        p = torch.softmax(s, -1)
        ref, A = p @ v[g], p @ v[g].abs()
        most = qd[:, g].abs().amax(-1, keepdim=True)
        low = torch.where(qd[:, g].abs() < 2.0 ** -8 * most, 2.0 ** -17 * most, 0.0)
        size = size + torch.einsum("rhd,kd->rhk", low, k[g].abs()) / 8 / (70 * 2.0 ** -23)
        top = p.amax(-1) * 2.0 ** (int(vs[g].max()) - 127)
        x = torch.where(sees[:, None], s - s.amax(-1, keepdim=True), 0.0).abs().clamp(max=40).amax(-1)
        e = 70 * 2.0 ** -23 * torch.where(sees[:, None], size, 0.0).amax(-1) + 2.0 ** -21 + 2.0 ** -22 * x
        bound = (2 * e + 2.0 ** -11 + 2 * (keys / 64 + 64) * 2.0 ** -23)[..., None] * A \
            + (keys * 2.0 ** -31 * 448 * top)[..., None]
        bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        got = out.view(rows, NKV, NQ // NKV, D)[:, g].double()
        err = (got - ref).abs()
        bad = ~(err <= bound)
        assert not bad.any(), (what, g, float(err[bad].max()), float((err / bound)[bad].max()),
                               torch.nonzero(bad)[:4].tolist())
