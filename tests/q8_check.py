"""Plain forms of the 8-bit cache's operators and the caches their tests run on.

Codes and scales are compared exactly: a scale is a power of two and a value divided by it is
rounded once, so that there is nothing to allow for.

Attention's bounds, derived before the first run.  The output is rounded once to bf16, off by
at most 2^-8 of it.  A weight enters the product with V as fp16, off by at most 2^-11 of it
or, below fp16's normal numbers, by half its smallest step, 2^-25, in units of 2^-7 of the
largest V scale vmax: 2^-32 vmax for weights relative to a row's maximum, whose sum is at
least 1, times a code of at most 448.  Logits are sums of 128 exact products in fp32
and two fp32 multiplications,
    E = 132 2^-23 scale max_t sum_i |q_i k_t,i|,
a weight is off by a factor exp(E) for itself and for the sum, ex2.approx adds 2^-22 and the
fp32 sums (64 partial ones of n / 64 terms, then theirs) n 2^-30 and 2^-18: E_w = 2 E + 2^-16
+ n 2^-30.  So
    |out - ref| <= (2^-11 + E_w) sum_t p_t |v_t| + 2^-8 (1 + E_w) |ref| + n 2^-32 448 vmax."""
from __future__ import annotations

import math

import torch

from two_stage_kv_snapkv_gb300 import workloads as W

D = 128
SCALE = 1.0 / math.sqrt(D)
LARGEST = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def scale_of(x, fmt):
    """x: a block's new values.  NaN when one is not finite."""
    if not torch.isfinite(x).all():
        return math.nan
    top = float(x.double().abs().max()) / LARGEST[fmt] if x.numel() else 0.0
    if top == 0.0:
        return 2.0 ** -126
    m, e = math.frexp(top)
    return max(2.0 ** (e - 1 if m == 0.5 else e), 2.0 ** -126)


def codes_of(x, s, fmt):
    """The codes (as fp64 values) of x / s: nearest, ties to even."""
    y = x.double() / s
    if fmt == "int8":
        return torch.round(y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def write_block(old, was, new, fmt):
    """A block of `old` codes (fp64 [h, D]) with scale `was` takes the new rows (bf16 [m, D]):
    (codes [h + m, D], scale); the codes of a NaN scale mean nothing."""
    s = scale_of(new, fmt)
    if old.shape[0]:
        if was != was or s != s:
            s = math.nan
        else:
            s = max(s, was)
            old = codes_of(old * was, s, fmt) if s > was else old
    if s != s:
        return torch.zeros(old.shape[0] + new.shape[0], D, dtype=torch.float64), s
    return torch.cat([old, codes_of(new, s, fmt)]), s


class Model:
    """The cache's contents, sequence after sequence: blocks[b][g] = list of (K codes, K scale,
    V codes, V scale)."""

    def __init__(self, B, Hkv, P, fmt):
        self.B, self.H, self.P, self.fmt = B, Hkv, P, fmt
        self.n = [0] * B
        self.blocks = [[[] for _ in range(Hkv)] for _ in range(B)]

    def append(self, b, k, v):  # [Hkv, m, D] bf16
        m = k.shape[1]
        for g in range(self.H):
            at, n = 0, self.n[b]
            while at < m:
                room = self.P - n % self.P
                kk, vv = k[g, at:at + room], v[g, at:at + room]
                if n % self.P:
                    ko, ks, vo, vs = self.blocks[b][g].pop()
                else:
                    ko = vo = torch.zeros(0, D, dtype=torch.float64)
                    ks = vs = 0.0
                k1, ks = write_block(ko, ks, kk, self.fmt)
                v1, vs = write_block(vo, vs, vv, self.fmt)
                if ks != ks or vs != vs:
                    ks = vs = math.nan
                self.blocks[b][g].append((k1, ks, v1, vs))
                n += kk.shape[0]
                at += kk.shape[0]
        self.n[b] += m

    def check(self, cache, what=""):
        assert cache.seq_len.cpu().tolist() == self.n, what
        kc, vc = cache.k_codes.float().double().cpu(), cache.v_codes.float().double().cpu()
        ks, vs = cache.k_scale.double().cpu(), cache.v_scale.double().cpu()
        pt = cache.page_table.cpu()
        for b in range(self.B):
            for g in range(self.H):
                for j, (k1, s1, v1, s2) in enumerate(self.blocks[b][g]):
                    ph = int(pt[b, j])
                    for got, s, c, ref, want in ((kc, ks, "K", k1, s1), (vc, vs, "V", v1, s2)):
                        where = f"{what} {c} sequence {b} head {g} page {j}"
                        if want != want:
                            assert math.isnan(float(s[ph, g])), where
                            continue
                        assert float(s[ph, g]) == want, (where, float(s[ph, g]), want)
                        assert torch.equal(got[ph, g, :ref.shape[0]], ref), where


def cache8(rkv, B, Hkv, P, pages, fmt, seed=0, junk=True):
    """An empty cache on permuted pages; everything in it is junk: NaN codes (e4m3) and scales,
    page ids far out of range behind what a sequence may use."""
    pages = (pages + 7) // 8 * 8
    pt = W.page_table(B, pages, seed, "cuda", spare=3)
    cache = rkv.PagedCache8(B, Hkv, P, pages, "cuda", page_table=pt, num_phys_pages=B * pages + 3, fmt=fmt)
    for t in (cache.k_codes, cache.v_codes):
        t.view(torch.uint8).fill_(0x7F if fmt == "e4m3" else 0x80)
    cache.k_scale.fill_(math.nan if junk else 1.0)
    cache.v_scale.fill_(math.nan if junk else 1.0)
    return cache


def filled(rkv, lens, Hkv, P, fmt, seed=0, room=0, spread=True):
    """A cache of the given lengths, written by torch from plain codes.  Returns (cache, K, V):
    per sequence the values [Hkv, n, D] fp64 on the GPU.  spread: pages' magnitudes differ."""
    B = len(lens)
    cache = cache8(rkv, B, Hkv, P, max(1, -(-(max(lens) + room) // P)), fmt, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 77)
    K, V = [], []
    for b, n in enumerate(lens):
        pages = -(-n // P)
        vals = []
        for codes, scale, base in ((cache.k_codes, cache.k_scale, 2.0 ** -7), (cache.v_codes, cache.v_scale, 2.0 ** -7)):
            x = torch.randn(pages, Hkv, P, D, generator=g, device="cuda")
            top = x.abs().amax((2, 3), keepdim=True)
            y = x * (LARGEST[fmt] / top).clamp(max=LARGEST[fmt])
            c = y.to(DTYPE[fmt]) if fmt == "e4m3" else y.round().to(torch.int8)
            e = torch.randint(-3, 3, (pages, Hkv), generator=g, device="cuda") if spread else torch.zeros(pages, Hkv, device="cuda")
            s = base * torch.exp2(e.float()) * (448.0 / LARGEST[fmt] if fmt == "e4m3" else 4.0)
            phys = cache.page_table[b, :pages].long()
            if pages:
                scale[phys] = s
                live = (torch.arange(pages * P, device="cuda") < n).view(pages, 1, P, 1)
                raw = codes.view(torch.uint8)
                raw[phys] = torch.where(live, c.view(torch.uint8), raw[phys])
            v = c.float().double() * s.double()[:, :, None, None]
            vals.append(v.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n])
        K.append(vals[0])
        V.append(vals[1])
    cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    return cache, K, V


def check_attention(cache, K, V, q, out, lse, rows, scale=SCALE, what="", sample=None):
    """Every row (or the sampled rows) of every sequence and head against the definition in fp64."""
    B, Hq, T, _ = q.shape
    G = Hq // cache.Hkv
    for b in range(B):
        n, m = K[b].shape[1], rows[b]
        vmax = float(V[b].abs().max()) if n else 0.0  # at least vmax's scale times 1
        unit = float(cache.v_scale[cache.page_table[b, :-(-n // cache.page_size)].long()].max()) if n else 0.0
        idx = torch.arange(m, device="cuda") if sample is None or m <= sample else torch.linspace(0, m - 1, sample, device="cuda").long()
        for h in range(Hq):
            k, v = K[b][h // G], V[b][h // G]
            qq = q[b, h, idx].double()
            where = f"{what} sequence {b} head {h}"
            got, gl = out[b, h, idx].double(), lse[b, h, idx].double() if lse is not None else None
            if m == 0:
                continue
            z = (qq @ k.T) * scale if n else torch.zeros(len(idx), 0, device="cuda").double()
            z = z.masked_fill(torch.arange(n, device="cuda")[None] > (n - m + idx)[:, None], -math.inf)
            ref_l = torch.logsumexp(z, 1) if n else torch.full((len(idx),), -math.inf, device="cuda").double()
            w = torch.where(ref_l[:, None] == -math.inf, torch.zeros_like(z), torch.exp(z - ref_l[:, None]))
            ref = w @ v
            E = 132 * 2.0 ** -23 * scale * float((qq.abs() @ k.abs().T).max()) if n else 0.0
            Ew = 2 * E + 2.0 ** -16 + n * 2.0 ** -30
            tol = (2.0 ** -11 + Ew) * (w @ v.abs()) + 2.0 ** -8 * (1 + Ew) * ref.abs() + n * 2.0 ** -32 * 448 * unit
            assert torch.isfinite(got).all(), f"{where}: not finite"
            bad = (got - ref).abs() > tol
            assert not bad.any(), f"{where}: {int(bad.sum())} outputs off, worst {float(((got - ref).abs() - tol).max()):.3e} of {vmax:.2f}"
            if gl is not None:
                empty = ref_l == -math.inf
                assert torch.equal(gl == -math.inf, empty), f"{where}: empty rows"
                d = (gl - ref_l)[~empty].abs()
                assert (d <= Ew + 2.0 ** -22 * ref_l[~empty].abs()).all(), f"{where}: lse off by {float(d.max()):.3e}"
