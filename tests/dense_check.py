"""Plain 64-bit forms of the dense cache operators (tree attention, accumulated weights,
eviction by them), the caches their tests run on, and the bounds they are held to.

Bounds, derived before the first run.  A rounding to bf16 is off by at most 2^-8 of the
value (half a step).  The softmax weights are rounded once before the product with V, and
the output once after it, so an output channel is off by at most
    2^-8 sum_t p_t |v_t| + 2^-8 |out| + fp32 terms.
fp32 terms: a logit is a sum of 128 products accumulated in fp32 (each partial sum off by
at most 2^-23 of the sum of magnitudes), so it is off by at most
    E = 128 2^-23 scale max_t sum_i |q_i k_t,i|,
a weight by a factor exp(E) each for itself and for the log-sum-exp, ex2.approx adds 2^-22
and the fp32 sums (their order is free) at most 2^-12 for 4096 terms, in practice far less;
E_w = 2 E + 2^-16 covers them for the sizes tested here.  An accumulated weight adds one
rounding of the sum, 2^-23 of its value."""
from __future__ import annotations

import math

import torch

from two_stage_kv_snapkv_gb300 import workloads as W

D = 128
SCALE = 1.0 / math.sqrt(D)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def make_cache(rkv, lens, Hkv, P, seed=0, room=0, max_pages=0, fill=float("nan"), sinks=True):
    """A cache of the given lengths on permuted pages, everything that is not a cached
    token's row filled with `fill`, its summaries rebuilt by the append.  Returns (cache,
    K, V): per sequence the bf16 rows [Hkv, n, 128] on the CPU."""
    g = gen(seed)
    B = len(lens)
    pages = max(max_pages, -(-(max(lens) + room) // P), 1)
    pages = (pages + 7) // 8 * 8
    pt = W.page_table(B, pages, seed, "cuda", spare=3)
    cache = rkv.PagedCache(B, Hkv, P, pages, "cuda", page_table=pt, num_phys_pages=B * pages + 3, fill=fill)
    K, V = [], []
    for b, n in enumerate(lens):
        k, v = randn(g, Hkv, n, D), randn(g, Hkv, n, D)
        if sinks and n > 2:
            k[:, :2] *= 3
        K.append(k)
        V.append(v)
        put_rows(cache, b, k, v)
    cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    cache.kmax.copy_(summaries(cache, K, True))
    cache.kmin.copy_(summaries(cache, K, False))
    return cache, K, V


def put_rows(cache, b, k, v):
    n, P = k.shape[1], cache.page_size
    at = torch.arange(n)
    phys = cache.page_table[b].cpu().long()[at // P]
    for pool, x in ((cache.k_pages, k), (cache.v_pages, v)):
        pool[phys.cuda(), :, (at % P).cuda()] = x.transpose(0, 1).cuda()


def summaries(cache, K, top, base=None):
    """kmax (or kmin) rebuilt from the rows; pages without tokens keep `base`."""
    out = (cache.kmax if top else cache.kmin).cpu().clone() if base is None else base.clone()
    P = cache.page_size
    for b, k in enumerate(K):
        for pg in range(-(-k.shape[1] // P)):
            x = k[:, pg * P:(pg + 1) * P].float()
            out[b, :, :, pg] = (x.amax(1) if top else x.amin(1)).to(torch.bfloat16)
    return out


def mask_words(sees):
    """[B, T, T] bool -> the bit words [B, T, ceil(T/32)] int32."""
    B, T, _ = sees.shape
    w = (T + 31) // 32
    bits = torch.zeros(B, T, w * 32, dtype=torch.int64)
    bits[..., :T] = sees
    words = (bits.view(B, T, w, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def ancestors(B, T, g):
    """A random tree: node t's parent is a node before it; a node sees itself and its
    ancestors."""
    sees = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            if t:
                par = int(torch.randint(0, t, (1,), generator=g))
                sees[b, t] = sees[b, par]
            sees[b, t, t] = True
    return sees


def attend(q, K, V, shown, scale=SCALE):
    """q [R, D], K, V [n, D], shown [R, n] -> out, lse, weights, E_w, all fp64."""
    q, K, V = q.double(), K.double(), V.double()
    if K.shape[0] == 0:
        R = q.shape[0]
        return torch.zeros(R, D).double(), torch.full((R,), -math.inf).double(), torch.zeros(R, 0).double(), 2.0 ** -16
    z = (q @ K.T) * scale
    z = z.masked_fill(~shown, -math.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.where(lse[:, None] == -math.inf, torch.zeros_like(z), torch.exp(z - lse[:, None]))
    E = 128 * 2.0 ** -23 * scale * float((q.abs() @ K.abs().T).max()) if q.shape[0] else 0.0
    return w @ V, lse, w, 2 * E + 2.0 ** -16


def check_out(got, ref, w, V, Ew, what=""):
    got = got.double()
    mag = w @ V.double().abs() if V.shape[0] else torch.zeros_like(ref)
    tol = (2.0 ** -8 * (1 + Ew) + Ew) * mag + 2.0 ** -8 * ref.abs() * (1 + Ew) + 1e-30
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} outputs off, worst {float(((got - ref).abs() - tol).max()):.3e}"


def check_lse(got, ref, Ew, what=""):
    got = got.double()
    empty = ref == -math.inf
    assert torch.equal(got == -math.inf, empty), f"{what}: empty rows"
    d = (got - ref)[~empty].abs()
    tol = Ew + 2.0 ** -22 * ref[~empty].abs()
    assert (d <= tol).all(), f"{what}: lse off by {float((d - tol).max()):.3e} too much"


def keep_set(acc, n, keep, recent):
    """The kept positions of one unit: the definition, on Python floats."""
    if n <= keep:
        return list(range(n))
    a = [math.inf if x != x else float(x) for x in acc[:n - recent].tolist()]
    nan_first = [0 if x == x else -1 for x in acc[:n - recent].tolist()]
    order = sorted(range(n - recent), key=lambda t: (nan_first[t], -a[t], t))
    return sorted(order[:keep - recent]) + list(range(n - recent, n))
