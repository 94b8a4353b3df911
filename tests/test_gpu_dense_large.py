"""The dense cache calls at the largest caches they take: 2^20 positions a sequence, lines of
more than 2^20 pieces, 2^20 query rows, and the eviction's limit.  A read-only cache maps its
pages onto a few physical ones, so that position t holds row t % 2048 and the 64-bit forms
stay small: a softmax over 2048 keys, each with the number of its positions."""
import math

import pytest
import torch

import dense_check as C
from dense_check import D, SCALE

pytestmark = pytest.mark.gpu

MOST = 1 << 20
BASE = 2048


@pytest.fixture(scope="module")
def rkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from two_stage_kv_snapkv_gb300 import build_lib
    build_lib.build()
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _status(rkv, cache):
    return rkv.rkv_get_device_status(cache)[1]


@pytest.fixture(scope="module")
def wide(rkv):
    """16 sequences of up to 2^20 positions with 8 KV heads over 32 pages."""
    B, Hkv, P = 16, 8, 64
    pages = MOST // P
    table = (torch.arange(pages, dtype=torch.int32, device="cuda") % (BASE // P)).repeat(B, 1).contiguous()
    cache = rkv.PagedCache(B, Hkv, P, pages, "cuda", page_table=table, num_phys_pages=BASE // P)
    g = C.gen(121)
    K, V = C.randn(g, Hkv, BASE, D), C.randn(g, Hkv, BASE, D)
    at = torch.arange(BASE)
    for pool, x in ((cache.k_pages, K), (cache.v_pages, V)):
        pool[(at // P).cuda(), :, (at % P).cuda()] = x.transpose(0, 1).cuda()
    lens = [MOST - 1 - 977 * b for b in range(B)]
    lens[0], lens[5], lens[9] = MOST, 1, 0
    cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    return cache, K, V, lens


def _counts(n):
    return torch.tensor([n // BASE + (j < n % BASE) for j in range(BASE)]).double()


def _attend(q, K, V, n, kt=None, vt=None, shown=None):
    """q [R, D] over the positions 0 .. n of the repeated rows and the nodes shown [R, T] ->
    (out, lse, weight of one position of each row [R, BASE], magnitude, E_w), fp64."""
    k, v, c = K.double(), V.double(), _counts(n)
    z = (q.double() @ k.T) * SCALE
    parts = [(z + c.log()[None], v)]
    if kt is not None:
        parts.append((((q.double() @ kt.double().T) * SCALE).masked_fill(~shown, -math.inf), vt.double()))
    every = torch.cat([x for x, _ in parts], 1)
    lse = torch.logsumexp(every, 1)
    w = torch.where(lse[:, None] == -math.inf, torch.zeros_like(every), torch.exp(every - lse[:, None]))
    vs = torch.cat([x for _, x in parts])
    E = 128 * 2.0 ** -23 * SCALE * float((q.double().abs() @ torch.cat([k] + ([kt.double()] if kt is not None else [])).abs().T).max())
    one = torch.where(lse[:, None] == -math.inf, torch.zeros_like(z), torch.exp(z - lse[:, None]))
    # fp32 sums: a warp adds its share's chunks one after the other, 2^20 / 16 of them at most
    # if all the line were one share; 152 shares of 8 warps hold fewer than 2^13 of a unit
    return w @ vs, lse, one, w, vs, 2 * E + 2.0 ** -16 + 2.0 ** 13 * 2.0 ** -24


@pytest.mark.parametrize("T,G", [(1, 1), (3, 4), (20, 4), (40, 4)])
def test_tree_attention_over_a_million_positions(rkv, wide, T, G):
    cache, K, V, lens = wide
    B, Hkv = cache.B, cache.Hkv
    g = C.gen(122)
    q, kt, vt = C.randn(g, B, Hkv * G, T, D), C.randn(g, B, Hkv, T, D), C.randn(g, B, Hkv, T, D)
    sees = C.ancestors(B, T, g)
    sees[9, 0] = False                                     # an empty cache and nothing to see
    out = torch.full((B, Hkv * G, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hkv * G, T), 7.0, device="cuda")
    rkv.rkv_tree_attention(cache, q.cuda(), kt.cuda(), vt.cuda(), C.mask_words(sees).cuda(), out, lse=lse)
    assert _status(rkv, cache) == 0
    out, lse = out.cpu(), lse.cpu()
    for b in (0, 1, 5, 9, 15):
        for h in range(0, Hkv * G, 3):
            ref, l, _, w, v, Ew = _attend(q[b, h], K[h // G], V[h // G], lens[b], kt[b, h // G], vt[b, h // G], sees[b])
            C.check_out(out[b, h], ref, w, v, Ew, f"b{b} h{h}")
            C.check_lse(lse[b, h], l, Ew, f"b{b} h{h}")


def test_decode_accum_over_a_million_positions(rkv, wide):
    cache, K, V, lens = wide
    B, Hkv = cache.B, cache.Hkv
    q = C.randn(C.gen(123), B, Hkv, D)
    out = torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device="cuda")
    lse, acc = torch.zeros(B, Hkv, device="cuda"), rkv.accum_sums(cache)
    rkv.rkv_decode_accum(cache, q.cuda(), out, acc, lse=lse)
    assert _status(rkv, cache) == 0
    for b in (0, 1, 5, 9, 15):
        n = lens[b]
        for h in range(Hkv):
            ref, l, one, w, v, Ew = _attend(q[b, h:h + 1], K[h], V[h], n)
            C.check_out(out[b, h:h + 1].cpu(), ref, w, v, Ew, f"b{b} h{h}")
            C.check_lse(lse[b, h:h + 1].cpu(), l, Ew, f"b{b} h{h}")
            want = one[0].cuda().repeat(MOST // BASE)[:n]
            got = acc[b, h].double()
            assert ((got[:n] - want).abs() <= want * (math.exp(Ew) - 1 + 2.0 ** -20)).all(), f"b{b} h{h}"
            assert (got[n:] == 0).all()


@pytest.mark.parametrize("T", [8, 300])
def test_accum_rows_over_a_million_positions(rkv, wide, T):
    cache, K, V, lens = wide
    B, Hkv = cache.B, cache.Hkv
    g = C.gen(124)
    q, lse = C.randn(g, B, Hkv, T, D), torch.rand(B, Hkv, T, generator=g) * 4 + 6
    m = [min(T, n) for n in lens]
    acc = rkv.accum_sums(cache)
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, row_len=_ints(m))
    assert _status(rkv, cache) == 0
    for b in (0, 1, 5, 9, 15):
        n = lens[b]
        for h in range(0, Hkv, 3):
            z = (q[b, h, :m[b]].double() @ K[h].double().T) * SCALE - lse[b, h, :m[b]].double()[:, None]
            w = z.exp().cuda()                             # [m, BASE]
            want = w.sum(0).repeat(MOST // BASE)[:n]       # what every row sees
            for t in range(max(n - m[b] + 1, 0), n):       # the last positions: rows t - (n - m) ..
                want[t] = w[t - (n - m[b]):, t % BASE].sum()
            E = 128 * 2.0 ** -23 * SCALE * float((q[b, h].double().abs() @ K[h].double().abs().T).max())
            got = acc[b, h].double()
            tol = want * (math.exp(E + 2.0 ** -22 * 30) - 1 + 2.0 ** -16)
            assert ((got[:n] - want).abs() <= tol).all(), f"b{b} h{h}"
            assert (got[n:] == 0).all()


def test_accum_rows_of_a_million_rows(rkv):
    # every row is the same: position t, seen by the rows from t on, has 2^20 - t equal weights
    P, n = 64, MOST
    table = (torch.arange(n // P, dtype=torch.int32, device="cuda") % (BASE // P)).view(1, -1).contiguous()
    cache = rkv.PagedCache(1, 1, P, n // P, "cuda", page_table=table, num_phys_pages=BASE // P)
    g = C.gen(125)
    K, one = C.randn(g, 1, BASE, D), C.randn(g, D)
    at = torch.arange(BASE)
    cache.k_pages[(at // P).cuda(), :, (at % P).cuda()] = K.transpose(0, 1).cuda()
    cache.v_pages.zero_()
    cache.seq_len.fill_(n)
    q = one.cuda().view(1, 1, 1, D).expand(1, 1, n, D).contiguous()
    lse = torch.full((1, 1, n), 14.0, device="cuda")
    acc = rkv.accum_sums(cache)
    rkv.rkv_accum_rows(cache, q, lse, acc)
    assert _status(rkv, cache) == 0
    w = torch.exp((K[0].double() @ one.double()) * SCALE - 14).cuda().repeat(n // BASE)
    want = w * (n - torch.arange(n, device="cuda")).double()
    E = 128 * 2.0 ** -23 * SCALE * float((K[0].double().abs() @ one.double().abs()).max())
    # a key's sum: 64 weights of a tile added in four chains of 16, then up to 8192 tiles one
    # after the other, each addition off by 2^-24
    tol = want * (math.exp(E + 2.0 ** -22 * 40) - 1 + (8192 + 64) * 2.0 ** -24)
    assert ((acc[0, 0].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_at_the_largest_cache(rkv, in_place):
    n, P, Hkv, keep, recent = 393216, 64, 2, 5000, 100
    cache = rkv.PagedCache(1, Hkv, P, n // P, "cuda")
    dev = torch.Generator(device="cuda").manual_seed(126)
    cache.k_pages.normal_(generator=dev)
    cache.v_pages.normal_(generator=dev)
    cache.seq_len.fill_(n)
    K, V = [x.clone() for x in cache.token_kv(0, n)]
    acc0 = torch.rand(1, Hkv, n, generator=C.gen(127))
    acc0[0, 1] = (acc0[0, 1] * 50).floor()                 # ties by the thousand
    acc = acc0.cuda()
    kept = torch.full((1, Hkv, keep), -7, dtype=torch.int32, device="cuda")
    to, sums = cache, acc
    if in_place:
        rkv.rkv_evict_accum(cache, acc, [keep], recent, kept)
    else:
        to = rkv.PagedCache(1, Hkv, P, 80, "cuda")
        sums = rkv.accum_sums(to)
        rkv.rkv_evict_accum(cache, acc, [keep], recent, kept, dst=to, dst_acc=sums)
    assert _status(rkv, cache) == 0 and to.seq_len.tolist() == [keep]
    gk, gv = to.token_kv(0, keep)
    for h in range(Hkv):
        want = C.keep_set(acc0[0, h], n, keep, recent)
        assert kept[0, h].tolist() == want
        at = torch.tensor(want, device="cuda")
        assert torch.equal(gk[h], K[h][at]) and torch.equal(gv[h], V[h][at])
        assert torch.equal(sums[0, h, :keep].cpu(), acc0[0, h][want]) and (sums[0, h, keep:] == 0).all()
