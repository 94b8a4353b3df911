"""The ends of what the dense cache calls accept: values that are not finite, scales at the
ends of their range, sequences that cannot be used, streams."""
import math

import pytest
import torch

import dense_check as C
from dense_check import D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from two_stage_kv_snapkv_gb300 import build_lib
    build_lib.build()
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def _status(rkv, cache):
    return rkv.rkv_get_device_status(cache)[1]


# ------------------------------------------------------------------ eviction: weights that are NaN
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n,nans,keep,recent,room", [
    (150, 143, 12, 0, 0), (1000, 100, 50, 4, 0), (1000, 999, 500, 0, 0), (300, 300, 20, 3, 0),
    (1000, 100, 50, 4, 20000), (3000, 2500, 700, 16, 20000), (9000, 8000, 4000, 0, 0)])
def test_evict_with_more_nan_weights_than_kept(rkv, n, nans, keep, recent, room, in_place):
    """One decoding step with a NaN leaves every sum of its KV head NaN; tokens appended later
    weigh something.  `room` above 8192 positions: a cluster selects instead of one CTA."""
    Hkv, P = 2, 16
    cache, K, V = C.make_cache(rkv, [n], Hkv, P, seed=81, room=room)
    g = C.gen(82)
    acc0 = torch.rand(1, Hkv, cache.max_pages * P, generator=g) + 2.0 ** -10    # no zero among them
    for h in range(Hkv):
        at = torch.randperm(n, generator=g)[:nans] if h else torch.arange(nans)
        acc0[0, h, at] = math.nan
    acc0[:, :, n:] = 0
    kept = torch.full((1, Hkv, keep + 1), -7, dtype=torch.int32, device="cuda")
    to, to_acc = None, None
    if not in_place:
        to, _, _ = C.make_cache(rkv, [0], Hkv, P, seed=83, room=keep)
        to_acc = rkv.accum_sums(to)
    acc = acc0.cuda()
    rkv.rkv_evict_accum(cache, acc, [keep], recent, kept, dst=to, dst_acc=to_acc)
    assert _status(rkv, cache) == 0
    got, sums = (cache, acc) if in_place else (to, to_acc)
    for h in range(Hkv):
        want = C.keep_set(acc0[0, h], n, keep, recent)
        assert kept[0, h].tolist() == want + [-7], f"g{h}"
        assert torch.equal(got.token_kv(0, keep)[0][h].cpu(), K[0][h][want])
        assert torch.equal(sums[0, h, :keep].cpu().view(torch.int32), acc0[0, h][want].view(torch.int32))


# ------------------------------------------------------------------ scales at the ends of their range
def _whole(g, *shape, sign):
    """Whole numbers: channels 1 .. 16 of -1, 0, 1 and one of 8 (its sign `sign`), so that
    every q . k is exact in fp32, lies in +-[48, 80] and often ties."""
    x = torch.zeros(*shape, D)
    x[..., 1:17] = torch.randint(-1, 2, (*shape, 16), generator=g).float()
    x[..., 0] = 8 * sign
    return x.to(torch.bfloat16)


def _attend_whole(q, K, V, shown, scale):
    """(out, lse, weights) in fp64.  The logits of different q . k differ by `scale` at least and
    equal ones are equal to the bit, so only the fp32 rounding of scale, log2(e) and their
    products enters, not the weights' ratios."""
    z = (q.double() @ K.double().T) * float(torch.tensor(scale))
    z = z.masked_fill(~shown, -math.inf)
    lse = torch.logsumexp(z, 1)
    top = z.max(1, keepdim=True).values.clamp_min(-1e300)
    w = torch.exp(z - top)
    w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return w @ V.double(), lse, w


def _check_whole(out, lse, ref, rlse, w, V, scale, what):
    # a logit's difference to the largest (at most 32 scale) is off by 2^-22 of the largest
    # logit (80 scale): below scale 1 / 16 that is a weight's error, from 60 on every weight is 0
    # or a tie.  Between them the test has no scale.  Then a rounding of the weights and one
    # of the output, 2^-8 each (dense_check).
    Ew = 2.0 ** -22 * 80 * scale + 2.0 ** -16 if scale < 1 else 2.0 ** -16
    C.check_out(out, ref, w, V, Ew, what)
    C.check_lse(lse, rlse, Ew, what)


SCALES = [1e-30, 1e-20, 1e-3, 1e3, 3e5, 1e7, 1e9, 1e20, 1e30]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("T,G,room", [(3, 4, 0), (3, 4, 40000), (20, 4, 40000), (70, 4, 40000)])
def test_tree_attention_over_the_range_of_scales(rkv, T, G, room, scale, sign):
    # clusters; 16-row tiles; 128 rows; 256 rows
    g = C.gen(91)
    lens, Hkv, P = [700, 0, 130], 1, 16
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=90, room=room)
    q, kt, vt = _whole(g, 3, Hkv * G, T, sign=1), _whole(g, 3, Hkv, T, sign=sign), C.randn(g, 3, Hkv, T, D)
    for b, n in enumerate(lens):
        K[b] = _whole(g, Hkv, n, sign=sign)
        C.put_rows(cache, b, K[b], V[b])
    sees = torch.rand(3, T, T, generator=g) < 0.5
    sees[:, 0] = False                                     # sequence 1's first node sees nothing
    out = torch.full((3, Hkv * G, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, Hkv * G, T), 7.0, device="cuda")
    rkv.rkv_tree_attention(cache, q.cuda(), kt.cuda(), vt.cuda(), C.mask_words(sees).cuda(), out, lse=lse, scale=scale)
    assert _status(rkv, cache) == 0
    for b, n in enumerate(lens):
        shown = torch.cat([torch.ones(T, n, dtype=torch.bool), sees[b]], 1)
        k, v = torch.cat([K[b][0], kt[b, 0]]), torch.cat([V[b][0], vt[b, 0]])
        for h in range(Hkv * G):
            ref, rlse, w = _attend_whole(q[b, h], k, v, shown, scale)
            _check_whole(out[b, h].cpu(), lse[b, h].cpu(), ref, rlse, w, v, scale, f"b{b} h{h}")


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("room", [0, 40000])
def test_decode_accum_over_the_range_of_scales(rkv, room, scale, sign):
    g = C.gen(93)
    lens, Hkv, G, P = [900, 1, 33], 2, 2, 16
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=92, room=room)
    for b, n in enumerate(lens):
        K[b] = _whole(g, Hkv, n, sign=sign)
        C.put_rows(cache, b, K[b], V[b])
    q = _whole(g, 3, Hkv * G, sign=1)
    out = torch.zeros(3, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    lse, acc = torch.zeros(3, Hkv * G, device="cuda"), rkv.accum_sums(cache)
    rkv.rkv_decode_accum(cache, q.cuda(), out, acc, lse=lse, scale=scale)
    assert _status(rkv, cache) == 0
    Ew = 2.0 ** -22 * 80 * scale + 2.0 ** -16 if scale < 1 else 2.0 ** -16
    for b, n in enumerate(lens):
        want = torch.zeros(Hkv, n).double()
        for h in range(Hkv * G):
            ref, rlse, w = _attend_whole(q[b, h:h + 1], K[b][h // G], V[b][h // G], torch.ones(1, n, dtype=torch.bool), scale)
            _check_whole(out[b, h:h + 1].cpu(), lse[b, h:h + 1].cpu(), ref, rlse, w, V[b][h // G], scale, f"b{b} h{h}")
            want[h // G] += w[0]
        got = acc[b, :, :n].cpu().double()
        assert ((got - want).abs() <= want * (math.exp(Ew) - 1 + 2.0 ** -20)).all(), f"b{b}"


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("T,G,room", [(3, 4, 0), (3, 4, 40000), (20, 4, 40000), (70, 4, 40000)])
def test_tree_attention_whose_maxima_lie_far_apart(rkv, T, G, room, late):
    """Rows of three kinds in every warp.  The first 256 keys have the logit -+2^40 scale or 0,
    the same for all of them; one key behind them, if `late`, +-2^42 scale or 0.  The rest is
    ordinary.  So a row's maximum stays far below or above the rest, or comes from far below
    to the rest and from there to far above."""
    n = 900
    cache, K, V = C.make_cache(rkv, [n], 1, 16, seed=107, room=room)
    g = C.gen(108)
    K[0][0, :, 0] = 0
    K[0][0, :256] = 0
    K[0][0, :256, 0] = -2.0 ** 40
    if late:
        K[0][0, 700] = 0
        K[0][0, 700, 0] = 2.0 ** 42
    C.put_rows(cache, 0, K[0], V[0])
    q, kt, vt = C.randn(g, 1, G, T, D), C.randn(g, 1, 1, T, D), C.randn(g, 1, 1, T, D)
    kt[..., 0] = 0
    kind = (torch.arange(G)[:, None] + torch.arange(T)[None]) % 3 - 1          # [G, T]: -1, 0, 1
    q[0, :, :, 0] = kind.to(torch.bfloat16)
    sees = C.ancestors(1, T, g)
    out = torch.full((1, G, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, G, T), 7.0, device="cuda")
    rkv.rkv_tree_attention(cache, q.cuda(), kt.cuda(), vt.cuda(), C.mask_words(sees).cuda(), out, lse=lse)
    assert _status(rkv, cache) == 0
    out, lse = out[0].cpu(), lse[0].cpu()
    k, v = torch.cat([K[0][0], kt[0, 0]]), torch.cat([V[0][0], vt[0, 0]])
    for h in range(G):
        for t in range(T):
            shown = torch.cat([torch.ones(n, dtype=torch.bool), sees[0, t]])
            if kind[h, t] < 0:                             # the first keys alone, all the same
                shown[256:] = False
            elif kind[h, t] > 0:                           # all but the first, or the late one alone
                shown[:256] = False
                if late:
                    shown[:] = False
                    shown[700] = True
            # the keys that count: their logits are exact where far, ordinary elsewhere
            at = torch.nonzero(shown)[:, 0]
            ref, l, w, Ew = C.attend(q[0, h, t:t + 1], k[at], v[at], torch.ones(1, len(at), dtype=torch.bool))
            if kind[h, t] < 0 or (kind[h, t] > 0 and late):
                Ew = 2.0 ** -16
            C.check_out(out[h, t:t + 1], ref, w, v[at], Ew, f"h{h} t{t}")
            C.check_lse(lse[h, t:t + 1], l, Ew, f"h{h} t{t}")


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("T,G,m", [(8, 4, [8, 3]), (40, 4, [40, 9]), (150, 1, [150, 60])])
def test_accum_rows_over_the_range_of_scales(rkv, T, G, m, scale):
    # 16-row blocks; tensor cores with 64 and with 128 rows a tile.  q . k is 0 in the even rows and in
    # [-80, -48] in the others, so that no weight overflows.
    g = C.gen(95)
    lens, Hkv, P = [400, 60], 2, 16
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=94)
    for b, n in enumerate(lens):
        K[b] = _whole(g, Hkv, n, sign=-1)
        C.put_rows(cache, b, K[b], V[b])
    q = _whole(g, 2, Hkv * G, T, sign=1)
    q[:, :, ::2] = 0
    lse = torch.rand(2, Hkv * G, T, generator=g) * 4 + 6
    lse[:, :, 1::5] = -math.inf                            # rows that saw nothing weigh nothing
    lse[:, 0, 2] = math.inf
    acc = rkv.accum_sums(cache)
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, scale=scale,
                       row_len=torch.tensor(m, dtype=torch.int32, device="cuda"))
    assert _status(rkv, cache) == 0
    # an exponent, of at most 80 scale + 10 before it is 0 all the same (from 120 on), is off by 2^-22
    # of it for each of its roundings (scale log2 e, the product, lse log2 e or its three terms)
    E = 4 * 2.0 ** -22 * min(80 * scale + 10, 130.0) + 2.0 ** -16
    for b, n in enumerate(lens):
        seen = torch.arange(n)[None] <= (n - m[b] + torch.arange(m[b]))[:, None]
        for h in range(Hkv):
            want = torch.zeros(n).double()
            for i in range(h * G, (h + 1) * G):
                z = (q[b, i, :m[b]].double() @ K[b][h].double().T) * float(torch.tensor(scale))
                l = lse[b, i, :m[b]].double()[:, None]
                want += torch.where(seen & (l != -math.inf), torch.exp(z - l), torch.zeros_like(z)).sum(0)
            got = acc[b, h, :n].cpu().double()
            assert ((got - want).abs() <= want * (math.exp(E) - 1) + 1e-37).all(), f"b{b} g{h}"


# ------------------------------------------------------------------ values that are not numbers
@pytest.mark.parametrize("T,G,room", [(3, 4, 0), (3, 4, 40000), (20, 4, 40000), (70, 4, 40000)])
def test_tree_attention_keeps_a_nan(rkv, T, G, room):
    # a query with a NaN: its row is NaN, the log-sum-exp too, and no other row is
    g = C.gen(97)
    cache, K, V = C.make_cache(rkv, [700, 90], 1, 16, seed=96, room=room)
    q, kt, vt = C.randn(g, 2, G, T, D), C.randn(g, 2, 1, T, D), C.randn(g, 2, 1, T, D)
    sees = C.ancestors(2, T, g)
    q[0, 1, T - 1, 77] = math.nan
    K[1][0, 40, 3] = math.nan                              # and a cached key: every row of its sequence
    C.put_rows(cache, 1, K[1], V[1])
    out = torch.full((2, G, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, G, T), 7.0, device="cuda")
    rkv.rkv_tree_attention(cache, q.cuda(), kt.cuda(), vt.cuda(), C.mask_words(sees).cuda(), out, lse=lse)
    assert _status(rkv, cache) == 0
    out, lse = out.cpu(), lse.cpu()
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert out[0, 1, T - 1].isnan().all() and lse[0, 1, T - 1].isnan()
    shown = torch.cat([torch.ones(T, 700, dtype=torch.bool), sees[0]], 1)
    k, v = torch.cat([K[0][0], kt[0, 0]]), torch.cat([V[0][0], vt[0, 0]])
    for h in range(G):
        rows = [t for t in range(T) if (h, t) != (1, T - 1)]
        ref, l, w, Ew = C.attend(q[0, h][rows], k, v, shown[rows])
        C.check_out(out[0, h][rows], ref, w, v, Ew, f"h{h}")
        C.check_lse(lse[0, h][rows], l, Ew, f"h{h}")


@pytest.mark.parametrize("room", [0, 40000])
def test_decode_accum_keeps_a_nan(rkv, room):
    g = C.gen(99)
    lens = [900, 65]
    cache, K, V = C.make_cache(rkv, lens, 2, 16, seed=98, room=room)
    K[0][1, 500, 9] = math.nan
    C.put_rows(cache, 0, K[0], V[0])
    q = C.randn(g, 2, 4, D)
    q[1, 3, 0] = math.nan
    out = torch.zeros(2, 4, D, dtype=torch.bfloat16, device="cuda")
    lse, acc = torch.zeros(2, 4, device="cuda"), rkv.accum_sums(cache)
    rkv.rkv_decode_accum(cache, q.cuda(), out, acc, lse=lse)
    assert _status(rkv, cache) == 0
    out, lse, acc = out.cpu(), lse.cpu(), acc.cpu()
    nan = torch.tensor([[False, False, True, True], [False, False, False, True]])
    assert torch.equal(lse.isnan(), nan) and torch.equal(out.isnan().all(-1), nan) and torch.equal(out.isnan().any(-1), nan)
    for b, n in enumerate(lens):
        assert acc[b, 1, :n].isnan().all() and (acc[b, :, n:] == 0).all()
        w = [C.attend(q[b, h:h + 1], K[b][0], V[b][0], torch.ones(1, n, dtype=torch.bool)) for h in range(2)]
        want, Ew = w[0][2][0] + w[1][2][0], max(w[0][3], w[1][3])
        assert ((acc[b, 0, :n].double() - want).abs() <= want * (math.exp(Ew) - 1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("T,G", [(8, 4), (40, 4), (150, 1)])
def test_accum_rows_keeps_a_nan(rkv, T, G):
    # a row whose log-sum-exp is NaN makes what it sees NaN, and nothing else
    g = C.gen(101)
    cache, K, V = C.make_cache(rkv, [300], 2, 16, seed=100)
    q, lse = C.randn(g, 1, 2 * G, T, D), torch.full((1, 2 * G, T), 7.0)
    lse[0, 0, T // 2] = math.nan
    acc = rkv.accum_sums(cache)
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc)
    assert _status(rkv, cache) == 0
    seen = 300 - T + T // 2 + 1
    assert acc[0, 0, :seen].isnan().all() and not acc[0, 0, seen:].isnan().any() and not acc[0, 1].isnan().any()


# ------------------------------------------------------------------ eviction: lengths that cannot be used
@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("bad", [-3, None])
def test_evict_in_place_leaves_a_sequence_of_unusable_length(rkv, bad, room):
    lens, P = [100, 90, 40], 16
    cache, K, V = C.make_cache(rkv, lens, 2, P, seed=103, room=room)
    acc0 = torch.rand(3, 2, cache.max_pages * P, generator=C.gen(104))
    acc, kept = acc0.cuda(), torch.full((3, 2, 30), -7, dtype=torch.int32, device="cuda")
    cache.seq_len[0] = cache.max_pages * P + 1 if bad is None else bad
    bits = lambda t: t.cpu().view(torch.int16)  # noqa: E731
    at = cache.page_table[0].long()
    before = [bits(t) for t in (cache.k_pages[at], cache.v_pages[at], cache.kmax[0], cache.kmin[0])]
    length = int(cache.seq_len[0])
    rkv.rkv_evict_accum(cache, acc, [30, 30, 30], 5, kept)
    assert _status(rkv, cache) == rkv.DEVERR_CAPACITY
    assert cache.seq_len.tolist() == [length, 30, 30]
    after = [bits(t) for t in (cache.k_pages[at], cache.v_pages[at], cache.kmax[0], cache.kmin[0])]
    assert all(torch.equal(x, y) for x, y in zip(before, after))
    assert torch.equal(acc[0].cpu(), acc0[0]) and (kept[0] == -7).all()
    for b in (1, 2):
        for h in range(2):
            want = C.keep_set(acc0[b, h], lens[b], 30, 5)
            assert kept[b, h].tolist() == want
            assert torch.equal(cache.token_kv(b, 30)[0][h].cpu(), K[b][h][want])


# ------------------------------------------------------------------ workspaces on another stream
def test_a_workspace_is_not_memory_that_the_current_stream_still_writes(rkv):
    """The reverse of a workspace handed out too early: what the current stream is still writing
    to has been freed on the host, and a call on another stream makes its workspace."""
    lens = [6000, 900]
    cache, K, V = C.make_cache(rkv, lens, 2, 16, seed=105, room=10000)
    q = C.randn(C.gen(106), 2, 8, D)
    qd = q.cuda()
    side = torch.cuda.Stream()
    acc, lse = rkv.accum_sums(cache), torch.zeros(2, 8, device="cuda")
    outs = [torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    size = rkv.accum_workspace(2, 8, 2, cache.max_pages, 16).numel()
    torch.cuda.synchronize()
    for o in outs:
        was = torch.empty(size, dtype=torch.uint8, device="cuda")
        for _ in range(60):
            was.fill_(255)
        del was
        rkv.rkv_decode_accum(cache, qd, o, acc, lse=lse, stream=side)
    torch.cuda.synchronize()
    assert _status(rkv, cache) == 0
    for o in outs:
        assert torch.equal(o, outs[0])
    for b, n in enumerate(lens):
        for h in range(8):
            ref, l, w, Ew = C.attend(q[b, h:h + 1], K[b][h // 4], V[b][h // 4], torch.ones(1, n, dtype=torch.bool))
            C.check_out(outs[0][b, h:h + 1].cpu(), ref, w, V[b][h // 4], Ew, f"b{b} h{h}")
            C.check_lse(lse[b, h:h + 1].cpu(), l, Ew, f"b{b} h{h}")
