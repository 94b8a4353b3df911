"""Tree attention, path commit, accumulated weights and the eviction by them, against plain
64-bit forms, at the sizes and masks where they can go wrong."""
import math

import pytest
import torch

import dense_check as C
from dense_check import D, SCALE

pytestmark = pytest.mark.gpu


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


# ------------------------------------------------------------------ tree attention
def _tree_case(rkv, lens, Hkv, G, P, T, nodes, kind, seed=1, scale=None, **kw):
    g = C.gen(seed + 100)
    B = len(lens)
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed, **kw)
    q = C.randn(g, B, Hkv * G, T, D)
    kt, vt = C.randn(g, B, Hkv, T, D), C.randn(g, B, Hkv, T, D)
    if kind == "tree":
        sees = C.ancestors(B, T, g)
    elif kind == "random":
        sees = torch.rand(B, T, T, generator=g) < 0.4
    elif kind == "full":
        sees = torch.ones(B, T, T, dtype=torch.bool)
    else:
        sees = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):                       # behind the last node anything may lie
        kt[b, :, nodes[b]:] = math.nan
        vt[b, :, nodes[b]:] = math.nan
        q[b, :, nodes[b]:] = math.nan
    return cache, K, V, q, kt, vt, sees, scale


def _run_tree(rkv, cache, q, kt, vt, sees, nodes, scale=None, ws=None, stream=None, lse=True):
    B, Hq, T, _ = q.shape
    out = torch.full((B, Hq, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B, Hq, T), 7.0, dtype=torch.float32, device="cuda") if lse else None
    rkv.rkv_tree_attention(cache, q.cuda(), kt.cuda(), vt.cuda(), C.mask_words(sees).cuda(), out, lse=ls,
                           tree_len=None if nodes is None else _ints(nodes), scale=scale, workspace=ws, stream=stream)
    return out, ls


def _check_tree(out, lse, K, V, q, kt, vt, sees, nodes, scale=None):
    B, Hq, T, _ = q.shape
    Hkv = kt.shape[1]
    G = Hq // Hkv
    out, lse = out.cpu(), lse.cpu()
    for b in range(B):
        t, n = nodes[b], K[b].shape[1]
        assert (out[b, :, t:] == 7).all() and (lse[b, :, t:] == 7).all(), "rows behind the last node changed"
        shown = torch.cat([torch.ones(t, n, dtype=torch.bool), sees[b, :t, :t]], 1)
        for h in range(Hq):
            k = torch.cat([K[b][h // G], kt[b, h // G, :t]])
            v = torch.cat([V[b][h // G], vt[b, h // G, :t]])
            ref, l, w, Ew = C.attend(q[b, h, :t], k, v, shown, scale or SCALE)
            C.check_out(out[b, h, :t], ref, w, v, Ew, f"b{b} h{h}")
            C.check_lse(lse[b, h, :t], l, Ew, f"b{b} h{h}")


@pytest.mark.parametrize("lens,Hkv,G,P,T,nodes,kind", [
    ([0], 1, 1, 16, 1, [1], "empty"),                       # a row that sees nothing at all
    ([0, 1], 1, 2, 16, 3, [3, 3], "empty"),
    ([0, 0], 2, 4, 32, 5, [5, 0], "random"),
    ([1, 15, 16, 17], 2, 4, 16, 4, [4, 3, 1, 0], "tree"),
    ([127, 128, 129, 255], 1, 8, 16, 9, [9, 8, 1, 9], "tree"),
    ([31, 33, 64, 65], 2, 2, 32, 31, [31, 30, 31, 16], "tree"),
    ([63, 64, 65], 1, 4, 64, 32, [32, 17, 31], "random"),
    ([300], 1, 1, 16, 33, [33], "tree"),
    ([515], 2, 4, 16, 8, None, "tree"),
    ([2000], 1, 4, 16, 64, [64], "tree"),
    ([1000, 20], 1, 8, 32, 65, [65, 64], "tree"),
    ([700], 1, 8, 64, 128, [127], "full"),
    ([400, 0, 90], 2, 1, 16, 129, [129, 128, 2], "tree"),
    ([130], 1, 8, 16, 256, [256], "random"),
    ([4099], 4, 4, 16, 17, [17], "tree"),
])
@pytest.mark.parametrize("room", [0, 40000])
def test_tree_attention(rkv, lens, Hkv, G, P, T, nodes, kind, room):
    # the room a cache has left decides which kernel takes a short one
    live = nodes or [T] * len(lens)
    cache, K, V, q, kt, vt, sees, _ = _tree_case(rkv, lens, Hkv, G, P, T, live, kind, room=room)
    out, lse = _run_tree(rkv, cache, q, kt, vt, sees, nodes)
    assert _status(rkv, cache) == 0
    _check_tree(out, lse, K, V, q, kt, vt, sees, live)


@pytest.mark.parametrize("T,G,room", [(3, 4, 0), (3, 4, 40000), (40, 4, 0)])
def test_tree_attention_large_logits_and_scale(rkv, T, G, room):
    # keys far from the mean: the running maximum moves late in the cache, by hundreds
    lens, nodes = [777], [T]
    cache, K, V, q, kt, vt, sees, _ = _tree_case(rkv, lens, 1, G, 16, T, nodes, "tree", seed=5, room=room)
    K[0][:, 700] *= 40
    K[0][:, 5] *= 20
    C.put_rows(cache, 0, K[0], V[0])
    out, lse = _run_tree(rkv, cache, q, kt, vt, sees, nodes, scale=0.3)
    _check_tree(out, lse, K, V, q, kt, vt, sees, nodes, 0.3)


@pytest.mark.parametrize("T,G,room", [(2, 4, 0), (2, 4, 40000), (24, 4, 0)])
def test_tree_attention_bad_lengths_and_pages_are_flagged(rkv, T, G, room):
    lens, nodes = [300, 40], [T, T]
    cache, K, V, q, kt, vt, sees, _ = _tree_case(rkv, lens, 1, G, 16, T, nodes, "tree", seed=6, room=room)
    out, lse = _run_tree(rkv, cache, q, kt, vt, sees, [T + 1, T])
    assert _status(rkv, cache) == rkv.DEVERR_TREE
    assert (out[0].cpu() == 7).all()
    _check_tree(out[1:], lse[1:], K[1:], V[1:], q[1:], kt[1:], vt[1:], sees[1:], [T])
    cache.seq_len[0] = cache.max_pages * 16 + 1
    out, lse = _run_tree(rkv, cache, q, kt, vt, sees, nodes)
    assert _status(rkv, cache) == rkv.DEVERR_CAPACITY
    _check_tree(out, lse, [K[0][:, :0], K[1]], [V[0][:, :0], V[1]], q, kt, vt, sees, nodes)
    cache.seq_len[0] = 300
    cache.page_table[0, 3] = cache.num_phys_pages          # 16 tokens that cannot be read
    cache.page_table[0, 18] = -1                           # the last, partial page
    out, lse = _run_tree(rkv, cache, q, kt, vt, sees, nodes)
    assert _status(rkv, cache) == rkv.DEVERR_PAGE_ID
    at = [t for t in range(300) if t // 16 not in (3, 18)]
    _check_tree(out, lse, [K[0][:, at], K[1]], [V[0][:, at], V[1]], q, kt, vt, sees, nodes)


def test_tree_attention_without_lse_and_twice_the_same(rkv):
    cache, K, V, q, kt, vt, sees, _ = _tree_case(rkv, [3000], 2, 4, 16, 30, [30], "tree", seed=7)
    a, la = _run_tree(rkv, cache, q, kt, vt, sees, [30])
    b, lb = _run_tree(rkv, cache, q, kt, vt, sees, [30], lse=False)
    assert torch.equal(a, b) and lb is None


# ------------------------------------------------------------------ one token with weights
def _check_decode(out, lse, got_acc, acc0, K, V, q, steps=1):
    B, Hq, _ = q.shape
    Hkv = K[0].shape[0]
    G = Hq // Hkv
    out, lse, got_acc = out.cpu(), lse.cpu(), got_acc.cpu()
    for b in range(B):
        n = K[b].shape[1]
        for g in range(Hkv):
            want, tol = acc0[b, g].double().clone(), torch.zeros(acc0.shape[2]).double()
            for h in range(g * G, (g + 1) * G):
                ref, l, w, Ew = C.attend(q[b, h:h + 1], K[b][g], V[b][g], torch.ones(1, n, dtype=torch.bool))
                C.check_out(out[b, h:h + 1], ref, w, V[b][g], Ew, f"b{b} h{h}")
                C.check_lse(lse[b, h:h + 1], l, Ew, f"b{b} h{h}")
                want[:n] += steps * w[0]
                tol[:n] += steps * w[0] * (math.exp(Ew) - 1 + 2.0 ** -20)
            tol[:n] += steps * 2.0 ** -23 * want[:n].abs()
            d = (got_acc[b, g].double() - want).abs()
            assert (d <= tol).all(), f"b{b} g{g}: weights off by {float((d - tol).max()):.3e} too much"


@pytest.mark.parametrize("lens,Hkv,G,P", [
    ([0], 1, 1, 16), ([1], 2, 8, 16), ([0, 5, 16], 1, 4, 16), ([17, 1000, 31], 2, 2, 32), ([64, 63, 129], 1, 8, 64),
    ([2563], 8, 4, 16), ([6000, 0], 1, 1, 16), ([40] * 70, 4, 4, 16), ([100, 7, 300], 30, 2, 16)])
@pytest.mark.parametrize("room", [0, 20000])
def test_decode_accum(rkv, lens, Hkv, G, P, room):
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=11, room=room)
    g = C.gen(12)
    B = len(lens)
    q = C.randn(g, B, Hkv * G, D)
    acc0 = torch.rand(B, Hkv, cache.max_pages * P + 5, generator=g)
    acc = acc0.cuda()
    out = torch.full((B, Hkv * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hkv * G), 7.0, device="cuda")
    ws = rkv.accum_workspace(B, Hkv * G, Hkv, cache.max_pages, P)
    ws.fill_(255)
    rkv.rkv_decode_accum(cache, q.cuda(), out, acc, lse=lse, workspace=ws)
    assert _status(rkv, cache) == 0
    _check_decode(out, lse, acc, acc0, K, V, q)
    rkv.rkv_decode_accum(cache, q.cuda(), out, acc, lse=lse, workspace=ws)
    _check_decode(out, lse, acc, acc0, K, V, q, steps=2)
    for b, n in enumerate(lens):  # behind the last token nothing moves
        assert torch.equal(acc[b, :, n:].cpu(), acc0[b, :, n:])


@pytest.mark.parametrize("room", [0, 20000])
def test_decode_accum_skips_a_bad_page(rkv, room):
    cache, K, V = C.make_cache(rkv, [100, 50], 1, 16, seed=13, room=room)
    q = C.randn(C.gen(14), 2, 4, D)
    acc = rkv.accum_sums(cache)
    out = torch.empty(2, 4, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 4, device="cuda")
    cache.page_table[0, 2] = -5
    rkv.rkv_decode_accum(cache, q.cuda(), out, acc, lse=lse)
    assert _status(rkv, cache) == rkv.DEVERR_PAGE_ID
    at = [t for t in range(100) if t // 16 != 2]
    assert (acc[0, 0, 32:48] == 0).all()
    got = torch.zeros(2, 1, acc.shape[2])
    got[0, 0, :len(at)] = acc[0, 0, at].cpu()
    got[1] = acc[1].cpu()
    _check_decode(out, lse, got, torch.zeros_like(got), [K[0][:, at], K[1]], [V[0][:, at], V[1]], q)


# ------------------------------------------------------------------ weights of given rows
def _rows_ref(K, q, lse, ids, m, G, acc0):
    """One (b, g): q [G, T, D], lse [G, T] -> (sums, tolerance)."""
    n = K.shape[0]
    want = acc0.double().clone()
    tol = torch.zeros_like(want)
    for h in range(G):
        x = (q[h][ids].double() @ K.double().T) * SCALE
        seen = torch.arange(n)[None] <= (n - m + torch.arange(m))[:, None]
        w = torch.where(seen, torch.exp(x - lse[h][ids].double()[:, None]), torch.zeros_like(x))
        w[lse[h][ids] == -math.inf] = 0
        E = 128 * 2.0 ** -23 * SCALE * float((q[h][ids].double().abs() @ K.double().abs().T).max()) if m else 0.0
        big = float(lse[h][ids].abs().nan_to_num(0, 0, 0).max()) if m else 0.0
        want[:n] += w.sum(0)
        tol[:n] += w.sum(0) * (math.exp(E + 2.0 ** -22 * (big + 20)) - 1 + 2.0 ** -16)
    tol[:n] += 2.0 ** -23 * want[:n].abs() * 4
    return want, tol


@pytest.mark.parametrize("lens,Hkv,G,P,T,m,ids", [
    ([1], 1, 1, 16, 1, [1], False),
    ([40, 17], 2, 4, 16, 5, [5, 0], False),
    ([16, 64, 200], 1, 2, 16, 16, [16, 16, 1], False),
    ([300, 33], 1, 8, 32, 30, [30, 29], False),
    ([129], 2, 4, 64, 129, [129], False),
    ([500], 1, 4, 16, 500, None, False),
    ([1000], 1, 1, 16, 700, [650], False),
    ([200, 31, 90], 2, 4, 16, 26, [6, 1, 0], True),
    ([2000], 1, 8, 32, 63, None, True),
    ([1500, 700], 2, 2, 64, 1024, [1000, 129], False),
])
def test_accum_rows(rkv, lens, Hkv, G, P, T, m, ids):
    B = len(lens)
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=21)
    g = C.gen(22)
    q = C.randn(g, B, Hkv * G, T, D)
    lse = torch.rand(B, Hkv * G, T, generator=g) * 4 + 6
    lse[:, :, T // 2] = -math.inf                      # a row that saw nothing weighs nothing
    row_ids = torch.randint(0, T, (B, 9), generator=g).to(torch.int32) if ids else None
    most = 9 if ids else T
    live = m or [most] * B
    if ids:
        row_ids[:, 1] = row_ids[:, 0]                  # the same row twice counts twice
    acc0 = torch.rand(B, Hkv, cache.max_pages * P, generator=g)
    acc = acc0.cuda()
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, row_len=None if m is None else _ints(m),
                       row_ids=None if row_ids is None else row_ids.cuda())
    assert _status(rkv, cache) == 0
    got = acc.cpu().double()
    for b in range(B):
        at = (row_ids[b, :live[b]] if ids else torch.arange(live[b])).long()
        for h in range(Hkv):
            want, tol = _rows_ref(K[b][h], q[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G], at, live[b], G, acc0[b, h])
            d = (got[b, h] - want).abs()
            assert (d <= tol).all(), f"b{b} g{h}: off by {float((d - tol).max()):.3e} too much"
            assert torch.equal(acc[b, h, lens[b]:].cpu(), acc0[b, h, lens[b]:])
    again = acc0.cuda()
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), again, row_len=None if m is None else _ints(m),
                       row_ids=None if row_ids is None else row_ids.cuda())
    assert torch.equal(again, acc), "the sums depend on the run"


def test_accum_rows_bad_counts_and_ids_are_flagged(rkv):
    cache, K, V = C.make_cache(rkv, [50, 60], 1, 16, seed=23)
    g = C.gen(24)
    q, lse = C.randn(g, 2, 4, 8, D), torch.full((2, 4, 8), 5.0)
    acc = rkv.accum_sums(cache)
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, row_len=_ints([9, 3]))
    assert _status(rkv, cache) == rkv.DEVERR_TREE
    assert (acc[0] == 0).all() and (acc[1, 0, :60] > 0).all()
    cache.seq_len[0] = 5                                # more rows than the cache holds tokens
    acc.zero_()
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, row_len=_ints([8, 3]))
    assert _status(rkv, cache) == rkv.DEVERR_TREE
    assert (acc[0] == 0).all()
    cache.seq_len[0] = 50
    acc.zero_()
    ids = torch.tensor([[0, 8, 2], [-1, 1, 1]], dtype=torch.int32)
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, row_ids=ids.cuda())
    assert _status(rkv, cache) == rkv.DEVERR_TREE
    bare = lse.clone()
    for b, row in ((0, 7), (1, 0)):                     # the rows with a bad id count as empty ones
        bare[b, :, row] = -math.inf
    good = torch.tensor([[0, 7, 2], [0, 1, 1]])
    for b in range(2):
        want, tol = _rows_ref(K[b][0], q[b], bare[b], good[b], 3, 4, torch.zeros(acc.shape[2]))
        assert ((acc[b, 0].cpu().double() - want).abs() <= tol).all()


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("lens,Hkv,P,T,path_lens", [
    ([0], 1, 16, 1, [1]), ([15, 16, 17, 0], 2, 16, 8, [1, 2, 8, 0]), ([30, 5], 8, 32, 63, [9, 0]),
    ([63], 3, 64, 256, [256]), ([10, 11], 1, 16, 40, [40, 39])])
def test_tree_commit_is_an_append_of_the_path(rkv, lens, Hkv, P, T, path_lens):
    B = len(lens)
    g = C.gen(31)
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=30, room=T)
    kt, vt = C.randn(g, B, Hkv, T, D), C.randn(g, B, Hkv, T, D)
    path = torch.randint(0, T, (B, max(path_lens)), generator=g).to(torch.int32)
    want = [cache.k_pages.cpu().clone(), cache.v_pages.cpu().clone()]
    grown = []
    for b, m in enumerate(path_lens):
        rows = path[b, :m].long()
        for pool, x in zip(want, (kt, vt)):
            for i in range(m):
                pos = lens[b] + i
                pool[int(cache.page_table[b, pos // P]), :, pos % P] = x[b, :, rows[i]]
        grown.append(torch.cat([K[b], kt[b][:, rows]], 1))
        path[b, m:] = -77                               # entries behind the path are not read
    rkv.rkv_tree_commit(cache, kt.cuda(), vt.cuda(), path.cuda(), _ints(path_lens))
    assert _status(rkv, cache) == 0
    bits = lambda t: t.cpu().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(cache.k_pages), bits(want[0])) and torch.equal(bits(cache.v_pages), bits(want[1]))
    assert cache.seq_len.tolist() == [n + m for n, m in zip(lens, path_lens)]
    assert torch.equal(bits(cache.kmax), bits(C.summaries(cache, grown, True)))
    assert torch.equal(bits(cache.kmin), bits(C.summaries(cache, grown, False)))


def test_tree_commit_refuses_on_the_device(rkv):
    cache, K, V = C.make_cache(rkv, [120, 120, 128, 9], 1, 16, seed=32, max_pages=8)
    before = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.kmax, cache.kmin, cache.seq_len)]
    g = C.gen(33)
    kt, vt = C.randn(g, 4, 1, 4, D).cuda(), C.randn(g, 4, 1, 4, D).cuda()
    path = torch.tensor([[0, 4, 1], [0, 1, -1], [0, 1, 2], [0, 1, 2]], dtype=torch.int32, device="cuda")
    rkv.rkv_tree_commit(cache, kt, vt, path, _ints([3, 3, 0, 4]))
    assert _status(rkv, cache) == rkv.DEVERR_TREE
    rkv.rkv_tree_commit(cache, kt, vt, path, _ints([1, 0, 1, -1]))
    assert _status(rkv, cache) == rkv.DEVERR_TREE | rkv.DEVERR_CAPACITY
    assert cache.seq_len.tolist() == [121, 120, 128, 9]
    cache.seq_len[0] = 120
    for got, ref in zip((cache.v_pages, cache.kmin, cache.seq_len), (before[1], before[3], before[4])):
        same = got.view(torch.int16 if got.dtype == torch.bfloat16 else got.dtype) == \
            ref.view(torch.int16 if ref.dtype == torch.bfloat16 else ref.dtype)
        assert int((~same).sum()) <= 128               # the one token of sequence 0


# ------------------------------------------------------------------ eviction
def _evict_case(rkv, lens, Hkv, P, seed, ties):
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=seed)
    g = C.gen(seed + 1)
    acc = torch.rand(len(lens), Hkv, cache.max_pages * P, generator=g)
    if ties:
        acc = torch.randint(0, 3, acc.shape, generator=g).float()
    for b, n in enumerate(lens):
        acc[b, :, n:] = 0
    return cache, K, V, acc


def _check_evicted(rkv, cache, acc, kept, K, V, acc0, lens, keep, recent):
    Hkv = K[0].shape[0]
    bits = lambda t: t.cpu().view(torch.int16)  # noqa: E731
    newK = []
    for b, n in enumerate(lens):
        m = min(n, keep[b])
        assert int(cache.seq_len[b]) == m
        gotK, gotV = cache.token_kv(b, m)
        rows = []
        for g in range(Hkv):
            want = C.keep_set(acc0[b, g], n, keep[b], recent)
            assert kept[b, g, :m].tolist() == want, f"b{b} g{g}"
            assert (kept[b, g, m:] == -7).all()
            assert torch.equal(bits(gotK[g]), bits(K[b][g][want])) and torch.equal(bits(gotV[g]), bits(V[b][g][want]))
            a = acc[b, g].cpu()
            assert torch.equal(a[:m].view(torch.int32), acc0[b, g][want].view(torch.int32))
            assert (a[m:] == 0).all()
            rows.append(K[b][g][want])
        newK.append(torch.stack(rows) if m else K[b][:, :0])
    for got, top in ((cache.kmax, True), (cache.kmin, False)):
        want = C.summaries(cache, newK, top)
        assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,Hkv,P,keep,recent,ties", [
    ([1], 1, 16, [1], 0, False), ([0, 40], 2, 16, [8, 8], 4, False), ([100, 17, 16], 1, 16, [20, 16, 16], 16, False),
    ([200, 300], 2, 32, [64, 33], 0, True), ([257], 3, 64, [256], 1, True), ([500, 64], 1, 16, [64, 64], 64, False),
    ([5000, 1234], 2, 16, [1500, 700], 100, False), ([9000], 1, 32, [8999], 0, True), ([50], 1, 16, [40], 0, None)])
def test_evict_accum(rkv, lens, Hkv, P, keep, recent, ties, in_place):
    cache, K, V, acc0 = _evict_case(rkv, lens, Hkv, P, 41, bool(ties))
    if ties is None:  # the heaviest stand first and in order: the kept rows stay where they are
        acc0[:, :, :lens[0]] = torch.arange(lens[0], 0, -1).float()
    acc = acc0.cuda()
    B = len(lens)
    kept = torch.full((B, Hkv, max(keep) + 3), -7, dtype=torch.int32, device="cuda")
    if in_place:
        rkv.rkv_evict_accum(cache, acc, keep, recent, kept)
        assert _status(rkv, cache) == 0
        _check_evicted(rkv, cache, acc, kept, K, V, acc0, lens, keep, recent)
        return
    before = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.kmax, cache.kmin, cache.seq_len)]
    dst, _, _ = C.make_cache(rkv, [0] * B, Hkv, P, seed=43, room=max(keep))
    dst_acc = torch.full((B, Hkv, dst.max_pages * P + 1), 3.0, device="cuda")
    rkv.rkv_evict_accum(cache, acc, keep, recent, kept, dst=dst, dst_acc=dst_acc)
    assert _status(rkv, cache) == 0 and _status(rkv, dst) == 0
    _check_evicted(rkv, dst, dst_acc, kept, K, V, acc0, lens, keep, recent)
    for got, ref in zip((cache.k_pages, cache.v_pages, cache.kmax, cache.kmin, cache.seq_len, acc), before + [acc0.cuda()]):
        as_int = {torch.bfloat16: torch.int16, torch.float32: torch.int32, torch.int32: torch.int32}[got.dtype]
        assert torch.equal(got.view(as_int), ref.view(as_int)), "the source changed"


def test_evict_accum_nan_and_infinite_weights(rkv):
    cache, K, V, acc0 = _evict_case(rkv, [64], 2, 16, 45, False)
    acc0[0, 0, 7] = math.nan
    acc0[0, 0, 9] = -math.nan
    acc0[0, 0, 20] = math.inf
    acc0[0, 0, 21:30] = -math.inf
    acc0[0, 1, 3] = -0.0
    acc0[0, 1, :64] = acc0[0, 1, :64].where(torch.arange(64) % 2 == 0, torch.tensor(0.0))
    acc0[0, 1, 0] = -0.0                               # equal to the zeros behind it
    acc = acc0.cuda()
    kept = torch.full((1, 2, 40), -7, dtype=torch.int32, device="cuda")
    rkv.rkv_evict_accum(cache, acc, [40], 2, kept)
    for g in range(2):
        assert kept[0, g].tolist() == C.keep_set(acc0[0, g], 64, 40, 2)


def test_evict_accum_flags_bad_lengths_and_pages(rkv):
    cache, K, V, acc0 = _evict_case(rkv, [100, 90], 1, 16, 46, False)
    kept = torch.full((2, 1, 30), -7, dtype=torch.int32, device="cuda")
    dst, _, _ = C.make_cache(rkv, [0, 0], 1, 16, seed=47, room=30)
    dst_acc = rkv.accum_sums(dst)
    cache.seq_len[0] = -3
    rkv.rkv_evict_accum(cache, acc0.cuda(), [30, 30], 0, kept, dst=dst, dst_acc=dst_acc)
    assert _status(rkv, cache) == rkv.DEVERR_CAPACITY
    assert dst.seq_len.tolist() == [0, 30] and (kept[0] == -7).all()
    cache.seq_len[0] = 100
    cache.page_table[0, 1] = cache.num_phys_pages + 4
    dst.page_table[1, 0] = -1
    rkv.rkv_evict_accum(cache, acc0.cuda(), [30, 30], 0, kept, dst=dst, dst_acc=dst_acc)
    assert _status(rkv, cache) == rkv.DEVERR_PAGE_ID and _status(rkv, dst) == rkv.DEVERR_PAGE_ID
    want = C.keep_set(acc0[0, 0], 100, 30, 0)
    assert kept[0, 0].tolist() == want
    got = dst.token_kv(0, 30)[0][0].cpu()
    for i, t in enumerate(want):
        if t // 16 != 1:
            assert torch.equal(got[i], K[0][0, t])


def test_evict_accum_in_place_skips_a_page_it_cannot_read(rkv):
    cache, K, V, acc0 = _evict_case(rkv, [100], 2, 16, 48, False)
    acc0[0, :, 32:48] += 2                             # the unreadable page's tokens are among the kept
    kept = torch.full((1, 2, 40), -7, dtype=torch.int32, device="cuda")
    acc = acc0.cuda()
    ws = rkv.evict_workspace(1, 2, 40)
    ws.fill_(255)                                      # NaN patterns, were they copied
    bad = int(cache.page_table[0, 2])
    cache.page_table[0, 2] = cache.num_phys_pages
    rkv.rkv_evict_accum(cache, acc, [40], 4, kept, workspace=ws)
    assert _status(rkv, cache) == rkv.DEVERR_PAGE_ID
    cache.page_table[0, 2] = bad
    for g in range(2):
        want = C.keep_set(acc0[0, g], 100, 40, 4)
        assert kept[0, g].tolist() == want
        got = cache.token_kv(0, 32)[0][g].cpu()        # rows 32.. would go to the bad page
        for i, t in enumerate(want[:32]):
            if t // 16 != 2:
                assert torch.equal(got[i], K[0][g, t])
        assert torch.equal(acc[0, g, :40].cpu(), acc0[0, g][want])


# ------------------------------------------------------------------ together
def _together(rkv, lens, Hkv, G, P, rounds, seed, stream=None):
    """Speculative decoding with a heavy-hitter budget: a prompt's weights, then rounds of a
    drafted tree, its accepted path, the path's weights, a plain step, and the eviction;
    everything against a 64-bit simulation that follows the library's kept sets."""
    B, Hq, T = len(lens), Hkv * G, 12
    g = C.gen(seed)
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=seed, room=4 * T * rounds)
    acc = rkv.accum_sums(cache)
    sums = [torch.zeros(Hkv, n).double() for n in lens]
    tols = [torch.zeros(Hkv, n).double() for n in lens]

    def add(b, w, Ew, m):
        """weights w [Hq, m rows, n]"""
        s = w.view(Hkv, G, m, -1).sum((1, 2))
        sums[b] += s
        tols[b] += s * (math.exp(Ew) - 1 + 2.0 ** -14) + 2.0 ** -22 * sums[b]

    # the prompt's rows, whose attention some prefill computed
    m = min(lens)
    q = C.randn(g, B, Hq, m, D)
    lse = torch.zeros(B, Hq, m)
    for b, n in enumerate(lens):
        shown = torch.arange(n)[None] <= (n - m + torch.arange(m))[:, None]
        ws = []
        for h in range(Hq):
            _, l, w, Ew = C.attend(q[b, h], K[b][h // G], V[b][h // G], shown)
            lse[b, h] = l.float()
            ws.append(w)
        add(b, torch.stack(ws), Ew, m)
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, stream=stream)
    for r in range(rounds):
        sees = C.ancestors(B, T, g)
        q, kt, vt = C.randn(g, B, Hq, T, D), C.randn(g, B, Hkv, T, D), C.randn(g, B, Hkv, T, D)
        out = torch.full((B, Hq, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, Hq, T), 7.0, device="cuda")
        qd, ktd, vtd = q.cuda(), kt.cuda(), vt.cuda()
        rkv.rkv_tree_attention(cache, qd, ktd, vtd, C.mask_words(sees).cuda(), out, lse=lse, stream=stream)
        _check_tree(out, lse, K, V, q, kt, vt, sees, [T] * B)
        # accept the chain that ends in some node
        path = torch.zeros(B, T, dtype=torch.int32)
        lens_p = []
        for b in range(B):
            chain = torch.nonzero(sees[b, (r * 5 + b) % T])[:, 0]
            path[b, :len(chain)] = chain.int()
            lens_p.append(len(chain))
        rkv.rkv_tree_commit(cache, ktd, vtd, path.cuda(), _ints(lens_p), stream=stream)
        rkv.rkv_accum_rows(cache, qd, lse, acc, row_len=_ints(lens_p), row_ids=path.cuda(), stream=stream)
        for b in range(B):
            m = lens_p[b]
            at = path[b, :m].long()
            K[b], V[b] = torch.cat([K[b], kt[b][:, at]], 1), torch.cat([V[b], vt[b][:, at]], 1)
            n = K[b].shape[1]
            sums[b] = torch.cat([sums[b], torch.zeros(Hkv, m).double()], 1)
            tols[b] = torch.cat([tols[b], torch.zeros(Hkv, m).double()], 1)
            shown = torch.arange(n)[None] <= (n - m + torch.arange(m))[:, None]
            ws = [C.attend(q[b, h, at], K[b][h // G], V[b][h // G], shown) for h in range(Hq)]
            add(b, torch.stack([x[2] for x in ws]), 2 * max(x[3] for x in ws), m)
        q1 = C.randn(g, B, Hq, D)
        o1 = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        rkv.rkv_decode_accum(cache, q1.cuda(), o1, acc, stream=stream)
        for b in range(B):
            ws = [C.attend(q1[b, h:h + 1], K[b][h // G], V[b][h // G], torch.ones(1, K[b].shape[1], dtype=torch.bool))
                  for h in range(Hq)]
            for h in range(Hq):
                C.check_out(o1[b, h:h + 1].cpu(), ws[h][0], ws[h][2], V[b][h // G], ws[h][3])
            add(b, torch.stack([x[2] for x in ws]), max(x[3] for x in ws), 1)
            n = K[b].shape[1]
            assert ((acc[b, :, :n].cpu().double() - sums[b]).abs() <= tols[b]).all(), f"round {r} b{b}"
            assert (acc[b, :, n:] == 0).all()
        keep = [max(20, K[b].shape[1] - 9 * (b + 1)) for b in range(B)]
        kept = torch.full((B, Hkv, max(keep)), -7, dtype=torch.int32, device="cuda")
        had = acc.cpu().clone()
        rkv.rkv_evict_accum(cache, acc, keep, 8, kept, stream=stream)
        for b in range(B):
            n = K[b].shape[1]
            at = [C.keep_set(had[b, h], n, keep[b], 8) for h in range(Hkv)]
            for h in range(Hkv):
                assert kept[b, h, :len(at[h])].tolist() == at[h]
            idx = torch.tensor(at)
            pick = lambda x: x.gather(1, idx)  # noqa: E731
            K[b] = K[b].gather(1, idx[..., None].expand(-1, -1, D))
            V[b] = V[b].gather(1, idx[..., None].expand(-1, -1, D))
            sums[b], tols[b] = pick(sums[b]), pick(tols[b])
            got = cache.token_kv(b, idx.shape[1])
            assert torch.equal(got[0].cpu(), K[b]) and torch.equal(got[1].cpu(), V[b])
    assert _status(rkv, cache) == 0


@pytest.mark.parametrize("lens,Hkv,G,P", [([60, 33], 2, 4, 16), ([150], 1, 8, 32), ([40, 70, 65], 1, 1, 64)])
def test_a_run_of_them(rkv, lens, Hkv, G, P):
    _together(rkv, lens, Hkv, G, P, 3, 51)


def test_the_sparse_step_goes_on_from_the_evicted_cache(rkv):
    # after an eviction the page summaries serve the sparse step as after a prefill: with
    # every channel and every page taken it is the dense step
    cache, K, V, acc0 = _evict_case(rkv, [400], 2, 16, 55, False)
    kept = torch.empty(1, 2, 100, dtype=torch.int32, device="cuda")
    acc = acc0.cuda()
    rkv.rkv_evict_accum(cache, acc, [100], 16, kept)
    q = C.randn(C.gen(56), 1, 8, D)
    o32 = torch.empty(1, 8, D, device="cuda")
    rkv.rkv_decode_hsa(cache, q.cuda(), [128], [7], o32)
    for h in range(8):
        at = kept[0, h // 4].cpu().long()
        k, v = K[0][h // 4][at], V[0][h // 4][at]
        ref, _, w, Ew = C.attend(q[0, h:h + 1], k, v, torch.ones(1, 100, dtype=torch.bool))
        C.check_out(o32[0, h:h + 1].cpu(), ref, w, v, Ew)


def test_another_stream_and_a_replayed_graph(rkv):
    """The calls on a side stream, captured once and replayed while the cache grows; two
    graphs with workspaces of their own."""
    Hkv, G, P, T = 2, 4, 16, 20
    cache, K, V = C.make_cache(rkv, [700, 90], Hkv, P, seed=61, room=64)
    g = C.gen(62)
    q, kt, vt = C.randn(g, 2, 8, T, D), C.randn(g, 2, Hkv, T, D), C.randn(g, 2, Hkv, T, D)
    sees = C.ancestors(2, T, g)
    path = torch.tensor([[0, 3, 5], [1, 1, 19]], dtype=torch.int32)
    dev = [t.cuda() for t in (q, kt, vt, C.mask_words(sees), path)]
    plen = _ints([3, 2])
    out = torch.zeros(2, 8, T, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 8, T, device="cuda")
    q1 = C.randn(g, 2, 8, D)
    q1d = q1.cuda()
    o1 = torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda")
    l1 = torch.zeros(2, 8, device="cuda")
    acc = rkv.accum_sums(cache)
    wt = rkv.tree_workspace(2, 8, Hkv, T, cache.max_pages, P)
    wa = rkv.accum_workspace(2, 8, Hkv, cache.max_pages, P)
    wr = rkv.accum_rows_workspace(2, 8, Hkv, T, cache.max_pages, P)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        rkv.rkv_tree_attention(cache, dev[0], dev[1], dev[2], dev[3], out, lse=lse, workspace=wt)
        rkv.rkv_tree_commit(cache, dev[1], dev[2], dev[4], plen)
        rkv.rkv_accum_rows(cache, dev[0], lse, acc, row_len=plen, row_ids=dev[4], workspace=wr)

    def token():
        rkv.rkv_decode_accum(cache, q1d, o1, acc, lse=l1, workspace=wa)

    with torch.cuda.stream(side):
        step()
        token()
        a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(a, stream=side):
            step()
        with torch.cuda.graph(b, stream=side):
            token()
        for _ in range(3):
            a.replay()
            b.replay()
    side.synchronize()
    torch.cuda.synchronize()
    for i in range(2):
        m = int(plen[i])
        at = path[i, :m].long()
        for _ in range(3):
            K[i], V[i] = torch.cat([K[i], kt[i][:, at]], 1), torch.cat([V[i], vt[i][:, at]], 1)
    _check_tree(out, lse, K, V, q, kt, vt, sees, [T, T])  # the last replay saw the first three paths
    for i in range(2):
        m = int(plen[i])
        at = path[i, :m].long()
        K[i], V[i] = torch.cat([K[i], kt[i][:, at]], 1), torch.cat([V[i], vt[i][:, at]], 1)
        for h in range(8):
            ref, l, w, Ew = C.attend(q1[i, h:h + 1], K[i][h // G], V[i][h // G],
                                     torch.ones(1, K[i].shape[1], dtype=torch.bool))
            C.check_out(o1[i, h:h + 1].cpu(), ref, w, V[i][h // G], Ew)
            C.check_lse(l1[i, h:h + 1].cpu(), l, Ew)
    assert cache.seq_len.tolist() == [700 + 12, 90 + 8]
    assert _status(rkv, cache) == 0


def test_workspaces_made_by_the_calls_on_another_stream(rkv):
    """Without a workspace argument each call makes its own; on a stream that is not the
    current one its memory must not be handed out while the call still runs."""
    cache, K, V = C.make_cache(rkv, [6000, 900], 2, 16, seed=65, room=10000)
    g = C.gen(66)
    q = C.randn(g, 2, 8, D)
    qd = q.cuda()
    side = torch.cuda.Stream()
    outs = [torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
    lse = torch.zeros(2, 8, device="cuda")
    acc = rkv.accum_sums(cache)
    torch.cuda.synchronize()
    for o in outs:
        rkv.rkv_decode_accum(cache, qd, o, acc, lse=lse, stream=side)
        torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")  # takes what was freed, on the current stream
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    _check_decode(outs[0], lse, acc, torch.zeros(2, 2, acc.shape[2]), K, V, q, steps=20)


def test_a_long_cache_with_offsets_past_32_bits(rkv):
    """Page pools of more than 2^31 elements: 4.6 GB each, the sequence on the last pages."""
    P, Hkv = 64, 8
    phys = 35200                                           # 35200 * 8 * 64 * 128 elements > 2^31
    pages = 24
    pt = torch.arange(phys - pages, phys, dtype=torch.int32, device="cuda").flip(0).view(1, pages).contiguous()
    cache = rkv.PagedCache(1, Hkv, P, pages, "cuda", page_table=pt, num_phys_pages=phys)
    g = C.gen(71)
    n, T, G = 1200, 10, 4
    K, V = C.randn(g, Hkv, n, D), C.randn(g, Hkv, n, D)
    C.put_rows(cache, 0, K, V)
    cache.seq_len.fill_(n)
    q, kt, vt = C.randn(g, 1, Hkv * G, T, D), C.randn(g, 1, Hkv, T, D), C.randn(g, 1, Hkv, T, D)
    sees = C.ancestors(1, T, g)
    out, lse = _run_tree(rkv, cache, q, kt, vt, sees, [T])
    _check_tree(out, lse, [K], [V], q, kt, vt, sees, [T])
    acc = rkv.accum_sums(cache)
    q1 = C.randn(g, 1, Hkv * G, D)
    o1 = torch.empty(1, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    l1 = torch.empty(1, Hkv * G, device="cuda")
    rkv.rkv_decode_accum(cache, q1.cuda(), o1, acc, lse=l1)
    _check_decode(o1, l1, acc, torch.zeros(1, Hkv, acc.shape[2]), [K], [V], q1)
    kept = torch.full((1, Hkv, 300), -7, dtype=torch.int32, device="cuda")
    had = acc.cpu().clone()
    rkv.rkv_evict_accum(cache, acc, [300], 10, kept)
    for h in range(Hkv):
        at = C.keep_set(had[0, h], n, 300, 10)
        assert kept[0, h].tolist() == at
        assert torch.equal(cache.token_kv(0, 300)[0][h].cpu(), K[h][at])
    assert _status(rkv, cache) == 0
