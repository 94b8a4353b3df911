"""Attention over the 8-bit cache against its definition in fp64 (bounds: tests/q8_check.py)."""
import math

import pytest
import torch

import q8_check as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rkv():
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _queries(B, Hq, T, seed=0, loud=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 13)
    q = torch.randn(B, Hq, T, C.D, generator=g, device="cuda")
    if loud:  # rows of very different size
        q *= torch.exp2(torch.randint(-3, 3, (B, Hq, T, 1), generator=g, device="cuda").float())
    return q.bfloat16()


def _run(rkv, cache, q, rows=None, **kw):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    rkv.rkv_q8_attention(cache, q, out, lse=lse, row_len=_ints(rows) if rows is not None else None, **kw)
    return out, lse


def _check(rkv, cache, K, V, q, rows=None, **kw):
    out, lse = _run(rkv, cache, q, rows)
    full = rows if rows is not None else [q.shape[2]] * q.shape[0]
    C.check_attention(cache, K, V, q, out, lse, full, **kw)
    for b, m in enumerate(full):  # rows behind the last are left as they were
        assert (out[b, :, m:] == 7.0).all() and (lse[b, :, m:] == 7.0).all()
    assert rkv.rkv_read_device_error(cache.error_word) == (rkv.RKV_OK, 0)
    return out, lse


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (3, 8), (8, 2)])
def test_one_token_at_every_length(rkv, Hkv, G, P, fmt):
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 2563]
    cache, K, V = C.filled(rkv, lens, Hkv, P, fmt, seed=P + G)
    _check(rkv, cache, K, V, _queries(len(lens), Hkv * G, 1, seed=G))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T,rows,lens,Hkv,G,P", [
    (2, [2, 1, 0], [40, 3, 90], 2, 4, 16),
    (4, [4, 4, 2], [4, 2, 1000], 1, 4, 32),          # rows before the first key see nothing
    (5, [5, 3, 5, 0, 1], [3000, 5, 1, 0, 700], 2, 8, 64),
    (17, [17, 9], [17, 300], 4, 1, 16),
    (33, [33, 1, 20], [20, 1, 4097], 1, 2, 16),       # more rows than keys
    (64, [64, 63], [64, 1111], 2, 8, 32),
    (100, [100, 7, 0], [257, 2000, 31], 2, 4, 64),
    (300, [300, 299], [301, 1500], 2, 4, 16),
    (700, [650, 700, 1], [650, 300, 128], 1, 8, 32)])
def test_the_last_rows(rkv, T, rows, lens, Hkv, G, P, fmt):
    cache, K, V = C.filled(rkv, lens, Hkv, P, fmt, seed=T)
    _check(rkv, cache, K, V, _queries(len(lens), Hkv * G, T, seed=T), rows)


@pytest.mark.parametrize("T", [1, 3, 50, 200])
def test_ragged_batches_of_many_sequences(rkv, T):
    lens = [(37 * b * b + 11 * b) % 900 for b in range(61)]
    rows = [(T - b % (T + 1)) for b in range(61)]
    cache, K, V = C.filled(rkv, lens, 2, 16, "e4m3", seed=T)
    _check(rkv, cache, K, V, _queries(61, 8, T, seed=T), rows)


@pytest.mark.parametrize("T,n", [(1, 70001), (3, 40000), (40, 30001), (1500, 9000)])
def test_long_caches(rkv, T, n):
    cache, K, V = C.filled(rkv, [n, n // 3], 2, 32, "e4m3", seed=n)
    _check(rkv, cache, K, V, _queries(2, 16, T, seed=n), sample=40)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_the_longest_cache(rkv, T):
    """2^20 positions, the most that a table holds."""
    cache, K, V = C.filled(rkv, [1 << 20], 1, 64, "e4m3", seed=T)
    assert cache.max_pages == 16384
    _check(rkv, cache, K, V, _queries(1, 8, T, seed=T), sample=8)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_far_pages(rkv, T):
    """Codes behind 2^31 bytes of their pools."""
    H, P, phys, n = 8, 64, 40000, 700
    pt = torch.arange(phys - 16, phys, dtype=torch.int32, device="cuda").view(1, 16)
    cache = rkv.PagedCache8(1, H, P, 16, "cuda", page_table=pt, num_phys_pages=phys, fmt="int8")
    g = torch.Generator(device="cuda").manual_seed(T)
    rkv.rkv_q8_append(cache, torch.randn(1, H, n, C.D, generator=g, device="cuda").bfloat16(),
                      torch.randn(1, H, n, C.D, generator=g, device="cuda").bfloat16())
    K, V = zip(*[[y.double() for y in cache.token_kv(0)]])
    _check(rkv, cache, K, V, _queries(1, 2 * H, T, seed=T))


@pytest.mark.parametrize("B,n", [(1, 3), (1, 900), (1, 8000), (3, 2000), (8, 1500), (19, 700), (20, 700)])
@pytest.mark.parametrize("T", [1, 2, 6])
def test_small_caches_by_clusters_of_every_size(rkv, B, n, T):
    lens = [n - (n * b) // (2 * B) for b in range(B)]
    if B > 2:
        lens[1] = 0
    cache, K, V = C.filled(rkv, lens, 8, 16, "e4m3" if T != 2 else "int8", seed=n)
    _check(rkv, cache, K, V, _queries(B, 32, T, seed=n), [T - (b % 2) * (T // 2) for b in range(B)])


@pytest.mark.parametrize("T", [1, 4, 70, 300])
def test_every_row_a_whole_prompt(rkv, T):
    """n = m: the causal triangle from its first row on."""
    cache, K, V = C.filled(rkv, [T, T], 2, 16, "int8", seed=T)
    _check(rkv, cache, K, V, _queries(2, 8, T, seed=T))


@pytest.mark.parametrize("T", [1, 2, 40, 90])
def test_page_scales_far_apart(rkv, T):
    """Pages whose scales differ by up to 2^20 either way, and pages of zeros."""
    n, P = 900, 16
    cache, K, V = C.filled(rkv, [n], 2, P, "e4m3", seed=1)
    g = C.gen(5)
    phys = cache.page_table[0, :-(-n // P)].long()
    kf = torch.exp2(torch.randint(-9, 1, (len(phys), 2), generator=g).float()).cuda()
    vf = torch.exp2(torch.randint(-12, 9, (len(phys), 2), generator=g).float()).cuda()
    vf[3], vf[20] = 0.0, 0.0
    cache.k_scale[phys] *= kf
    cache.v_scale[phys] = torch.where(vf == 0, torch.tensor(2.0 ** -126, device="cuda"), cache.v_scale[phys] * vf)
    zero = phys[[3, 20]]
    cache.v_codes.view(torch.uint8)[zero] = 0
    K, V = zip(*[[x.double() for x in cache.token_kv(0)]])
    _check(rkv, cache, K, V, _queries(1, 8, T, seed=T))


@pytest.mark.parametrize("T", [1, 3, 40, 90])
def test_logits_far_from_zero(rkv, T):
    """Queries that make one key outweigh all others, and rows whose logits are all far below zero."""
    cache, K, V = C.filled(rkv, [777], 1, 32, "e4m3", seed=2, spread=False)
    q = _queries(1, 4, T, seed=3, loud=False)
    q[:, 0] *= 64
    q[:, 1] *= 1e-3
    q[:, 2] = -K[0][0, :1].float().mean(0).bfloat16() * 16
    q[:, 3] = 0
    _check(rkv, cache, K, V, q)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1.0, 40.0])
@pytest.mark.parametrize("T", [1, 90])
def test_scales_of_the_softmax(rkv, scale, T):
    cache, K, V = C.filled(rkv, [400], 2, 16, "int8", seed=2)
    q = _queries(1, 4, T, seed=5, loud=False)
    out, lse = _run(rkv, cache, q, scale=scale)
    C.check_attention(cache, K, V, q, out, lse, [T], scale=scale)


@pytest.mark.parametrize("T", [1, 3, 40, 200])
@pytest.mark.parametrize("P", [16, 64])
def test_pages_of_nan_reach_who_sees_them_alone(rkv, T, P):
    n = 330
    cache, K, V = C.filled(rkv, [n, n], 2, P, "e4m3", seed=T)
    page = (n - 1) // P - (1 if T > P else 0)  # a page that the first rows of a long tail do not see
    ph = cache.page_table[0, page].long()
    cache.k_scale[ph, 1] = math.nan
    cache.v_scale[ph, 1] = math.nan
    q = _queries(2, 8, T, seed=T)
    out, lse = _run(rkv, cache, q)
    sees = torch.arange(T, device="cuda") + n - T >= page * P
    assert torch.isnan(out[0, 4:, sees]).all() and torch.isnan(lse[0, 4:, sees]).all()
    keep = (~sees).nonzero().flatten()
    # the rows that do not see the page, and every other head and sequence
    for b, heads in ((0, range(4)), (0, range(4, 8)), (1, range(8))):
        for h in heads:
            idx = keep if b == 0 and h >= 4 else torch.arange(T, device="cuda")
            if not len(idx):
                continue
            zz = (q[b, h, idx].double() @ K[b][h // 4].T) * C.SCALE
            zz = zz.masked_fill(torch.arange(n, device="cuda")[None] > (n - T + idx)[:, None], -math.inf)
            ref = torch.softmax(zz, 1) @ V[b][h // 4]
            assert torch.isfinite(out[b, h, idx]).all()
            assert ((out[b, h, idx].double() - ref).abs() <= 2.0 ** -6 * (torch.softmax(zz, 1) @ V[b][h // 4].abs()) + 1e-6).all()


@pytest.mark.parametrize("T", [1, 3, 6, 40, 200])
@pytest.mark.parametrize("page", [2, 20])
def test_pages_of_nan_among_logits_far_from_zero(rkv, T, page):
    """Logits beyond 2^30 of either sign: a page of NaN makes every row that sees it NaN, none else."""
    n, P = 330, 16
    cache, K, V = C.filled(rkv, [n], 2, P, "e4m3", seed=T)
    ph = cache.page_table[0, page].long()
    cache.k_scale[ph] = math.nan
    cache.v_scale[ph] = math.nan
    q = _queries(1, 8, T, seed=T)
    q[:, 1::2] = -q[:, ::2]
    out, lse = _run(rkv, cache, q, scale=2.0 ** 34)
    sees = torch.arange(T, device="cuda") + n - T >= page * P
    assert torch.isnan(out[0, :, sees]).all() and torch.isnan(lse[0, :, sees]).all()
    assert torch.isfinite(out[0, :, ~sees]).all() and torch.isfinite(lse[0, :, ~sees]).all()


@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T,n,P,at,room", [
    (3, 306, 16, 304, 0),       # clusters; the page begins inside 32 keys that are taken together
    (6, 308, 16, 304, 0),
    (6, 322, 64, 320, 0),
    (2, 305, 16, 304, 9000),    # the flat split on mma.sync: 8, 16 and 24 rows
    (3, 306, 16, 304, 9000),
    (6, 307, 16, 304, 9000),
    (6, 321, 64, 320, 9000),
    (32, 322, 16, 320, 0),      # 128-row tiles
    (32, 322, 16, 304, 0),
    (32, 322, 64, 320, 0),
    (100, 322, 16, 320, 0),     # 256-row tiles
    (100, 322, 16, 256, 0),
    (300, 700, 16, 512, 0),
])
def test_pages_that_a_row_does_not_see(rkv, T, n, P, at, room, fmt, which):
    """A page with 2^100 times its neighbours' scales has no part in the results of rows that end before it."""
    cache, K, V = C.filled(rkv, [n], 2, P, fmt, seed=T, room=room)
    ph = cache.page_table[0, at // P].long()
    unit = float(cache.v_scale[cache.page_table[0, :at // P].long()].max())
    for t, s in (("k", cache.k_scale), ("v", cache.v_scale)):
        if t in which:
            s[ph] *= 2.0 ** 100
    q = _queries(1, 8, T, seed=T)
    out, lse = _run(rkv, cache, q)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    pos = torch.arange(n - T, n, device="cuda")
    idx = (pos < at).nonzero().flatten()
    assert len(idx)
    for h in range(8):
        k, v = K[0][h // 4][:at], V[0][h // 4][:at]
        qq = q[0, h, idx].double()
        hidden = torch.arange(at, device="cuda")[None] > pos[idx][:, None]
        z = (qq @ k.T * C.SCALE).masked_fill(hidden, -math.inf)
        ref_l, w = torch.logsumexp(z, 1), torch.softmax(z, 1)
        ref = w @ v
        E = 132 * 2.0 ** -23 * C.SCALE * float((qq.abs() @ k.abs().T).max())
        Ew = 2 * E + 2.0 ** -16 + n * 2.0 ** -30
        tol = (2.0 ** -11 + Ew) * (w @ v.abs()) + 2.0 ** -8 * (1 + Ew) * ref.abs() + n * 2.0 ** -32 * 448 * unit
        assert ((out[0, h, idx].double() - ref).abs() <= tol).all(), f"head {h}"
        assert ((lse[0, h, idx].double() - ref_l).abs() <= Ew + 2.0 ** -22 * ref_l.abs()).all(), f"head {h}"


@pytest.mark.parametrize("T", [1, 3, 40])
def test_queries_with_a_nan_or_an_infinity(rkv, T):
    cache, K, V = C.filled(rkv, [200], 2, 16, "e4m3", seed=T)
    q = _queries(1, 8, T, seed=T)
    q[0, 2, T - 1, 5], q[0, 5, 0, 9] = math.nan, math.inf
    out, lse = _run(rkv, cache, q)
    bad = torch.zeros(8, T, dtype=torch.bool, device="cuda")
    bad[2, T - 1], bad[5, 0] = True, True
    assert torch.equal(torch.isnan(lse[0]), bad) and torch.equal(torch.isnan(out[0]).all(2), bad)
    assert torch.isfinite(out[0][~bad]).all()


@pytest.mark.parametrize("T", [1, 3, 40, 200])
def test_pages_that_cannot_be_read(rkv, T):
    """Bad ids are flagged and their tokens are not there; other sequences are not touched."""
    P, n = 16, 310
    cache, K, V = C.filled(rkv, [n, n, 900], 2, P, "e4m3", seed=T)
    q = _queries(3, 8, T, seed=T)
    cache.page_table[0, 2], cache.page_table[0, 9] = -1, cache.num_phys_pages
    cache.seq_len[2] = cache.max_pages * P + 1
    out, lse = _run(rkv, cache, q, [T, T, T])
    assert rkv.rkv_read_device_error(cache.error_word)[1] == rkv.DEVERR_PAGE_ID | rkv.DEVERR_CAPACITY
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    # the split of the work, and so the order of sums, depends on all lengths: bounds, not bits
    none = [torch.zeros(2, 0, C.D, device="cuda").double()] * 2
    C.check_attention(cache, [none[0], K[1], none[0]], [none[1], V[1], none[1]], q, out, lse, [0, T, 0])
    gone = torch.zeros(n, dtype=torch.bool, device="cuda")
    gone[2 * P:3 * P] = gone[9 * P:10 * P] = True
    for h in range(8):
        z = (q[0, h].double() @ K[0][h // 4].T) * C.SCALE
        i = torch.arange(T, device="cuda")
        z = z.masked_fill((torch.arange(n, device="cuda")[None] > (n - T + i)[:, None]) | gone[None], -math.inf)
        w = torch.softmax(z, 1)
        ref_o = w @ V[0][h // 4]
        assert ((out[0, h].double() - ref_o).abs() <= 2.0 ** -6 * (w @ V[0][h // 4].abs()) + 1e-6).all()
    cache.seq_len[2] = 900
    rkv.rkv_q8_attention(cache, q, out, row_len=_ints([T, T + 1, -1]))
    assert rkv.rkv_read_device_error(cache.error_word)[1] & rkv.DEVERR_TREE


@pytest.mark.parametrize("T", [1, 6, 130])
def test_without_lse_on_another_stream_and_twice(rkv, T):
    cache, K, V = C.filled(rkv, [1000, 20], 2, 16, "int8", seed=T)
    q = _queries(2, 8, T, seed=T)
    ref, ref_l = _check(rkv, cache, K, V, q)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
    for _ in range(3):
        rkv.rkv_q8_attention(cache, q, o1, stream=a)
        rkv.rkv_q8_attention(cache, q, o2, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(o1, ref) and torch.equal(o2, ref)


def test_a_captured_step_follows_the_cache(rkv):
    """Reserve, rotate, append and attend, captured once and replayed as the cache grows; at
    every step against the plain forms of all four."""
    B, Hkv, G, P, pages = 3, 2, 4, 16, 16
    pool = rkv.PagePool(B * pages, B, "cuda")
    table = torch.zeros(B, pages, dtype=torch.int32, device="cuda")
    cache = rkv.PagedCache8(B, Hkv, P, pages, "cuda", page_table=table, num_phys_pages=B * pages)
    assert cache.page_table.data_ptr() == table.data_ptr()
    plan = rkv.rotary_plan(128, 10000.0)
    model = C.Model(B, Hkv, P, "e4m3")
    g = torch.Generator(device="cuda").manual_seed(1)
    offset = _ints([0, 1000, 50000])  # the positions of a compressed cache's tokens lie ahead of its rows
    at, lens = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")

    def state(T):
        x = torch.zeros(B, T, Hkv * (G + 2), C.D, dtype=torch.bfloat16, device="cuda")
        return dict(x=x, q=torch.zeros(B, Hkv * G, T, C.D, dtype=torch.bfloat16, device="cuda"),
                    k=torch.zeros(B, Hkv, T, C.D, dtype=torch.bfloat16, device="cuda"),
                    out=torch.zeros(B, Hkv * G, T, C.D, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros(B, Hkv * G, T, device="cuda"), new=torch.zeros(B, dtype=torch.int32, device="cuda"),
                    ws=rkv.q8_workspace(B, Hkv * G, Hkv, T, cache.max_pages, P))

    def step(s, T):
        torch.add(cache.seq_len, s["new"], out=lens)
        rkv.rkv_reserve_pages(pool, table, P, lens)
        torch.add(cache.seq_len, offset, out=at)
        x = s["x"]
        rkv.rkv_rotary(plan, x[:, :, :Hkv * G].transpose(1, 2), x[:, :, Hkv * G:Hkv * (G + 1)].transpose(1, 2), at, s["q"], s["k"])
        rkv.rkv_q8_append(cache, s["k"], x[:, :, Hkv * (G + 1):].transpose(1, 2), new_len=s["new"])
        rkv.rkv_q8_attention(cache, s["q"], s["out"], lse=s["lse"], row_len=s["new"], workspace=s["ws"])

    def check(s, T):
        torch.cuda.synchronize()
        new = s["new"].tolist()
        for b in range(B):
            model.append(b, s["k"][b, :, :new[b]].cpu(), s["x"][b, :new[b], Hkv * (G + 1):].transpose(0, 1).cpu())
        model.check(cache)
        K, V = zip(*[[y.double() for y in cache.token_kv(b)] for b in range(B)])
        C.check_attention(cache, K, V, s["q"], s["out"], s["lse"], new)

    prompt = state(37)
    prompt["x"].copy_(torch.randn(prompt["x"].shape, generator=g, device="cuda"))
    prompt["new"].copy_(_ints([37, 5, 0]))
    step(prompt, 37)
    check(prompt, 37)
    one = state(1)
    one["new"].copy_(_ints([1, 1, 1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one, 1)
    for i in range(20):
        one["x"].copy_(torch.randn(one["x"].shape, generator=g, device="cuda") * (1 + i))
        one["new"].copy_(_ints([1, 1, i % 2]))
        graph.replay()
        check(one, 1)
    assert rkv.rkv_read_device_error(cache.error_word) == (rkv.RKV_OK, 0)
    assert rkv.rkv_read_device_error(pool.error_word) == (rkv.RKV_OK, 0)


def test_an_evicted_prompt_goes_on_in_8_bits(rkv):
    """Stage 1 keeps a prompt's tokens in a bf16 cache; the 8-bit one made of it decodes on."""
    B, Hkv, G, L, w, P = 2, 2, 4, 600, 8, 16
    g = C.gen(3)
    k, v = C.randn(g, B, Hkv, L, C.D).cuda(), C.randn(g, B, Hkv, L, C.D).cuda()
    q_win = C.randn(g, B, Hkv * G, w, C.D).cuda()
    keep = [150, 90]
    src = rkv.PagedCache(B, Hkv, P, 16)
    kept = torch.empty(B, Hkv, 150, dtype=torch.int32, device="cuda")
    rkv.rkv_prefill_evict(q_win, k, v, [L, L], keep, [5, 5], src, kept)
    cache = rkv.PagedCache8(B, Hkv, P, 16, page_table=src.page_table, num_phys_pages=src.num_phys_pages, fmt="int8")
    rkv.rkv_q8_load(cache, src)
    model = C.Model(B, Hkv, P, "int8")
    for b in range(B):
        kk, vv = src.token_kv(b)
        model.append(b, kk.cpu(), vv.cpu())
    model.check(cache)
    for _ in range(3):
        kn, vn = C.randn(g, B, Hkv, 1, C.D), C.randn(g, B, Hkv, 1, C.D)
        rkv.rkv_q8_append(cache, kn.cuda(), vn.cuda())
        for b in range(B):
            model.append(b, kn[b], vn[b])
        model.check(cache)
        K, V = zip(*[[y.double() for y in cache.token_kv(b)] for b in range(B)])
        _check(rkv, cache, K, V, _queries(B, Hkv * G, 1))
