"""Branches of the dense cache kernels that a well-formed batch does not enter: pages that
cannot be read, sequences without rows between others, refused paths."""
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


def _rows_want(K, q, lse, m, scale=SCALE):
    """The weights of the m last rows of one (sequence, KV head): q [G, m, D], lse [G, m] ->
    (sums [n], tolerance), bounds as dense_check derives them."""
    n = K.shape[0]
    want, tol = torch.zeros(n).double(), torch.zeros(n).double()
    seen = torch.arange(n)[None] <= (n - m + torch.arange(m))[:, None]
    for h in range(q.shape[0]):
        z = (q[h].double() @ K.double().T) * scale
        w = torch.where(seen, torch.exp(z - lse[h].double()[:, None]), torch.zeros_like(z)).sum(0)
        E = 128 * 2.0 ** -23 * scale * float((q[h].double().abs() @ K.double().abs().T).max()) if m else 0.0
        big = float(lse[h].abs().max()) if m else 0.0
        want += w
        tol += w * (math.exp(E + 2.0 ** -22 * (big + 20)) - 1 + 2.0 ** -16)
    return want, tol + 2.0 ** -21 * want


# (T, G): 16 rows; 32; blocks of 64; tensor cores with 64 rows a tile, with 128, several tiles
@pytest.mark.parametrize("T,G", [(4, 4), (8, 4), (26, 4), (40, 4), (64, 8), (130, 1), (300, 2)])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("bad", [False, True])
def test_accum_rows_ragged_and_with_pages_it_cannot_read(rkv, T, G, P, bad):
    lens = [0, 700, 300, 0, 515, 301, 0]
    m = [0, min(T, 700), 0, 0, T, 1, 0]
    Hkv = 2
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=110 + P)
    g = C.gen(111)
    q = C.randn(g, len(lens), Hkv * G, T, D)
    lse = torch.rand(len(lens), Hkv * G, T, generator=g) * 4 + 6
    for b in range(len(lens)):                             # behind the last row anything may lie
        q[b, :, m[b]:] = math.nan
        lse[b, :, m[b]:] = math.nan
    lost = {1: [], 4: [], 5: []}
    if bad:
        lost = {1: [3, 699 // P], 4: [0, 256 // P], 5: [300 // P]}
        for b, pages in lost.items():
            for i, pg in enumerate(pages):
                cache.page_table[b, pg] = -1 if i else cache.num_phys_pages
    acc0 = torch.rand(len(lens), Hkv, cache.max_pages * P, generator=g)
    acc = acc0.cuda()
    rkv.rkv_accum_rows(cache, q.cuda(), lse.cuda(), acc, row_len=_ints(m))
    assert _status(rkv, cache) == (rkv.DEVERR_PAGE_ID if bad else 0)
    acc = acc.cpu()
    for b, n in enumerate(lens):
        if m[b] == 0:
            assert torch.equal(acc[b], acc0[b]), f"b{b}: no row, and sums that moved"
            continue
        gone = torch.tensor([t // P in lost[b] for t in range(n)])
        for h in range(Hkv):
            rows = slice(h * G, (h + 1) * G)
            want, tol = _rows_want(K[b][h], q[b, rows, :m[b]], lse[b, rows, :m[b]], m[b])
            got = acc[b, h, :n]
            assert torch.equal(got[gone], acc0[b, h, :n][gone]), f"b{b} g{h}: an unreadable page's sums moved"
            d = (got.double() - acc0[b, h, :n].double() - want).abs()[~gone]
            lim = (tol + 2.0 ** -23 * (acc0[b, h, :n].double() + want))[~gone]
            assert (d <= lim).all(), f"b{b} g{h}: off by {float((d - lim).max()):.3e} too much"
            assert torch.equal(acc[b, h, n:], acc0[b, h, n:])


@pytest.mark.parametrize("T,G,P", [(70, 4, 16), (70, 4, 64), (33, 8, 32), (256, 1, 16), (60, 1, 16), (90, 1, 64)])
def test_tree_attention_with_pages_it_cannot_read(rkv, T, G, P):
    # one and two row slots of the tensor-core form, a middle page and the last, partial one
    g = C.gen(113)
    lens = [700, 0, 150]
    cache, K, V = C.make_cache(rkv, lens, 2, P, seed=112, room=40000)
    q, kt, vt = C.randn(g, 3, 2 * G, T, D), C.randn(g, 3, 2, T, D), C.randn(g, 3, 2, T, D)
    sees = C.ancestors(3, T, g)
    nodes = [T, T - 3, 1]
    for b in range(3):
        kt[b, :, nodes[b]:] = math.nan
        vt[b, :, nodes[b]:] = math.nan
        q[b, :, nodes[b]:] = math.nan
    pages = [2, 699 // P]
    cache.page_table[0, pages[0]] = cache.num_phys_pages
    cache.page_table[0, pages[1]] = -4
    out = torch.full((3, 2 * G, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 2 * G, T), 7.0, device="cuda")
    rkv.rkv_tree_attention(cache, q.cuda(), kt.cuda(), vt.cuda(), C.mask_words(sees).cuda(), out, lse=lse,
                           tree_len=_ints(nodes))
    assert _status(rkv, cache) == rkv.DEVERR_PAGE_ID
    out, lse = out.cpu(), lse.cpu()
    for b, n in enumerate(lens):
        at = [t for t in range(n) if b or t // P not in pages]
        t = nodes[b]
        shown = torch.cat([torch.ones(t, len(at), dtype=torch.bool), sees[b, :t, :t]], 1)
        assert (out[b, :, t:] == 7).all() and (lse[b, :, t:] == 7).all()
        for h in range(2 * G):
            k, v = torch.cat([K[b][h // G][at], kt[b, h // G, :t]]), torch.cat([V[b][h // G][at], vt[b, h // G, :t]])
            ref, l, w, Ew = C.attend(q[b, h, :t], k, v, shown)
            C.check_out(out[b, h, :t], ref, w, v, Ew, f"b{b} h{h}")
            C.check_lse(lse[b, h, :t], l, Ew, f"b{b} h{h}")


def test_tree_commit_changes_nothing_but_the_accepted_rows(rkv):
    lens, P, Hkv = [120, 120, 128, 9, 37], 16, 2
    cache, K, V = C.make_cache(rkv, lens, Hkv, P, seed=114, max_pages=8)
    g = C.gen(115)
    kt, vt = C.randn(g, 5, Hkv, 4, D), C.randn(g, 5, Hkv, 4, D)
    path = torch.tensor([[2, 4, 1], [0, 1, -1], [0, 1, 2], [0, 1, 2], [3, 3, 0]], dtype=torch.int32)
    pools = lambda: [t.cpu().view(torch.int16).clone() for t in (cache.k_pages, cache.v_pages, cache.kmax, cache.kmin)]  # noqa: E731
    want = pools()
    # refused: a node outside the tree (1), no room (2), a negative count (3); taken: 0 and 4
    m = [1, 3, 1, -1, 3]
    rkv.rkv_tree_commit(cache, kt.cuda(), vt.cuda(), path.cuda(), _ints(m))
    assert _status(rkv, cache) == rkv.DEVERR_TREE | rkv.DEVERR_CAPACITY
    assert cache.seq_len.tolist() == [121, 120, 128, 9, 40]
    table = cache.page_table.cpu()
    for b in (0, 4):
        for i in range(m[b]):
            pos, node = lens[b] + i, int(path[b, i])
            for pool, x in zip(want[:2], (kt, vt)):
                pool[int(table[b, pos // P]), :, pos % P] = x[b, :, node].view(torch.int16)
        rows = torch.cat([K[b], kt[b][:, path[b, :m[b]].long()]], 1)
        for pg in range(lens[b] // P, (lens[b] + m[b] - 1) // P + 1):
            x = rows[:, pg * P:(pg + 1) * P].float()
            want[2][b, :, :, pg] = x.amax(1).to(torch.bfloat16).view(torch.int16)
            want[3][b, :, :, pg] = x.amin(1).to(torch.bfloat16).view(torch.int16)
    for name, got, ref in zip(("k_pages", "v_pages", "kmax", "kmin"), pools(), want):
        assert torch.equal(got, ref), f"{name}: {int((got != ref).sum())} values differ"


def test_the_same_call_twice_gives_the_same_bits(rkv):
    """Parts of split units are joined in a fixed order: over every kernel."""
    g = C.gen(117)
    for lens, T, G, room in (([2000, 100], 3, 4, 0), ([5000, 100], 3, 4, 40000), ([5000, 0, 900], 30, 4, 40000),
                             ([5000, 900], 70, 4, 40000)):
        cache, K, V = C.make_cache(rkv, lens, 2, 16, seed=116, room=room)
        B = len(lens)
        q, kt, vt = C.randn(g, B, 2 * G, T, D).cuda(), C.randn(g, B, 2, T, D).cuda(), C.randn(g, B, 2, T, D).cuda()
        mask = C.mask_words(C.ancestors(B, T, g)).cuda()
        runs = []
        for _ in range(3):
            out = torch.zeros(B, 2 * G, T, D, dtype=torch.bfloat16, device="cuda")
            lse, acc = torch.zeros(B, 2 * G, T, device="cuda"), rkv.accum_sums(cache)
            one = torch.zeros(B, 2 * G, D, dtype=torch.bfloat16, device="cuda")
            rkv.rkv_tree_attention(cache, q, kt, vt, mask, out, lse=lse)
            rkv.rkv_decode_accum(cache, q[:, :, 0].contiguous(), one, acc)
            runs.append([out.cpu(), lse.cpu(), one.cpu(), acc.cpu()])
        for other in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(runs[0], other)), (lens, T)
        assert _status(rkv, cache) == 0


def _round(rkv, seed, lens, T, G, P=16, room=20000):
    """A cache of its own, what a round of decoding over it needs, and the round: tree, commit,
    the path's weights, a prompt's weights, one token, eviction in place."""
    Hkv, B = 2, len(lens)
    g = C.gen(seed)
    cache, _, _ = C.make_cache(rkv, lens, Hkv, P, seed=seed, room=room)
    q, kt, vt = C.randn(g, B, Hkv * G, T, D).cuda(), C.randn(g, B, Hkv, T, D).cuda(), C.randn(g, B, Hkv, T, D).cuda()
    mask = C.mask_words(C.ancestors(B, T, g)).cuda()
    path = torch.randint(0, T, (B, 5), generator=g).to(torch.int32).cuda()
    plen = torch.randint(1, 6, (B,), generator=g).to(torch.int32).cuda()
    rows = 150
    qr, lr = C.randn(g, B, Hkv * G, rows, D).cuda(), (torch.rand(B, Hkv * G, rows, generator=g) * 4 + 6).cuda()
    few = torch.full((B,), rows - 7, dtype=torch.int32, device="cuda")
    q1 = C.randn(g, B, Hkv * G, D).cuda()
    out = torch.zeros(B, Hkv * G, T, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(B, Hkv * G, T, device="cuda")
    one = torch.zeros(B, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    acc = rkv.accum_sums(cache)
    keep = [max(200, n - 3) for n in lens]
    kept = torch.zeros(B, Hkv, max(keep), dtype=torch.int32, device="cuda")
    size = (B, Hkv * G, Hkv)
    ws = [rkv.tree_workspace(*size, T, cache.max_pages, P), rkv.accum_rows_workspace(*size, T, cache.max_pages, P),
          rkv.accum_rows_workspace(*size, rows, cache.max_pages, P), rkv.accum_workspace(*size, cache.max_pages, P),
          rkv.evict_workspace(B, Hkv, max(keep))]

    def run():
        rkv.rkv_tree_attention(cache, q, kt, vt, mask, out, lse=lse, workspace=ws[0])
        rkv.rkv_tree_commit(cache, kt, vt, path, plen)
        rkv.rkv_accum_rows(cache, q, lse, acc, row_len=plen, row_ids=path, workspace=ws[1])
        rkv.rkv_accum_rows(cache, qr, lr, acc, row_len=few, workspace=ws[2])
        rkv.rkv_decode_accum(cache, q1, one, acc, workspace=ws[3])
        rkv.rkv_evict_accum(cache, acc, keep, 20, kept, workspace=ws[4])

    def state():
        assert _status(rkv, cache) == 0
        return [t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).clone() for t in
                (out, lse, one, acc, kept, cache.seq_len, cache.k_pages, cache.v_pages, cache.kmax, cache.kmin)]

    return run, state


SHAPES = [(201, [3000, 250, 900], 30, 4), (202, [2500], 70, 4), (203, [400, 700], 3, 4), (204, [5000, 300], 16, 8)]


def test_calls_on_several_streams_at_once(rkv):
    want = []
    for shape in SHAPES:
        run, state = _round(rkv, *shape)
        for _ in range(4):
            run()
        want.append(state())
    rounds = [_round(rkv, *shape) for shape in SHAPES]
    streams = [torch.cuda.Stream() for _ in SHAPES]
    torch.cuda.synchronize()
    for _ in range(4):
        for (run, _), s in zip(rounds, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for i, (_, state) in enumerate(rounds):
        for j, (a, b) in enumerate(zip(state(), want[i])):
            assert torch.equal(a, b), f"shape {i}, tensor {j}"


@pytest.mark.parametrize("shape", SHAPES)
def test_a_round_with_its_eviction_captured_and_replayed(rkv, shape):
    run, state = _round(rkv, *shape)
    for _ in range(4):
        run()
    want = state()
    run, state = _round(rkv, *shape)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    for j, (a, b) in enumerate(zip(state(), want)):
        assert torch.equal(a, b), f"tensor {j}"
