"""The 8-bit cache's write side against its definition, code for code (tests/q8_check.py)."""
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


def _rows(g, B, H, T, loud=True):
    x = C.randn(g, B, H, T, C.D)
    if loud:
        x[..., 3] *= 9
        x *= torch.exp2(torch.randint(-6, 7, (B, H, T, 1), generator=g).float()).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,P,steps", [
    (1, 1, 16, [1] * 20), (3, 2, 32, [5, 1, 16, 3, 1, 17, 2]), (2, 9, 64, [16, 1, 63, 70, 1, 200]),
    (5, 8, 16, [100, 1, 4, 33]), (1, 3, 64, [1, 1, 1, 40, 130])])
def test_appends_of_every_length(rkv, B, H, P, steps, fmt):
    g = C.gen(B * 1000 + P)
    cache = C.cache8(rkv, B, H, P, -(-sum(steps) // P) + 1, fmt, seed=P)
    model = C.Model(B, H, P, fmt)
    for i, T in enumerate(steps):
        k, v = _rows(g, B, H, T), _rows(g, B, H, T)
        new = [T - (b + i) % 3 * T // 3 for b in range(B)] if B > 1 else [T]
        if B > 2:
            new[(i + 1) % B] = 0
        raw = [t.view(torch.uint8).clone() for t in (cache.k_codes, cache.v_codes)]
        rkv.rkv_q8_append(cache, k.cuda(), v.cuda(), new_len=None if new == [T] * B else _ints(new))
        for b in range(B):
            model.append(b, k[b, :, :new[b]], v[b, :, :new[b]])
        model.check(cache, f"step {i}")
        # nothing else was written
        for t, old in zip((cache.k_codes, cache.v_codes), raw):
            keep = torch.ones(t.shape[0], P, dtype=torch.bool)
            for b in range(B):
                pt = cache.page_table[b].cpu()
                for j in range(-(-model.n[b] // P)):
                    keep[int(pt[j]), :model.n[b] - j * P] = False
            keep = keep.cuda()[:, None, :, None].expand(t.shape)
            assert torch.equal(t.view(torch.uint8)[keep], old[keep])
        assert (cache.sync == 0).all()
    assert rkv.rkv_read_device_error(cache.error_word) == (rkv.RKV_OK, 0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rounding_and_scales_at_their_borders(rkv, fmt):
    """Magnitudes on both sides of a power of two times the largest code, ties, zeros, the
    smallest and the largest numbers."""
    top = C.LARGEST[fmt]
    rows = []
    for x in (top, top * 2 ** -20, top * (1 + 2 ** -7), top * (1 - 2 ** -8), 1.0, 2.0 ** -126, 2.0 ** -133, 3.3e38, 0.0):
        row = torch.zeros(C.D)
        row[0] = x
        row[1:64] = x * torch.arange(63) / 64.0
        row[64:] = -x * torch.linspace(0, 1, 64) ** 4
        rows.append(row)
    x = torch.stack(rows).to(torch.bfloat16).view(1, len(rows), 1, C.D)
    cache = C.cache8(rkv, 1, len(rows), 16, 8, fmt)
    model = C.Model(1, len(rows), 16, fmt)
    y = (x.float() * 2.0 ** -3).to(torch.bfloat16)
    for k, v in ((y, x), (x, y)):  # the second token raises one scale and not the other
        rkv.rkv_q8_append(cache, k.cuda(), v.cuda())
        model.append(0, k[0], v[0])
        model.check(cache)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [3, 40])
def test_pages_with_a_nan_or_an_infinity(rkv, fmt, T):
    g = C.gen(T)
    cache, model = C.cache8(rkv, 1, 2, 32, 8, fmt), C.Model(1, 2, 32, fmt)
    for step, bad in enumerate((None, math.nan, None, None, -math.inf, None)):
        k, v = _rows(g, 1, 2, T), _rows(g, 1, 2, T)
        if bad is not None:
            (k if step == 1 else v)[0, 1, T // 2, 77] = bad
        rkv.rkv_q8_append(cache, k.cuda(), v.cuda())
        model.append(0, k[0], v[0])
        model.check(cache, f"step {step}")
    gone = [math.isnan(x[1]) for x in model.blocks[0][1]]
    assert any(gone) and not any(math.isnan(x[1]) for x in model.blocks[0][0])


def test_rows_where_a_projection_leaves_them(rkv):
    B, H, T = 2, 4, 21
    g = C.gen(4)
    x = C.randn(g, B, T, 2 * H + 3, C.D).cuda()
    k, v = x[:, :, 1:1 + H].transpose(1, 2), x[:, :, H + 2:2 * H + 2].transpose(1, 2)
    cache, model = C.cache8(rkv, B, H, 16, 8, "e4m3"), C.Model(B, H, 16, "e4m3")
    rkv.rkv_q8_append(cache, k, v)
    for b in range(B):
        model.append(b, k[b].cpu(), v[b].cpu())
    model.check(cache)


def test_what_cannot_be_written(rkv):
    """A sequence with a bad count or no room stays as it is; a bad page is skipped."""
    g = C.gen(6)
    for T in (4, 40):
        cache, model = C.cache8(rkv, 4, 2, 16, 8, "e4m3"), C.Model(4, 2, 16, "e4m3")
        cache.seq_len.copy_(_ints([0, 0, 128 - T + 1, -1]))
        k, v = _rows(g, 4, 2, T), _rows(g, 4, 2, T)
        rkv.rkv_q8_append(cache, k.cuda(), v.cuda(), new_len=_ints([T, T + 1, T, 1]))
        assert rkv.rkv_read_device_error(cache.error_word)[1] == rkv.DEVERR_TREE | rkv.DEVERR_CAPACITY
        model.append(0, k[0], v[0])
        assert cache.seq_len.tolist() == [T, 0, 128 - T + 1, -1]
        cache.seq_len.copy_(_ints([T, 0, 0, 0]))
        model.check(cache)
        other = cache.k_codes.view(torch.uint8).clone()
        cache.page_table[1, 0] = cache.num_phys_pages
        rkv.rkv_q8_append(cache, k.cuda(), v.cuda(), new_len=_ints([0, T, 0, 0]))
        assert rkv.rkv_read_device_error(cache.error_word)[1] == rkv.DEVERR_PAGE_ID
        assert cache.seq_len.tolist() == [T, T, 0, 0]
        if T <= 16:
            assert torch.equal(cache.k_codes.view(torch.uint8), other)
        assert (cache.sync == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("P,lens", [(16, [33]), (32, [1, 0, 95]), (64, [300, 64, 0, 1000, 7])])
def test_a_bf16_cache_becomes_an_8_bit_one(rkv, P, lens, fmt):
    import dense_check as DC
    H = 3
    src, K, V = DC.make_cache(rkv, lens, H, P, seed=P)
    cache, model = C.cache8(rkv, len(lens), H, P, src.max_pages + 8, fmt, seed=1), C.Model(len(lens), H, P, fmt)
    cache.seq_len.fill_(9)
    before = src.k_pages.view(torch.int16).clone()
    rkv.rkv_q8_load(cache, src)
    for b in range(len(lens)):
        model.append(b, K[b], V[b])
    model.check(cache)
    assert torch.equal(src.k_pages.view(torch.int16), before)
    # appending one row at a time gives the same up to codes that were rounded twice
    rkv.rkv_q8_append(cache, K[0][:, :1].unsqueeze(0).expand(len(lens), -1, -1, -1).contiguous().cuda(),
                      V[0][:, :1].unsqueeze(0).expand(len(lens), -1, -1, -1).contiguous().cuda())
    for b in range(len(lens)):
        model.append(b, K[0][:, :1], V[0][:, :1])
    model.check(cache)
    # lengths that neither side holds, pages that cannot be read
    src.seq_len[0] = src.max_pages * P + 1
    if len(lens) > 2:
        src.page_table[2, 0] = -5
    rkv.rkv_q8_load(cache, src)
    want = rkv.DEVERR_CAPACITY | (rkv.DEVERR_PAGE_ID if len(lens) > 2 and lens[2] else 0)
    assert rkv.rkv_read_device_error(cache.error_word)[1] == want
    assert cache.seq_len.tolist() == [0] + lens[1:]
    if len(lens) > 2 and lens[2]:
        assert torch.isnan(cache.k_scale[cache.page_table[2, 0].long()]).all()


def test_far_pages(rkv):
    """Codes behind 2^31 bytes."""
    H, P, phys = 8, 64, 40000  # 2.6 GB of codes in each pool
    pt = torch.arange(phys - 8, phys, dtype=torch.int32, device="cuda").view(1, 8)
    cache = rkv.PagedCache8(1, H, P, 8, "cuda", page_table=pt, num_phys_pages=phys)
    model = C.Model(1, H, P, "e4m3")
    g = C.gen(8)
    for T in (70, 3):
        k, v = C.randn(g, 1, H, T, C.D), C.randn(g, 1, H, T, C.D)
        rkv.rkv_q8_append(cache, k.cuda(), v.cuda())
        model.append(0, k[0], v[0])
    assert cache.seq_len.tolist() == [73]
    got_k, got_v = cache.token_kv(0)
    for g_ in range(H):
        ref = torch.cat([x[0] * x[1] for x in model.blocks[0][g_]])
        assert torch.equal(got_k[g_].double().cpu(), ref)
