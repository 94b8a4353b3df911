"""Refusals and host-side arithmetic of the page, rotary and 8-bit calls: no GPU, nothing is launched."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def rkv():
    from two_stage_kv_snapkv_gb300 import build_lib
    build_lib.build()
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def _cache8(rkv, **kw):
    base = dict(k_codes=0x10000, v_codes=0x20000, k_scale=0x30000, v_scale=0x40000, page_table=0x50000, seq_len=0x60000,
                error_word=0x70000, sync=0x80000, B=2, Hkv=2, head_dim=128, page_size=16, max_pages=64,
                num_phys_pages=128, format=0)
    base.update(kw)
    return rkv.RkvCache8Struct(**base)


def _pool(rkv, **kw):
    base = dict(free_pages=0x10000, free_count=0x20000, held=0x30000, sync=0x40000, error_word=0x50000, num_phys_pages=64)
    base.update(kw)
    return rkv.RkvPagePoolStruct(**base)


def _st(*v):
    return (ctypes.c_int64 * 3)(*v)


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
CACHES = [(dict(k_codes=0), INVALID), (dict(v_scale=0), INVALID), (dict(sync=0), INVALID), (dict(k_codes=0x10008), INVALID),
          (dict(k_scale=0x30002), INVALID), (dict(B=0), INVALID), (dict(B=257), INVALID), (dict(Hkv=0), INVALID),
          (dict(head_dim=64), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(max_pages=12), INVALID),
          (dict(max_pages=16392), UNSUPPORTED), (dict(num_phys_pages=0), INVALID),
          (dict(num_phys_pages=1 << 27), UNSUPPORTED), (dict(format=2), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_every_call_refuses_a_bad_cache(rkv, kw, status):
    lib = rkv.lib()
    c = ctypes.byref(_cache8(rkv, **kw))
    assert lib.rkv_q8_append(c, 0x1000, _st(0, 0, 128), 0x2000, _st(0, 0, 128), 1, None, None) == status
    assert lib.rkv_q8_attention(c, 0x1000, 8, 1, None, 0.1, 0x2000, None, 0x3000, 1 << 40, None) == status
    src = rkv.RkvCacheStruct(k_pages=0x10000, v_pages=0x20000, page_table=0x30000, seq_len=0x40000, kmax=0x50000,
                             kmin=0x60000, error_word=0x70000, B=2, Hkv=2, head_dim=128, page_size=16, max_pages=64,
                             num_phys_pages=128)
    assert lib.rkv_q8_load(c, ctypes.byref(src), None) == status
    assert rkv.rkv_last_error()


@pytest.mark.parametrize("args,status", [
    ((None, _st(0, 0, 128), 0x2000, _st(0, 0, 128), 1, None), INVALID),
    ((0x1008, _st(0, 0, 128), 0x2000, _st(0, 0, 128), 1, None), INVALID),
    ((0x1000, None, 0x2000, _st(0, 0, 128), 1, None), INVALID),
    ((0x1000, _st(0, 0, 132), 0x2000, _st(0, 0, 128), 1, None), INVALID),
    ((0x1000, _st(0, 0, 128), 0x2000, _st(0, -128, 128), 1, None), INVALID),
    ((0x1000, _st(0, 0, 128), 0x2000, _st(0, 0, 128), 0, None), INVALID),
    ((0x1000, _st(0, 0, 128), 0x2000, _st(0, 0, 128), (1 << 20) + 1, None), INVALID),
    ((0x1000, _st(0, 0, 128), 0x2000, _st(0, 0, 128), 1, 0x3002), INVALID)])
def test_append_refuses(rkv, args, status):
    assert rkv.lib().rkv_q8_append(ctypes.byref(_cache8(rkv)), *args, None) == status


def test_load_refuses(rkv):
    lib = rkv.lib()
    base = dict(k_pages=0x10000, v_pages=0x20000, page_table=0x30000, seq_len=0x40000, kmax=0x50000, kmin=0x60000,
                error_word=0x70000, B=2, Hkv=2, head_dim=128, page_size=16, max_pages=64, num_phys_pages=128)
    for kw in (dict(B=3), dict(Hkv=4), dict(page_size=32), dict(seq_len=0x60000), dict(k_pages=0)):
        assert lib.rkv_q8_load(ctypes.byref(_cache8(rkv)), ctypes.byref(rkv.RkvCacheStruct(**{**base, **kw})), None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(q=0x1004), INVALID),
    (dict(lse=0x2002), INVALID), (dict(rows=0x2001), INVALID), (dict(Hq=3), INVALID), (dict(Hq=32), UNSUPPORTED),
    (dict(T=0), INVALID), (dict(T=(1 << 20) + 1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=1e31), INVALID), (dict(scale=-1.0), INVALID), (dict(ws_bytes=16), WORKSPACE)])
def test_attention_refuses(rkv, kw, status):
    a = dict(q=0x1000, Hq=8, T=1, rows=None, scale=0.1, out=0x2000, lse=None, ws=0x3000, ws_bytes=1 << 40)
    a.update(kw)
    got = rkv.lib().rkv_q8_attention(ctypes.byref(_cache8(rkv)), a["q"], a["Hq"], a["T"], a["rows"], a["scale"], a["out"],
                                     a["lse"], a["ws"], a["ws_bytes"], None)
    assert got == status


def test_attention_refuses_rows_beyond_31_bits(rkv):
    c = _cache8(rkv, B=256, Hkv=8, page_size=16, num_phys_pages=1024)
    assert rkv.lib().rkv_q8_attention(ctypes.byref(c), 0x1000, 64, 1 << 20, None, 0.1, 0x2000, None, 0x3000, 1 << 60,
                                      None) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(free_pages=0), INVALID), (dict(held=0x30001), INVALID), (dict(num_phys_pages=0), INVALID),
    (dict(num_phys_pages=1 << 28), UNSUPPORTED)])
def test_reserve_refuses_a_bad_pool(rkv, kw, status):
    got = rkv.lib().rkv_reserve_pages(ctypes.byref(_pool(rkv, **kw)), 0x1000, 2, 64, 16, 0x2000, None, None, 0, None,
                                      0x3000, 0x4000, None)
    assert got == status


@pytest.mark.parametrize("args,status", [
    ((None, 2, 64, 16, 0x2000, None, None, 0, None, 0x3000, 0x4000), INVALID),
    ((0x1000, 0, 64, 16, 0x2000, None, None, 0, None, 0x3000, 0x4000), INVALID),
    ((0x1000, 257, 64, 16, 0x2000, None, None, 0, None, 0x3000, 0x4000), INVALID),
    ((0x1000, 2, 60, 16, 0x2000, None, None, 0, None, 0x3000, 0x4000), INVALID),
    ((0x1000, 2, 16392, 16, 0x2000, None, None, 0, None, 0x3000, 0x4000), UNSUPPORTED),
    ((0x1000, 2, 64, 17, 0x2000, None, None, 0, None, 0x3000, 0x4000), UNSUPPORTED),
    ((0x1000, 2, 64, 16, None, None, None, 0, None, 0x3000, 0x4000), INVALID),
    ((0x1000, 2, 64, 16, 0x2000, 0x2100, None, 0, 0x2200, 0x3000, 0x4000), INVALID),
    ((0x1000, 2, 64, 16, 0x2000, 0x2100, 0x2400, 8, None, 0x3000, 0x4000), INVALID),
    ((0x1000, 2, 64, 16, 0x2000, 0x2100, 0x2400, -1, 0x2200, 0x3000, 0x4000), INVALID),
    ((0x1000, 2, 64, 16, 0x2000, None, None, 0, None, None, 0x4000), INVALID)])
def test_reserve_refuses(rkv, args, status):
    assert rkv.lib().rkv_reserve_pages(ctypes.byref(_pool(rkv)), *args, None) == status


def _frequency(i, rot, base, scaling, factor, n0, low, high):
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "none":
        return f
    r = n0 * f / (2 * math.pi)
    if scaling == "logs":
        r, low, high = math.log(r), math.log(low), math.log(high)
    w = min(1.0, max(0.0, (r - low) / (high - low)))
    return f * (w + (1 - w) / factor)


@pytest.mark.parametrize("scaling", ["none", "linear", "turns", "logs"])
@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (16, 1.5), (112, 1e9)])
def test_rotary_frequencies(rkv, rot, base, scaling):
    p = rkv.rotary_plan(rot, base, interleaved=True, scaling=scaling, factor=8.0, original_len=4096, low=1.0, high=32.0,
                        amplitude=1.5)
    assert p.rot_dim == rot and p.interleaved == 1 and p.amplitude == 1.5
    for i in range(64):
        if i >= rot // 2:
            assert p.turns[i] == 0
            continue
        f = _frequency(i, rot, base, scaling, 8.0, 4096, 1.0, 32.0)
        # a few roundings of 2^-53, and half of the fraction's last place
        assert abs(p.turns[i] / 2.0 ** 64 * 2 * math.pi - f) <= 2.0 ** -50 * f + 2.0 ** -62
    # the ramp's ends: untouched above `high` turns, divided by the factor below `low`
    if scaling in ("turns", "logs"):
        q = rkv.rotary_plan(rot, base)
        for i in range(rot // 2):
            turns = 4096 * base ** (-2.0 * i / rot) / (2 * math.pi)
            if turns > 33:
                assert p.turns[i] == q.turns[i]
            if turns < 0.99:
                assert abs(p.turns[i] * 8 - q.turns[i]) <= 8 + q.turns[i] * 2.0 ** -50


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), UNSUPPORTED), (dict(rot_dim=24), UNSUPPORTED), (dict(rot_dim=144), UNSUPPORTED),
    (dict(base=1.0), INVALID), (dict(base=math.inf), INVALID), (dict(base=math.nan), INVALID),
    (dict(scaling="linear", factor=0.5), INVALID), (dict(scaling="turns", factor=2.0, original_len=0), INVALID),
    (dict(scaling="logs", factor=2.0, original_len=10, low=4.0, high=4.0), INVALID),
    (dict(scaling="logs", factor=2.0, original_len=10, low=0.0), INVALID), (dict(amplitude=0.0), INVALID),
    (dict(amplitude=math.inf), INVALID)])
def test_rotary_plans_that_cannot_be(rkv, kw, status):
    with pytest.raises(rkv.RkvError) as e:
        rkv.rotary_plan(**kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q_out=None), dict(k=None), dict(ko=None), dict(B=0), dict(T=0), dict(Hq=0), dict(Hkv=0),
    dict(q=0x1008), dict(pos=None), dict(pos=0x5002), dict(qs=_st(0, 0, 4)), dict(qs=None), dict(kos=_st(0, 64, 128)),
    dict(qos=_st(0, 0, 128)), dict(qos=_st(8 * 128, 0, 128)), dict(qos=_st(1 << 20, 128, 512)),
    dict(kos=_st(1 << 20, 1 << 10, 64))])
def test_rotary_refuses(rkv, kw):
    plan = rkv.rotary_plan()
    a = dict(q=0x1000, qs=_st(1 << 20, 1 << 10, 128), k=0x2000, ks=_st(1 << 20, 1 << 10, 128), B=2, Hq=8, Hkv=2, T=8,
             pos=0x5000, q_out=0x3000, qos=_st(1 << 20, 1 << 10, 128), ko=0x4000, kos=_st(1 << 20, 1 << 10, 128))
    a.update(kw)
    got = rkv.lib().rkv_rotary(ctypes.byref(plan), a["q"], a["qs"], a["k"], a["ks"], a["B"], a["Hq"], a["Hkv"], a["T"],
                               a["pos"], 0, 0, a["q_out"], a["qos"], a["ko"], a["kos"], None)
    assert got == INVALID


def test_rotary_refuses_a_plan_that_was_not_filled(rkv):
    st = _st(1 << 20, 1 << 10, 128)
    got = rkv.lib().rkv_rotary(ctypes.byref(rkv.RkvRotaryPlan()), 0x1000, st, None, None, 1, 1, 0, 1, 0x5000, 0, 0, 0x3000,
                               st, None, None, None)
    assert got == INVALID


def test_the_binding_checks_tensors(rkv):
    cpu = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rkv.rkv_rotary(rkv.rotary_plan(), cpu, None, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        rkv.rkv_rotary(rkv.rotary_plan(), cpu[0], None, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        rkv.rotary_plan(scaling="other")
    with pytest.raises(ValueError):
        rkv.PagedCache8(1, 1, 16, 8, "cpu", fmt="e5m2")
    with pytest.raises(ValueError):
        rkv.PagedCache8(1, 1, 16, 8, "cpu", page_table=torch.zeros(1, 16, dtype=torch.int32))
    cache = rkv.PagedCache8(1, 2, 16, 8, "cpu")
    with pytest.raises(ValueError):
        rkv.rkv_q8_append(cache, cpu.float(), cpu)
    with pytest.raises(ValueError):
        rkv.rkv_q8_append(cache, cpu, cpu[:, :1])
    with pytest.raises(ValueError):
        rkv.rkv_q8_append(cache, torch.zeros(1, 2, 1, 256, dtype=torch.bfloat16)[..., ::2], cpu)
    with pytest.raises(ValueError):
        rkv.rkv_q8_attention(cache, cpu[0], cpu)
    with pytest.raises(ValueError):
        rkv.rkv_q8_attention(cache, cpu, cpu.float())
    pool = rkv.PagePool(8, 1, "cpu")
    with pytest.raises(ValueError):
        rkv.rkv_reserve_pages(pool, torch.zeros(8, dtype=torch.int32), 16, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        rkv.rkv_reserve_pages(pool, torch.zeros(1, 8, dtype=torch.int32), 16, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        rkv.PagePool(8, 1, "cpu", free_pages=torch.zeros(7, dtype=torch.int32))


def test_workspace_sizes(rkv):
    lib = rkv.lib()
    assert lib.rkv_q8_workspace_size(0, 8, 2, 1, 8, 16) == 0
    small, large = lib.rkv_q8_workspace_size(1, 8, 2, 1, 8, 16), lib.rkv_q8_workspace_size(1, 8, 2, 1000, 8, 16)
    assert 0 < small <= large


def test_products_given_up_are_waited_for_in_the_tiles_of_codes():
    # as for the other tensor-core kernels: after a timeout a commit behind the last product is
    # waited for before TMEM is freed; and a warp that gives up frees its partner's barrier
    import os
    import re

    from two_stage_kv_snapkv_gb300 import build_lib
    text = open(os.path.join(build_lib.CSRC, "rkv_q8_tiles.cu")).read()
    stop = text.index("if (abort_flag) {")
    branch = text[stop:text.index("tmem_dealloc(", stop)]
    assert "tc_commit_if(elect_lane(), &sh.drained);" in branch and "mbar_wait(&sh.drained, 0);" in branch
    assert text.count("mbar_init(&sh.drained, 1)") == 1
    reds, leave = text.count("barrier.cta.red"), re.search(r"if \(!ok\) asm volatile\(\"barrier\.cta\.arrive", text)
    assert reds == 1 and leave
