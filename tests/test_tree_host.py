"""Refusals of the tree and accumulated-weight calls: nothing is launched (no GPU)."""
import ctypes

import pytest
import torch

VP = ctypes.c_void_p
F = ctypes.c_float


@pytest.fixture(scope="module")
def rkv():
    from two_stage_kv_snapkv_gb300 import build_lib
    build_lib.build()
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def _cache(rkv, **kw):
    base = dict(k_pages=0x10000, v_pages=0x20000, page_table=0x30000, seq_len=0x40000, kmax=0x50000,
                kmin=0x60000, error_word=0x70000, B=2, Hkv=2, head_dim=128, page_size=16, max_pages=64,
                num_phys_pages=128)
    base.update(kw)
    return rkv.RkvCacheStruct(**base)


def _refused(rkv, call, cases):
    before = rkv.rkv_launch_count()
    for kw, expect in cases:
        assert call(**kw) == getattr(rkv, "RKV_ERR_" + expect), (kw, rkv.rkv_last_error())
        assert rkv.rkv_last_error()
    assert rkv.rkv_launch_count() == before


def test_tree_attention_refusals(rkv):
    lib = rkv.lib()

    def call(c=None, q=0x100000, kt=0x200000, vt=0x300000, mask=0x400000, Hq=8, T=8, tl=None, scale=0.1, out=0x500000,
             lse=None, ws=0x600000, short=0):
        c = c or _cache(rkv)
        need = lib.rkv_tree_workspace_size(c.B, Hq, c.Hkv, T, c.max_pages, c.page_size)
        return lib.rkv_tree_attention(ctypes.byref(c), VP(q), VP(kt), VP(vt), VP(mask), Hq, T, VP(tl), F(scale), VP(out),
                                      VP(lse), VP(ws), max(need, 1) - short, None)

    _refused(rkv, call, [
        (dict(c=_cache(rkv, head_dim=64)), "UNSUPPORTED"), (dict(c=_cache(rkv, page_size=24)), "UNSUPPORTED"),
        (dict(c=_cache(rkv, max_pages=0)), "INVALID_ARG"), (dict(Hq=6), "UNSUPPORTED"), (dict(Hq=7), "INVALID_ARG"),
        (dict(Hq=32), "UNSUPPORTED"), (dict(T=0), "INVALID_ARG"), (dict(T=257), "INVALID_ARG"),
        (dict(q=None), "INVALID_ARG"), (dict(kt=None), "INVALID_ARG"), (dict(vt=None), "INVALID_ARG"),
        (dict(mask=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
        (dict(q=0x100008), "INVALID_ARG"), (dict(vt=0x300002), "INVALID_ARG"), (dict(mask=0x400002), "INVALID_ARG"),
        (dict(lse=0x700001), "INVALID_ARG"), (dict(tl=0x700002), "INVALID_ARG"),
        (dict(scale=0.0), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
        (dict(scale=float("inf")), "INVALID_ARG"), (dict(scale=1e-38), "INVALID_ARG"), (dict(scale=1e31), "INVALID_ARG"),
        (dict(short=1), "WORKSPACE")])


def test_tree_commit_refusals(rkv):
    lib = rkv.lib()

    def call(c=None, kt=0x200000, vt=0x300000, T=8, path=0x400000, stride=4, plen=0x500000):
        c = c or _cache(rkv)
        return lib.rkv_tree_commit(ctypes.byref(c), VP(kt), VP(vt), T, VP(path), stride, VP(plen), None)

    _refused(rkv, call, [
        (dict(c=_cache(rkv, error_word=0)), "INVALID_ARG"), (dict(kt=None), "INVALID_ARG"), (dict(vt=0x300004), "INVALID_ARG"),
        (dict(path=None), "INVALID_ARG"), (dict(plen=None), "INVALID_ARG"), (dict(path=0x400001), "INVALID_ARG"),
        (dict(T=0), "INVALID_ARG"), (dict(T=300), "INVALID_ARG"), (dict(stride=0), "INVALID_ARG"),
        (dict(stride=257), "INVALID_ARG")])


def test_decode_accum_refusals(rkv):
    lib = rkv.lib()

    def call(c=None, q=0x100000, Hq=8, scale=0.1, out=0x200000, lse=None, acc=0x300000, stride=1024, ws=0x400000, short=0):
        c = c or _cache(rkv)
        need = lib.rkv_accum_workspace_size(c.B, Hq, c.Hkv, c.max_pages, c.page_size)
        return lib.rkv_decode_accum(ctypes.byref(c), VP(q), Hq, F(scale), VP(out), VP(lse), VP(acc), stride, VP(ws),
                                    max(need, 1) - short, None)

    _refused(rkv, call, [
        (dict(c=_cache(rkv, B=257)), "INVALID_ARG"), (dict(Hq=6), "UNSUPPORTED"), (dict(q=None), "INVALID_ARG"),
        (dict(out=None), "INVALID_ARG"), (dict(acc=None), "INVALID_ARG"), (dict(acc=0x300002), "INVALID_ARG"),
        (dict(stride=1023), "INVALID_ARG"), (dict(out=0x200008), "INVALID_ARG"), (dict(lse=0x3), "INVALID_ARG"),
        (dict(scale=0.0), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"), (dict(short=1), "WORKSPACE")])


def test_accum_rows_refusals(rkv):
    lib = rkv.lib()

    def call(c=None, q=0x100000, lse=0x200000, Hq=8, T=8, rl=None, ids=None, stride=0, scale=0.1, acc=0x300000, acs=1024,
             ws=0x400000, short=0):
        c = c or _cache(rkv)
        need = lib.rkv_accum_rows_workspace_size(c.B, Hq, c.Hkv, T, c.max_pages, c.page_size)
        return lib.rkv_accum_rows(ctypes.byref(c), VP(q), VP(lse), Hq, T, VP(rl), VP(ids), stride, F(scale), VP(acc), acs,
                                  VP(ws), max(need, 1) - short, None)

    _refused(rkv, call, [
        (dict(c=_cache(rkv, kmax=0)), "INVALID_ARG"), (dict(Hq=12), "UNSUPPORTED"), (dict(q=None), "INVALID_ARG"),
        (dict(lse=None), "INVALID_ARG"), (dict(T=0), "INVALID_ARG"), (dict(T=(1 << 20) + 1), "INVALID_ARG"),
        (dict(ids=0x500000, stride=0), "INVALID_ARG"), (dict(ids=0x500001, stride=4), "INVALID_ARG"),
        (dict(rl=0x500002), "INVALID_ARG"), (dict(acs=1000), "INVALID_ARG"), (dict(acc=None), "INVALID_ARG"),
        (dict(scale=float("nan")), "INVALID_ARG"), (dict(short=1), "WORKSPACE")])


def test_evict_accum_refusals(rkv):
    lib = rkv.lib()
    other = dict(k_pages=0x110000, v_pages=0x120000, page_table=0x130000, seq_len=0x140000, kmax=0x150000,
                 kmin=0x160000, error_word=0x170000)

    def call(c=None, acc=0x200000, acs=1024, keep=(100, 50), recent=10, kept=0x300000, stride=100, dst=None, dacc=None,
             das=0, ws=0x400000, short=0):
        c = c or _cache(rkv)
        need = lib.rkv_evict_workspace_size(c.B, c.Hkv, max(1, max(keep)), 1 if dst is None else 0)
        return lib.rkv_evict_accum(ctypes.byref(c), VP(acc), acs, (ctypes.c_int32 * len(keep))(*keep), recent, VP(kept),
                                   stride, ctypes.byref(dst) if dst is not None else None, VP(dacc), das, VP(ws),
                                   need - short, None)

    dst = _cache(rkv, max_pages=8, **other)
    _refused(rkv, call, [
        (dict(c=_cache(rkv, v_pages=0)), "INVALID_ARG"), (dict(acc=None), "INVALID_ARG"), (dict(acs=512), "INVALID_ARG"),
        (dict(keep=(100, 0)), "INVALID_ARG"), (dict(keep=(1025, 50)), "INVALID_ARG"), (dict(recent=51), "INVALID_ARG"),
        (dict(recent=-1), "INVALID_ARG"), (dict(stride=99), "INVALID_ARG"), (dict(kept=None), "INVALID_ARG"),
        (dict(kept=0x300002), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"), (dict(short=1), "WORKSPACE"),
        (dict(dst=dst), "INVALID_ARG"), (dict(dacc=0x500000, das=1024), "INVALID_ARG"),
        (dict(dst=dst, dacc=0x500000, das=127), "INVALID_ARG"),
        (dict(dst=dst, dacc=0x500000, das=128, keep=(129, 50), stride=200), "INVALID_ARG"),
        (dict(dst=dst, dacc=0x200000, das=128), "INVALID_ARG"),
        (dict(dst=_cache(rkv, max_pages=8), dacc=0x500000, das=128), "INVALID_ARG"),
        (dict(dst=_cache(rkv, max_pages=8, page_size=32, **other), dacc=0x500000, das=256), "INVALID_ARG"),
        (dict(dst=_cache(rkv, max_pages=8, B=1, **other), dacc=0x500000, das=128), "INVALID_ARG"),
        (dict(c=_cache(rkv, max_pages=16384, page_size=64), acs=1 << 20), "UNSUPPORTED"),
        (dict(c=_cache(rkv, Hkv=40000, num_phys_pages=64)), "UNSUPPORTED")])


def test_workspace_sizes_of_bad_sizes_are_zero(rkv):
    lib = rkv.lib()
    assert lib.rkv_tree_workspace_size(0, 8, 2, 8, 64, 16) == 0
    assert lib.rkv_accum_workspace_size(1, 8, 2, 0, 16) == 0
    assert lib.rkv_accum_rows_workspace_size(1, 8, 2, 0, 64, 16) == 0
    assert lib.rkv_evict_workspace_size(1, 2, 0, 1) == 0


class _CpuCache:
    """What the binding's checks look at of a PagedCache."""

    def __init__(self):
        self.B, self.Hkv, self.page_size, self.max_pages = 2, 2, 16, 8
        self.k_pages = torch.zeros(1)


def test_binding_refuses_wrong_shapes_types_and_devices(rkv):
    c = _CpuCache()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    tree = dict(q=bf(2, 8, 5, 128), k_tree=bf(2, 2, 5, 128), v_tree=bf(2, 2, 5, 128), tree_mask=i32(2, 5, 1),
                out=bf(2, 8, 5, 128))
    for bad in (dict(q=bf(2, 8, 128)), dict(q=f32(2, 8, 5, 128)), dict(k_tree=bf(2, 2, 4, 128)), dict(tree_mask=i32(2, 5, 2)),
                dict(tree_mask=torch.zeros(2, 5, 1, dtype=torch.int64)), dict(out=f32(2, 8, 5, 128)),
                dict(lse=f32(2, 8)), dict(tree_len=i32(3)), dict(q=bf(3, 8, 5, 128)),
                dict(v_tree=bf(2, 2, 5, 128).to("meta"))):
        with pytest.raises(ValueError):
            rkv.rkv_tree_attention(c, **{**tree, **bad})
    with pytest.raises(ValueError):
        rkv.rkv_tree_commit(c, bf(2, 2, 5, 128), bf(2, 2, 5, 128), i32(2, 3), i32(1))
    with pytest.raises(ValueError):
        rkv.rkv_decode_accum(c, bf(2, 8, 128), bf(2, 8, 128), f32(2, 3, 128))
    with pytest.raises(ValueError):
        rkv.rkv_decode_accum(c, bf(2, 8, 64), bf(2, 8, 64), f32(2, 2, 128))
    with pytest.raises(ValueError):
        rkv.rkv_accum_rows(c, bf(2, 8, 5, 128), f32(2, 8, 4), f32(2, 2, 128))
    with pytest.raises(ValueError):
        rkv.rkv_accum_rows(c, bf(2, 8, 5, 128), f32(2, 8, 5), f32(2, 2, 128), row_ids=i32(2))
    with pytest.raises(ValueError):
        rkv.rkv_evict_accum(c, f32(2, 2, 128), [5], 0, i32(2, 2, 5))
    with pytest.raises(ValueError):
        rkv.rkv_evict_accum(c, f32(2, 2, 128), [5, 5], 0, i32(2, 5))
