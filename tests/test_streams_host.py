"""Where the binding's calls take the workspaces they make for themselves (no GPU)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def rkv():
    from two_stage_kv_snapkv_gb300 import build_lib
    build_lib.build()
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


MAKERS = ["prefill_workspace", "prefill_chunk_workspace", "decode_workspace", "sparq_workspace", "tree_workspace",
          "accum_workspace", "accum_rows_workspace", "evict_workspace"]


def _calls(rkv, stream):
    c = SimpleNamespace(B=2, Hkv=2, page_size=16, max_pages=8, struct=rkv.RkvCacheStruct(), k_pages=torch.zeros(1))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, two = bf(2, 8, 128), [4, 4]
    return dict(
        prefill=lambda: rkv.rkv_prefill_evict(bf(2, 8, 8, 128), bf(2, 2, 40, 128), bf(2, 2, 40, 128), [40, 40], two, two, c,
                                              i32(2, 2, 4), stream=stream),
        chunk=lambda: rkv.rkv_prefill_chunk(bf(2, 8, 8, 128), bf(2, 2, 40, 128), bf(2, 2, 40, 128), [40, 40], [0, 0], two,
                                            two, c, i32(2, 2, 4), stream=stream),
        hsa=lambda: rkv.rkv_decode_hsa(c, q, two, two, f32(2, 8, 128), stream=stream),
        step=lambda: rkv.rkv_decode_step(c, q, bf(2, 2, 128), bf(2, 2, 128), two, two, f32(2, 8, 128), stream=stream),
        sparq=lambda: rkv.rkv_decode_sparq(c, q, two, two, f32(2, 8, 128), stream=stream),
        tree=lambda: rkv.rkv_tree_attention(c, bf(2, 8, 5, 128), bf(2, 2, 5, 128), bf(2, 2, 5, 128), i32(2, 5, 1),
                                            bf(2, 8, 5, 128), stream=stream),
        accum=lambda: rkv.rkv_decode_accum(c, q, bf(2, 8, 128), f32(2, 2, 128), stream=stream),
        rows=lambda: rkv.rkv_accum_rows(c, bf(2, 8, 5, 128), f32(2, 8, 5), f32(2, 2, 128), stream=stream),
        evict=lambda: rkv.rkv_evict_accum(c, f32(2, 2, 128), [5, 5], 0, i32(2, 2, 5), stream=stream))


@pytest.mark.parametrize("name", ["prefill", "chunk", "hsa", "step", "sparq", "tree", "accum", "rows", "evict"])
def test_a_workspace_belongs_to_the_stream_of_its_call(rkv, monkeypatch, name):
    # memory of the current stream may still be in use there when another stream writes to it
    side, inside, made = SimpleNamespace(cuda_stream=77), [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    def maker(*a, device=None, **kw):
        made.append(inside[-1] if inside else None)
        return torch.empty(8, dtype=torch.uint8)

    monkeypatch.setattr(torch.cuda, "stream", on)
    for m in MAKERS:
        monkeypatch.setattr(rkv, m, maker)
    done = []
    monkeypatch.setattr(rkv, "_lib", SimpleNamespace(**{
        f: lambda *a, f=f: done.append(f) or 0 for f in rkv.EXPORTED if f.startswith("rkv_")}))
    monkeypatch.setattr(rkv, "_call_on", lambda dev, stream, fn, *a: fn(*a))
    _calls(rkv, side)[name]()
    assert made == [side] and len(done) == 1
