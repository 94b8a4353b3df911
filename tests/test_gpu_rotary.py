"""Rotary positions against the formula in fp64.

Bound: the result is rounded once to bf16 (2^-8 of it at most).  Before that an angle's part of
a turn is cut to 32 bits and rounded to fp32 (2^-24 of at most pi), sincospif is off by an
ulp or two, the amplitude, two products and a sum round: 2^-20 of amplitude (|a| + |b|) covers
them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128
SCALINGS = {"none": {}, "linear": dict(factor=4.0), "turns": dict(factor=8.0, original_len=8192, low=1.0, high=4.0),
            "logs": dict(factor=32.0, original_len=4096, low=1.0, high=32.0, amplitude=1.25)}


@pytest.fixture(scope="module")
def rkv():
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def frequencies(rot, base, scaling):
    p, out = SCALINGS[scaling], []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= p["factor"]
        elif scaling != "none":
            r = p["original_len"] * f / (2 * math.pi)
            lo, hi = p["low"], p["high"]
            if scaling == "logs":
                r, lo, hi = math.log(r), math.log(lo), math.log(hi)
            w = min(1.0, max(0.0, (r - lo) / (hi - lo)))
            f *= w + (1 - w) / p["factor"]
        out.append(f)
    return out


def check(x, got, pos, rot, base, inter, scaling, inverse=False):
    """x, got [B, H, T, D]; pos [B, T] int64."""
    x, got = x.double(), got.double()
    amp = SCALINGS[scaling].get("amplitude", 1.0)
    a = pos.double()[:, :, None] * torch.tensor(frequencies(rot, base, scaling), dtype=torch.float64, device=x.device)
    cos, sin = (torch.cos(a) * amp)[:, None], (torch.sin(a) * (-amp if inverse else amp))[:, None]
    if inter:
        u, v = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    else:
        u, v = torch.arange(rot // 2), torch.arange(rot // 2) + rot // 2
    p, q = x[..., u], x[..., v]
    for ref, at in ((p * cos - q * sin, u), (q * cos + p * sin, v)):
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * amp * (p.abs() + q.abs())
        bad = (got[..., at] - ref).abs() > tol
        assert not bad.any(), f"{int(bad.sum())} off, worst {float(((got[..., at] - ref).abs() - tol).max()):.3e}"
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("B,Hq,Hkv,T,rot", [(1, 1, 1, 1, 128), (2, 8, 1, 33, 64), (3, 32, 8, 5, 96), (1, 5, 3, 100, 16),
                                            (2, 9, 9, 65, 112)])
def test_against_the_formula(rkv, B, Hq, Hkv, T, rot, scaling, inter):
    g = torch.Generator(device="cuda").manual_seed(B * 100 + T)
    q = torch.randn(B, Hq, T, D, generator=g, device="cuda").bfloat16()
    k = torch.randn(B, Hkv, T, D, generator=g, device="cuda").bfloat16()
    plan = rkv.rotary_plan(rot, 10000.0, interleaved=inter, scaling=scaling, **SCALINGS[scaling])
    at = torch.randint(0, 1 << 20, (B,), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    rkv.rkv_rotary(plan, q, k, at, qo, ko)
    pos = at.long()[:, None] + torch.arange(T, device="cuda")
    check(q, qo, pos, rot, 10000.0, inter, scaling)
    check(k, ko, pos, rot, 10000.0, inter, scaling)
    # a position for every token, in place, and back again
    each = torch.randint(-5000, 1 << 24, (B, T), generator=g, device="cuda", dtype=torch.int32)
    q2, k2 = q.clone(), k.clone()
    rkv.rkv_rotary(plan, q2, k2, each)
    check(q, q2, each.long(), rot, 10000.0, inter, scaling)
    check(k, k2, each.long(), rot, 10000.0, inter, scaling)
    q3 = torch.empty_like(q)
    rkv.rkv_rotary(plan, q2, None, each, q3, inverse=True)
    check(q2, q3, each.long(), rot, 10000.0, inter, scaling, inverse=True)


@pytest.mark.parametrize("pos", [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789])
def test_far_positions(rkv, pos):
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(1, 4, 1, D, generator=g, device="cuda").bfloat16()
    plan = rkv.rotary_plan(128, 500000.0)
    out = torch.empty_like(q)
    at = torch.tensor([pos], dtype=torch.int32, device="cuda")
    rkv.rkv_rotary(plan, q, None, at, out)
    # cos and sin of a far angle: reduced with integers, 2 pi to 200 bits
    two_pi = 0x6487ED5110B4611A62633145C06E0E68948127044533E63A0105DF531D89CD91  # 2 pi 2^252
    x, y = q.double(), out.double()
    for i, f in enumerate(frequencies(128, 500000.0, "none")):
        fn, fd = f.as_integer_ratio()
        a = (pos * fn << 252) // fd % two_pi / 2.0 ** 252
        c, s = math.cos(a), math.sin(a)
        p, r = x[..., i], x[..., i + 64]
        for got, ref in ((y[..., i], p * c - r * s), (y[..., i + 64], r * c + p * s)):
            # a frequency in turns is a double (2^-53 of it): the position's angle is off by 2^-52 of itself
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -20 + abs(pos) * f * 2.0 ** -52) * (p.abs() + r.abs())
            assert ((got - ref).abs() <= tol).all(), (i, pos)


def test_rows_where_a_projection_leaves_them(rkv):
    """Slices of one fused output, read in place and written elsewhere, or rotated where they lie."""
    B, T, Hq, Hkv = 2, 37, 8, 2
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    whole = x.clone()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    plan = rkv.rotary_plan(128, 10000.0)
    at = torch.tensor([0, 70000], dtype=torch.int32, device="cuda")
    pos = at.long()[:, None] + torch.arange(T, device="cuda")
    qo = torch.empty(B, Hq, T, D, dtype=torch.bfloat16, device="cuda")
    ko = torch.empty(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda")
    rkv.rkv_rotary(plan, q, k, at, qo, ko)
    assert torch.equal(x, whole)
    check(q, qo, pos, 128, 10000.0, False, "none")
    check(k, ko, pos, 128, 10000.0, False, "none")
    rkv.rkv_rotary(plan, q, k, at)
    assert torch.equal(x[:, :, :Hq].transpose(1, 2), qo) and torch.equal(x[:, :, Hq:Hq + Hkv].transpose(1, 2), ko)
    assert torch.equal(x[:, :, Hq + Hkv:], whole[:, :, Hq + Hkv:])


def test_nan_and_infinity_stay_in_their_pair(rkv):
    x = torch.ones(1, 1, 3, D, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0, 5], x[0, 0, 1, 70] = math.nan, math.inf
    out = torch.empty_like(x)
    rkv.rkv_rotary(rkv.rotary_plan(), x, None, torch.tensor([9], dtype=torch.int32, device="cuda"), out)
    bad = ~torch.isfinite(out[0, 0])
    assert bad[0].nonzero().flatten().tolist() == [5, 69] and bad[1].nonzero().flatten().tolist() == [6, 70]
    assert not bad[2].any()


def test_on_another_stream_and_captured(rkv):
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(2, 4, 9, D, generator=g, device="cuda").bfloat16()
    plan, at = rkv.rotary_plan(64, 10000.0, interleaved=True), torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    ref, out = torch.empty_like(q), torch.zeros_like(q)
    rkv.rkv_rotary(plan, q, None, at, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rkv.rkv_rotary(plan, q, None, at, out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rkv.rkv_rotary(plan, q, None, at, out)
        at += 1
    for step in range(3):
        at.copy_(torch.tensor([step, 1000 * step], dtype=torch.int32))
        graph.replay()
        check(q, out, torch.tensor([step, 1000 * step], device="cuda")[:, None] + torch.arange(9, device="cuda"), 64,
              10000.0, True, "none")
