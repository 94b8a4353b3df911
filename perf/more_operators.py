"""Timing cases of librkv's 8-bit cache and of what a step does around it.

Every case is one call for one attention layer (see include/rkv.h for the layouts).  `run`
computes the operator in elementary torch operations, or, where `own` is set, through the
library's entry points:

  reserve  rkv_reserve_pages   page tables and slot maps from the requests' new lengths
  rotary   rkv_rotary          rotary positions of a step's queries and keys
  append   rkv_q8_append       new keys and values enter the 8-bit cache
  load     rkv_q8_load         a bf16 cache (a prompt after stage 1) becomes an 8-bit one
  attend   rkv_q8_attention    the last rows' attention over the 8-bit cache

The cache holds a code of 8 bits for each value (e4m3 or a signed integer) and, for each page
and KV head, one power of two for K and one for V: value = code * scale.  A page's scale is the
smallest power of two that brings its largest magnitude into the codes' range; a page that
already holds tokens keeps the larger of its scale and the new tokens' and, where that is the
latter, its old codes are rounded again to it.

Shapes are those of an 8B-class layer (32 query and 8 KV heads of 128 channels) and of the
small layer that the parity tests use; prompts, page sizes and batches are those of
workloads.py.
"""
import math

import torch

own = False
DEV = "cuda"
D = 128
INF = float("inf")
LARGEST = {"e4m3": 448.0, "int8": 127.0}
LOWEST = 2.0 ** -126                                   # the scale of a block of zeros


# ------------------------------------------------------------------ cases
def listed():
    def reserve(name, B, P, n, m, ragged=False):
        return dict(name=name, op="reserve", B=B, P=P, n=n, T=m, ragged=ragged)

    def rotary(name, B, Hkv, G, T, at, rot, pairs, scaling, fused):
        return dict(name=name, op="rotary", B=B, Hkv=Hkv, G=G, T=T, at=at, rot=rot, pairs=pairs, scaling=scaling,
                    fused=fused)

    def append(name, B, Hkv, P, n, T, fmt, ragged=False):
        return dict(name=name, op="append", B=B, Hkv=Hkv, P=P, n=n, T=T, fmt=fmt, ragged=ragged)

    def load(name, B, Hkv, P, n, fmt, ragged=False):
        return dict(name=name, op="load", B=B, Hkv=Hkv, P=P, n=n, T=1, fmt=fmt, ragged=ragged)

    def attend(name, B, Hkv, G, P, n, T, fmt, ragged=False):
        return dict(name=name, op="attend", B=B, Hkv=Hkv, G=G, P=P, n=n, T=T, fmt=fmt, ragged=ragged)

    return [
        # a full batch's decode step: a page for some of the sequences
        reserve("reserve_step_b64", 64, 32, 4001, 1, True),
        # a batch of prompts admitted at once: all their pages, and a slot for every token
        reserve("reserve_prompts_b128", 128, 16, 0, 32000, True),
        # one token of a full batch at its positions, as the projections leave it
        rotary("rotary_step_b64", 64, 8, 4, 1, 4001, 128, "half", "none", True),
        # a long prompt with frequencies stretched for it
        rotary("rotary_prompt_16k", 1, 8, 4, 16384, 100000, 128, "half", "turns", True),
        # a ragged chunk, half of the head rotated, neighbouring channels paired
        rotary("rotary_chunk_part", 3, 2, 8, 1025, 1000000, 64, "neighbours", "logs", False),
        # one token for every sequence of a full batch, and a batch of prompts
        append("append_step_b64", 64, 8, 32, 4001, 1, "e4m3", True),
        append("append_prompt_b8", 8, 8, 16, 0, 16384, "int8", True),
        # the survivors of a ragged batch of prompts move to 8 bits
        load("load_b16_ragged", 16, 8, 32, 9675, "e4m3", True),
        # a single token over stage 1's survivors of a 32K prompt, and over a ragged batch
        attend("attend_b1_2k", 1, 8, 4, 16, 2563, 1, "e4m3"),
        attend("attend_b16_ragged", 16, 8, 4, 32, 32000, 1, "e4m3", True),
        # a few drafted tokens in a chain over the ragged batch
        attend("attend_draft5_b16", 16, 8, 4, 32, 32000, 5, "int8", True),
        # a prompt's chunk over what came before it
        attend("attend_chunk_2k", 1, 8, 4, 16, 32768, 2048, "e4m3"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reserve", "rotary", "append", "load", "attend", "attend", "attend"])
    P, B = rng.choice([16, 32, 64]), _log_int(rng, 1, 64)
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    if op == "reserve":
        c = dict(op=op, B=_log_int(rng, 1, 256), P=P, n=_log_int(rng, 1, 32000) - 1, T=_log_int(rng, 1, 32000),
                 ragged=rng.random() < 0.7)
    elif op == "rotary":
        c = dict(op=op, B=B, Hkv=Hkv, G=G, T=_log_int(rng, 1, 16384), at=_log_int(rng, 1, 1 << 20),
                 rot=rng.choice([16, 32, 64, 96, 128, 128]), pairs=rng.choice(["half", "neighbours"]),
                 scaling=rng.choice(["none", "linear", "turns", "logs"]), fused=rng.random() < 0.5)
    else:
        c = dict(op=op, B=min(B, 32), Hkv=Hkv, P=P, n=_log_int(rng, 1, 65536), T=1, fmt=rng.choice(["e4m3", "int8"]),
                 ragged=rng.random() < 0.6)
        if op == "append":
            c["n"] -= 1
            c["T"] = _log_int(rng, 1, 16384)
        if op == "attend":
            c["G"] = G
            c["T"] = _log_int(rng, 1, rng.choice([8, 64, 2048]))
    # no dearer than the largest listed case of the kind
    kinds = [x for x in listed() if x["op"] == op]
    most = {m: max(work(x)[m] for x in kinds) for m in ("bytes", "flops")}
    while any(work(c)[m] > most[m] for m in most):
        at = "B" if c["B"] > 4 else ("n" if op in ("load", "attend") and c["n"] > c["T"] else "T")
        c[at] = c[at] * 3 // 4
    return c


def _lens(c):
    """Cached tokens of the case's sequences; the first is the longest, one of a ragged batch
    of three or more is empty."""
    n, B = c["n"], c["B"]
    if not c["ragged"]:
        return [n] * B
    out = [n] + [int(n * (0.25 + 0.75 * ((b * 0.6180339887498949) % 1.0))) for b in range(1, B)]
    if B >= 3 and c["op"] != "reserve":
        out[B // 2] = 0
    return out


def _rows(c):
    """New tokens (reserve, append) or query rows (attend) of each sequence: ragged batches
    have fewer here and there, and a sequence of a batch of five or more has none."""
    T, B = c["T"], c["B"]
    if not c["ragged"]:
        return [T] * B
    out = [T] + [max(1, int(T * (1.0 - 0.5 * ((b * 0.7548776662466927) % 1.0)))) for b in range(1, B)]
    if B >= 5:
        out[B - 2] = 0
    return out


def work(c):
    B, T = c["B"], c["T"]
    if c["op"] == "reserve":
        pages = sum(-(-(n + m) // c["P"]) - -(-n // c["P"]) for n, m in zip(_lens(c), _rows(c)))
        return {"bytes": 4 * (2 * pages + sum(_rows(c)) + 6 * B), "flops": sum(_rows(c)) + pages}
    if c["op"] == "rotary":
        heads = c["Hkv"] * (1 + c["G"])
        return {"bytes": B * T * heads * D * 4 + B * 4, "flops": B * T * heads * c["rot"] * 3}
    lens, H = _lens(c), c["Hkv"]
    if c["op"] == "append":
        m = sum(_rows(c))
        blocks = sum(-(-(n + x) // c["P"]) - n // c["P"] for n, x in zip(lens, _rows(c)) if x) * H
        return {"bytes": m * H * D * 6 + blocks * 16, "flops": m * H * D * 4}
    blocks = sum(-(-n // c["P"]) for n in lens) * H
    if c["op"] == "load":
        return {"bytes": sum(lens) * H * D * 6 + blocks * 8, "flops": sum(lens) * H * D * 4}
    pairs = sum(max(0, r) * n - r * (r - 1) // 2 for n, r in zip(lens, [min(x, n) for x, n in zip(_rows(c), lens)]))
    return {"bytes": sum(lens) * H * D * 2 + blocks * 8 + sum(_rows(c)) * H * c["G"] * (D * 4 + 4),
            "flops": pairs * H * c["G"] * 4 * D}


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _table(g, B, pages, spare):
    return torch.randperm(B * pages + spare, generator=g, device=DEV)[:B * pages].view(B, pages).to(torch.int32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _scale(top, fmt):
    """The smallest power of two that brings a block's largest magnitude into the codes' range."""
    m, e = torch.frexp(top.float() / LARGEST[fmt])      # m in [0.5, 1): a power of two has m = 0.5
    e = torch.where(m > 0.5, e, e - 1).clamp(min=-126)
    return torch.where(top > 0, ((e + 127) << 23).view(torch.float32), LOWEST)


def _codes(x, fmt):
    """x rounded to the codes (it lies in their range): to the nearest, ties to even."""
    return x.to(torch.float8_e4m3fn) if fmt == "e4m3" else x.round().to(torch.int8)


def _pool(g, phys, H, P, fmt, loud):
    """A pool of pages that other requests have written before: codes and scales."""
    x = torch.randn((phys, H, P, D), generator=g, device=DEV)
    if loud is not None:
        x[..., loud] *= 2                              # outlier channels
    s = _scale(x.abs().amax((2, 3)), fmt)
    return _codes(x / s[:, :, None, None], fmt), s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 29)
    B, T = c["B"], c["T"]
    s = dict(case=c)
    if own:
        from two_stage_kv_snapkv_gb300 import rkv
        s["rkv"] = rkv
    if c["op"] == "reserve":
        lens, new, P = _lens(c), _rows(c), c["P"]
        s["start"], s["lens"] = _ints(lens), _ints([n + m for n, m in zip(lens, new)])
        have = [-(-n // P) for n in lens]
        pages = -(-(c["n"] + c["T"]) // P // 8) * 8 + 8
        phys = B * pages + 5
        order = torch.randperm(phys, generator=g, device=DEV).to(torch.int32)
        left = phys - sum(have)
        s["held"], s["count"] = _ints(have), _ints([left])
        s["table"] = torch.full((B, pages), -1, dtype=torch.int32, device=DEV)
        s["table"][torch.arange(pages, device=DEV) < s["held"].view(B, 1)] = order[left:]
        s["free"] = torch.where(torch.arange(phys, device=DEV) < left, order, -1)
        s["slots"] = torch.full((B * T,), -1, dtype=torch.int32, device=DEV)
        s["first"] = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
        s["held_out"], s["count_out"] = torch.zeros_like(s["held"]), torch.zeros_like(s["count"])
        if own:
            s["pool"] = rkv.PagePool(phys, B, DEV, free_pages=s["free"], free_count=s["count"], held=s["held"])
        return s
    if c["op"] == "rotary":
        H, G = c["Hkv"], c["G"]
        s["at"] = torch.randint(0, c["at"], (B,), generator=g, device=DEV, dtype=torch.int32)
        if c["fused"]:                                 # one projection's output, token after token
            x = _normal(g, B, T, H * (G + 2), D)
            s["q"], s["k"] = x[:, :, :H * G].transpose(1, 2), x[:, :, H * G:H * (G + 1)].transpose(1, 2)
        else:
            s["q"], s["k"] = _normal(g, B, H * G, T, D), _normal(g, B, H, T, D)
        s["q_out"] = torch.empty((B, H * G, T, D), dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty((B, H, T, D), dtype=torch.bfloat16, device=DEV)
        s["freq"] = torch.tensor(_frequencies(c), dtype=torch.float64, device=DEV)
        if own:
            p = SCALINGS[c["scaling"]]
            s["plan"] = rkv.rotary_plan(c["rot"], BASE, interleaved=c["pairs"] == "neighbours", scaling=c["scaling"],
                                        **p)
        return s

    H, P, fmt = c["Hkv"], c["P"], c["fmt"]
    lens = _lens(c)
    s["lens"], s["seq_len"], s["n0"] = lens, _ints(lens), _ints(lens)
    more = T if c["op"] == "append" else 0
    pages = -(-(c["n"] + more) // P // 8) * 8 + 8
    phys = B * pages + 5
    s["page_table"] = _table(g, B, pages, 5)
    loud = torch.randint(0, D, (4,), generator=g, device=DEV)
    s["k_codes"], s["k_scale"] = _pool(g, phys, H, P, fmt, loud)
    s["v_codes"], s["v_scale"] = _pool(g, phys, H, P, fmt, None)
    if own:  # the cache's handle, which a program makes once; s then names the handle's own tensors
        cache = rkv.PagedCache8(B, H, P, pages, DEV, page_table=s["page_table"], num_phys_pages=phys, fmt=fmt)
        for name in ("k_codes", "v_codes", "k_scale", "v_scale", "seq_len"):
            getattr(cache, name).copy_(s[name])
            s[name] = getattr(cache, name)
        s["cache"] = cache
    if c["op"] == "append":
        s["k_new"], s["v_new"] = _normal(g, B, H, T, D), _normal(g, B, H, T, D)
        s["k_new"][..., loud] *= 2
        s["k_new"][:, :, :, :] *= torch.where(torch.rand(B, H, T, 1, generator=g, device=DEV) < 0.05, 3.0, 1.0).to(torch.bfloat16)
        s["new"] = _ints(_rows(c))
    elif c["op"] == "load":
        s["src_table"] = _table(g, B, pages, 5)
        s["src_k"], s["src_v"] = _normal(g, phys, H, P, D), _normal(g, phys, H, P, D)
        s["src_k"][..., loud] *= 2
        if own:
            src = rkv.PagedCache(B, H, P, pages, DEV, page_table=s["src_table"], num_phys_pages=phys)
            src.k_pages.copy_(s["src_k"])
            src.v_pages.copy_(s["src_v"])
            src.seq_len.copy_(s["n0"])
            s["src"] = src
    else:
        HQ = H * c["G"]
        s["q"] = _normal(g, B, HQ, T, D)
        s["rows"] = _ints(_rows(c))
        s["out"] = torch.zeros((B, HQ, T, D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((B, HQ, T), dtype=torch.float32, device=DEV)
        if own:
            s["ws"] = rkv.q8_workspace(B, HQ, H, T, pages, P, DEV)
    return s


BASE = 500000.0
SCALINGS = {"none": {}, "linear": dict(factor=4.0), "turns": dict(factor=8.0, original_len=8192, low=1.0, high=4.0),
            "logs": dict(factor=32.0, original_len=4096, low=1.0, high=32.0, amplitude=0.1 * math.log(32.0) + 1.0)}


def _frequencies(c):
    """Radians a position, for each pair of channels: base^(-2 i / rot), slowed down by `factor`
    where the original context holds few turns, by a ramp in the turns or in their logarithm."""
    p, out = SCALINGS[c["scaling"]], []
    for i in range(c["rot"] // 2):
        f = BASE ** (-2.0 * i / c["rot"])
        if c["scaling"] == "linear":
            f /= p["factor"]
        elif c["scaling"] != "none":
            turns = p["original_len"] * f / (2 * math.pi)
            way = math.log if c["scaling"] == "logs" else float
            ramp = (way(turns) - way(p["low"])) / (way(p["high"]) - way(p["low"]))
            ramp = min(1.0, max(0.0, ramp))
            f *= ramp + (1 - ramp) / p["factor"]
        out.append(f)
    return out


# ------------------------------------------------------------------ the operators
def run(s):
    c = s["case"]
    if own:
        rkv = s["rkv"]
        if c["op"] == "reserve":
            rkv.rkv_reserve_pages(s["pool"], s["table"], c["P"], s["lens"], start=s["start"], slots=s["slots"],
                                  first=s["first"], held_out=s["held_out"], free_count_out=s["count_out"])
            return s["table"], s["slots"], s["first"], s["held_out"], s["count_out"]
        if c["op"] == "rotary":
            rkv.rkv_rotary(s["plan"], s["q"], s["k"], s["at"], s["q_out"], s["k_out"])
            return s["q_out"], s["k_out"]
        if c["op"] == "append":
            s["seq_len"].copy_(s["n0"])
            rkv.rkv_q8_append(s["cache"], s["k_new"], s["v_new"], new_len=s["new"])
            return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["seq_len"]
        if c["op"] == "load":
            rkv.rkv_q8_load(s["cache"], s["src"])
            return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["seq_len"]
        rkv.rkv_q8_attention(s["cache"], s["q"], s["out"], lse=s["lse"], row_len=s["rows"], workspace=s["ws"])
        return s["out"], s["lse"]
    return {"reserve": _reserve, "rotary": _rotary, "append": _append, "load": _load, "attend": _attend}[c["op"]](s)


def _reserve(s):
    """Every sequence's table grows to the pages that its new length needs, taken from the top
    of the stack of free pages in the sequences' order; positions start .. length - 1 get their
    slots, page id * page size + place in the page."""
    c, table = s["case"], s["table"]
    B, P = c["B"], c["P"]
    need = (s["lens"].long() + P - 1) // P
    held = s["held"].long()
    take = need - held
    before = take.cumsum(0) - take
    b, j = torch.nonzero(torch.arange(table.shape[1], device=DEV) < take.view(B, 1), as_tuple=True)
    table[b, held[b] + j] = s["free"][s["count"].long() - 1 - before[b] - j]
    s["held_out"].copy_(need)
    s["count_out"].copy_(s["count"] - take.sum())
    m = (s["lens"] - s["start"]).long()
    end = m.cumsum(0)
    s["first"][1:] = end
    x = torch.arange(s["slots"].numel(), device=DEV)
    b = torch.searchsorted(end, x, right=True).clamp(max=B - 1)
    pos = s["start"][b].long() + x - (end - m)[b]
    live = x < end[-1]
    slot = table[b, torch.where(live, pos, 0) // P].long() * P + pos % P
    s["slots"].copy_(torch.where(live, slot, s["slots"].long()))
    return table, s["slots"], s["first"], s["held_out"], s["count_out"]


def _rotary(s):
    c = s["case"]
    T, rot = c["T"], c["rot"]
    angle = (s["at"].view(-1, 1).double() + torch.arange(T, device=DEV))[..., None] * s["freq"]     # [B, T, rot / 2]
    size = SCALINGS[c["scaling"]].get("amplitude", 1.0)
    cos, sin = (angle.cos() * size).float()[:, None], (angle.sin() * size).float()[:, None]
    outs = []
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        x = x.float()
        if c["pairs"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out[..., :rot] = y.to(torch.bfloat16)
        out[..., rot:] = x[..., rot:].to(torch.bfloat16)
        outs.append(out)
    return tuple(outs)


def _append(s):
    c, fmt = s["case"], s["case"]["fmt"]
    B, P = c["B"], c["P"]
    s["seq_len"].copy_(s["n0"])
    n, m = s["n0"].long(), s["new"].long()
    end = n + m
    page = (n // P).view(B, 1) + torch.arange(-(-c["T"] // P) + 1, device=DEV)         # the pages that may be touched
    b, j = torch.nonzero((page * P < end.view(B, 1)) & (m > 0).view(B, 1), as_tuple=True)
    page = page[b, j]
    phys = s["page_table"][b, page].long()
    pos = page.view(-1, 1) * P + torch.arange(P, device=DEV)                           # [touched, P]
    first = n[b].view(-1, 1)
    fresh = ((pos >= first) & (pos < end[b].view(-1, 1))).view(-1, 1, P, 1)
    old = (pos < first).view(-1, 1, P, 1)
    for codes, scale, new in ((s["k_codes"], s["k_scale"], s["k_new"]), (s["v_codes"], s["v_scale"], s["v_new"])):
        x = new[b.view(-1, 1), :, (pos - first).clamp(0, c["T"] - 1)].transpose(1, 2).float()   # [touched, H, P, D]
        was = scale[phys]
        s1 = _scale(torch.where(fresh, x.abs(), 0.0).amax((2, 3)), fmt)
        s1 = torch.where(old.view(-1, 1, P).any(2), torch.maximum(s1, was), s1)
        held = codes[phys]
        y = torch.where(fresh, x, torch.where(old, held.float() * was[:, :, None, None], 0.0)) / s1[:, :, None, None]
        y = _codes(y, fmt).view(torch.uint8)
        codes.view(torch.uint8)[phys] = torch.where(fresh | old, y, held.view(torch.uint8))
        scale[phys] = s1
    s["seq_len"].copy_(end)
    return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["seq_len"]


def _load(s):
    c, fmt = s["case"], s["case"]["fmt"]
    B, P = c["B"], c["P"]
    b, page = torch.nonzero(torch.arange(s["page_table"].shape[1], device=DEV) * P < s["n0"].view(B, 1), as_tuple=True)
    src, dst = s["src_table"][b, page].long(), s["page_table"][b, page].long()
    live = (page.view(-1, 1) * P + torch.arange(P, device=DEV) < s["n0"][b].view(-1, 1)).view(-1, 1, P, 1)
    for codes, scale, pool in ((s["k_codes"], s["k_scale"], s["src_k"]), (s["v_codes"], s["v_scale"], s["src_v"])):
        x = torch.where(live, pool[src].float(), 0.0)
        s1 = _scale(x.abs().amax((2, 3)), fmt)
        y = _codes(x / s1[:, :, None, None], fmt).view(torch.uint8)
        codes.view(torch.uint8)[dst] = torch.where(live, y, codes.view(torch.uint8)[dst])
        scale[dst] = s1
    s["seq_len"].copy_(s["n0"])
    return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["seq_len"]


def _cached(s, which, used):
    """[B, H, used * P, D] fp32: the values that the sequences' codes stand for."""
    at = s["page_table"][:, :used].long()
    x = s[which + "_codes"][at].float() * s[which + "_scale"][at][..., None, None]     # [B, used, H, P, D]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, D)


def _attend(s):
    c = s["case"]
    B, H, G, T, P = c["B"], c["Hkv"], c["G"], c["T"], c["P"]
    used = max(1, -(-max(s["lens"]) // P))
    q = s["q"].view(B, H, G * T, D).float()
    z = (q @ _cached(s, "k", used).transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, H, G, T, -1)
    i, rows, n = torch.arange(T, device=DEV).view(1, T, 1), s["rows"].view(B, 1, 1), s["seq_len"].view(B, 1, 1)
    hidden = torch.arange(used * P, device=DEV) > n - rows + i                          # row i lies at n - rows + i
    z.masked_fill_(hidden.view(B, 1, 1, T, -1), -INF)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -INF, 0.0, m)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    w = e.div_(torch.where(total == 0, 1.0, total)).view(B, H, G * T, -1)
    out = (w @ _cached(s, "v", used)).view(B, H * G, T, D).to(torch.bfloat16)
    lse = (total.log() + m)[..., 0].view(B, H * G, T)
    live = torch.arange(T, device=DEV) < s["rows"].view(B, 1)
    return (torch.where(live.view(B, 1, T, 1), out, s["out"]), torch.where(live.view(B, 1, T), lse, s["lse"]))


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions, in fp64, a sequence (and a KV head) at a time."""
    c = dict(case)
    if c["op"] == "reserve":
        return None                                    # it computes whole numbers alone
    s = prepare(c, seed)
    f8 = torch.float64
    if c["op"] == "rotary":
        outs = []
        for x in (s["q"], s["k"]):
            y = x.to(f8).contiguous()
            rot, size = c["rot"], SCALINGS[c["scaling"]].get("amplitude", 1.0)
            for b in range(c["B"]):
                at = (int(s["at"][b]) + torch.arange(c["T"], device=DEV)).to(f8)
                for i, f in enumerate(_frequencies(c)):
                    u, v = (i, i + rot // 2) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
                    cos, sin = torch.cos(at * f) * size, torch.sin(at * f) * size
                    p, r = y[b, :, :, u].clone(), y[b, :, :, v].clone()
                    y[b, :, :, u], y[b, :, :, v] = p * cos - r * sin, p * sin + r * cos
            outs.append(y)
        return tuple(outs)
    B, H, P, fmt = c["B"], c["Hkv"], c["P"], c["fmt"]
    if c["op"] in ("append", "load"):
        return _exact_codes(s)
    G, T = c["G"], c["T"]
    rows = _rows(c)
    out = s["out"].to(f8)
    lse = s["lse"].to(f8)
    for b in range(B):
        n, m = s["lens"][b], rows[b]
        at = torch.arange(n, device=DEV)
        phys = s["page_table"][b].long()[at // P]
        for h in range(H):
            K, V = (s[w + "_codes"][phys, h, at % P].to(f8) * s[w + "_scale"][phys, h].to(f8)[:, None] for w in "kv")
            for hq in range(h * G, (h + 1) * G):
                for lo in range(0, m, 512):
                    i = torch.arange(lo, min(lo + 512, m), device=DEV)
                    x = (s["q"][b, hq, i].to(f8) @ K.T) / math.sqrt(D)
                    x[at[None] > (n - m + i)[:, None]] = -INF
                    total = torch.logsumexp(x, 1) if n else torch.full((len(i),), -INF, dtype=f8, device=DEV)
                    w = torch.exp(x - torch.where(total == -INF, 0.0, total)[:, None])
                    out[b, hq, i] = w @ V
                    lse[b, hq, i] = total
    return out, lse


def _exact_codes(s):
    """(k codes, v codes, k scales, v scales, nothing for the lengths), from what a code is."""
    c = s["case"]
    power = torch.tensor([2.0 ** e for e in range(-200, 200)], dtype=torch.float64, device=DEV)

    def exponent(v):                                   # floor(log2 v)
        return torch.frexp(v)[1].long() - 1

    B, P = c["B"], c["P"]
    got = {}
    for w in "kv":
        codes, scale = s[w + "_codes"].to(torch.float64), s[w + "_scale"].to(torch.float64)
        for b in range(B):
            if c["op"] == "append":
                n, m = s["lens"][b], _rows(c)[b]
                new = s[w + "_new"][b, :, :m].to(torch.float64)
            else:
                n, m = 0, s["lens"][b]
                at = torch.arange(m, device=DEV)
                new = s["src_" + w][s["src_table"][b].long()[at // P], :, at % P].to(torch.float64).transpose(0, 1)
            if m == 0:
                continue
            lo = n // P * P                            # the first touched page's first position
            pages = -(-(n + m - lo) // P)
            phys = s["page_table"][b, lo // P:lo // P + pages].long()
            x = torch.zeros(new.shape[0], pages * P, D, dtype=torch.float64, device=DEV)
            if n > lo:
                x[:, :n - lo] = codes[phys[0], :, :n - lo] * scale[phys[0]][:, None, None]
            x[:, n - lo:n - lo + m] = new
            top = x.clone()
            top[:, :n - lo] = 0
            top = top.view(-1, pages, P, D).abs().amax((2, 3)).clamp(min=2.0 ** -140) / LARGEST[c["fmt"]]
            s1 = power[200 + exponent(top)]
            s1 = torch.where(s1 < top, s1 * 2, s1).clamp(min=LOWEST)
            if n > lo:
                s1[:, 0] = torch.maximum(s1[:, 0], scale[phys[0]])
            y = x.view(-1, pages, P, D) / s1[:, :, None, None]
            # e4m3: three bits behind the leading one, which stands for 2^-6 at least
            step = power[200 + exponent(y.abs().clamp(min=2.0 ** -6)) - 3] if c["fmt"] == "e4m3" else 1.0
            y = (torch.round(y / step) * step).view(-1, pages * P, D)
            at = torch.arange(n + m - lo, device=DEV)
            codes[phys[at // P], :, at % P] = y[:, :n + m - lo].transpose(0, 1)
            scale[phys] = s1.T
        got[w] = codes, scale
    return got["k"][0], got["v"][0], got["k"][1], got["v"][1], None
