"""Timing cases of the tree-decoding and accumulated-weight operators of librkv.

Every case is one call on the paged cache of one attention layer (see include/rkv.h for
the layout).  `run` computes the operator in elementary torch operations, or, where `own`
is set, through the library's entry points:

  tree     rkv_tree_attention   attention of a tree of drafted tokens over the cache
  commit   rkv_tree_commit      the accepted path's keys and values join the cache
  decode   rkv_decode_accum     one-token attention that adds up each position's weight
  rows     rkv_accum_rows       the weights of given query rows, added to the same sums
  evict    rkv_evict_accum      the cache cut down to its heaviest and its latest tokens

Shapes are those of an 8B-class layer (32 query and 8 KV heads of 128 channels) and of the
small layer that the parity tests use; the prompts, page sizes and batches are those of
workloads.py.
"""
import math

import torch

own = False
DEV = "cuda"
D = 128
INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    def tree(name, B, Hkv, G, P, n, T, ragged=False):
        return dict(name=name, op="tree", B=B, Hkv=Hkv, G=G, P=P, n=n, T=T, ragged=ragged)

    def commit(name, B, Hkv, P, n, T, path):
        return dict(name=name, op="commit", B=B, Hkv=Hkv, G=4, P=P, n=n, T=T, path=path, ragged=B > 1)

    def decode(name, B, Hkv, G, P, n, ragged=False):
        return dict(name=name, op="decode", B=B, Hkv=Hkv, G=G, P=P, n=n, ragged=ragged)

    def rows(name, B, Hkv, G, P, n, T, ids, ragged=False):
        return dict(name=name, op="rows", B=B, Hkv=Hkv, G=G, P=P, n=n, T=T, ids=ids, ragged=ragged)

    def evict(name, B, Hkv, P, n, keep, recent, ragged=False):
        return dict(name=name, op="evict", B=B, Hkv=Hkv, G=4, P=P, n=n, keep=keep, recent=recent, ragged=ragged)

    return [
        # a chat turn's short cache, a draft head's few nodes: latency alone
        tree("tree_small", 1, 2, 4, 16, 515, 8),
        # one long request, a mid-sized tree: the cache has to be split over the whole GPU
        tree("tree_b1_32k", 1, 8, 4, 16, 32768, 26),
        # batched serving with ragged lengths and the widest tree
        tree("tree_b16_ragged", 16, 8, 4, 32, 32000, 63, True),
        # the 64K-prompt batch, every node drafted
        tree("tree_b8_64k", 8, 8, 4, 16, 65536, 64),
        # one request accepts a few nodes, and a full batch does
        commit("commit_b1", 1, 8, 16, 2563, 26, 4),
        commit("commit_b64", 64, 8, 32, 4001, 63, 9),
        # a single token over stage 1's survivors of a 32K prompt, and over the ragged batch
        decode("decode_b1_2k", 1, 8, 4, 16, 2563),
        decode("decode_b16_ragged", 16, 8, 4, 32, 32000, True),
        # an accepted path's rows, and a whole prompt's
        rows("rows_path_b16", 16, 8, 4, 32, 32000, 63, 6, True),
        rows("rows_prompt_16k", 1, 8, 4, 16, 16384, 16384, 0),
        # a chat turn's cache cut to a quarter, and the batch cut to its budget
        evict("evict_b1_4k", 1, 2, 16, 4096, 1024, 32),
        evict("evict_b16_ragged", 16, 8, 32, 32000, 8192, 128, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "decode", "decode", "rows", "rows", "commit", "evict"])
    c = dict(op=op, B=_log_int(rng, 1, 16), Hkv=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 4, 8]),
             P=rng.choice([16, 32, 64]), n=_log_int(rng, 1, 65536), ragged=rng.random() < 0.6)
    if op == "tree":
        c["T"] = _log_int(rng, 1, 128)
    elif op == "commit":
        c["T"] = _log_int(rng, 1, 128)
        c["path"] = min(c["T"], _log_int(rng, 1, 16))
    elif op == "rows":
        if rng.random() < 0.5:
            c["T"] = _log_int(rng, 1, 128)
            c["ids"] = min(c["T"], c["n"], _log_int(rng, 1, 16))
        else:
            c["n"] = min(c["n"], 16384)
            c["T"] = _log_int(rng, 1, c["n"])
            c["ids"] = 0
    elif op == "evict":
        c["keep"] = _log_int(rng, 1, max(1, c["n"]))
        c["recent"] = rng.randrange(0, min(c["keep"], 256) + 1)
    # no dearer than the largest listed case of the kind
    kinds = [x for x in listed() if x["op"] == op]
    most = {m: max(work(x)[m] for x in kinds) for m in ("bytes", "flops")}
    while c["n"] > 1 and any(work(c)[m] > most[m] for m in most):
        c["n"] = c["n"] * 3 // 4
        if op == "rows":
            c["T"] = min(c["T"], c["n"]) if not c["ids"] else c["T"]
            c["ids"] = min(c["ids"], c["n"])
        if op == "evict":
            c["keep"] = min(c["keep"], c["n"])
            c["recent"] = min(c["recent"], c["keep"])
    return c


def _lens(c):
    """Cache lengths of the case's sequences; the first is the longest, one of a ragged
    batch of three or more is empty (but for `rows`, whose rows lie in the cache)."""
    n, B = c["n"], c["B"]
    if not c["ragged"]:
        return [n] * B
    out = [n] + [int(n * (0.25 + 0.75 * ((b * 0.6180339887498949) % 1.0))) for b in range(1, B)]
    if B >= 3 and c["op"] != "rows":
        out[B // 2] = 0
    if c["op"] == "rows":
        out = [max(x, 1) for x in out]
    return out


def _nodes(c):
    """Drafted nodes of each sequence (ragged batches draft fewer here and there)."""
    return [c["T"] - (b % 3) * (c["T"] // 4) if c["ragged"] else c["T"] for b in range(c["B"])]


def _path_lens(c, lens=None):
    """Accepted nodes (`commit`) or rows taken (`rows`) of each sequence."""
    most = c["path"] if c["op"] == "commit" else (c["ids"] or c["T"])
    got = [most - (b % 4) * most // 4 if c["ragged"] else most for b in range(c["B"])]
    return [min(x, y) for x, y in zip(got, lens)] if lens else got


def work(c):
    lens, H, G = _lens(c), c["Hkv"], c["G"]
    row = D * 2
    if c["op"] == "tree":
        nodes = _nodes(c)
        kv = sum(x + t for x, t in zip(lens, nodes)) * H * 2 * row
        qo = sum(nodes) * H * G * (2 * row + 4)
        fl = sum((x * t + t * t) * H * G * 4 * D for x, t in zip(lens, nodes))
        return {"bytes": kv + qo, "flops": fl}
    if c["op"] == "commit":
        m = sum(_path_lens(c))
        return {"bytes": m * H * 4 * row + c["B"] * H * 4 * row, "flops": m * H * 2 * D}
    if c["op"] == "decode":
        return {"bytes": sum(lens) * H * (2 * row + 8) + c["B"] * H * G * (2 * row + 4),
                "flops": sum(lens) * H * G * 4 * D}
    if c["op"] == "rows":
        m = _path_lens(c, lens)
        pairs = sum(x * r - r * (r - 1) // 2 for x, r in zip(lens, m))
        return {"bytes": sum(lens) * H * (row + 8) + sum(m) * H * G * (row + 4), "flops": pairs * H * G * 2 * D}
    kept = [min(x, c["keep"]) for x in lens]
    return {"bytes": sum(lens) * H * 4 + sum(kept) * H * (4 * row + 8) + sum(-(-x // c["P"]) for x in kept) * H * 2 * row,
            "flops": sum(lens) * H}


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _table(g, B, pages, spare):
    return torch.randperm(B * pages + spare, generator=g, device=DEV)[:B * pages].view(B, pages).to(torch.int32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _capacity(c):
    more = c["T"] if c["op"] in ("tree", "commit") else 1
    return -(-(c["n"] + more) // c["P"] // 8) * 8 + 8


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    B, H, G, P = c["B"], c["Hkv"], c["G"], c["P"]
    lens = _lens(c)
    pages = _capacity(c)
    s = dict(case=c, scale=1.0 / math.sqrt(D), lens=lens, pages=pages)
    # recycled pages: what lies behind a sequence's end is another request's data
    s["k_pages"] = _normal(g, B * pages + 5, H, P, D)
    s["v_pages"] = _normal(g, B * pages + 5, H, P, D)
    s["page_table"] = _table(g, B, pages, 5)
    loud = torch.randint(0, D, (4,), generator=g, device=DEV)
    s["k_pages"][..., loud] *= 2                       # outlier channels
    if max(lens) > 8:                                  # attention sinks: each first page's first tokens
        s["k_pages"][s["page_table"][:, 0].long(), :, :4] *= 3
    s["seq_len"] = _ints(lens)
    s["n0"] = _ints(lens)
    if c["op"] in ("commit", "evict"):
        x = s["k_pages"][s["page_table"].long()]       # [B, pages, H, P, D]
        live = torch.arange(pages * P, device=DEV).view(1, pages, 1, P, 1) < s["n0"].view(B, 1, 1, 1, 1)
        s["kmax"] = x.masked_fill(~live, -INF).amax(3).permute(0, 2, 3, 1).contiguous()
        s["kmin"] = x.masked_fill(~live, INF).amin(3).permute(0, 2, 3, 1).contiguous()
    else:
        s["kmax"] = torch.zeros(B, H, D, pages, dtype=torch.bfloat16, device=DEV)
        s["kmin"] = torch.zeros(B, H, D, pages, dtype=torch.bfloat16, device=DEV)

    if c["op"] in ("tree", "commit"):
        T = c["T"]
        s["q"] = _normal(g, B, H * G, T, D)
        s["k_tree"] = _normal(g, B, H, T, D)
        s["v_tree"] = _normal(g, B, H, T, D)
        nodes = _nodes(c)
        if c["op"] == "tree":
            # each node's parent among the nodes before it; a node sees itself and its ancestors
            parent = (torch.rand(B, T, generator=g, device=DEV) * torch.arange(T, device=DEV)).long()
            sees = torch.zeros(B, T, T, dtype=torch.bool, device=DEV)
            sees[:, 0, 0] = True
            for t in range(1, T):
                sees[:, t] = sees.gather(1, parent[:, t].view(B, 1, 1).expand(B, 1, T))[:, 0]
                sees[:, t, t] = True
            W = (T + 31) // 32
            bits = torch.zeros(B, T, W * 32, dtype=torch.int64, device=DEV)
            bits[..., :T] = sees
            words = (bits.view(B, T, W, 32) << torch.arange(32, device=DEV)).sum(-1)
            s["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
            s["tree_len"] = _ints(nodes)
            s["out"] = torch.zeros(B, H * G, T, D, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.zeros(B, H * G, T, dtype=torch.float32, device=DEV)
        else:
            s["path"] = torch.rand(B, T, generator=g, device=DEV).argsort(1)[:, :c["path"]].sort(1)[0].to(torch.int32).contiguous()
            s["path_len"] = _ints(_path_lens(c))
    if c["op"] == "decode":
        s["q"] = _normal(g, B, H * G, D)
        s["out"] = torch.zeros(B, H * G, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(B, H * G, dtype=torch.float32, device=DEV)
    if c["op"] == "rows":
        T = c["T"]
        s["q"] = _normal(g, B, H * G, T, D)
        s["row_len"] = _ints(_path_lens(c, lens))
        s["row_ids"] = None
        if c["ids"]:
            s["row_ids"] = torch.rand(B, T, generator=g, device=DEV).argsort(1)[:, :c["ids"]].sort(1)[0].to(torch.int32).contiguous()
        s["lse"] = _rows_lse(s)
    if c["op"] in ("decode", "rows", "evict"):
        live = torch.arange(pages * P, device=DEV).view(1, 1, -1) < s["n0"].view(B, 1, 1)
        w = torch.rand(B, H, pages * P, generator=g, device=DEV) ** 8 * 30
        w = torch.where(torch.rand(B, H, pages * P, generator=g, device=DEV) < 0.05, 0.0, w)  # tokens nobody looked at yet
        s["acc0"] = torch.where(live, w, 0.0)
        s["acc"] = s["acc0"].clone()
    if c["op"] == "evict":
        dp = -(-c["keep"] // P // 8) * 8 + 8
        s["dst"] = dict(pages=dp, page_table=_table(g, B, dp, 5),
                        k_pages=torch.zeros(B * dp + 5, H, P, D, dtype=torch.bfloat16, device=DEV),
                        v_pages=torch.zeros(B * dp + 5, H, P, D, dtype=torch.bfloat16, device=DEV),
                        kmax=torch.zeros(B, H, D, dp, dtype=torch.bfloat16, device=DEV),
                        kmin=torch.zeros(B, H, D, dp, dtype=torch.bfloat16, device=DEV),
                        seq_len=torch.zeros(B, dtype=torch.int32, device=DEV),
                        acc=torch.zeros(B, H, dp * P, dtype=torch.float32, device=DEV))
        s["kept"] = torch.full((B, H, c["keep"]), -1, dtype=torch.int32, device=DEV)
    if own:  # the cache's handle and the workspace, which a program makes once
        from two_stage_kv_snapkv_gb300 import rkv
        s["rkv"] = rkv
        s["cache"] = _handle(rkv, s, B, H, P, pages)
        if c["op"] == "tree":
            s["ws"] = rkv.tree_workspace(B, H * G, H, c["T"], pages, P, DEV)
        elif c["op"] == "decode":
            s["ws"] = rkv.accum_workspace(B, H * G, H, pages, P, DEV)
        elif c["op"] == "rows":
            s["ws"] = rkv.accum_rows_workspace(B, H * G, H, c["T"], pages, P, DEV)
        elif c["op"] == "evict":
            s["dst_cache"] = _handle(rkv, s["dst"], B, H, P, s["dst"]["pages"])
            s["ws"] = rkv.evict_workspace(B, H, c["keep"], DEV, in_place=False)
    return s


def _handle(rkv, s, B, H, P, pages):
    """A PagedCache holding s's data; s then names the cache's own tensors."""
    cache = rkv.PagedCache(B, H, P, pages, DEV, page_table=s["page_table"], num_phys_pages=s["k_pages"].shape[0])
    for name in ("k_pages", "v_pages", "kmax", "kmin", "seq_len"):
        getattr(cache, name).copy_(s[name])
        s[name] = getattr(cache, name)
    return cache


def _rows_lse(s):
    """The log-sum-exp that the attention over these rows left behind, for every row that
    is taken; a head at a time, since this is input and not the operator."""
    c = s["case"]
    B, H, G, T = c["B"], c["Hkv"], c["G"], c["T"]
    lse = torch.zeros(B, H * G, T, dtype=torch.float32, device=DEV)
    for b in range(B):
        n, m = s["lens"][b], int(s["row_len"][b])
        ids = torch.arange(m, device=DEV) if s["row_ids"] is None else s["row_ids"][b, :m].long()
        K = s["k_pages"][s["page_table"][b, :-(-n // c["P"])].long()].transpose(0, 1).reshape(H, -1, D)[:, :n].float()
        hidden = torch.arange(n, device=DEV)[None] > torch.arange(n - m, n, device=DEV)[:, None]
        for h in range(H * G):
            x = (s["q"][b, h, ids].float() @ K[h // G].T) * s["scale"]
            lse[b, h, ids] = x.masked_fill_(hidden, -INF).logsumexp(1)
    return lse


# ------------------------------------------------------------------ the operators
def run(s):
    c = s["case"]
    if own:
        rkv = s["rkv"]
        if c["op"] == "tree":
            rkv.rkv_tree_attention(s["cache"], s["q"], s["k_tree"], s["v_tree"], s["mask"], s["out"], lse=s["lse"],
                                   tree_len=s["tree_len"], workspace=s["ws"])
            return s["out"], s["lse"]
        if c["op"] == "commit":
            s["seq_len"].copy_(s["n0"])
            rkv.rkv_tree_commit(s["cache"], s["k_tree"], s["v_tree"], s["path"], s["path_len"])
            return s["k_pages"], s["v_pages"], s["kmax"], s["kmin"], s["seq_len"]
        if c["op"] == "decode":
            s["acc"].copy_(s["acc0"])
            rkv.rkv_decode_accum(s["cache"], s["q"], s["out"], s["acc"], lse=s["lse"], workspace=s["ws"])
            return s["out"], s["lse"], s["acc"]
        if c["op"] == "rows":
            s["acc"].copy_(s["acc0"])
            rkv.rkv_accum_rows(s["cache"], s["q"], s["lse"], s["acc"], row_len=s["row_len"], row_ids=s["row_ids"],
                               workspace=s["ws"])
            return s["acc"]
        d = s["dst"]
        rkv.rkv_evict_accum(s["cache"], s["acc"], [c["keep"]] * c["B"], c["recent"], s["kept"], dst=s["dst_cache"],
                            dst_acc=d["acc"], workspace=s["ws"])
        return s["kept"], d["acc"], d["k_pages"], d["v_pages"], d["kmax"], d["kmin"], d["seq_len"]
    return {"tree": _tree, "commit": _commit, "decode": _decode, "rows": _rows, "evict": _evict}[c["op"]](s)


def _cached(s, pool, used):
    """[B, H, used * P, D] fp32: the sequences' cached rows, page after page."""
    B, H = s["case"]["B"], s["case"]["Hkv"]
    return s[pool][s["page_table"][:, :used].long()].permute(0, 2, 1, 3, 4).reshape(B, H, -1, D).float()


def _softmax(z):
    """(weights, log-sum-exp) over the last axis; a row of nothing but -inf weighs nothing."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -INF, 0.0, m)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    return e.div_(torch.where(total == 0, 1.0, total)), (total.log() + m)[..., 0]


def _tree(s):
    c = s["case"]
    B, H, G, T, P = c["B"], c["Hkv"], c["G"], c["T"], c["P"]
    used = -(-max(s["lens"]) // P)
    K = torch.cat([_cached(s, "k_pages", used), s["k_tree"].float()], 2)
    V = torch.cat([_cached(s, "v_pages", used), s["v_tree"].float()], 2)
    bits = (s["mask"][..., None] >> torch.arange(32, device=DEV)) & 1
    sees = bits.reshape(B, T, -1)[..., :T] == 1
    sees = sees & (torch.arange(T, device=DEV) < s["tree_len"].view(B, 1, 1))
    cached = torch.arange(used * P, device=DEV) < s["seq_len"].view(B, 1, 1)
    shown = torch.cat([cached.expand(B, T, used * P), sees], 2)
    q = s["q"].view(B, H, G * T, D).float()
    z = (q @ K.transpose(2, 3)).mul_(s["scale"])
    z.view(B, H, G, T, -1).masked_fill_(~shown.view(B, 1, 1, T, -1), -INF)
    w, lse = _softmax(z)
    out = (w @ V).view(B, H * G, T, D).to(torch.bfloat16)
    drafted = torch.arange(T, device=DEV) < s["tree_len"].view(B, 1)
    lse = lse.view(B, H * G, T)
    return (torch.where(drafted.view(B, 1, T, 1), out, s["out"]), torch.where(drafted.view(B, 1, T), lse, s["lse"]))


def _commit(s):
    c = s["case"]
    B, H, P, m = c["B"], c["Hkv"], c["P"], c["path"]
    s["seq_len"].copy_(s["n0"])
    i = torch.arange(m, device=DEV)
    b, i = torch.nonzero(i < s["path_len"].view(B, 1), as_tuple=True)
    pos = s["seq_len"][b].long() + i
    phys, slot, node = s["page_table"][b, pos // P].long(), pos % P, s["path"][b, i].long()
    s["k_pages"][phys, :, slot] = s["k_tree"][b, :, node]
    s["v_pages"][phys, :, slot] = s["v_tree"][b, :, node]
    end = s["seq_len"] + s["path_len"]
    page = s["seq_len"].view(B, 1) // P + torch.arange((m + P - 1) // P + 1, device=DEV)  # the pages that may be touched
    b, j = torch.nonzero((page * P < end.view(B, 1)) & (s["path_len"].view(B, 1) > 0), as_tuple=True)
    page = page[b, j].long()
    x = s["k_pages"][s["page_table"][b, page].long()].float()                         # [touched, H, P, D]
    live = (page.view(-1, 1) * P + torch.arange(P, device=DEV) < end[b].view(-1, 1)).view(-1, 1, P, 1)
    s["kmax"][b, :, :, page] = torch.where(live, x, -INF).amax(2).to(torch.bfloat16)
    s["kmin"][b, :, :, page] = torch.where(live, x, INF).amin(2).to(torch.bfloat16)
    s["seq_len"].copy_(end)
    return s["k_pages"], s["v_pages"], s["kmax"], s["kmin"], s["seq_len"]


def _decode(s):
    c = s["case"]
    B, H, G, P = c["B"], c["Hkv"], c["G"], c["P"]
    s["acc"].copy_(s["acc0"])
    used = -(-max(s["lens"]) // P)
    z = (s["q"].view(B, H, G, D).float() @ _cached(s, "k_pages", used).transpose(2, 3)).mul_(s["scale"])
    z.masked_fill_(torch.arange(used * P, device=DEV) >= s["seq_len"].view(B, 1, 1, 1), -INF)
    w, lse = _softmax(z)
    s["acc"][..., :used * P] += w.sum(2)
    return (w @ _cached(s, "v_pages", used)).view(B, H * G, D).to(torch.bfloat16), lse.reshape(B, H * G), s["acc"]


def _rows(s):
    c = s["case"]
    B, H, G, P = c["B"], c["Hkv"], c["G"], c["P"]
    s["acc"].copy_(s["acc0"])
    used = -(-max(s["lens"]) // P)
    q, lse = s["q"], s["lse"]
    if s["row_ids"] is not None:
        ids = s["row_ids"].long().view(B, 1, -1).expand(B, H * G, -1)
        q, lse = q.gather(2, ids[..., None].expand(-1, -1, -1, D)), lse.gather(2, ids)
    m = q.shape[2]
    z = (q.reshape(B, H, G * m, D).float() @ _cached(s, "k_pages", used).transpose(2, 3)).mul_(s["scale"])
    z.sub_(lse.reshape(B, H, G * m, 1)).exp_()
    i, first = torch.arange(m, device=DEV).view(1, m, 1), (s["seq_len"] - s["row_len"]).view(B, 1, 1)
    hidden = (torch.arange(used * P, device=DEV) > first + i) | (i >= s["row_len"].view(B, 1, 1))
    z.view(B, H, G, m, -1).masked_fill_(hidden.view(B, 1, 1, m, -1), 0.0)
    s["acc"][..., :used * P] += z.sum(2)
    return s["acc"]


def _evict(s):
    c, d = s["case"], s["dst"]
    B, H, P, keep = c["B"], c["Hkv"], c["P"], c["keep"]
    used = -(-max(s["lens"]) // P)
    pos = torch.arange(used * P, device=DEV).view(1, 1, -1)
    n = s["seq_len"].view(B, 1, 1)
    a = s["acc"][..., :used * P]
    rank = torch.where(pos >= n, -INF, torch.where(pos >= n - c["recent"], INF, a))
    order = rank.sort(dim=2, descending=True, stable=True)[1][..., :keep]
    count = torch.clamp(n, max=keep)                                                   # [B, 1, 1]
    i = torch.arange(order.shape[2], device=DEV).view(1, 1, -1)
    kept = torch.where(i < count, order, used * P).sort(2)[0]                          # ascending, the rest behind
    s["kept"][..., :order.shape[2]] = torch.where(i < count, kept, -1).to(torch.int32)
    d["acc"].zero_()
    b, h, i = torch.nonzero((i < count).expand(B, H, -1), as_tuple=True)
    src = kept[b, h, i]
    d["acc"][b, h, i] = a[b, h, src]
    phys, to = s["page_table"][b, src // P].long(), d["page_table"][b, i // P].long()
    d["k_pages"][to, h, i % P] = s["k_pages"][phys, h, src % P]
    d["v_pages"][to, h, i % P] = s["v_pages"][phys, h, src % P]
    full = -(-keep // P)
    x = d["k_pages"][d["page_table"][:, :full].long()].float()                         # [B, full, H, P, D]
    at = torch.arange(full * P, device=DEV).view(1, full, 1, P, 1)
    live = at < count.view(B, 1, 1, 1, 1)
    some = (torch.arange(full, device=DEV).view(1, 1, 1, full) * P < count.view(B, 1, 1, 1))
    for_max = torch.where(live, x, -INF).amax(3).permute(0, 2, 3, 1).to(torch.bfloat16)
    for_min = torch.where(live, x, INF).amin(3).permute(0, 2, 3, 1).to(torch.bfloat16)
    d["kmax"][..., :full] = torch.where(some, for_max, d["kmax"][..., :full])
    d["kmin"][..., :full] = torch.where(some, for_min, d["kmin"][..., :full])
    d["seq_len"].copy_(count.view(B))
    return s["kept"], d["acc"], d["k_pages"], d["v_pages"], d["kmax"], d["kmin"], d["seq_len"]


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions, in fp64, one sequence and one KV head at a time."""
    c = dict(case)
    if c["op"] in ("commit", "evict"):
        return None                                    # they move values and compute none
    s = prepare(c, seed)
    B, H, G, P = c["B"], c["Hkv"], c["G"], c["P"]
    f8 = torch.float64

    def unit(pool, b, h, n):
        at = torch.arange(n, device=DEV)
        return s[pool][s["page_table"][b].long()[at // P], h, at % P].to(f8)

    if c["op"] == "rows":
        acc = s["acc0"].to(f8)
        for b in range(B):
            n, m = s["lens"][b], int(s["row_len"][b])
            ids = list(range(m)) if s["row_ids"] is None else s["row_ids"][b, :m].tolist()
            for h in range(H):
                K = unit("k_pages", b, h, n)
                for hq in range(h * G, (h + 1) * G):
                    for lo in range(0, m, 2048):
                        part = ids[lo:lo + 2048]
                        x = (s["q"][b, hq][part].to(f8) @ K.T) / math.sqrt(D)
                        w = torch.exp(x - s["lse"][b, hq][part].to(f8)[:, None])
                        w = w.tril_(n - m + lo)        # row lo + r lies at n - m + lo + r
                        acc[b, h, :n] += w.sum(0)
        return acc
    T = c["T"] if c["op"] == "tree" else 1
    out = torch.zeros(B, H * G, T, D, dtype=f8, device=DEV)
    lse = torch.zeros(B, H * G, T, dtype=f8, device=DEV)
    acc = s["acc0"].to(f8) if c["op"] == "decode" else None
    q = s["q"].view(B, H * G, T, D)
    nodes = _nodes(c) if c["op"] == "tree" else [1] * B
    for b in range(B):
        n, t = s["lens"][b], nodes[b]
        if c["op"] == "tree":
            words = s["mask"][b, :t].tolist()
            sees = torch.tensor([[(words[i][j // 32] >> (j % 32)) & 1 for j in range(t)] for i in range(t)],
                                dtype=torch.bool, device=DEV).view(t, t)
        for h in range(H):
            K, V = unit("k_pages", b, h, n), unit("v_pages", b, h, n)
            if c["op"] == "tree":
                K = torch.cat([K, s["k_tree"][b, h, :t].to(f8)])
                V = torch.cat([V, s["v_tree"][b, h, :t].to(f8)])
            if K.shape[0] == 0:
                lse[b, h * G:(h + 1) * G, :t] = -INF
                continue
            for hq in range(h * G, (h + 1) * G):
                x = (q[b, hq, :t].to(f8) @ K.T) / math.sqrt(D)
                if c["op"] == "tree":
                    x[:, n:] = x[:, n:].masked_fill(~sees, -INF)
                total = torch.logsumexp(x, 1)
                w = torch.exp(x - total[:, None])
                out[b, hq, :t] = w @ V
                lse[b, hq, :t] = total
                if acc is not None:
                    acc[b, h, :n] += w[0]
    if c["op"] == "decode":
        return out.view(B, H * G, D), lse.view(B, H * G), acc
    return out, lse
