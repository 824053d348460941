"""The operators of the attention layers that stand beside the GDN layers of a hybrid decoder, as measured cases.

Three operators over one paged key/value cache:

  prologue   per new token and head: RMS norm of q and k (optional), rotary positions (half or interleaved pairs, part of
             the head), then k and v appended to the pages of the token's sequence
  attention  a chunk of new tokens of every sequence (one token in decode) over the sequence's cached keys and values
  pages      forking rows that share pages (with a copy of the partial page), freeing them, and compacting the pool

`run` computes them in plain torch operations in 32 bits where `own` is false, and calls the framework where it is true.

A cache row r holds seq_len[r] tokens (the chunk's own included) in pages table[r][0 .. ceil(seq_len / page_size)); page 0 is
the null page.  Pools are [layers][pages][kv heads][page_size][d].  New tokens are packed: row r's are cu[r] .. cu[r+1], and
token i of n sits at position seq_len[r] - n + i.  A row of length 0 is padding: its outputs are zero and it touches no page.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
DEV = "cuda"


def listed():
    def prologue(name, **k):
        return dict({"name": name, "op": "prologue", "dtype": "bf16", "hq": 16, "hkv": 4, "d": 128, "rot": 128, "page": 16, "norm": True,
                     "interleaved": False, "rows": 1, "new_lo": 1, "new_hi": 1, "ctx_lo": 0, "ctx_hi": 0, "pad": 0}, **k)

    def attention(name, **k):
        return dict({"name": name, "op": "attention", "dtype": "bf16", "hq": 16, "hkv": 4, "d": 128, "page": 16, "rows": 1, "new_lo": 1,
                     "new_hi": 1, "ctx_lo": 0, "ctx_hi": 0, "pad": 0}, **k)

    def pages(name, **k):
        return dict({"name": name, "op": "fork", "dtype": "bf16", "hkv": 4, "d": 128, "page": 16, "layers": 1, "rows": 1, "kids": 1,
                     "ctx_lo": 1, "ctx_hi": 1, "live": 0.5}, **k)

    return [
        # one decode step of a 64-row batch, an eighth of it padding: a launch of latency, quarter-head rotation as hybrid decoders use
        prologue("prologue decode 64 rows", rows=64, ctx_lo=3, ctx_hi=5000, pad=8, hkv=2, d=256, rot=64),
        # fp32 activations, interleaved pairs, no norms, ragged short chunks: a speculative batch of a small model
        prologue("prologue f32 interleaved", dtype="f32", hq=12, hkv=4, d=64, rot=64, norm=False, interleaved=True, rows=37, new_lo=2,
                 new_hi=9, ctx_lo=1, ctx_hi=3000),
        # the prefill of eight prompts, about 16 k tokens in all: the bandwidth-bound end
        prologue("prologue prefill 8 prompts", rows=8, new_lo=1500, new_hi=2600, ctx_lo=0, ctx_hi=4000),
        # a single stream in decode: the smallest call, where latency counts
        attention("attention decode 1 row", ctx_lo=776, ctx_hi=776),
        # the headline batch of the decode step: 64 rows, ragged contexts, padding rows
        attention("attention decode 64 rows", rows=64, ctx_lo=500, ctx_hi=8000, pad=8),
        # two very long contexts: few rows, so the key axis has to be split over the GPU
        attention("attention decode long context", rows=2, ctx_lo=180001, ctx_hi=210000, hq=32, hkv=4, page=64),
        # speculative verification, four tokens a row, 256-wide heads
        attention("attention verify 32 rows d256", rows=32, new_lo=4, new_hi=4, ctx_lo=1000, ctx_hi=6000, hkv=2, d=256),
        # one prompt's chunk over what earlier chunks left in the cache: the compute-bound end
        attention("attention prefill chunk", rows=1, new_lo=2048, new_hi=2048, ctx_lo=16000, ctx_hi=16000, page=32),
        # a mixed step in fp32: decode rows beside short chunks, odd sizes
        attention("attention mixed f32", dtype="f32", rows=13, new_lo=1, new_hi=250, ctx_lo=1, ctx_hi=1900, hq=12, hkv=4, d=64),
        # one prompt sampled twice: the smallest fork
        pages("fork 1 row", rows=1, kids=1, ctx_lo=1001, ctx_hi=1001),
        # 48 prompts sampled four times each over eight layers' pages, then released
        pages("fork 48 rows x 4", rows=48, kids=4, ctx_lo=100, ctx_hi=6000, layers=8),
        # a pool half full after many requests came and went, squeezed to its low pages
        pages("compact 4 layers", op="compact", rows=150, ctx_lo=300, ctx_hi=6000, layers=4, hkv=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = rng.choice([(16, 4, 128), (32, 8, 128), (16, 2, 256), (8, 8, 64), (12, 4, 64), (10, 2, 128), (7, 1, 128), (6, 2, 256)])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["prologue", "attention", "attention", "attention", "fork", "compact"])
    hq, hkv, d = heads
    c = {"op": op, "dtype": dtype, "hkv": hkv, "d": d, "page": page}
    if op == "prologue":
        new = _log(rng, 1, 2000)
        hi = _log(rng, 1, 6000)
        c.update(hq=hq, rot=rng.choice([d, d // 2, d // 4]), norm=rng.random() < 0.6, interleaved=rng.random() < 0.5,
                 rows=max(1, min(_log(rng, 1, 128), 12000 // new)), new_lo=max(1, new // 2), new_hi=new, ctx_lo=rng.randint(0, hi), ctx_hi=hi, pad=rng.choice([0, 0, 9]))
    elif op == "attention":
        kind = rng.choice(["decode", "long", "verify", "chunk"])
        if dtype == "f32" and kind == "long":
            kind = "decode"
        if kind == "decode":
            rows, new, hi = _log(rng, 1, 64), 1, _log(rng, 20, 8000)
        elif kind == "long":
            rows, new, hi = 1, 1, _log(rng, 20000, 200000)
        elif kind == "verify":
            rows, new, hi = _log(rng, 2, 32), rng.randint(2, 9), _log(rng, 100, 5000)
        else:
            rows, new, hi = rng.randint(1, 3), _log(rng, 65, 900 if dtype == "bf16" else 300), _log(rng, 100, 9000 if dtype == "bf16" else 2500)
        lo = max(0, int(hi * rng.uniform(0.1, 1.0)))
        c.update(hq=hq, rows=rows, new_lo=max(1, new - new // 3), new_hi=new, ctx_lo=lo, ctx_hi=hi, pad=rng.choice([0, 0, 7]))
    elif op == "fork":
        rows, hi = _log(rng, 1, 48), _log(rng, 17, 4000)
        c.update(layers=rng.randint(1, 4), rows=rows, kids=rng.randint(1, 5), ctx_lo=max(1, hi // 5), ctx_hi=hi, live=0.5)
    else:
        rows, hi = _log(rng, 5, 100), _log(rng, 50, 3000)
        c.update(layers=rng.randint(1, 3), rows=rows, kids=0, ctx_lo=max(1, hi // 5), ctx_hi=hi, live=rng.uniform(0.3, 0.8))
    return c


# ---- what a case's sizes and tables are (from the case alone) ----------------------------------------------------------------


def _lengths(c):
    """(new tokens, lengths) of the rows; a padding row brings one token and has length 0."""
    rng = random.Random("%d %d %d" % (c["rows"], c["ctx_hi"], c["page"]))
    new, length = [], []
    for r in range(c["rows"]):
        n = rng.randint(c.get("new_lo", 0), c.get("new_hi", 0))
        t = rng.randint(c["ctx_lo"], c["ctx_hi"])
        if c.get("pad") and r % c["pad"] == c["pad"] - 1:
            n, t = 1, -1
        new.append(n)
        length.append(t + n)
    return new, length


def _layout(c):
    """new tokens, lengths, table, refs and pages of a case: its rows' pages are scattered over the pool."""
    new, length = _lengths(c)
    page, rows = c["page"], c["rows"]
    held = [-(-n // page) for n in length]
    most = max(held + [1])
    spare = rows * c["kids"] if c["op"] == "fork" else 0
    used = sum(held)
    pages = 1 + (int(used / c["live"]) + spare + 2 if c["op"] in ("fork", "compact") else used + 2 + used // 16)
    order = 1 + np.random.RandomState(used % 65521).permutation(pages - 1)
    table = np.zeros((rows * (1 + c.get("kids", 0)), most), np.int32)
    at = 0
    for r in range(rows):
        table[r, : held[r]] = order[at : at + held[r]]
        at += held[r]
    if c["op"] == "compact":  # neighbours share their first pages, as forked rows do
        for r in range(1, rows, 2):
            s = min(held[r - 1], held[r]) // 3
            table[r, :s] = table[r - 1, :s]
    refs = np.bincount(table.ravel(), minlength=pages).astype(np.int32)
    refs[0] = 0
    return {"new": new, "length": length, "table": table, "refs": refs, "pages": pages}


def _moves(refs):
    """(source, destination) pages of a compaction: the live pages past the live count, in order, to the holes below it, in order."""
    live = refs > 0
    live[0] = True
    n = int(live.sum())
    at = np.arange(len(refs))
    return at[live & (at >= n)], at[~live & (at < n)]


# ---- inputs ------------------------------------------------------------------------------------------------------------------


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV, dtype=TYPES[dtype])
    return x.mul_(scale) if scale != 1.0 else x


def prepare(c, seed):
    lay = _layout(c)
    t = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    layers = c.get("layers", 1)
    shape = (layers, lay["pages"], c["hkv"], c["page"], c["d"])
    # pages that no row holds keep what earlier requests left in them; the null page is zero
    s = {"case": c, "k": _randn(shape, c["dtype"], 8 * seed + 1), "v": _randn(shape, c["dtype"], 8 * seed + 2), "table": t(lay["table"])}
    s["k"][:, 0] = 0
    s["v"][:, 0] = 0
    if c["op"] in ("prologue", "attention"):
        cu = np.concatenate([[0], np.cumsum(lay["new"])])
        s.update(cu=t(cu), length=t(lay["length"]), most_new=max(lay["new"]), most=max(max(lay["length"]), 1))
        tokens = int(cu[-1])
    if c["op"] == "prologue":
        # the layer's packed projection [q | k | v], of which q, k and v are views; norm weights near one
        width = (c["hq"] + 2 * c["hkv"]) * c["d"]
        x = _randn((tokens, width), c["dtype"], 8 * seed + 3, 1.5)
        nq, nk = c["hq"] * c["d"], c["hkv"] * c["d"]
        s["q"] = x[:, :nq].view(tokens, c["hq"], c["d"])
        s["kn"] = x[:, nq : nq + nk].view(tokens, c["hkv"], c["d"])
        s["vn"] = x[:, nq + nk :].view(tokens, c["hkv"], c["d"])
        s["qw"] = 1 + 0.2 * _randn((c["d"],), "f32", 8 * seed + 4) if c["norm"] else None
        s["kw"] = 1 + 0.2 * _randn((c["d"],), "f32", 8 * seed + 5) if c["norm"] else None
        # the program's rotation table, [positions][cos | sin], frequencies of base 1e6 stretched fourfold for a long context
        half = c["rot"] // 2
        f = torch.arange(half, device=DEV, dtype=torch.float64).mul_(-2.0 / c["rot"])
        angle = torch.arange(s["most"], device=DEV, dtype=torch.float64)[:, None] * torch.pow(1e6, f) / 4
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    elif c["op"] == "attention":
        s["q"] = _randn((tokens, c["hq"], c["d"]), c["dtype"], 8 * seed + 3, 2.0)
        s["scale"] = c["d"] ** -0.5
    else:
        s["refs"] = t(lay["refs"])
        if c["op"] == "fork":
            rows, kids = c["rows"], c["kids"]
            s["length"] = t(lay["length"] + [0] * (rows * kids))
            s["src"] = t(np.repeat(np.arange(rows), kids))
            s["dst"] = t(rows + np.arange(rows * kids))
        else:
            s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------------------


def _places(s):
    """Of every new token: its row, its number in the row, its position, and whether its row is real."""
    cu, length = s["cu"].long(), s["length"].long()
    tok = torch.arange(s["q"].shape[0], device=DEV)
    row = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    i = tok - cu[row]
    return row, i, length[row] - (cu[row + 1] - cu[row]) + i, length[row] > 0


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2 : rot])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _prologue(s):
    c = s["case"]
    row, _, pos, real = _places(s)
    turn = s["rope"][pos.clamp(min=0)][:, None]
    cos, sin = turn[..., : c["rot"] // 2], turn[..., c["rot"] // 2 :]
    q, k = s["q"].float(), s["kn"].float()
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["qw"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["kw"]
    q = _rotate(q, cos, sin, c["rot"], c["interleaved"]) * real[:, None, None]
    k = _rotate(k, cos, sin, c["rot"], c["interleaved"])
    pos = pos.clamp(min=0)
    # a padding token rewrites the null page's zeros
    page = torch.where(real, s["table"][row, pos // c["page"]].long(), 0)
    at = (page[:, None], torch.arange(c["hkv"], device=DEV)[None], (pos % c["page"])[:, None])
    s["k"][0].index_put_(at, (k * real[:, None, None]).to(s["k"].dtype))
    s["v"][0].index_put_(at, s["vn"] * real[:, None, None])
    return {"q": q.to(s["q"].dtype), "k": s["k"], "v": s["v"]}


def _attention(s):
    c = s["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    rows, g, n, held = c["rows"], hq // hkv, s["most_new"], -(-s["most"] // page)
    row, i, _, real = _places(s)
    cu, length = s["cu"].long(), s["length"].long()
    q = torch.zeros((rows, n, hq, d), device=DEV)
    q[row, i] = s["q"].float()
    q = q.view(rows, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(rows, hkv, g * n, d)
    at = s["table"][:, :held].long()
    k = s["k"][0][at].float().transpose(1, 2).reshape(rows, hkv, held * page, d)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(rows, hkv, g, n, held * page)
    seen = (length - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device=DEV) + 1  # keys before this are seen
    seen = torch.where((length > 0)[:, None], seen, 0)
    hidden = torch.arange(held * page, device=DEV) >= seen[:, :, None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(torch.isinf(top), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v"][0][at].float().transpose(1, 2).reshape(rows, hkv, held * page, d)
    o = torch.matmul(p.view(rows, hkv, g * n, held * page), v).view(rows, hkv, g, n, d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(rows, n, hq, d)[row, i]
    return {"out": o.to(s["q"].dtype)}


def _fork(s):
    c = s["case"]
    table, refs, length, src, dst, page = s["table"], s["refs"], s["length"], s["src"].long(), s["dst"].long(), c["page"]
    n = length[src]
    at = torch.arange(table.shape[1], device=DEV)
    shared = torch.where(at < (n // page)[:, None], table[src], 0)
    part = n % page > 0
    # free pages, lowest first; the null page is never free
    taken = refs > 0
    taken[0] = True
    free = torch.argsort(taken.int(), stable=True)[: len(src)]
    rank = torch.cumsum(part, 0) - 1
    new = torch.where(part, free[rank.clamp(min=0)], 0).int()
    last = (n // page).clamp(max=table.shape[1] - 1).long()
    old = torch.where(part, table[src, last], 0)
    table[dst] = shared
    table[dst, last] += new
    length[dst] = n
    refs.index_add_(0, table[dst].flatten().long(), torch.ones_like(table[dst]).flatten())
    refs[0] = 0
    # the pairs to copy, in front of zeros
    front = torch.argsort((~part).int(), stable=True)
    move_src, move_dst, count = old[front], new[front], part.sum().int().reshape(1)
    s["k"][:, move_dst.long()] = s["k"][:, move_src.long()]
    s["v"][:, move_dst.long()] = s["v"][:, move_src.long()]
    # the copies are released
    refs.index_add_(0, table[dst].flatten().long(), -torch.ones_like(table[dst]).flatten())
    refs[0] = 0
    table[dst] = 0
    length[dst] = 0
    return {"src": move_src, "dst": move_dst, "count": count, "k": s["k"], "v": s["v"], "table": table, "refs": refs, "length": length}


def _compact(s):
    refs = s["refs"]
    live = refs > 0
    live[0] = True
    at = torch.arange(len(refs), device=DEV, dtype=torch.int32)
    n = live.sum()
    src = torch.nonzero(live & (at >= n)).flatten()
    dst = torch.nonzero(~live & (at < n)).flatten()
    remap = torch.where(live, at, 0)
    remap[src] = dst.int()
    s["table_out"].copy_(remap[s["table"].long()])
    s["refs_out"].copy_(refs)
    s["refs_out"][dst] = refs[src]
    s["refs_out"][src] = 0
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    count = torch.full((1,), len(src), dtype=torch.int32, device=DEV)
    return {"remap": remap, "count": count, "table": s["table_out"], "refs": s["refs_out"], "k": s["k"], "v": s["v"]}


# ---- the framework's operators -----------------------------------------------------------------------------------------------


def _own(s):
    import gated_deltanet_decode_gb300 as G

    c = s["case"]
    if "pool" not in s:  # a program makes the handles of its pool and its move list once
        s["pool"] = G.KVPagePool(s["k"].shape[1], c["page"], c["hkv"], c["d"], layers=s["k"].shape[0], dtype=s["k"].dtype, k=s["k"], v=s["v"])
        if c["op"] in ("fork", "compact"):
            s["moves"] = G.KVPageMoves(len(s["src"]) if c["op"] == "fork" else len(s["refs"]))
    pool = s["pool"]
    if c["op"] == "prologue":
        q = G.attn_prologue(s["q"], s["kn"], s["vn"], pool, s["rope"], s["table"], s["length"], s["cu"], q_norm=s["qw"], k_norm=s["kw"],
                            eps=EPS, interleaved=c["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if c["op"] == "attention":
        return {"out": G.paged_attention(s["q"], pool, s["table"], s["length"], s["cu"], scale=s["scale"])}
    m = s["moves"]
    if c["op"] == "fork":
        G.kv_pages_fork(s["table"], s["length"], s["refs"], s["src"], s["dst"], c["page"], m)
        G.kv_pages_copy(pool, m)
        G.kv_pages_free(s["table"], s["length"], s["refs"], s["dst"])
        return {"src": m.src, "dst": m.dst, "count": m.count, "k": s["k"], "v": s["v"], "table": s["table"], "refs": s["refs"], "length": s["length"]}
    remap = G.kv_pages_compact(s["table"], s["refs"], m, table_out=s["table_out"], refs_out=s["refs_out"])
    G.kv_pages_copy(pool, m)
    return {"remap": remap, "count": m.count, "table": s["table_out"], "refs": s["refs_out"], "k": s["k"], "v": s["v"]}


def run(s):
    if own:
        return _own(s)
    return {"prologue": _prologue, "attention": _attention, "fork": _fork, "compact": _compact}[s["case"]["op"]](s)


# ---- the same in 64 bits, from the definitions -------------------------------------------------------------------------------


def exact(c, seed):
    s = prepare(c, seed)
    lay = _layout(c)
    if c["op"] == "attention":
        return {"out": _exact_attention(c, s, lay)}
    k, v = s["k"].double(), s["v"].double()
    if c["op"] == "prologue":
        return dict(_exact_prologue(c, s, lay, k, v), k=k, v=v)
    if c["op"] == "fork":
        src, dst, refs = [], [], lay["refs"]
        free = iter([p for p in range(1, lay["pages"]) if refs[p] == 0])
        for r in range(c["rows"]):
            for _ in range(c["kids"]):
                if lay["length"][r] % c["page"]:
                    src.append(int(lay["table"][r, lay["length"][r] // c["page"]]))
                    dst.append(next(free))
    else:
        src, dst = (list(map(int, x)) for x in _moves(lay["refs"]))
    k[:, dst], v[:, dst] = k[:, src], v[:, src]
    return {"k": k, "v": v}


def _exact_attention(c, s, lay):
    g, at, out = c["hq"] // c["hkv"], 0, torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for r, (n, length) in enumerate(zip(lay["new"], lay["length"])):
        if length:
            held = s["table"][r, : -(-length // c["page"])].long()
            see = torch.arange(length, device=DEV)[None] <= (length - n + torch.arange(n, device=DEV))[:, None]
            for h in range(c["hkv"]):
                k = s["k"][0, held, h].double().reshape(-1, c["d"])[:length]
                v = s["v"][0, held, h].double().reshape(-1, c["d"])[:length]
                for j in range(h * g, (h + 1) * g):
                    w = (s["q"][at : at + n, j].double() @ k.T) * s["scale"]
                    w = torch.softmax(torch.where(see, w, -math.inf), -1)
                    out[at : at + n, j] = w @ v
        at += n
    return out


def _exact_prologue(c, s, lay, k, v):
    half, at = c["rot"] // 2, 0
    first = torch.arange(half, device=DEV) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)

    def turn(x, w, places):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * w.double()
        y, r = x.clone(), s["rope"][places].double()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(r[:, :half], r[:, half:])[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    for r, (n, length) in enumerate(zip(lay["new"], lay["length"])):
        if length:
            places = torch.arange(length - n, length, device=DEV)
            page, slot = s["table"][r].long()[places // c["page"]], places % c["page"]
            out[at : at + n] = turn(s["q"][at : at + n], s["qw"], places)
            k[0, page, :, slot] = turn(s["kn"][at : at + n], s["kw"], places)
            v[0, page, :, slot] = s["vn"][at : at + n].double()
        at += n
    return {"q": out}


# ---- what a pass cannot do without -------------------------------------------------------------------------------------------


def work(c):
    es = SIZE[c["dtype"]]
    if c["op"] in ("prologue", "attention"):
        new, length = _lengths(c)
        tokens = sum(new)
        live = [(n, t) for n, t in zip(new, length) if t]
        fresh = sum(n for n, _ in live)
        tables = 4 * (sum(-(-t // c["page"]) for t in length) + 2 * c["rows"] + 1)
        if c["op"] == "prologue":
            # q in and out, k and v in and into their pages, a row of the rotation table a token
            moved = (fresh * (c["hq"] + 4 * c["hkv"]) + tokens * c["hq"]) * c["d"] * es + fresh * c["rot"] * 4
            return {"bytes": moved + 8 * c["rows"] + 4 * fresh, "flops": fresh * (c["hq"] + c["hkv"]) * (3 * c["rot"] + (5 * c["d"] if c["norm"] else 0))}
        pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in live)
        moved = (fresh + tokens) * c["hq"] * c["d"] * es + 2 * sum(length) * c["hkv"] * c["d"] * es + tables
        return {"bytes": moved, "flops": 4 * pairs * c["hq"] * c["d"]}
    lay = _layout(c)
    if c["op"] == "fork":
        copied = c["kids"] * sum(t % c["page"] > 0 for t in lay["length"])
        # the forked rows' entries are read, written and cleared, their pages' counts go up and down
        tables = 4 * c["kids"] * sum(-(-t // c["page"]) for t in lay["length"]) * 5 + 4 * lay["pages"]
    else:
        copied = len(_moves(lay["refs"])[0])
        tables = 8 * lay["table"].size + 12 * lay["pages"]
    return {"bytes": 2 * 2 * copied * c["layers"] * c["hkv"] * c["page"] * c["d"] * es + tables, "flops": 0}
