"""Linear attention with a decay for each head, and attention over prefixes that forked rows share, as measured cases.

Operators of a hybrid decoder that stand beside the gated delta rule and the paged attention:

  decode    linear attention, one token a row:     S' = a S + v k^T,  o = scale S' q, over slots of a state pool
  prefill   the same over many tokens a sequence (prompts), packed
  attention new tokens of rows that share their first pages, the shared keys and values read once for a group of rows
  shared    which pages the rows of each group share, from the page table

`run` computes them in plain torch operations in 32 bits where `own` is false, and calls the framework where it is true.

The state pool is [slots][hv][dv][dk] in 32 bits, slot 0 the null slot; a row or sequence reads its state from one slot and
writes the next one to another, so a pass can be repeated.  The decay is a = exp(log_decay), a number a head (fixed) or a head
and token.  Value head h reads query and key head h / (hv / hk).  A row on slot 0 is padding: its outputs are zero.

The page pool is [pages][kv heads][page_size][d].  Rows come in groups of neighbours; the rows of a group have the same pages
first, then pages of their own.  Row r holds length[r] tokens, its new ones included; a row of length 0 is padding.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
DEV = "cuda"
CHUNK = 64  # tokens of a chunk in the plain prefill


def listed():
    def decode(name, **k):
        return dict({"name": name, "op": "decode", "dtype": "bf16", "hk": 16, "hv": 16, "dk": 128, "dv": 128, "rows": 1, "pad": 0,
                     "fixed": False}, **k)

    def prefill(name, **k):
        return dict({"name": name, "op": "prefill", "dtype": "bf16", "hk": 16, "hv": 16, "dk": 128, "dv": 128, "rows": 1, "new_lo": 1,
                     "new_hi": 1, "pad": 0, "fixed": False}, **k)

    def attention(name, **k):
        return dict({"name": name, "op": "attention", "dtype": "bf16", "hq": 16, "hkv": 4, "d": 128, "page": 16, "groups": 1, "members": 16,
                     "new_lo": 1, "new_hi": 1, "pre_lo": 512, "pre_hi": 512, "ctx_lo": 0, "ctx_hi": 100, "pad": 0}, **k)

    def shared(name, **k):
        return dict({"name": name, "op": "shared", "page": 16, "groups": 1, "members": 16, "new_lo": 1, "new_hi": 1, "pre_lo": 512,
                     "pre_hi": 512, "ctx_lo": 0, "ctx_hi": 100, "pad": 0}, **k)

    return [
        # a single stream in decode: the smallest call, where latency counts
        decode("linear decode 1 row", fixed=True),
        # a decode step's batch of 64, an eighth of it padding, a decay a token
        decode("linear decode 64 rows", rows=64, pad=8),
        # fp32 activations, few qk heads over many narrow value heads, an odd number of rows
        decode("linear decode 203 rows f32", dtype="f32", rows=203, hk=2, hv=32, dk=128, dv=64),
        # a speculative batch's few tokens a row: hardly a chunk each
        prefill("linear prefill 37 short", rows=37, new_lo=1, new_hi=9, hk=8, hv=16),
        # the prompts of a batch
        prefill("linear prefill 8 prompts", rows=8, new_lo=1500, new_hi=2600),
        # one long prompt: few chains, so the tokens have to be split over the GPU
        prefill("linear prefill one long", rows=1, new_lo=16000, new_hi=16000, fixed=True),
        # fp32 activations and narrow heads, a ragged batch
        prefill("linear prefill f32", dtype="f32", rows=5, new_lo=200, new_hi=900, hk=4, hv=8, dk=64, dv=64, pad=5),
        # a short prompt sampled sixteen times: a call of latency
        attention("shared attention 16 samples"),
        # 64 samples of one long prompt, an eighth of them done and released
        attention("shared attention 64 samples", members=64, pre_lo=16000, pre_hi=16000, ctx_lo=1, ctx_hi=900, pad=8),
        # four prompts in fp32, eight samples each, four tokens of every one to be verified
        attention("shared attention f32 verify", dtype="f32", groups=4, members=8, new_lo=4, new_hi=4, pre_lo=300, pre_hi=2000, ctx_lo=0,
                  ctx_hi=300, hq=12, hkv=4, d=64),
        # one step's look at the table for the smallest batch, and for a large one of long prompts
        shared("shared pages 16 rows"),
        shared("shared pages 1024 rows", groups=32, members=32, pre_lo=1000, pre_hi=16000, ctx_lo=0, ctx_hi=1500, pad=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prefill", "prefill", "attention", "attention", "shared"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op in ("decode", "prefill"):
        hk, hv, dk, dv = rng.choice([(16, 16, 128, 128), (8, 16, 128, 128), (16, 32, 128, 128), (4, 8, 64, 64), (1, 24, 128, 64), (6, 6, 64, 128),
                                     (3, 3, 32, 40), (4, 4, 256, 128)])
        c = {"op": op, "dtype": dtype, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "pad": rng.choice([0, 0, 6]), "fixed": rng.random() < 0.4}
        if op == "decode":
            return dict(c, rows=max(1, min(_log(rng, 1, 190), 190 * 2 ** 18 // (hv * dk * dv))))
        slow = dtype == "f32" or (dk, dv) not in ((128, 128), (64, 64), (128, 64), (64, 128))
        most = _log(rng, 2, 700 if slow else 6000)
        tokens = 3000 if slow else 16000 * 2 ** 18 // max(hv * dk * dv, 2 ** 18)
        return dict(c, rows=max(1, min(_log(rng, 1, 48), tokens // most)), new_lo=max(1, most // 3), new_hi=most)
    page = rng.choice([16, 32, 64, 128])
    groups = _log(rng, 1, 8)
    members = max(1, min(_log(rng, 2, 64), 96 // groups))
    pre = _log(rng, 100, 12000 // groups)
    ctx = _log(rng, 2, 1000)
    new = rng.choice([1, 1, 1, 3, 5])
    c = {"op": op, "page": page, "groups": groups, "members": members, "new_lo": max(1, new - 1), "new_hi": new, "pre_lo": pre // 2, "pre_hi": pre,
         "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx, "pad": rng.choice([0, 0, 5])}
    if op == "attention":
        hq, hkv, d = rng.choice([(16, 4, 128), (32, 8, 128), (16, 2, 256), (8, 8, 64), (12, 4, 64), (10, 2, 128), (7, 1, 128), (6, 2, 256)])
        c.update(dtype=dtype, hq=hq, hkv=hkv, d=d)
        if dtype == "f32":
            c.update(pre_lo=min(c["pre_lo"], 1500), pre_hi=min(pre, 3000))
    return c


# ---- what a case's sizes and tables are (from the case alone) ----------------------------------------------------------------


def _padding(c, r):
    return bool(c["pad"]) and r % c["pad"] == c["pad"] - 1


def _tokens(c):
    """New tokens of every sequence of a prefill."""
    rng = random.Random("%d %d %d" % (c["rows"], c["new_hi"], c["hv"]))
    return [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["rows"])]


def _slots(c):
    """Read and write slots: distinct, in no order; padding rows on slot 0."""
    order = 1 + np.random.RandomState(c["rows"]).permutation(2 * c["rows"])
    pad = np.array([_padding(c, r) for r in range(c["rows"])])
    return [np.where(pad, 0, order[i :: 2]).astype(np.int32) for i in (0, 1)]


def _layout(c):
    """New tokens, lengths, shared pages and the table of a case of rows in groups; a padding row brings one token, has length 0
    and no pages (it was released)."""
    rng = random.Random("%d %d %d" % (c["groups"], c["pre_hi"], c["members"]))
    page, rows = c["page"], c["groups"] * c["members"]
    shared = [rng.randint(c["pre_lo"], c["pre_hi"]) // page for _ in range(c["groups"])]
    new, length = [], []
    for r in range(rows):
        n = rng.randint(c["new_lo"], c["new_hi"])
        t = shared[r // c["members"]] * page + rng.randint(c["ctx_lo"], c["ctx_hi"]) + n
        new.append(1 if _padding(c, r) else n)
        length.append(0 if _padding(c, r) else t)
    held = [-(-t // page) for t in length]
    pages = 1 + sum(shared) + sum(held)
    order = 1 + np.random.RandomState(pages % 65521).permutation(pages - 1)
    table = np.zeros((rows, max(held + [1])), np.int32)
    at = 0
    for g in range(c["groups"]):
        first = order[at : at + shared[g]]
        at += shared[g]
        for r in range(g * c["members"], (g + 1) * c["members"]):
            if length[r]:
                own_pages = held[r] - shared[g]
                table[r, : shared[g]] = first
                table[r, shared[g] : held[r]] = order[at : at + own_pages]
                at += own_pages
    return {"new": new, "length": length, "shared": shared, "table": table, "pages": pages}


def _prefix(c, lay):
    """Of every row: its group's first live row, and the pages that the group's live rows share (none where one row is live)."""
    out = np.zeros((len(lay["new"]), 2), np.int32)
    for g in range(c["groups"]):
        rows = range(g * c["members"], (g + 1) * c["members"])
        live = [r for r in rows if lay["length"][r]]
        out[rows.start : rows.stop] = (live[0] if live else rows.start, lay["shared"][g] if len(live) > 1 else 0)
    return out


# ---- inputs ------------------------------------------------------------------------------------------------------------------


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV, dtype=TYPES[dtype])
    return x.mul_(scale) if scale != 1.0 else x


def _ints(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)


def prepare(c, seed):
    if c["op"] in ("decode", "prefill"):
        return _prepare_linear(c, seed)
    return _prepare_paged(c, seed)


def _prepare_linear(c, seed):
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    new = _tokens(c) if c["op"] == "prefill" else [1] * c["rows"]
    tokens = sum(new)
    # the layer's packed projection [q | k | v], of which q, k and v are views
    x = _randn((tokens, 2 * hk * dk + hv * dv), c["dtype"], 8 * seed + 1)
    x[:, hk * dk : 2 * hk * dk] *= dk ** -0.5
    s = {"case": c, "q": x[:, : hk * dk].view(tokens, hk, dk), "k": x[:, hk * dk : 2 * hk * dk].view(tokens, hk, dk),
         "v": x[:, 2 * hk * dk :].view(tokens, hv, dv), "scale": dk ** -0.5}
    if c["fixed"]:  # a decay a head, from a memory of some tens of tokens to one of thousands
        memory = torch.pow(2.0, 4 + 8 * torch.arange(hv, device=DEV, dtype=torch.float64) / hv)
        s["log_decay"] = torch.log1p(-1 / memory).float()
    else:  # a rate a head, a step a token
        rate = 1 + 15 * torch.rand((hv,), generator=torch.Generator(device=DEV).manual_seed(8 * seed + 2), device=DEV)
        s["log_decay"] = -rate * torch.log1p(torch.exp(_randn((tokens, hv), "f32", 8 * seed + 3) - 4))
    slots = 2 * c["rows"] + 1
    s["state"] = _randn((slots, hv, dv, dk), "f32", 8 * seed + 4, 0.5)
    s["state"][0] = 0
    s["read"], s["write"] = (_ints(a) for a in _slots(c))
    if c["op"] == "prefill":
        s.update(cu=_ints(np.concatenate([[0], np.cumsum(new)])), most=max(new))
    return s


def _prepare_paged(c, seed):
    lay = _layout(c)
    rows = len(lay["new"])
    cu = np.concatenate([[0], np.cumsum(lay["new"])])
    s = {"case": c, "table": _ints(lay["table"]), "cu": _ints(cu), "bounds": _ints(np.arange(c["groups"] + 1) * c["members"])}
    if c["op"] == "shared":
        # the pages' numbers are the inputs, and what became of the rows: another seed deals the pages out anew, the first rows of a
        # group are done by now, and one row went its own way within the last half of what the others share
        order = np.random.RandomState(seed).permutation(lay["pages"] - 1) + 1
        table = np.concatenate([[0], order])[lay["table"]].astype(np.int32)
        length = list(lay["length"])
        rng = random.Random(seed)
        for g in range(c["groups"]):
            first, last = g * c["members"], (g + 1) * c["members"] - 1
            for r in range(first, first + rng.randint(0, c["members"] // 2)):
                table[r], length[r] = 0, 0
            if lay["shared"][g] > 1 and length[last]:
                table[last, rng.randrange(lay["shared"][g] // 2, lay["shared"][g])] = lay["pages"] + last
        s.update(table=_ints(table), length=_ints(length))
        return s
    tokens = int(cu[-1])
    shape = (1, lay["pages"], c["hkv"], c["page"], c["d"])
    s.update(k=_randn(shape, c["dtype"], 8 * seed + 1), v=_randn(shape, c["dtype"], 8 * seed + 2), length=_ints(lay["length"]),
             prefix=_ints(_prefix(c, lay)), q=_randn((tokens, c["hq"], c["d"]), c["dtype"], 8 * seed + 3, 2.0), scale=c["d"] ** -0.5,
             most_new=max(lay["new"]), most_shared=max(lay["shared"]), rows=rows,
             most_own=max(max([-(-t // c["page"]) - lay["shared"][r // c["members"]] for r, t in enumerate(lay["length"])]), 1))
    s["k"][:, 0] = 0
    s["v"][:, 0] = 0
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------------------


def _heads(x, hv):
    """[...][hk][dk] as [...][hv][dk], a query or key head for each value head."""
    return x.repeat_interleave(hv // x.shape[-2], -2)


def _decode(s):
    c = s["case"]
    real = (s["read"] > 0)[:, None, None, None]
    q, k, v = _heads(s["q"].float(), c["hv"]), _heads(s["k"].float(), c["hv"]), s["v"].float()
    decay = torch.exp(s["log_decay"]).expand(c["rows"], c["hv"])
    state = decay[..., None, None] * s["state"][s["read"].long()] + v[..., :, None] * k[..., None, :]
    state = state * real
    out = torch.matmul(state, q[..., None])[..., 0] * s["scale"]
    s["state"][s["write"].long()] = state  # a padding row rewrites the null slot's zeros
    return {"out": out.to(s["q"].dtype), "state": s["state"]}


def _prefill(s):
    c = s["case"]
    hv, cu = c["hv"], s["cu"].long()
    n = -(-s["most"] // CHUNK)  # chunks of the longest sequence
    at = torch.arange(n * CHUNK, device=DEV)
    there = (at < (cu[1:] - cu[:-1])[:, None])
    token = torch.where(there, cu[:-1, None] + at, 0)

    def chunks(x):  # [tokens][hv][d] -> [rows][hv][chunks][CHUNK][d], zeros past a sequence's end
        x = torch.where(there[..., None, None], x.float()[token], 0.0)
        return x.view(c["rows"], n, CHUNK, hv, -1).permute(0, 3, 1, 2, 4)

    q, k, v = chunks(_heads(s["q"], hv)), chunks(_heads(s["k"], hv)), chunks(s["v"])
    g = s["log_decay"].double().expand(s["q"].shape[0], hv)[token]
    g = torch.where(there[..., None], g, 0.0).view(c["rows"], n, CHUNK, hv).permute(0, 3, 1, 2)
    upto = torch.cumsum(g, -1)  # within a chunk
    chunk = upto[..., -1]
    total = torch.cumsum(chunk, -1)  # to a chunk's end
    # within the chunks
    i = torch.arange(CHUNK, device=DEV)
    seen = i[:, None] >= i
    decay = torch.where(seen, torch.exp(torch.where(seen, upto[..., :, None] - upto[..., None, :], 0.0)).float(), 0.0)
    out = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * decay, v)
    # what each chunk adds to the state, and the states before every chunk and after the last
    add = torch.matmul((v * torch.exp(chunk[..., None] - upto).float()[..., None]).transpose(-1, -2), k)
    start = s["state"][s["read"].long()]
    begin = torch.cat([torch.zeros_like(total[..., :1]), total], -1)
    j = torch.arange(n, device=DEV)
    before = torch.arange(n + 1, device=DEV)[:, None] > j
    carry = torch.where(before, torch.exp(torch.where(before, begin[..., :, None] - total[..., None, :], 0.0)).float(), 0.0)
    states = torch.matmul(carry, add.flatten(-2)).view(*begin.shape, c["dv"], c["dk"])
    states = states + torch.exp(begin).float()[..., None, None] * start[:, :, None]
    out = out + torch.exp(upto).float()[..., None] * torch.matmul(q, states[:, :, :n].transpose(-1, -2))
    real = (s["read"] > 0)[:, None, None, None]
    s["state"][s["write"].long()] = states[:, :, n] * real
    out = (out * s["scale"] * real[..., None]).permute(0, 2, 3, 1, 4).reshape(-1, hv, c["dv"])
    # back to packed tokens
    row = torch.searchsorted(cu[1:].contiguous(), torch.arange(s["q"].shape[0], device=DEV), right=True)
    return {"out": out[row * n * CHUNK + torch.arange(len(row), device=DEV) - cu[row]].to(s["q"].dtype), "state": s["state"]}


def _attention(s):
    c = s["case"]
    hq, hkv, d, page, rows, n, members = c["hq"], c["hkv"], c["d"], c["page"], s["rows"], s["most_new"], c["members"]
    g, groups = hq // hkv, c["groups"]
    cu, length = s["cu"].long(), s["length"].long()
    token = torch.arange(s["q"].shape[0], device=DEV)
    row = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    i = token - cu[row]
    q = torch.zeros((rows, n, hq, d), device=DEV)
    q[row, i] = s["q"].float()
    q = q.view(rows, n, hkv, g, d).permute(2, 0, 3, 1, 4)  # [hkv][rows][g][n][d]
    lead, pages = s["prefix"][:, 0].long(), s["prefix"][:, 1].long()
    # the shared keys, once a group
    first = torch.arange(groups, device=DEV) * members
    at = s["table"][lead[first], : max(s["most_shared"], 1)].long()
    pk = s["k"][0][at].float().permute(2, 0, 1, 3, 4).reshape(hkv, groups, -1, d)
    pv = s["v"][0][at].float().permute(2, 0, 1, 3, 4).reshape(hkv, groups, -1, d)
    ps = torch.matmul(q.reshape(hkv, groups, members * g * n, d), pk.transpose(-1, -2)).mul_(s["scale"])
    ps.masked_fill_((torch.arange(pk.shape[2], device=DEV) >= (pages[first] * page)[:, None])[None, :, None], -math.inf)
    # every row's own keys
    held = torch.arange(s["most_own"] + s["most_shared"], device=DEV)[: s["most_own"]] + pages[:, None]
    at = torch.gather(s["table"].long(), 1, held.clamp(max=s["table"].shape[1] - 1))
    ok = s["k"][0][at].float().permute(2, 0, 1, 3, 4).reshape(hkv, rows, -1, d)
    ov = s["v"][0][at].float().permute(2, 0, 1, 3, 4).reshape(hkv, rows, -1, d)
    os = torch.matmul(q.reshape(hkv, rows, g * n, d), ok.transpose(-1, -2)).mul_(s["scale"]).view(hkv, rows, g, n, -1)
    seen = (length - (cu[1:] - cu[:-1]) - pages * page)[:, None] + torch.arange(n, device=DEV) + 1
    seen = torch.where((length > 0)[:, None], seen, 0)
    os.masked_fill_((torch.arange(ok.shape[2], device=DEV) >= seen[..., None])[None, :, None], -math.inf)
    # one softmax over both
    ps = ps.view(hkv, rows, g, n, -1)
    top = torch.maximum(ps.amax(-1, keepdim=True), os.amax(-1, keepdim=True))
    top = torch.where(torch.isinf(top), 0.0, top)
    pp, po = ps.sub_(top).exp_(), os.sub_(top).exp_()
    total = pp.sum(-1) + po.sum(-1)
    o = torch.matmul(pp.view(hkv, groups, members * g * n, -1), pv).view(hkv, rows, g, n, d)
    o = (o + torch.matmul(po.reshape(hkv, rows, g * n, -1), ov).view(hkv, rows, g, n, d)) / torch.where(total > 0, total, 1.0)[..., None]
    o = o.permute(1, 3, 0, 2, 4).reshape(rows, n, hq, d)[row, i]
    return {"out": (o * (length > 0)[row, None, None]).to(s["q"].dtype)}


def _shared(s):
    table, bounds, cu, length = s["table"], s["bounds"].long(), s["cu"].long(), s["length"].long()
    rows, groups = table.shape[0], len(bounds) - 1
    at = torch.arange(rows, device=DEV)
    group = torch.searchsorted(bounds[1:].contiguous(), at, right=True)
    before = length - (cu[1:] - cu[:-1])  # tokens that a row held before the new ones
    live = (length > 0) & (before >= 0)
    lead = torch.full((groups,), rows, device=DEV).scatter_reduce(0, group, torch.where(live, at, rows), "amin")
    lead = torch.where(lead < rows, lead, bounds[:-1])
    count = torch.zeros((groups,), dtype=torch.long, device=DEV).scatter_reduce(0, group, live.long(), "sum")
    alike = torch.cumprod((table == table[lead[group]]).int(), 1).sum(1)
    alike = torch.where(live, torch.minimum(alike, before // s["case"]["page"]), table.shape[1])
    pages = torch.full((groups,), table.shape[1], device=DEV).scatter_reduce(0, group, alike, "amin")
    pages = torch.where(count > 1, pages, 0)
    return {"prefix": torch.stack([lead[group], pages[group]], 1).int()}


# ---- the framework's operators -----------------------------------------------------------------------------------------------


def _own(s):
    import gated_deltanet_decode_gb300 as G

    c = s["case"]
    if c["op"] in ("decode", "prefill"):
        if "pool" not in s:  # a program makes the handle of its pool once
            s["pool"] = G.GDNStatePool(s["state"].shape[0], c["hk"], c["hv"], c["dk"], c["dv"], tensor=s["state"])
        if c["op"] == "decode":
            out = G.linear_attention_decode(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], s["read"], s["write"], scale=s["scale"])
        else:
            out = G.linear_attention_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], s["cu"], s["read"], s["write"],
                                             scale=s["scale"])
        return {"out": out, "state": s["state"]}
    if c["op"] == "shared":
        return {"prefix": G.kv_pages_shared(s["table"], s["length"], s["cu"], s["bounds"], c["page"])}
    if "pool" not in s:
        s["pool"] = G.KVPagePool(s["k"].shape[1], c["page"], c["hkv"], c["d"], dtype=s["k"].dtype, k=s["k"], v=s["v"])
    return {"out": G.paged_attention_shared(s["q"], s["pool"], s["table"], s["length"], s["cu"], s["bounds"], s["prefix"], scale=s["scale"])}


def run(s):
    if own:
        return _own(s)
    return {"decode": _decode, "prefill": _prefill, "attention": _attention, "shared": _shared}[s["case"]["op"]](s)


# ---- the same in 64 bits, from the definitions -------------------------------------------------------------------------------


def exact(c, seed):
    if c["op"] == "shared":
        return None
    s = prepare(c, seed)
    return {"out": _exact_attention(c, s)} if c["op"] == "attention" else _exact_linear(c, s)


def _exact_linear(c, s):
    new = _tokens(c) if c["op"] == "prefill" else [1] * c["rows"]
    g, rows = c["hv"] // c["hk"], [r for r in range(c["rows"]) if not _padding(c, r)]
    first = [sum(new[:r]) for r in range(c["rows"])]
    by_length = sorted(rows, key=lambda r: -new[r])  # so that the sequences that go on are in front
    read, write = (a[by_length] for a in _slots(c))
    state = s["state"].double()
    S = state[torch.as_tensor(read, dtype=torch.long, device=DEV)]
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    where = torch.as_tensor([first[r] for r in by_length], device=DEV)
    head = torch.arange(c["hv"], device=DEV) // g
    rate = s["log_decay"].double()
    for t in range(max([new[r] for r in rows] + [0])):
        n = sum(new[r] > t for r in by_length)
        at = where[:n] + t
        a = torch.exp(rate if c["fixed"] else rate[at]).expand(n, c["hv"])
        k, q = s["k"][at].double()[:, head], s["q"][at].double()[:, head]
        S[:n] *= a[..., None, None]
        S[:n] += torch.einsum("rhv,rhk->rhvk", s["v"][at].double(), k)
        out[at] = torch.einsum("rhvk,rhk->rhv", S[:n], q) * s["scale"]
    state[torch.as_tensor(write, dtype=torch.long, device=DEV)] = S
    return {"out": out, "state": state}


def _exact_attention(c, s):
    lay, g, at = _layout(c), c["hq"] // c["hkv"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for r, (n, length) in enumerate(zip(lay["new"], lay["length"])):
        if length:
            held = s["table"][r, : -(-length // c["page"])].long()
            see = torch.arange(length, device=DEV)[None] <= (length - n + torch.arange(n, device=DEV))[:, None]
            k = s["k"][0, held].double().transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :length]
            v = s["v"][0, held].double().transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :length]
            q = s["q"][at : at + n].double().view(n, c["hkv"], g, c["d"])
            w = torch.einsum("nhgd,hkd->hgnk", q, k) * s["scale"]
            w = torch.softmax(torch.where(see, w, -math.inf), -1)
            out[at : at + n] = torch.einsum("hgnk,hkd->nhgd", w, v).reshape(n, c["hq"], c["d"])
        at += n
    return out


# ---- what a pass cannot do without -------------------------------------------------------------------------------------------


def work(c):
    if c["op"] in ("decode", "prefill"):
        es, hk, hv, dk, dv = SIZE[c["dtype"]], c["hk"], c["hv"], c["dk"], c["dv"]
        new = _tokens(c) if c["op"] == "prefill" else [1] * c["rows"]
        live = [n for r, n in enumerate(new) if not _padding(c, r)]
        moved = sum(live) * ((2 * hk * dk + hv * dv) * es + (0 if c["fixed"] else 4 * hv)) + sum(new) * hv * dv * es
        moved += 2 * len(live) * hv * dv * dk * 4 + 12 * c["rows"] + (4 * hv if c["fixed"] else 0)
        # an outer product added, and a product with q, a token
        return {"bytes": moved, "flops": 4 * sum(live) * hv * dv * dk}
    lay = _layout(c)
    live = [(r, n, t) for r, (n, t) in enumerate(zip(lay["new"], lay["length"])) if t]
    prefix = _prefix(c, lay)
    if c["op"] == "shared":
        return {"bytes": 4 * sum(int(prefix[r, 1]) + 1 for r, _, _ in live) + 16 * len(lay["new"]) + 4 * c["groups"], "flops": 0}
    es, row_bytes = SIZE[c["dtype"]], 2 * c["hkv"] * c["d"] * SIZE[c["dtype"]]
    once = sum(int(prefix[g * c["members"], 1]) for g in range(c["groups"])) * c["page"]
    apart = sum(t - int(prefix[r, 1]) * c["page"] for r, _, t in live)
    moved = (sum(n for _, n, _ in live) + sum(lay["new"])) * c["hq"] * c["d"] * es + (once + apart) * row_bytes
    tables = 4 * ((once + apart) // c["page"] + 5 * len(lay["new"]))
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for _, n, t in live)
    return {"bytes": moved + tables, "flops": 4 * pairs * c["hq"] * c["d"]}
