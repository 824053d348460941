"""A small hybrid decoder's serving steps: GDN layers and attention layers over one set of rows.

Three of four layers are GDN layers (a conv window and a recurrent state a row, in slots), every fourth is an attention
layer (keys and values a row, in pages).  Each step takes some new tokens of every row: a prompt's chunk, one token in
decode, or several to be verified, mixed as they come.  Rows are forked (sampled several times), released, and the page
pool is squeezed together, while decoding goes on.

    python examples/hybrid_step.py

The projections are random and stand for a model's; everything between them is the library's.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_decode_gb300 as G  # noqa: E402

HIDDEN, LAYERS = 256, 8
HK, HV, DK, DV, WIDTH = 2, 4, 64, 64, 4           # GDN layers
HQ, HKV, D, ROT, PAGE = 8, 2, 64, 32, 16          # attention layers
BF16 = torch.bfloat16


def is_attention(layer):
    return layer % 4 == 3


class Decoder:
    """Weights, and the rows' state: slot r + 1 of the GDN pools and row r of the page table are row r's."""

    def __init__(self, rows, max_tokens, pages, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s, scale=1.0: torch.randn(s, generator=gen, device=device, dtype=torch.float32) * scale  # noqa: E731
        self.rows, self.device = rows, torch.device(device)
        self.weights, self.gdn = [], {}
        channels = 2 * HK * DK + HV * DV
        for layer in range(LAYERS):
            if is_attention(layer):
                self.weights.append(dict(
                    qkv=rand(HIDDEN, (HQ + 2 * HKV) * D, scale=HIDDEN ** -0.5).to(BF16),
                    out=rand(HQ * D, HIDDEN, scale=(HQ * D) ** -0.5).to(BF16),
                    q_norm=1 + 0.1 * rand(D), k_norm=1 + 0.1 * rand(D)))
            else:
                self.weights.append(dict(
                    x=rand(HIDDEN, channels, scale=HIDDEN ** -0.5).to(BF16), ab=rand(HIDDEN, 2 * HV, scale=HIDDEN ** -0.5).to(BF16),
                    out=rand(HV * DV, HIDDEN, scale=(HV * DV) ** -0.5).to(BF16),
                    conv=rand(channels, WIDTH, scale=0.5).to(BF16), bias=rand(channels, scale=0.1).to(BF16),
                    A_log=rand(HV, scale=0.5), dt_bias=rand(HV, scale=0.5)))
                self.gdn[layer] = (G.ConvStatePool(rows + 1, channels, WIDTH, device=device),
                                   G.GDNStatePool(rows + 1, HK, HV, DK, DV, device=device))
        i32 = dict(dtype=torch.int32, device=device)
        self.pool = G.KVPagePool(pages, PAGE, HKV, D, layers=LAYERS // 4, device=device)
        self.table = torch.zeros((rows, -(-max_tokens // PAGE)), **i32)
        self.length = torch.zeros(rows, **i32)
        self.refs = torch.zeros(pages, **i32)
        self.moves = G.KVPageMoves(pages, device=device)
        self.rope = G.rope_table(ROT, max_tokens, base=10000.0, scaling={"type": "linear", "factor": 2}, device=device)
        self.slots = torch.arange(1, rows + 1, **i32)
        self.all_rows = torch.arange(rows, **i32)

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def step(self, x, new):
        """x [sum(new)][HIDDEN]: new[r] tokens of row r (0 for a row that rests).  Returns the last layer's output.  A row
        that gets no pages (self.status) rests too: its length, pages and states stay, and its outputs mean nothing."""
        counts = self.ints(new)
        cu = torch.zeros(self.rows + 1, dtype=torch.int32, device=self.device)
        torch.cumsum(counts, 0, out=cu[1:])
        # the attention layers' rows: lengths with the new tokens, pages for them
        held = self.length + counts
        status = G.kv_pages_reserve(self.table, self.refs, self.all_rows, held, PAGE)
        served = status == 0
        self.length.copy_(torch.where(served, held, self.length))
        seen = torch.where(served, held, 0)  # a padding row, where there are no pages for its tokens
        busy = torch.where(served & (counts > 0), self.slots, 0).to(torch.int32)
        decode = all(n == 1 for n in new)
        for layer, w in enumerate(self.weights):
            if is_attention(layer):
                y = (x @ w["qkv"]).view(len(x), HQ + 2 * HKV, D)
                q, k, v = y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:]
                q = G.attn_prologue(q, k, v, self.pool, self.rope, self.table, seen, cu, layer=layer // 4,
                                    q_norm=w["q_norm"], k_norm=w["k_norm"])
                o = G.paged_attention(q, self.pool, self.table, seen, cu, layer=layer // 4)
            else:
                conv, state = self.gdn[layer]
                y, ab = x @ w["x"], x @ w["ab"]
                a, b = ab[:, :HV].contiguous(), ab[:, HV:].contiguous()
                if decode:
                    o = G.gdn_layer_decode(y, conv, w["conv"], w["bias"], w["A_log"], w["dt_bias"], a, b, state, busy,
                                           keep_in_place=True)
                else:
                    y = G.causal_conv1d_prefill(y, conv, cu, busy, w["conv"], w["bias"])
                    q, k, v = y.split([HK * DK, HK * DK, HV * DV], 1)
                    o = G.gdn_prefill(q.contiguous(), k.contiguous(), v.contiguous(), a, b, w["A_log"], w["dt_bias"], state,
                                      cu, busy, keep_in_place=True)
            x = x + o.reshape(len(x), -1) @ w["out"]
        self.status = status
        return x

    def fork(self, src, dst):
        """Rows dst (empty) go on from where rows src are: slots and partial pages copied, full pages shared.  Where the
        status is not 0 nothing is done."""
        moves = G.KVPageMoves(len(src), device=self.device)
        G.kv_pages_fork(self.table, self.length, self.refs, self.ints(src), self.ints(dst), PAGE, moves)
        G.kv_pages_copy(self.pool, moves)
        done = moves.status == 0
        src, dst = self.slots[self.ints(src)[done]], self.slots[self.ints(dst)[done]]
        for conv, state in self.gdn.values():
            for pool in (conv, state):
                pool.copy_slots(src, dst)
        return moves.status

    def release(self, rows):
        G.kv_pages_free(self.table, self.length, self.refs, self.ints(rows))
        for conv, state in self.gdn.values():
            for pool in (conv, state):
                pool.zero_slots(self.ints([r + 1 for r in rows]))

    def compact(self):
        """Squeeze the pages in use to the lowest numbers."""
        G.kv_pages_compact(self.table, self.refs, self.moves)
        G.kv_pages_copy(self.pool, self.moves)


def main():
    rows = 6
    model = Decoder(rows, max_tokens=512, pages=160)
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = lambda n: torch.randn((n, HIDDEN), generator=gen, device="cuda").to(BF16)  # noqa: E731
    model.step(tokens(37 + 120 + 5), [37, 120, 5, 0, 0, 0])          # three prompts
    model.step(tokens(1 + 64 + 4), [1, 64, 4, 0, 0, 0])              # decode, a prompt's next chunk, a verification
    status = model.fork([1, 1], [3, 4])                              # row 1 sampled three times
    x = tokens(3)
    y = model.step(torch.cat([x, x[1:2], x[1:2]]), [1, 1, 1, 1, 1, 0])
    same = torch.equal(y[1], y[3]) and torch.equal(y[1], y[4])
    model.release([0, 1])
    model.compact()
    for _ in range(3):
        y = model.step(tokens(3), [0, 0, 1, 1, 1, 0])
    torch.cuda.synchronize()
    used = int((model.refs > 0).sum())
    print(f"forks {status.tolist()}, forked rows alike: {same}; pages in use {used}, the highest "
          f"{int(model.table.max())}; lengths {model.length.tolist()}; error word {G.get_device_error()}")
    return same and torch.isfinite(y).all().item()


if __name__ == "__main__":
    sys.exit(0 if main() else 1)
