"""Linear attention layers and attention over shared prefixes as a decoder uses them together: one prompt, forked into
samples that decode, are released and forked again, against the same samples decoded apart."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HIDDEN, HK, HV, DK, DV = 128, 2, 4, 64, 64  # linear attention layers
HQ, HKV, D, PAGE = 8, 2, 64, 16             # attention layers
LAYERS = 4                                  # every second one is an attention layer
DEV = "cuda"


class Decoder:
    """Slot r + 1 of every state pool and row r of the page table are row r's."""

    def __init__(self, G, rows, pages, dtype, shared):
        self.G, self.rows, self.shared = G, rows, shared
        gen = torch.Generator().manual_seed(0)
        rand = lambda *s: (torch.randn(s, generator=gen) * s[0] ** -0.5).to(dtype).to(DEV)  # noqa: E731
        self.w, self.states = [], {}
        for i in range(LAYERS):
            if i % 2:
                self.w.append((rand(HIDDEN, (HQ + 2 * HKV) * D), rand(HQ * D, HIDDEN)))
            else:
                self.w.append((rand(HIDDEN, 2 * HK * DK + HV * DV), rand(HV * DV, HIDDEN), rand(HIDDEN, HV)))
                self.states[i] = G.GDNStatePool(rows + 1, HK, HV, DK, DV)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.pool = G.KVPagePool(pages, PAGE, HKV, D, layers=LAYERS // 2, dtype=dtype)
        self.table, self.length, self.refs = torch.zeros((rows, 40), **i32), torch.zeros(rows, **i32), torch.zeros(pages, **i32)
        self.rope = G.rope_table(32, 640)
        self.every = torch.arange(rows, **i32)

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def step(self, x, new, bounds):
        G = self.G
        counts = self.ints(new)
        cu = torch.zeros(self.rows + 1, dtype=torch.int32, device=DEV)
        torch.cumsum(counts, 0, out=cu[1:])
        self.length += counts
        assert (G.kv_pages_reserve(self.table, self.refs, self.every, self.length, PAGE) == 0).all()
        seen = torch.where(counts > 0, self.length, 0)
        slots = torch.where(counts > 0, self.every + 1, 0).to(torch.int32)
        if self.shared:
            bounds = self.ints(bounds)
            prefix = G.kv_pages_shared(self.table, seen, cu, bounds, PAGE)
        for i, w in enumerate(self.w):
            y = x @ w[0]
            if i % 2:
                y = y.view(len(x), HQ + 2 * HKV, D)
                q = G.attn_prologue(y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:], self.pool, self.rope, self.table, seen, cu, layer=i // 2)
                if self.shared:
                    o = G.paged_attention_shared(q, self.pool, self.table, seen, cu, bounds, prefix, layer=i // 2)
                else:
                    o = G.paged_attention(q, self.pool, self.table, seen, cu, layer=i // 2)
            else:
                a, b = HK * DK, 2 * HK * DK
                q, k, v = y[:, :a].view(-1, HK, DK), y[:, a:b].view(-1, HK, DK) * DK ** -0.5, y[:, b:].view(-1, HV, DV)
                g = -torch.nn.functional.softplus((x @ w[2]).float() - 2)
                if len(x) == self.rows and all(n == 1 for n in new):
                    o = G.linear_attention_decode(q, k, v, g, self.states[i], slots, keep_in_place=True)
                else:
                    o = G.linear_attention_prefill(q, k, v, g, self.states[i], cu, slots, keep_in_place=True)
            x = x + o.reshape(len(x), -1) @ w[1]
        return x

    def fork(self, src, dst):
        G, s, d = self.G, self.ints(src), self.ints(dst)
        moves = G.KVPageMoves(len(src))
        G.kv_pages_fork(self.table, self.length, self.refs, s, d, PAGE, moves)
        G.kv_pages_copy(self.pool, moves)
        assert (moves.status == 0).all()
        for p in self.states.values():
            p.copy_slots(s + 1, d + 1)

    def release(self, rows):
        self.G.kv_pages_free(self.table, self.length, self.refs, self.ints(rows))
        for p in self.states.values():
            p.zero_slots(self.ints([r + 1 for r in rows]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_samples_of_a_prompt(gdn, dtype):
    rows, prompt = 6, 171
    gen = torch.Generator().manual_seed(1)
    tokens = lambda n: torch.randn(n, HIDDEN, generator=gen).to(dtype).to(DEV)  # noqa: E731
    p, other = tokens(prompt), tokens(40)
    together, apart = Decoder(gdn, rows, 120, dtype, True), Decoder(gdn, rows, 120, dtype, False)
    # rows 0 .. 3 sample one prompt, rows 4 and 5 another: forked here, each by itself there
    a = together.step(torch.cat([p, other]), [prompt, 0, 0, 0, 40, 0], [0, 4, 6])
    b = apart.step(torch.cat([p, p, p, p, other, other]), [prompt] * 4 + [40] * 2, [0, 4, 6])
    together.fork([0, 0, 0, 4], [1, 2, 3, 5])

    # A layer is two products and an operator; in fp32 all are right to some 2^-20 of their size, in bf16 each rounds its
    # result and its factors to 2^-8; their norms add up over eight of these and three steps of feeding back.
    bound = 2.0 ** -14 if dtype == torch.float32 else 24 * 2.0 ** -8

    def alike(x, y):
        x, y = x.double(), y.double()
        assert torch.isfinite(x).all() and (x - y).norm() <= bound * y.norm()

    alike(a[:prompt], b[:prompt])
    for new in ([1] * 6, [1, 3, 1, 2, 1, 4], [1] * 6):
        x = tokens(sum(new))
        alike(together.step(x, new, [0, 4, 6]), apart.step(x, new, [0, 4, 6]))
    for d in (together, apart):
        d.release([0, 5])
    together.fork([2], [0])
    apart.step(torch.cat([p] + [tokens(0)]), [prompt, 0, 0, 0, 0, 0], [0, 4, 6])  # row 0 anew, from the prompt
    for d in (together, apart):
        d.release([0])
    new = [0, 1, 1, 1, 1, 0]
    x = tokens(4)
    alike(together.step(x, new, [0, 4, 6]), apart.step(x, new, [0, 4, 6]))
    assert gdn.get_device_error() == 0
