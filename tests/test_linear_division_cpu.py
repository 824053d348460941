"""How linear_attention_prefill divides sequences into segments, seen in its workspace: against every number of pieces looked at
one by one, and in little host time.  No GPU."""
import ctypes
import random
import time

import pytest

from gated_deltanet_decode_gb300 import _lib

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
F32, BF16 = 0, 1
SMS = 152


@pytest.fixture(scope="module")
def L():
    return _lib.load()


def make_pool(L, *dims):
    h = ctypes.c_void_p()
    assert L.gdn_state_pool_wrap(FAKE, 9, _lib.gdn_dims(*dims), ctypes.byref(h)) == 0
    return h


def segment(hv, dk, dv, dtype, nseq, tokens):
    """Tokens of a segment, by the rules of linear_attn_tc.cu and linear_attn_f32.cu."""
    tc = dtype == BF16 and dk in (64, 128) and dv in (64, 128)
    C = 128 if tc else 64
    m = -(-tokens // (nseq * C))
    vb = 32 if dk == 256 else 64
    blocks = nseq * hv * (1 if tc else -(-dv // vb))
    at_once = SMS if tc or dk > 64 else 2 * SMS
    begin, part, more = (1.0, 0.5, 3.0) if tc else (0.5, 0.25, 1.0)
    best, least = None, 1e30
    for cuts in range(1, min(m, SMS if tc else 2 * at_once) + 1):
        n = -(-m // cuts)
        segs = -(-m // n)
        cost = -(-segs * blocks // at_once) * (n + begin)
        if segs > 1:
            cost += -(-(segs - 1) * blocks // at_once) * (part * n + begin) + more
        if cost < least:
            least, best = cost, n
    if tc and best == m:
        best = max(2 * m, 4)
    return C * min(best, 1 << 20)


def test_the_same_as_every_number_of_pieces(L):
    rng = random.Random(1)
    for dims in ((1, 2, 128, 128), (16, 16, 64, 64), (2, 32, 128, 64), (4, 4, 256, 136), (3, 6, 32, 40), (1, 1, 16, 8)):
        pool = make_pool(L, *dims)
        hv, dk, dv = dims[1:]
        for dtype in (F32, BF16):
            for _ in range(60):
                nseq = int(2 ** rng.uniform(0, 7))
                tokens = int(2 ** rng.uniform(0, 18)) + rng.randrange(3)
                tokens = max(tokens, 1)
                span = segment(hv, dk, dv, dtype, nseq, tokens)
                want = 0 if tokens <= 20 or tokens <= span else 4 * (tokens // span + nseq + 1) * hv * (dv * dk + 1)
                assert L.linear_attention_prefill_workspace_bytes(pool, nseq, tokens, dtype) == want, (dims, dtype, nseq, tokens)
        L.gdn_state_pool_destroy(pool)


def test_a_long_sequence_costs_no_host_time(L):
    """Tried one by one, the pieces of 40,000 tokens took nine microseconds, five times as long as the rest of the call."""
    pool = make_pool(L, 8, 8, 64, 64)
    best = {100: 1e9, 40000: 1e9}
    for _ in range(30):
        for tokens in best:
            t = time.perf_counter()
            for _ in range(100):
                L.linear_attention_prefill_workspace_bytes(pool, 1, tokens, F32)
            best[tokens] = min(best[tokens], time.perf_counter() - t)
    L.gdn_state_pool_destroy(pool)
    assert best[40000] < 3 * best[100], best
