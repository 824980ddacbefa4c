"""A bounded wait of dec_paged_attention that runs out, without a fault: one
warp of the grid withholds the copies of its first tile.  The call returns with
DEC_DEV_TIMEOUT, the outputs that need the tile are left, the others are right,
and the next call on the same context is whole."""
import pytest
import torch

from decoder_greedy_decode_b200 import capi
from test_gpu_paged_attention import build

pytestmark = pytest.mark.gpu

# lens, q heads, kv heads, D, page
CASES = [
    ([700, 33, 260, 0, 40], 8, 2, 128, 16),          # runs of one tile: 44 states of the first sequence
    ([5, 3, 130] + [17] * 40, 96, 96, 64, 8),        # few workers: a run holds whole sequences
    ([8000, 5], 96, 96, 64, 64),                     # runs of 14 tiles: the ring laps
]


@pytest.fixture
def stalled():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    capi.dec_paged_attention_set_timeout_ns(20_000_000)   # 20 ms

    def stall(warp):
        capi.dec_paged_attention_set_debug_stall(0 if warp is None else warp + 1)

    yield stall
    stall(None)
    capi.dec_paged_attention_set_timeout_ns(2_000_000_000)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P", CASES)
def test_a_wait_that_runs_out_is_reported(lens, Hq, Hkv, D, P, fmt, stalled):
    c = build(lens, Hkv, D, P, fmt, seed=41)
    B, rep = len(lens), Hq // Hkv
    q = torch.randn((B, Hq, D), generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    want, want_lse = c.attend(0, q, return_lse=True)
    assert c.check() == 0
    for warp in (0, Hkv):          # KV head 0 of the first run, and of the second
        out = torch.full((B, Hq, D), 7.0, device="cuda")
        stalled(warp)
        c.attend(0, q, out=out)
        assert c.check() == capi.DEC_DEV_TIMEOUT
        left = (out == 7).flatten(2).all(2)
        right = (out == want).flatten(2).all(2)
        assert bool((left | right).all())
        # (an output is one query head's; the KV head of the late warp is 0)
        if warp == 0:
            assert bool(left[0, :rep].all())
        assert bool(left[:, :rep].any())
        # (of the joins by a whole CTA, the late one has only this head's)
        assert bool(right[:, rep:].all())
        stalled(None)
        again, lse = c.attend(0, q, return_lse=True)
        assert c.check() == 0 and torch.equal(again, want) and torch.equal(lse, want_lse)


def test_a_captured_call_keeps_its_limit(stalled):
    c = build([100, 20], 2, 64, 16, "bf16", seed=42)
    q = torch.randn((2, 4, 64)).bfloat16().cuda()
    want = c.attend(0, q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = c.attend(0, q)
    stalled(0)
    g.replay()                      # (captured before: nothing is withheld)
    assert c.check() == 0 and torch.equal(got, want)


def test_limits_that_are_refused():
    L = capi.lib()
    assert L.dec_paged_attention_set_timeout_ns(999_999) == -9
    assert L.dec_paged_attention_set_debug_stall(-1) == -9
