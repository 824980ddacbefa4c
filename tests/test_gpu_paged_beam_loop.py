"""The operators run together as they are used: beam search over a paged cache.

Every step selects beams, forks their pages, reserves the next row, appends the
new (normalised, rotated) rows and attends.  The attention of every beam is
compared with a 64-bit recompute over the beam's own history, kept on the host
as plain lists of raw keys and values."""
import math

import pytest
import torch

import paged_ref as ref
from decoder_greedy_decode_b200 import beam
from decoder_greedy_decode_b200.paged import PagedKV
from decoder_greedy_decode_b200.rotary import Rope

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,D,P,window", [("bf16", 128, 8, 0), ("fp8", 64, 16, 0), ("bf16", 64, 8, 12)])
def test_beam_search_over_pages(fmt, D, P, window):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G, W, H, Hq, V, prompt, steps, L = 2, 3, 2, 6, 500, 13, 20, 2
    S = G * W
    g = torch.Generator().manual_seed(D + P)
    c = PagedKV.create(L, 6 + S * 6, P, H, D, S, prompt + steps + P, dtype=fmt)
    rope = Rope(D // 2, theta=1e4, scaling="linear", factor=2.0)
    f = ref.inv_freq(D // 2, 1e4, "linear", 2.0)
    gk = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16()
    raw_k = [[] for _ in range(S)]   # per sequence: [H, D] float64 rows as appended
    raw_v = [[] for _ in range(S)]

    def rows_now(n):
        return torch.full((S,), n, dtype=torch.int32, device="cuda")

    # prompts: sequence g * W holds them, its beams fork from it
    first = torch.tensor([i * W if i * W == s else -1 for s in range(S) for i in [s // W]])
    target = torch.where(first >= 0, prompt, 0).int().cuda()
    c.resize(target)
    k = torch.randn((G * prompt, H, D), generator=g).bfloat16()
    v = torch.randn((G * prompt, H, D), generator=g).bfloat16()
    seq = torch.arange(G).repeat_interleave(prompt).int() * W
    pos = torch.arange(prompt).repeat(G).int()
    for layer in range(L):
        c.append(layer, k.cuda(), v.cuda(), pos.cuda(), seqs=seq.cuda(), rope=rope, k_norm=gk.cuda())
    turned = ref.rotate(ref.rms_norm(k.double(), gk, 1e-6), pos, f, False, 1.0)
    for i in range(G):
        raw_k[i * W] = list(turned[i * prompt:(i + 1) * prompt])
        raw_v[i * W] = list(v[i * prompt:(i + 1) * prompt].double())
    c.fork(torch.tensor([s // W * W for s in range(S)], dtype=torch.int32).cuda())
    for s in range(S):
        raw_k[s], raw_v[s] = list(raw_k[s // W * W]), list(raw_v[s // W * W])

    scores = torch.full((G, W), -math.inf, device="cuda")
    scores[:, 0] = 0
    base = (torch.arange(G) * W).repeat_interleave(W).int().cuda()
    n = prompt
    for t in range(steps):
        logits = (2 * torch.randn((G, W, V), generator=g)).cuda()
        r = beam.beam_select(logits, scores, out_scores=scores)
        parents = (r.parents.view(-1) + base).contiguous()
        c.fork(parents)
        n += 1
        c.resize(rows_now(n))
        pl = parents.cpu().tolist()
        raw_k, raw_v = [list(raw_k[p]) for p in pl], [list(raw_v[p]) for p in pl]
        k = torch.randn((S, H, D), generator=g).bfloat16()
        v = torch.randn((S, H, D), generator=g).bfloat16()
        q = torch.randn((S, Hq, D), generator=g).bfloat16()
        pos = torch.full((S,), n - 1, dtype=torch.int32)
        for layer in range(L):
            q_out = c.append(layer, k.cuda(), v.cuda(), pos.cuda(), rope=rope, q=q.cuda(), k_norm=gk.cuda())
        turned = ref.rotate(ref.rms_norm(k.double(), gk, 1e-6), pos, f, False, 1.0)
        for s in range(S):
            raw_k[s].append(turned[s])
            raw_v[s].append(v[s].double())
        out, lse = c.attend(t % L, q_out, window=window, return_lse=True)
        assert c.check() == 0
        lo = max(0, n - window) if window else 0
        for s in range(S):
            kk, vv = torch.stack(raw_k[s], 1), torch.stack(raw_v[s], 1)
            o, l, pv, mag = ref.attention(q_out[s].double().cpu(), kk, vv, lo, n)
            # stored keys are off by half a step of their type (bf16 2^-8, E4M3
            # 2^-4 and subnormal codes), which moves every score by at most
            # that share of sum |q k|, and values by the same share
            half = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -4 + 2.0 ** -10
            bound = (2 * half * mag + half) * pv.amax(-1, keepdim=True) + vv.abs().max() * (2.0 ** -10 if fmt == "fp8" else 0)
            assert bool(((out[s].double().cpu() - o).abs() <= bound + 1e-6).all()), (t, s)
        if t % 7 == 3:
            live = c.compact()
            assert int(live) == int((c.refs > 0).sum()) and c.check() == 0
    # the pages hold exactly what the sequences name
    held = c.table.cpu().flatten()
    assert torch.equal(torch.bincount(held[held >= 0].long(), minlength=c.n_pages).int(), c.refs.cpu())
    c.resize(rows_now(0))
    assert int(c.refs.sum()) == 0 and int((c.table >= 0).sum()) == 0


def search_state(fmt):
    """A cache of two groups of two beams with 21 shared rows (a page and a
    part of the next), and the buffers of a step."""
    g = torch.Generator().manual_seed(5)
    G, W, H, Hq, D, P, V = 2, 2, 2, 4, 64, 16, 300
    S = G * W
    c = PagedKV.create(1, 24, P, H, D, S, 64, dtype=fmt)
    c.resize(torch.tensor([21, 0, 21, 0], dtype=torch.int32).cuda())
    seq = torch.tensor([0] * 21 + [2] * 21, dtype=torch.int32).cuda()
    pos = torch.arange(21, dtype=torch.int32).repeat(2).cuda()
    k, v = (torch.randn((42, H, D), generator=g).bfloat16().cuda() for _ in range(2))
    c.append(0, k, v, pos, seqs=seq)
    c.fork(torch.tensor([0, 0, 2, 2], dtype=torch.int32).cuda())
    steps = [dict(logits=torch.randn((G, W, V), generator=g).cuda(),
                  k=torch.randn((S, H, D), generator=g).bfloat16().cuda(),
                  v=torch.randn((S, H, D), generator=g).bfloat16().cuda(),
                  q=torch.randn((S, Hq, D), generator=g).bfloat16().cuda()) for _ in range(14)]
    return c, Rope(D, theta=1e4), torch.tensor([[0.0, -1.0]] * G).cuda(), \
        torch.tensor([0, 0, 2, 2], dtype=torch.int32).cuda(), \
        torch.full((S,), 21, dtype=torch.int32).cuda(), steps


def search_step(c, rope, scores, base, pos, x, stream=None):
    r = beam.beam_select(x["logits"], scores, out_scores=scores, stream=stream)
    with torch.cuda.stream(stream):
        parents = r.parents.view(-1) + base
        rows = pos + 1
    c.fork(parents, stream=stream)
    c.resize(rows, stream=stream)
    q = c.append(0, x["k"], x["v"], pos, rope=rope, q=x["q"], stream=stream)
    out = c.attend(0, q, stream=stream)
    with torch.cuda.stream(stream):
        pos.copy_(rows)
    return r.tokens, out


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_the_same_search_on_a_side_stream_and_in_a_graph(fmt):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c, *rest, steps = search_state(fmt)
    want = [search_step(c, *rest, x) for x in steps]
    assert c.check() == 0
    end = c.table.clone()

    c, *rest, _ = search_state(fmt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [search_step(c, *rest, x, stream=side) for x in steps]
    side.synchronize()
    for (t, o), (t0, o0) in zip(got, want):
        assert torch.equal(t, t0) and torch.equal(o, o0)
    assert torch.equal(c.table, end) and c.check() == 0

    c, *rest, _ = search_state(fmt)
    now = {n: x.clone() for n, x in steps[0].items()}
    t, o = search_step(c, *rest, now)   # (the first call sets up what a capture may not)
    assert torch.equal(t, want[0][0]) and torch.equal(o, want[0][1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t, o = search_step(c, *rest, now)
    for x, (t0, o0) in zip(steps[1:], want[1:]):
        for n in now:
            now[n].copy_(x[n])
        graph.replay()
        assert torch.equal(t, t0) and torch.equal(o, o0)
    assert torch.equal(c.table, end) and c.check() == 0
