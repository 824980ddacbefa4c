"""dec_beam_select, dec_kv_reorder, dec_beam_backtrace and Decoder.beam_search.

Scores: the row's sum of exponentials is off by less than 2^-20 (each term
2^-21 relative, fp32 sums), so its log by 2^-20 absolute; the score is rounded
once, 2^-24 of its value.  Choices must be the reference's wherever the
reference's scores are further apart than that.
"""
import pytest
import torch

import paged_ref as ref
from decoder_greedy_decode_b200 import beam, capi, synth
from decoder_greedy_decode_b200.decoder import Decoder, to_device

pytestmark = pytest.mark.gpu
LSE = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def check(x, scores, k, done=None, eos=-1, got=None):
    G, W, V = x.shape
    if got is None:
        got = beam.beam_select(x.cuda(), scores.cuda(), k=k, done=None if done is None else done.cuda(), eos=eos)
    s, p, t, d = ref.beam(x.cpu().float(), scores, k, done, eos)
    gs = got.scores.cpu().double()
    ws = torch.from_numpy(s)
    fine = torch.isfinite(ws)
    assert bool((torch.isfinite(gs) == fine).all())
    assert bool(((gs - ws).abs()[fine] <= (LSE + 2.0 ** -24 * ws.abs())[fine]).all())
    # equal choices, but for neighbours closer than the scores' error that
    # belong to different rows (within a row the order is the logits')
    gp, gt = got.parents.cpu(), got.tokens.cpu()
    for g in range(G):
        for i in range(k):
            if (int(gp[g, i]), int(gt[g, i])) != (p[g, i], t[g, i]):
                near = [j for j in range(k) if j != i and p[g, j] != p[g, i] and abs(s[g, j] - s[g, i]) <= 4 * LSE]
                assert near or i == k - 1, (g, i, gp[g], gt[g], p[g], t[g])
    if eos >= 0:
        fd = done.bool() if done is not None else torch.zeros((G, W), dtype=torch.bool)
        want = fd.gather(1, gp.long()) | (gt == eos)
        assert torch.equal(got.done.cpu().bool(), want)
    return got


SIZES = [(1, 1, 1, 1), (1, 4, 151936, 4), (16, 4, 151936, 8), (3, 5, 1000, 7), (2, 32, 5003, 32),
         (5, 3, 33, 32), (1, 1, 50257, 1), (7, 2, 8191, 2), (1, 8, 1000000, 3), (40, 6, 2047, 6)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,W,V,k", SIZES)
def test_selection(G, W, V, k, dtype):
    if G * W * V > 6e6 and dtype == torch.bfloat16:
        G = 2
    g = torch.Generator().manual_seed(G + W + V + k)
    x = (2.5 * torch.randn((G, W, V), generator=g)).to(dtype)
    scores = -20 * torch.rand((G, W), generator=g)
    done = (torch.rand((G, W), generator=g) < 0.3).to(torch.uint8)
    eos = V // 2
    a = check(x, scores, k)
    assert a.done is None
    b = check(x, scores, k, done, eos)
    again = beam.beam_select(x.cuda(), scores.cuda(), k=k, done=done.cuda(), eos=eos)
    assert all(torch.equal(u, v) for u, v in zip(b, again))


@pytest.mark.parametrize("k", [1, 8, 32])
@pytest.mark.parametrize("order", ["random", "rising", "late"])
def test_many_rows_of_one_long_chunk(k, order):
    """Enough rows that a CTA takes each whole: thousands of logits reach the
    first bound, or the largest ones all come late."""
    G, W, V = 40, 8, 120007
    g = torch.Generator(device="cuda").manual_seed(k)
    x = torch.randn((G, W, V), generator=g, device="cuda")
    if order == "rising":
        x = x.sort(-1).values
    elif order == "late":
        x[..., V // 2:] += 1.5      # about a tenth of the second half
    scores = -3 * torch.rand((G, W), generator=g, device="cuda")
    r = beam.beam_select(x, scores, k=k)
    lse = torch.stack([row.double().logsumexp(-1) for row in x.unbind(0)])
    # the scores are those of the candidates named, and the k largest there are
    at = x[torch.arange(G, device="cuda")[:, None], r.parents.long(), r.tokens.long()].double()
    own = (scores.double() - lse).gather(1, r.parents.long()) + at
    bound = LSE + 2.0 ** -24 * own.abs()
    assert bool(((r.scores.double() - own).abs() <= bound).all())
    best = (x.topk(k, -1).values.double() + (scores.double() - lse)[..., None]).flatten(1).topk(k, -1).values
    assert bool(((own - best).abs() <= 4 * LSE).all())
    named = r.parents.long() * V + r.tokens
    assert all(len(set(row)) == k for row in named.tolist())


def test_ties_go_to_the_lowest_index():
    x = torch.zeros((2, 3, 20000))
    x[1, :, 777] = 1.0
    x[1, :, 19999] = 1.0
    got = check(x, torch.zeros((2, 3)), 5)
    assert got.parents.cpu().tolist() == [[0] * 5, [0, 0, 1, 1, 2]]
    assert got.tokens.cpu().tolist() == [[0, 1, 2, 3, 4], [777, 19999, 777, 19999, 777]]
    # zero has one value
    x = torch.full((1, 1, 100), -1.0)
    x[0, 0, 3], x[0, 0, 70] = -0.0, 0.0
    assert check(x, torch.zeros((1, 1)), 2).tokens.cpu().tolist() == [[3, 70]]


@pytest.mark.parametrize("order", [1, -1])
def test_sorted_logits(order):
    """Every chunk's largest logits sit with one thread's neighbours."""
    x = torch.linspace(-30, 10, 70001)[None, None].repeat(2, 2, 1)
    check(x if order > 0 else x.flip(-1), torch.tensor([[0.0, -1.0], [-3.0, -3.5]]), 32)


def test_masked_infinite_and_nan_rows():
    inf, nan = float("inf"), float("nan")
    x = torch.randn((6, 2, 3000), generator=torch.Generator().manual_seed(1))
    x[0, 0, 5:] = -inf                 # five tokens allowed
    x[0, 1] = -inf                     # none
    x[1, 0, 17] = nan
    x[2, 0, 2999] = inf
    x[3] = -inf                        # a whole group without candidates
    scores = torch.tensor([[-1.0, 0.0], [-1.0, -9.0], [0.0, -2.0], [0.0, 0.0], [-inf, -3.0], [nan, -4.0]])
    got = check(x, scores, 8)
    assert got.parents[3].tolist() == [0] * 8 and got.tokens[3].tolist() == list(range(8))
    assert bool((got.parents[[1, 2, 4, 5]] == 1).all())
    assert got.parents[0].tolist()[:5] == [0] * 5 and got.tokens[0].tolist()[5:] == [5, 6, 7]


def test_finished_beams():
    x = torch.randn((3, 3, 500), generator=torch.Generator().manual_seed(2))
    scores = torch.tensor([[-0.5, -30.0, -0.25], [0.0, -1.0, -2.0], [-1.0, float("-inf"), -2.0]])
    done = torch.tensor([[1, 0, 1], [1, 1, 1], [0, 1, 0]], dtype=torch.uint8)
    for eos in (0, 2, 499):
        got = check(x, scores, 6, done, eos)
        assert got.tokens[0, :2].tolist() == [eos, eos] and got.parents[0, :2].tolist() == [2, 0]
        # three finished beams: their own scores, then nothing, lowest tokens first
        rest = [t for t in range(5) if t != eos][:3]
        assert got.tokens[1].tolist() == [eos] * 3 + rest and got.scores[1].tolist()[3:] == [float("-inf")] * 3


def test_strided_unaligned_and_in_place():
    G, W, V = 3, 4, 4099
    big = torch.randn((G * W, V + 6), generator=torch.Generator().manual_seed(3))
    for dt in (torch.float32, torch.bfloat16):
        for off in (0, 1, 3):
            x = big.to(dt).cuda()[:, off:off + V].unflatten(0, (G, W))
            scores = -torch.rand((G, W))
            check(x.cpu(), scores, 3, got=beam.beam_select(x, scores.cuda(), k=3))
    scores = -torch.rand((G, W))
    done = torch.zeros((G, W), dtype=torch.uint8)
    done[1, 2] = 1
    s, d = scores.cuda(), done.cuda()
    x = big[:, :V].contiguous().view(G, W, V)
    want = beam.beam_select(x.cuda(), s.clone(), done=d.clone(), eos=5)
    got = beam.beam_select(x.cuda(), s, done=d, eos=5, out_scores=s, out_done=d)
    assert got.scores is s and all(torch.equal(u, v) for u, v in zip(got, want))
    check(x, scores, 4, done, 5, got=want)


def test_python_refusals():
    x, s = torch.zeros((2, 3, 64), device="cuda"), torch.zeros((2, 3), device="cuda")
    for bad in (dict(k=65), dict(k=0), dict(eos=64), dict(done=torch.zeros((2, 3), dtype=torch.uint8, device="cuda"))):
        with pytest.raises(capi.DecError):
            beam.beam_select(x, s, **bad)
    for xx, ss in ((x.transpose(0, 1), s.t()), (x.double(), s), (x, s.double()), (x, s[:1]), (x, s.cpu()),
                   (x[:, :, ::2], s)):
        with pytest.raises(ValueError):
            beam.beam_select(xx, ss)


def test_selection_replays_in_a_graph():
    x = torch.randn((2, 4, 9000), device="cuda")
    s = torch.zeros((2, 4), device="cuda")
    beam.beam_select(x, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = beam.beam_select(x, s)
    for seed in range(2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        check(x.cpu(), s.cpu(), 4, got=got)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("L,B,kvb,H,ctx,D", [(1, 1, 1, 1, 16, 64), (2, 8, 8, 2, 48, 128), (3, 5, 7, 3, 32, 64),
                                             (1, 64, 64, 1, 64, 128)])
def test_reorder(L, B, kvb, H, ctx, D, fmt):
    g = torch.Generator().manual_seed(B + ctx)
    shape = (L, 2, kvb, H, ctx, D)
    dt = torch.int16 if fmt == "bf16" else torch.uint8
    host = torch.randint(0, 200, shape, generator=g).to(dt)
    scale = torch.rand(shape[:-1], generator=g) if fmt == "fp8" else None
    for trial in range(3):
        parents = torch.randint(0, B, (B,), generator=g).int()
        if trial == 1:
            parents = torch.randperm(B, generator=g).int()      # cycles
        rows = torch.randint(0, ctx + 1, (B,), generator=g).int()
        if trial == 2:
            rows[:] = ctx
        dev = host.cuda()
        sd = scale.cuda() if scale is not None else None
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        beam.kv_reorder(dev.view(torch.bfloat16) if fmt == "bf16" else dev, parents.cuda(), rows.cuda(), scales=sd, status=st)
        want, ws = host.clone(), scale.clone() if scale is not None else None
        for b in range(B):
            p, n = int(parents[b]), int(rows[b])
            want[:, :, b, :, :n] = host[:, :, p, :, :n]
            if ws is not None:
                ws[:, :, b, :, :n] = scale[:, :, p, :, :n]
        assert int(st) == 0 and torch.equal(dev.cpu(), want)
        assert ws is None or torch.equal(sd.cpu(), ws)


def test_reorder_errors_change_nothing():
    x = torch.randn((1, 2, 3, 1, 16, 64), device="cuda").bfloat16()
    was = x.clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for par, rows, bit in (([0, 1, 3], [5, 5, 5], 8), ([1, -1, 0], [5, 5, 5], 8), ([1, 2, 0], [5, 17, 5], 1),
                           ([1, 2, 0], [-1, 5, 5], 1)):
        st.zero_()
        beam.kv_reorder(x, torch.tensor(par, dtype=torch.int32).cuda(), torch.tensor(rows, dtype=torch.int32).cuda(),
                        status=st)
        assert int(st) == bit and torch.equal(x, was)


def test_backtrace():
    g = torch.Generator().manual_seed(5)
    for n, G, W in ((1, 1, 1), (7, 3, 4), (40, 2, 32)):
        par = torch.randint(0, W, (n, G, W), generator=g).int()
        tok = torch.randint(0, 1000, (n, G, W), generator=g).int()
        got = beam.backtrace(par.cuda(), tok.cuda()).cpu()
        for a in range(G):
            for w in range(W):
                at, seq = w, []
                for t in reversed(range(n)):
                    seq.append(int(tok[t, a, at]))
                    at = int(par[t, a, at])
                assert got[a, w].tolist() == seq[::-1]
    par[3, 0, :] = 99
    assert bool((beam.backtrace(par.cuda(), tok.cuda())[0, :, :3] == -1).all())


# ------------------------------------------------------------- beam search
def _search_by_steps(dec, s, kv_host, tok, pos, n, W, eos):
    """Beam search by single-sequence steps: every hypothesis is decoded from
    the prompt again, token by token, on a cache of its own."""
    kv = dec.kv_cache(1, kv_host.shape[4])
    out, logits = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((1, s.vocab), device="cuda")

    def last_logits(seq):
        kv.values.copy_(kv_host.cuda())
        for i, t in enumerate([tok] + seq):
            dec.step(kv, torch.tensor([t], dtype=torch.int32, device="cuda"),
                     torch.tensor([pos + i], dtype=torch.int32, device="cuda"), out, logits)
        return torch.log_softmax(logits[0].double(), 0).cpu()

    hyps = [([], 0.0, False)]
    margin = float("inf")
    for _ in range(n):
        cand = []
        for seq, sc, done in hyps:
            if done:
                cand.append((sc, seq + [eos], True))
                continue
            lp = last_logits(seq)
            top = torch.topk(lp, W + 1)
            cand += [(sc + float(v), seq + [int(i)], int(i) == eos) for v, i in zip(top.values, top.indices)]
        cand.sort(key=lambda c: -c[0])
        margin = min([margin] + [cand[i][0] - cand[i + 1][0] for i in range(min(W, len(cand) - 1))])
        hyps = [(seq, sc, d) for sc, seq, d in cand[:W]]
    return hyps, margin


@pytest.mark.parametrize("eos", [-1, 7])
@pytest.mark.parametrize("batch", [4, 8])
def test_beam_search_equals_decoding_every_hypothesis(batch, eos):
    """Two groups (one for the persistent step's batches): the sequences and
    scores are those of a search that decodes each hypothesis alone."""
    s = synth.TINY
    W, n = 4, 6
    w = synth.model_weights(s, seed=3)
    G = batch // W
    lens = [20, 33][:G]
    dec = Decoder(s, to_device(w), batch)
    host, _ = synth.kv_prefill(s, batch, 64, [lens[b // W] if b % W == 0 else 0 for b in range(batch)], seed=4)
    kv = dec.kv_cache(batch, 64)
    kv.values.copy_(host.cuda())
    tok = synth.tokens(s.vocab, G, seed=5)
    if eos >= 0:   # an end token that the search meets: the best second token of the first group
        free, _ = dec.beam_search(kv, tok.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 2, W)
        eos = int(free[0, 0, 1])
        kv.values.copy_(host.cuda())
    seqs, scores = dec.beam_search(kv, tok.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), n, W, eos=eos)
    assert dec.check() == 0
    one = Decoder(s, to_device(w), 1)
    for g in range(G):
        want, margin = _search_by_steps(one, s, host[:, :, g * W: g * W + 1], int(tok[g]), lens[g], n, W, eos)
        # logits of the two paths differ by rounding only
        got = scores[g].cpu().double()
        assert bool(((got - torch.tensor([h[1] for h in want], dtype=torch.float64)).abs() <= 1e-3).all())
        if margin > 1e-3:
            assert seqs[g].cpu().tolist() == [h[0] for h in want]
    dec.close(), one.close()


def test_beam_search_on_an_e4m3_cache():
    """Every beam's cache and score agree with feeding its tokens one by one."""
    s = synth.TINY
    w = synth.model_weights(s, seed=13)
    dec = Decoder(s, to_device(w), 8)
    codes, scales = synth.kv_prefill(s, 8, 64, [25, 0, 0, 0, 40, 0, 0, 0], seed=8, kind="fp8")
    tok, pos = synth.tokens(s.vocab, 2, seed=9).cuda(), torch.tensor([25, 40], dtype=torch.int32).cuda()
    kv = dec.kv_cache(8, 64, "fp8")
    kv.codes.copy_(codes.cuda()), kv.scales.copy_(scales.cuda())
    n = 5
    seqs, scores = dec.beam_search(kv, tok, pos, n, 4)
    assert dec.check() == 0
    one = dec.kv_cache(8, 64, "fp8")
    for a in (one.codes, one.scales):
        src = codes if a is one.codes else scales
        for b in range(8):
            a[:, :, b].copy_(src[:, :, b // 4 * 4].cuda())
    total = torch.zeros(8, dtype=torch.float64)
    ids, logits = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros((8, s.vocab), device="cuda")
    feed, at = tok.repeat_interleave(4), pos.repeat_interleave(4)
    for t in range(n):
        dec.step(one, feed, at, ids, logits)
        feed = seqs.view(8, n)[:, t].contiguous()
        lp = torch.log_softmax(logits.double(), 1).cpu()
        total += lp.gather(1, feed.cpu().long()[:, None])[:, 0]
        at = at + 1
    # (the same kernels on the same rows: the logits are equal, a score is a
    # sum of n fp32 values of at most 64 off by 2^-19 + 2^-24 64 each)
    assert bool(((scores.view(8).cpu().double() - total).abs() <= n * (LSE + 2.0 ** -18)).all())
    for b in range(8):
        m = int(pos[b // 4]) + n
        assert torch.equal(kv.codes[:, :, b, :, :m], one.codes[:, :, b, :, :m])
        assert torch.equal(kv.scales[:, :, b, :, :m], one.scales[:, :, b, :, :m])
    dec.close()


def test_beam_search_of_one_beam_is_greedy():
    s = synth.TINY
    w = synth.model_weights(s, seed=9)
    dec = Decoder(s, to_device(w), 2)
    host, _ = synth.kv_prefill(s, 2, 64, [10, 30], seed=6)
    tok, pos = synth.tokens(s.vocab, 2, seed=7).cuda(), torch.tensor([10, 30], dtype=torch.int32).cuda()
    kv = dec.kv_cache(2, 64)
    kv.values.copy_(host.cuda())
    seqs, _ = dec.beam_search(kv, tok, pos, 8, 1)
    kv.values.copy_(host.cuda())
    out = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    dec.generate(kv, tok, pos.clone(), out)
    assert dec.check() == 0 and torch.equal(seqs[:, 0].t(), out)
    with pytest.raises(ValueError):
        dec.beam_search(kv, tok, pos, 4, 2)
    with pytest.raises(ValueError):
        dec.beam_search(kv, tok, pos, 0, 1)
    dec.close()
