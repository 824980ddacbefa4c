"""Beam search over a paged cache, row by row: every stored row is read back
right after its append and kept with its beam on the host; forks, copies on
write and compaction have to keep it bit for bit, and attention is compared
with a 64-bit softmax over exactly these rows (so E4M3 pages are checked as
closely as bf16 ones)."""
import math

import pytest
import torch

import paged_ref as ref
from decoder_greedy_decode_b200 import beam
from decoder_greedy_decode_b200.paged import PagedKV
from decoder_greedy_decode_b200.rotary import Rope
from test_gpu_paged_attention_rounding import eps

pytestmark = pytest.mark.gpu


class History:
    """The stored rows of every sequence: per sequence a list of [L, H, D]
    values (or codes with scales [L, H])."""

    def __init__(self, c):
        self.c = c
        self.pools = [c.k, c.v] + ([c.k_scale, c.v_scale] if c.k_scale is not None else [])
        self.rows = [[] for _ in range(c.n_seqs)]

    def stored(self, seqs, pos):
        """What stands at (sequence, row), for every pool [tokens, L, H, ...]."""
        page = self.c.table[seqs, pos // self.c.page_rows].long()
        assert bool((page >= 0).all())
        return [x[:, page, :, pos % self.c.page_rows].cpu() for x in self.pools]

    def add(self, seqs, pos):
        got = self.stored(seqs.cuda(), pos.cuda())
        for i, s in enumerate(seqs.tolist()):
            assert len(self.rows[s]) == int(pos[i])
            self.rows[s].append([x[i].clone() for x in got])

    def fork(self, parents):
        self.rows = [list(self.rows[p]) for p in parents]

    def check(self):
        """Every row that a sequence holds is as it was stored."""
        at = [(s, r) for s, rows in enumerate(self.rows) for r in range(len(rows))]
        seqs, pos = torch.tensor(at).cuda().unbind(1)
        for k, x in enumerate(self.stored(seqs, pos)):
            want = torch.stack([self.rows[s][r][k] for s, r in at])
            assert torch.equal(x.view(torch.uint8), want.view(torch.uint8))

    def values(self, s, layer):
        """Keys and values [H, rows, D] float64."""
        out = []
        for k in range(2):
            x = torch.stack([r[k][layer] for r in self.rows[s]], 1)
            if len(self.pools) == 4:
                x = ref.decode(x, torch.stack([r[2 + k][layer] for r in self.rows[s]], 1))
            out.append(x.double())
        return out


@pytest.mark.parametrize("fmt,D,P,window", [("bf16", 128, 8, 0), ("fp8", 64, 16, 0), ("fp8", 128, 8, 11)])
def test_every_row_of_every_beam(fmt, D, P, window):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G, W, H, Hq, V, prompt, steps, L = 2, 3, 2, 6, 500, 13, 20, 2
    S = G * W
    g = torch.Generator().manual_seed(D + P)
    c = PagedKV.create(L, 6 + S * 6, P, H, D, S, prompt + steps + P, dtype=fmt)
    h = History(c)
    rope = Rope(D // 2, theta=1e4, scaling="linear", factor=2.0)
    gk = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16().cuda()
    c.resize(torch.tensor([prompt if s % W == 0 else 0 for s in range(S)], dtype=torch.int32).cuda())
    seq = torch.arange(G).repeat_interleave(prompt) * W
    pos = torch.arange(prompt).repeat(G)
    k, v = (torch.randn((L, G * prompt, H, D), generator=g).bfloat16().cuda() for _ in range(2))
    for layer in range(L):
        c.append(layer, k[layer], v[layer], pos.int().cuda(), seqs=seq.int().cuda(), rope=rope, k_norm=gk)
    h.add(seq, pos)
    parents = [s // W * W for s in range(S)]
    c.fork(torch.tensor(parents, dtype=torch.int32).cuda())
    h.fork(parents)
    scores = torch.full((G, W), -math.inf, device="cuda")
    scores[:, 0] = 0
    base = (torch.arange(G) * W).repeat_interleave(W).int().cuda()
    n = prompt
    for t in range(steps):
        r = beam.beam_select((2 * torch.randn((G, W, V), generator=g)).cuda(), scores, out_scores=scores)
        parents = (r.parents.view(-1) + base).contiguous()
        c.fork(parents)
        h.fork(parents.cpu().tolist())
        n += 1
        c.resize(torch.full((S,), n, dtype=torch.int32, device="cuda"))
        k, v = (torch.randn((L, S, H, D), generator=g).bfloat16().cuda() for _ in range(2))
        q = torch.randn((S, Hq, D), generator=g).bfloat16().cuda()
        pos = torch.full((S,), n - 1)
        for layer in range(L):
            q_out = c.append(layer, k[layer], v[layer], pos.int().cuda(), rope=rope, q=q, k_norm=gk)
        h.add(torch.arange(S), pos)
        if t % 7 == 3:
            c.compact()
        assert c.check() == 0
        h.check()
        layer = t % L
        out, _ = c.attend(layer, q_out, window=window, return_lse=True)
        assert c.check() == 0
        lo = max(0, n - window) if window else 0
        for s in range(S):
            kk, vv = h.values(s, layer)
            qd = q_out[s].double().cpu()
            o, _, pv, mag = ref.attention(qd, kk, vv, lo, n)
            bound = eps(D, n, mag, fmt) * pv + (2.0 ** -39 * n * vv.abs().max() if fmt == "fp8" else 0.0)
            assert bool(((out[s].double().cpu() - o).abs() <= bound).all()), (t, s)
            # what a mistake would give is far outside: nothing, and the newest row missed
            missed = ref.attention(qd, kk, vv, lo, n - 1)[0]
            assert bool((o.abs() > bound).any()) and bool(((missed - o).abs() > bound).any())
