"""Plain 64-bit definitions of the paged-cache and beam-search operators (CPU,
numpy / Python lists), written from their formulas for the tests."""
import math

import numpy as np
import torch


class RefMap:
    """Pages of sequences as Python lists, changed one sequence at a time."""

    def __init__(self, n_pages, n_seqs, width, P):
        self.P, self.width = P, width
        self.refs = [0] * n_pages
        self.pages = [[] for _ in range(n_seqs)]
        self.rows = [0] * n_seqs
        self.copies = []      # (from, to, rows) of the last resize / compact

    def need(self, rows):
        return -(-rows // self.P)

    def resize(self, target):
        """False (and nothing changed) if the pages do not suffice."""
        refs = list(self.refs)
        tgt = [o if n < 0 else n for o, n in zip(self.rows, target)]
        for s, n in enumerate(tgt):
            for p in self.pages[s][self.need(n):]:
                refs[p] -= 1
        free = [i for i, r in enumerate(refs) if r == 0]
        pages, copies = [], []
        for s, n in enumerate(tgt):
            mine = list(self.pages[s][: self.need(n)])
            old = self.rows[s]
            if n > old:
                if old % self.P and refs[mine[-1]] > 1:
                    if not free:
                        return False
                    new = free.pop(0)
                    copies.append((mine[-1], new, old % self.P))
                    refs[mine[-1]] -= 1
                    refs[new] = 1
                    mine[-1] = new
                while len(mine) < self.need(n):
                    if not free:
                        return False
                    mine.append(free.pop(0))
                    refs[mine[-1]] = 1
            pages.append(mine)
        self.refs, self.pages, self.rows, self.copies = refs, pages, tgt, copies
        return True

    def fork(self, parents):
        self.pages = [[] if p < 0 else list(self.pages[p]) for p in parents]
        self.rows = [0 if p < 0 else self.rows[p] for p in parents]
        self.recount()

    def recount(self):
        self.refs = [0] * len(self.refs)
        for pp in self.pages:
            for p in pp:
                self.refs[p] += 1

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        src = [i for i, r in enumerate(self.refs) if r > 0 and i >= n]
        dst = [i for i, r in enumerate(self.refs) if r == 0 and i < n]
        to = dict(zip(src, dst))
        self.copies = [(a, b, self.P) for a, b in to.items()]
        self.pages = [[to.get(p, p) for p in pp] for pp in self.pages]
        self.recount()
        return n

    def table(self):
        return [pp + [-1] * (self.width - len(pp)) for pp in self.pages]

    def move(self, *pools):
        """Apply the last copies to pools [L, n_pages, H, P, ...] (CPU tensors)."""
        for x in pools:
            was = x.clone()
            for a, b, r in self.copies:
                x[:, b, :, :r] = was[:, a, :, :r]


def decode(codes, scales):
    """E4M3 codes [..., D] and scales [...] -> float64."""
    return codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None]


def attention(q, k, v, lo, n):
    """q [Hq, D], k, v [H, rows, D] float64; rows lo .. n-1.  Returns out, lse
    and, per element, sum p |v| and the largest sum |q k| / sqrt(D)."""
    Hq, D = q.shape
    rep = Hq // k.shape[0]
    if n <= lo:
        return torch.zeros(Hq, D, dtype=torch.float64), torch.full((Hq,), -math.inf, dtype=torch.float64), None, 0.0
    k = k[:, lo:n].repeat_interleave(rep, 0)
    v = v[:, lo:n].repeat_interleave(rep, 0)
    s = torch.einsum("hd,hjd->hj", q, k) / math.sqrt(D)
    mag = (torch.einsum("hd,hjd->hj", q.abs(), k.abs()) / math.sqrt(D)).max().item()
    p = torch.softmax(s, 1)
    return (torch.einsum("hj,hjd->hd", p, v), torch.logsumexp(s, 1),
            torch.einsum("hj,hjd->hd", p, v.abs()), mag)


def attention_eps(D, n, mag):
    """Error of out relative to sum p |v| (see dec_paged_attention): P in two
    bf16 planes, the rest p - bf16(p) (at most 2^-8 p) rounded to half a step,
    2^-9 of p 2^-8 = 2^-17; each score a sum of D exact products in fp32 and three
    more roundings, D + 3 of 2^-24 of sum |q k|, entering numerator and
    denominator; fp32 sums over tiles of 16 rows; the exponentials 2^-21."""
    return 2.0 ** -17 + 2 * (D + 3) * 2.0 ** -24 * mag + (n / 16 + 32) * 2.0 ** -23 + 2.0 ** -20


def inv_freq(R, theta=1e6, scaling="none", factor=1.0, orig_ctx=0.0, alpha=1.0, beta=32.0):
    if scaling == "ntk":
        theta = theta * factor ** (R / (R - 2))
    f = np.array([theta ** (-2.0 * i / R) for i in range(R // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        g = np.clip((orig_ctx * f / (2 * np.pi) - alpha) / (beta - alpha), 0.0, 1.0)
        f = g * f + (1 - g) * f / factor
    return f


def rotate(x, pos, f, inter, mscale):
    """x float64 [T, H, D], pos [T]."""
    R = 2 * len(f)
    ang = pos.double()[:, None] * torch.from_numpy(f)
    c, s = (mscale * torch.cos(ang))[:, None], (mscale * torch.sin(ang))[:, None]
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rms_norm(x, gain, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()


def beam(logits, scores, k, done, eos):
    """[G, W, V] -> scores float64, parents, tokens, done, by full sort."""
    G, W, V = logits.shape
    x = logits.double().numpy()
    out = []
    for g in range(G):
        cand = np.full((W, V), -np.inf)
        for w in range(W):
            s = float(scores[g, w])
            if done is not None and done[g, w]:
                cand[w, eos] = s
                continue
            with np.errstate(all="ignore"):
                m = x[g, w].max()
                lse = m + np.log(np.exp(x[g, w] - m).sum())
                cand[w] = s + x[g, w] - lse
        cand[np.isnan(cand)] = -np.inf
        flat = cand.reshape(-1)
        at = np.argsort(-flat, kind="stable")[:k]
        out.append((flat[at], at // V, at % V,
                    [bool(done is not None and done[g, a // V]) or (eos >= 0 and a % V == eos) for a in at]))
    return [np.array(z) for z in zip(*out)]
