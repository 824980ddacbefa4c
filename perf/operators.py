"""The measured cases of the paged-cache and beam-search operators.

Six kinds of case, each a call that a serving program makes:

  attend   one new token per sequence over a paged KV cache
  append   rotary positions of q and k, and the new rows into the pages
  rope     rotary positions alone, of a tensor of heads
  fork     beams take their parents' pages, then reserve the next row
  compact  the live pages of a pool to its lowest ids
  beam     the k best continuations of every group of beams
  reorder  sequences of a contiguous cache take their parents' rows

`run` computes them with elementary torch operations, or with `own` set by the
calls of this package.  `exact` computes the outputs again in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
NEG = float("-inf")


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the 0.6B decoder's prompt of 795 rows, one live sequence: latency of one layer's attention
        dict(name="attend_1x795", kind="attend", batch=1, lo=795, hi=795, heads=16, kv=8, dim=128, page=16, fmt="bf16",
             window=0, layers=2),
        # 64 concurrent 30 s windows, contexts of 200 to 420 rows
        dict(name="attend_64x420", kind="attend", batch=64, lo=200, hi=420, heads=16, kv=8, dim=128, page=16, fmt="bf16",
             window=0, layers=2),
        # 64 long contexts on an E4M3 cache with large pages
        dict(name="attend_64x4080_fp8", kind="attend", batch=64, lo=2048, hi=4080, heads=16, kv=8, dim=128, page=64,
             fmt="fp8", window=0, layers=1),
        # the longest contexts of the attention grid, ragged
        dict(name="attend_32x32768", kind="attend", batch=32, lo=16384, hi=32768, heads=16, kv=8, dim=128, page=32,
             fmt="bf16", window=0, layers=1),
        # one decode step's rows of 64 sequences: per-head norms, half layout, bf16 pages
        dict(name="append_64", kind="append", tokens=64, seqs=64, far=420, heads=16, kv=8, dim=128, rot=128, inter=False,
             scaling="none", factor=1.0, norm=True, page=16, fmt="bf16", dtype="bf16", pad=0),
        # prompts of a batch of windows appended at once, scaled positions, E4M3 pages
        dict(name="append_16384_fp8", kind="append", tokens=16384, seqs=21, far=795, heads=16, kv=8, dim=128, rot=128,
             inter=False, scaling="parts", factor=4.0, norm=True, page=64, fmt="fp8", dtype="bf16", pad=37),
        # rotation alone, interleaved pairs of half of each head, far positions
        dict(name="rope_8192_far", kind="rope", tokens=8192, far=1 << 20, heads=32, dim=128, rot=64, inter=True,
             scaling="ntk", factor=8.0, dtype="f32", pad=0),
        # one step of beam search over all layers of the 0.6B cache: 16 groups of 4 beams
        dict(name="fork_16x4", kind="fork", groups=16, beams=4, lo=200, hi=420, kv=8, dim=128, page=16, layers=28,
             grow=1),
        # a pool after many requests came and went: live pages to the front
        dict(name="compact_1024", kind="compact", pages=1024, live=0.5, seqs=32, kv=8, dim=128, page=16, layers=28),
        # one group of 4 beams over the 0.6B vocabulary: latency
        dict(name="beam_1x4", kind="beam", groups=1, beams=4, vocab=151936, k=4, dtype="f32", done=0),
        # a full batch: 16 groups of 4 beams, twice as many candidates kept, some beams finished
        dict(name="beam_16x4", kind="beam", groups=16, beams=4, vocab=151936, k=8, dtype="f32", done=5),
        # the contiguous cache of the same batch follows the chosen beams
        dict(name="reorder_16x4", kind="reorder", groups=16, beams=4, lo=200, hi=420, ctx=512, kv=8, dim=128, layers=28,
             fmt="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    kind = rng.choice(["attend", "attend", "append", "rope", "fork", "compact", "beam", "reorder"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    fmt = rng.choice(["bf16", "fp8"])
    if kind == "attend":
        batch, hi = _log(rng, 1, 64), _log(rng, 1, 32768)
        while batch * hi * kv * dim > 16 * 32768 * 8 * 128:
            hi = max(1, hi // 2)
        return dict(kind=kind, batch=batch, lo=rng.choice([0, (hi + 1) // 2, hi]), hi=hi, heads=kv * rng.randint(1, 8),
                    kv=kv, dim=dim, page=page, fmt=fmt, window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    layers=rng.randint(1, 2))
    if kind == "append":
        tokens = _log(rng, 1, 16384)
        rot = rng.choice([dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
        scaling = rng.choice(["none", "linear", "ntk", "parts"]) if rot > 2 else rng.choice(["none", "linear"])
        return dict(kind=kind, tokens=tokens, seqs=rng.randint(1, min(64, tokens)), far=_log(rng, 1, 4096),
                    heads=kv * rng.randint(1, 8), kv=kv, dim=dim, rot=rot, inter=rng.random() < 0.5, scaling=scaling,
                    factor=float(rng.choice([2, 4, 8])), norm=rng.random() < 0.5, page=page, fmt=fmt,
                    dtype=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 0, 3]) if tokens > 8 else 0)
    if kind == "rope":
        rot = rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        return dict(kind=kind, tokens=_log(rng, 1, 8192), far=_log(rng, 16, 1 << 20), heads=rng.randint(1, 32), dim=dim,
                    rot=rot, inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "parts"]) if rot > 2 else "none",
                    factor=float(rng.choice([2, 4, 8])), dtype=rng.choice(["bf16", "f32"]), pad=0)
    if kind == "fork":
        return dict(kind=kind, groups=rng.randint(1, 16), beams=rng.randint(1, 4), lo=_log(rng, 1, 100),
                    hi=_log(rng, 100, 420), kv=kv, dim=dim, page=page, layers=_log(rng, 1, 28), grow=rng.randint(1, 40))
    if kind == "compact":
        return dict(kind=kind, pages=_log(rng, 16, 1024), live=rng.uniform(0.1, 0.9), seqs=rng.randint(1, 32), kv=kv, dim=dim,
                    page=rng.choice([8, 16]), layers=_log(rng, 1, 28))
    if kind == "beam":
        groups, beams = rng.randint(1, 16), rng.randint(1, 4)
        return dict(kind=kind, groups=groups, beams=beams, vocab=_log(rng, 50, 151936), k=rng.randint(1, 8),
                    dtype=rng.choice(["bf16", "f32"]), done=rng.randint(0, groups * beams))
    return dict(kind=kind, groups=rng.randint(1, 16), beams=rng.randint(1, 4), lo=_log(rng, 1, 100), hi=_log(rng, 100, 420),
                ctx=rng.choice([432, 448, 512]), kv=kv, dim=dim, layers=_log(rng, 1, 28), fmt=fmt)


# ------------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _spread(n, lo, hi, g):
    """n whole numbers evenly over [lo, hi], in an order drawn from g (so that their sum is the case's)."""
    v = torch.linspace(lo, hi, n, device=DEV).round().int()
    return v[torch.randperm(n, generator=g, device=DEV)]


def _mean_rows(c):
    return sum(round(x) for x in torch.linspace(c["lo"], c["hi"], c.get("batch", c.get("groups"))).tolist())


def _codes(g, *shape):
    """E4M3 codes of N(0,1) * 32 and one scale per row."""
    z = torch.randn(shape, generator=g, device=DEV) * 32.0
    return (z.to(torch.float8_e4m3fn).view(torch.uint8),
            0.02 + 0.02 * torch.rand(shape[:-1], generator=g, device=DEV))


def _pool(g, c, pages):
    """Keys and values [layers, pages, kv, page, dim], and their scales for an E4M3 pool."""
    shape = (c.get("layers", 1), pages, c["kv"], c["page"], c["dim"])
    if c.get("fmt", "bf16") == "bf16":
        return dict(k=_randn(g, *shape, dtype=torch.bfloat16), v=_randn(g, *shape, dtype=torch.bfloat16), ks=None, vs=None)
    k, ks = _codes(g, *shape)
    v, vs = _codes(g, *shape)
    return dict(k=k, v=v, ks=ks, vs=vs)


def _table(rows, page, order, width):
    """Page table of sequences of `rows` rows: ids from `order`, -1 behind the last page."""
    need = (rows.long() + page - 1) // page
    start = torch.cumsum(need, 0) - need
    j = torch.arange(width, device=DEV)
    has = j[None] < need[:, None]
    ids = order[(start[:, None] + j[None]).clamp(max=order.numel() - 1)]
    return torch.where(has, ids, -1).int().contiguous()


def _pages_of(rows, page):
    return -(-rows // page)


def _paged(s, c, g, rows, n):
    width = _pages_of(max(1, int(s["max_rows"])), c["page"])
    order = torch.randperm(n, generator=g, device=DEV)
    s["table"] = _table(rows, c["page"], order, width)
    s["rows"] = rows.int().contiguous()
    held = s["table"].flatten()
    s["refs"] = torch.bincount(held[held >= 0].long(), minlength=n).int()
    s.update(_pool(g, c, n))


def _rope_of(c):
    return dict(rot_dim=c["rot"], theta=1e6, interleaved=c["inter"], scaling=c["scaling"], factor=c["factor"],
                orig_ctx=32768 if c["scaling"] == "parts" else 0)


def prepare(case, seed):
    c, g, kind = case, _gen(seed), case["kind"]
    s = dict(c=c)
    if kind == "attend":
        rows = _spread(c["batch"], c["lo"], c["hi"], g)
        s["max_rows"] = c["hi"]
        _paged(s, c, g, rows, sum(_pages_of(r, c["page"]) for r in rows.tolist()) + 3)
        s["q"] = _randn(g, c["batch"], c["heads"], c["dim"], dtype=torch.bfloat16)
    elif kind == "append":
        T, S = c["tokens"], c["seqs"]
        # every sequence holds up to `far` rows and gets an even share of the tokens behind them
        held = _spread(S, 0, c["far"], g).long()
        share = torch.full((S,), T // S, device=DEV)
        share[: T % S] += 1
        seq = torch.repeat_interleave(torch.arange(S, device=DEV), share, output_size=T)
        first = torch.cumsum(share, 0) - share
        pos = held[seq] + torch.arange(T, device=DEV) - first[seq]
        if c["pad"]:
            pos[torch.randperm(T, generator=g, device=DEV)[: c["pad"]]] = -1
        s["max_rows"] = c["far"] + T // S + 1
        _paged(s, c, g, held + share, sum(_pages_of(r + T // S + 1, c["page"]) for r in held.tolist()))
        s["seqs"], s["pos"] = seq.int().contiguous(), pos.int().contiguous()
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        # q, k and v are slices of one projection's output
        qkv = _randn(g, T, (c["heads"] + 2 * c["kv"]) * c["dim"], dtype=dt)
        a, b = c["heads"] * c["dim"], (c["heads"] + c["kv"]) * c["dim"]
        s["q"] = qkv[:, :a].unflatten(1, (c["heads"], c["dim"]))
        s["k_new"] = qkv[:, a:b].unflatten(1, (c["kv"], c["dim"]))
        s["v_new"] = qkv[:, b:].unflatten(1, (c["kv"], c["dim"]))
        s["gq"] = (1 + 0.1 * _randn(g, c["dim"])).bfloat16() if c["norm"] else None
        s["gk"] = (1 + 0.1 * _randn(g, c["dim"])).bfloat16() if c["norm"] else None
        s["q_out"] = torch.zeros((T, c["heads"], c["dim"]), dtype=torch.bfloat16, device=DEV)
    elif kind == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["x"] = _randn(g, c["tokens"], c["heads"], c["dim"], dtype=dt)
        s["pos"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device=DEV).int()
    elif kind == "fork":
        G, W, P = c["groups"], c["beams"], c["page"]
        rows = _spread(G, c["lo"], c["hi"], g).long()
        shared = (rows // P) // 2                       # pages of the common prefix
        need = (rows + P - 1) // P
        tail = need - shared
        width = _pages_of(c["hi"] + c["grow"], P) + 1
        per = shared + W * tail
        n = int(per.sum()) + G * W * (_pages_of(c["grow"], P) + 1) + 5
        order = torch.randperm(n, generator=g, device=DEV)
        start = torch.cumsum(per, 0) - per
        j = torch.arange(width, device=DEV)[None, None]
        w = torch.arange(W, device=DEV)[None, :, None]
        sh, ta, st = shared[:, None, None], tail[:, None, None], start[:, None, None]
        at = torch.where(j < sh, st + j, st + sh + w * ta + (j - sh))
        tab = torch.where(j < need[:, None, None], order[at.clamp(0, n - 1)], -1)
        s["table"] = tab.reshape(G * W, width).int().contiguous()
        s["rows"] = rows[:, None].expand(G, W).reshape(-1).int().contiguous()
        held = s["table"].flatten()
        s["refs"] = torch.bincount(held[held >= 0].long(), minlength=n).int()
        # half of the beams survive, each with about two continuations
        s["parents"] = _parents(g, G, W)
        s["target"] = (s["rows"] + c["grow"]).int()
        s["max_rows"] = width * P
        s.update(_pool(g, c, n))
    elif kind == "compact":
        n, S, P = c["pages"], c["seqs"], c["page"]
        live = max(1, int(n * c["live"]))
        cut = torch.linspace(0, live, S + 1, device=DEV).round().long()
        rows = (cut[1:] - cut[:-1]) * P
        order = torch.randperm(n, generator=g, device=DEV)
        s["max_rows"] = max(P, int(rows.max()))
        s["table"] = _table(rows, P, order, s["max_rows"] // P)
        s["rows"] = rows.int().contiguous()
        held = s["table"].flatten()
        s["refs"] = torch.bincount(held[held >= 0].long(), minlength=n).int()
        s.update(_pool(g, c, n))
    elif kind == "beam":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        G, W = c["groups"], c["beams"]
        s["logits"] = (_randn(g, G, W, c["vocab"]) * 2.5).to(dt)
        s["scores"] = -20.0 * torch.rand((G, W), generator=g, device=DEV)
        done = torch.zeros(G * W, dtype=torch.uint8, device=DEV)
        done[torch.randperm(G * W, generator=g, device=DEV)[: c["done"]]] = 1
        s["done"] = done.view(G, W)
        s["eos"] = c["vocab"] // 3
    else:
        G, W = c["groups"], c["beams"]
        shape = (c["layers"], 2, G * W, c["kv"], c["ctx"], c["dim"])
        if c["fmt"] == "bf16":
            s["cache"], s["scale"] = _randn(g, *shape, dtype=torch.bfloat16), None
        else:
            s["cache"], s["scale"] = _codes(g, *shape)
        s["rows"] = _spread(G, c["lo"], c["hi"], g)[:, None].expand(G, W).reshape(-1).int().contiguous()
        s["parents"] = _parents(g, G, W)
    if own:
        _handles(s, kind)
    return s


def _parents(g, G, W):
    """Parents of every beam, within its group: ceil(W / 2) beams survive."""
    keep = (W + 1) // 2
    alive = torch.rand((G, W), generator=g, device=DEV).argsort(1)[:, :keep]
    pick = alive[:, torch.arange(W, device=DEV) % keep]
    pick = pick.gather(1, torch.rand((G, W), generator=g, device=DEV).argsort(1))
    return (pick + W * torch.arange(G, device=DEV)[:, None]).reshape(-1).int().contiguous()


def _handles(s, kind):
    """The objects that a program keeps between calls."""
    if kind in ("attend", "append", "fork", "compact"):
        from decoder_greedy_decode_b200.paged import PagedKV
        if kind in ("fork", "compact"):
            meta = [s[n].clone() for n in ("table", "rows", "refs")]
        else:
            meta = [s[n] for n in ("table", "rows", "refs")]
        s["paged"] = PagedKV(s["k"], s["v"], meta[0], meta[1], meta[2], k_scale=s["ks"], v_scale=s["vs"])
    if kind in ("append", "rope"):
        from decoder_greedy_decode_b200.rotary import Rope
        s["rope"] = Rope(**_rope_of(s["c"]), device=DEV)


# ----------------------------------------------------------------- own calls
def _run_own(s):
    from decoder_greedy_decode_b200 import beam
    c, kind = s["c"], s["c"]["kind"]
    if kind == "attend":
        out, lse = s["paged"].attend(c["layers"] - 1, s["q"], s["rows"], window=c["window"], return_lse=True)
        return dict(out=out, lse=lse)
    if kind == "append":
        s["paged"].append(0, s["k_new"], s["v_new"], s["pos"], seqs=s["seqs"], rope=s["rope"], q=s["q"], q_out=s["q_out"],
                          q_norm=s["gq"], k_norm=s["gk"], eps=1e-6)
        return _pool_out(s, s["q_out"])
    if kind == "rope":
        return s["rope"].apply(s["x"], s["pos"])
    if kind == "fork":
        p = s["paged"]
        p.table.copy_(s["table"]), p.rows.copy_(s["rows"]), p.refs.copy_(s["refs"])
        p.fork(s["parents"])
        p.resize(s["target"])
        return dict(table=p.table, rows=p.rows, refs=p.refs, k=p.k, v=p.v)
    if kind == "compact":
        p = s["paged"]
        p.table.copy_(s["table"]), p.refs.copy_(s["refs"])
        live = p.compact()
        return dict(table=p.table, refs=p.refs, live=live, k=p.k, v=p.v)
    if kind == "beam":
        r = beam.beam_select(s["logits"], s["scores"], k=c["k"], done=s["done"], eos=s["eos"])
        return dict(scores=r.scores, parents=r.parents, tokens=r.tokens, done=r.done)
    beam.kv_reorder(s["cache"], s["parents"], s["rows"], scales=s["scale"])
    return _cache_out(s)


def _pool_out(s, q_out):
    if s["ks"] is None:
        return dict(q=q_out, k=s["k"], v=s["v"])
    return dict(q=q_out, k=s["k"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), ks=s["ks"], vs=s["vs"])


def _cache_out(s):
    if s["scale"] is None:
        return dict(cache=s["cache"])
    return dict(cache=s["cache"].view(torch.float8_e4m3fn), scale=s["scale"])


# --------------------------------------------------------------- plain forms
def run(state):
    if own:
        return _run_own(state)
    return dict(attend=_attend, append=_append, rope=_rope, fork=_fork, compact=_compact, beam=_beam,
                reorder=_reorder)[state["c"]["kind"]](state)


def _gathered(x, scale, table, layer):
    """Rows of every sequence, fp32 [batch, kv, width * page, dim]."""
    t = table.clamp(min=0).long()
    r = x[layer][t].permute(0, 2, 1, 3, 4)                  # [B, kv, width, page, dim]
    if scale is None:
        return r.float().flatten(2, 3)
    sc = scale[layer][t].permute(0, 2, 1, 3)
    return (r.view(torch.float8_e4m3fn).float() * sc[..., None]).flatten(2, 3)


def _attend(s):
    c = s["c"]
    B, rep, D = c["batch"], c["heads"] // c["kv"], c["dim"]
    k = _gathered(s["k"], s["ks"], s["table"], c["layers"] - 1)
    v = _gathered(s["v"], s["vs"], s["table"], c["layers"] - 1)
    n = s["rows"].long()
    j = torch.arange(k.shape[2], device=DEV)[None]
    first = (n - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(n)
    hide = ((j >= n[:, None]) | (j < first[:, None]))[:, None, None]
    q = s["q"].float().view(B, c["kv"], rep, D) / math.sqrt(D)
    x = torch.matmul(q, k.transpose(2, 3)).masked_fill(hide, NEG)
    m = x.amax(3, keepdim=True)
    safe = torch.where(m == NEG, torch.zeros_like(m), m)
    e = torch.exp(x - safe)
    z = e.sum(3, keepdim=True)
    v = v.masked_fill(hide[:, 0, 0, :][:, None, :, None], 0.0)
    out = torch.matmul(e, v) / torch.where(z > 0, z, torch.ones_like(z))
    lse = torch.where(z > 0, safe + torch.log(z), torch.full_like(z, NEG))
    return dict(out=out.reshape(B, c["heads"], D), lse=lse.reshape(B, c["heads"]))


def _inv_freq(c):
    """Angle per position of every pair, 64 bits, and the factor of the rotated values."""
    R, theta, f = c["rot"], 1e6, c["factor"]
    i = torch.arange(R // 2, dtype=torch.float64, device=DEV)
    if c["scaling"] == "ntk":
        theta = theta * f ** (R / (R - 2))
    w = torch.exp(-2 * i / R * math.log(theta))
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "parts":
        ramp = ((32768 * w / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        w = ramp * w + (1 - ramp) * w / f
    return w, (0.1 * math.log(f) + 1.0 if c["scaling"] == "parts" else 1.0)


def _rotated(x, pos, c):
    """x fp32 [tokens, heads, dim], the first rot elements of every head rotated."""
    w, m = _inv_freq(c)
    a = pos.double()[:, None] * w
    cs, sn = (torch.cos(a) * m).float()[:, None], (torch.sin(a) * m).float()[:, None]
    R = c["rot"]
    u, rest = x[..., :R], x[..., R:]
    if c["inter"]:
        a, b = u[..., 0::2], u[..., 1::2]
        y = torch.stack((a * cs - b * sn, b * cs + a * sn), -1).flatten(-2)
    else:
        a, b = u[..., : R // 2], u[..., R // 2:]
        y = torch.cat((a * cs - b * sn, b * cs + a * sn), -1)
    return torch.cat((y, rest), -1)


def _normed(x, gain):
    return x if gain is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain.float()


def _append(s):
    c = s["c"]
    pos = s["pos"].long()
    at = (pos >= 0).nonzero().flatten()
    pos, seq = pos[at], s["seqs"].long()[at]
    q = _rotated(_normed(s["q"][at].float(), s["gq"]), pos, c)
    k = _rotated(_normed(s["k_new"][at].float(), s["gk"]), pos, c)
    v = s["v_new"][at].float()
    s["q_out"][at] = q.bfloat16()
    page, row = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    if c["fmt"] == "bf16":
        s["k"][0][page, :, row] = k.bfloat16()
        s["v"][0][page, :, row] = v.bfloat16()
    else:
        ks, vs = (x.abs().amax(-1).clamp(min=2.0 ** -126) / 448.0 for x in (k, v))
        s["k"][0][page, :, row] = (k / ks[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"][0][page, :, row] = (v / vs[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["ks"][0][page, :, row] = ks
        s["vs"][0][page, :, row] = vs
    return _pool_out(s, s["q_out"])


def _rope(s):
    return _rotated(s["x"].float(), s["pos"], s["c"]).to(s["x"].dtype)


def _fork(s):
    c, P = s["c"], s["c"]["page"]
    table, n = s["table"][s["parents"].long()].long(), s["refs"].numel()
    old = s["rows"][s["parents"].long()].long()
    held = table.flatten()
    refs = torch.bincount(held[held >= 0], minlength=n)
    new = s["target"].long()
    # a sequence that grows writes into its last page: unless it is the last holder, it gets a copy
    b = torch.arange(old.numel(), device=DEV)
    slot = (old // P).clamp(max=table.shape[1] - 1)
    last = torch.where((new > old) & (old % P > 0), table[b, slot], -1 - b)
    rank = torch.tril(last[:, None] == last[None], -1).sum(1)
    copy = (last >= 0) & (rank < refs[last.clamp(min=0)] - 1)
    j = torch.arange(table.shape[1], device=DEV)[None]
    want = (copy[:, None] & (j == slot[:, None])) | ((j >= ((old + P - 1) // P)[:, None]) & (j < ((new + P - 1) // P)[:, None]))
    free = (refs == 0).nonzero().flatten()
    ids = free[(want.flatten().cumsum(0) - 1).clamp(0, free.numel() - 1)].view_as(table)
    refs.index_add_(0, last[copy], -torch.ones_like(last[copy]))
    table = torch.where(want, ids, table)
    refs.index_add_(0, ids[want], torch.ones_like(ids[want]))
    src, dst = last[copy], ids[b[copy], slot[copy]]
    fill = (torch.arange(P, device=DEV)[None] < (old % P)[copy][:, None])[None, :, None, :, None]
    s["k"][:, dst] = torch.where(fill, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(fill, s["v"][:, src], s["v"][:, dst])
    return dict(table=table.int(), rows=new.int(), refs=refs.int(), k=s["k"], v=s["v"])


def _compact(s):
    refs = s["refs"]
    held = refs > 0
    live = held.sum()
    ids = torch.arange(refs.numel(), device=DEV)
    src, dst = (held & (ids >= live)).nonzero().flatten(), (~held & (ids < live)).nonzero().flatten()
    to = ids.clone()
    to[src] = dst
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    new = torch.where(ids < live, refs, 0)
    new[dst] = refs[src]
    table = torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].int(), -1)
    return dict(table=table, refs=new, live=live.int().reshape(1), k=s["k"], v=s["v"])


def _beam(s):
    c = s["c"]
    G, W, V, k = c["groups"], c["beams"], c["vocab"], min(c["k"], c["beams"] * c["vocab"])
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    base = s["scores"].double()[..., None]
    cand = base + x - lse
    # a finished beam has one continuation: its end token, at its own score
    over = s["done"].bool()[..., None]
    stop = torch.arange(V, device=DEV) == s["eos"]
    cand = torch.where(over, torch.where(stop, base, NEG), cand)
    flat = torch.where(torch.isnan(cand), NEG, cand).view(G, W * V)
    # the k largest, the lowest index first among equals
    t = torch.topk(flat, k).values[:, -1:]
    above, same = flat > t, flat == t
    room = k - above.sum(1, keepdim=True)
    take = above | (same & (same.cumsum(1) <= room))
    at = take.nonzero()[:, 1].view(G, k)
    val, order = torch.sort(flat.gather(1, at), dim=1, descending=True, stable=True)
    at = at.gather(1, order)
    parent, token = at // V, at % V
    done = s["done"].bool().gather(1, parent) | (token == s["eos"])
    return dict(scores=val.float(), parents=parent.int(), tokens=token.int(), done=done.to(torch.uint8))


def _reorder(s):
    j = torch.arange(s["cache"].shape[4], device=DEV)
    fill = (j[None] < s["rows"][:, None])[None, None, :, None, :]
    p = s["parents"].long()
    s["cache"].copy_(torch.where(fill[..., None], s["cache"][:, :, p], s["cache"]))
    if s["scale"] is not None:
        s["scale"].copy_(torch.where(fill, s["scale"][:, :, p], s["scale"]))
    return _cache_out(s)


# ---------------------------------------------------------------------- work
def work(case):
    c, kind = case, case["kind"]
    if kind == "attend":
        rows = [round(x) for x in torch.linspace(c["lo"], c["hi"], c["batch"]).tolist()]
        n = sum(min(r, c["window"]) if c["window"] else r for r in rows)
        row = 2 * c["dim"] if c["fmt"] == "bf16" else c["dim"] + 4
        return dict(bytes=2 * n * c["kv"] * row + c["batch"] * c["heads"] * (6 * c["dim"] + 4),
                    flops=4 * n * c["heads"] * c["dim"])
    if kind == "append":
        e = 2 if c["dtype"] == "bf16" else 4
        row = 2 * c["dim"] if c["fmt"] == "bf16" else c["dim"] + 4
        return dict(bytes=c["tokens"] * ((c["heads"] + 2 * c["kv"]) * c["dim"] * e + c["heads"] * c["dim"] * 2 + 2 * c["kv"] * row),
                    flops=c["tokens"] * (c["heads"] + c["kv"]) * c["dim"] * 6)
    if kind == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=2 * c["tokens"] * c["heads"] * c["dim"] * e, flops=3 * c["tokens"] * c["heads"] * c["rot"])
    if kind == "fork":
        rows = [round(x) for x in torch.linspace(c["lo"], c["hi"], c["groups"]).tolist()]
        moved = sum(r % c["page"] for r in rows) * (c["beams"] - (c["beams"] + 1) // 2)
        width = _pages_of(c["hi"] + c["grow"], c["page"]) + 1
        return dict(bytes=2 * 2 * moved * c["layers"] * c["kv"] * c["dim"] * 2 + 8 * c["groups"] * c["beams"] * width, flops=0)
    if kind == "compact":
        live = max(1, int(c["pages"] * c["live"]))
        moved = live * (c["pages"] - live) / c["pages"]
        return dict(bytes=2 * 2 * moved * c["layers"] * c["kv"] * c["page"] * c["dim"] * 2 + 16 * c["pages"], flops=0)
    if kind == "beam":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["groups"] * c["beams"] * c["vocab"]
        return dict(bytes=n * e, flops=3 * n)
    rows = _mean_rows(c) * (c["beams"] - (c["beams"] + 1) // 2)
    row = 2 * c["dim"] if c["fmt"] == "bf16" else c["dim"] + 4
    return dict(bytes=2 * rows * c["layers"] * 2 * c["kv"] * row + 8 * c["groups"] * c["beams"], flops=0)


# --------------------------------------------------------------------- exact
def exact(case, seed):
    c, kind = case, case["kind"]
    s = prepare(case, seed)
    if kind == "attend":
        out = torch.zeros((c["batch"], c["heads"], c["dim"]), dtype=torch.float64, device=DEV)
        lse = torch.full((c["batch"], c["heads"]), NEG, dtype=torch.float64, device=DEV)
        rep = c["heads"] // c["kv"]
        for b, n in enumerate(s["rows"].tolist()):
            first = max(0, n - c["window"]) if c["window"] else 0
            if n <= first:
                continue
            at = torch.arange(first, n, device=DEV)
            page, r = s["table"][b].long()[at // c["page"]], at % c["page"]
            k, v = (s[x][c["layers"] - 1][page, :, r] for x in ("k", "v"))
            if s["ks"] is not None:
                k, v = (x.view(torch.float8_e4m3fn).double() * y[c["layers"] - 1][page, :, r].double()[..., None]
                        for x, y in ((k, s["ks"]), (v, s["vs"])))
            k, v = (x.double().repeat_interleave(rep, 1) for x in (k, v))
            w = (k * s["q"][b].double()).sum(-1) / math.sqrt(c["dim"])           # [rows, heads]
            lse[b] = torch.logsumexp(w, 0)
            out[b] = (torch.softmax(w, 0)[..., None] * v).sum(0)
        return dict(out=out, lse=lse)
    if kind == "rope":
        return _exact_turn(s["x"].double(), s["pos"], c)
    if kind == "append":
        def head(x, gain):
            x = x.double()
            if gain is not None:
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain.double()
            return _exact_turn(x, s["pos"], c)
        live = s["pos"] >= 0
        q = torch.where(live[:, None, None], head(s["q"], s["gq"]), s["q_out"].double())
        new = dict(k=head(s["k_new"], s["gk"]), v=s["v_new"].double())
        at = live.nonzero().flatten()
        pos, seq = s["pos"].long()[at], s["seqs"].long()[at]
        page, row = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
        r = dict(q=q)
        for n in ("k", "v"):
            x = new[n][at]
            if c["fmt"] == "bf16":
                r[n] = s[n].double()
                r[n][0][page, :, row] = x
                continue
            sc = x.abs().amax(-1).clamp(min=2.0 ** -126) / 448
            r[n] = s[n].view(torch.float8_e4m3fn).double()
            r[n][0][page, :, row] = x / sc[..., None]
            r[n + "s"] = s[n + "s"].double()
            r[n + "s"][0][page, :, row] = sc
        return r
    if kind == "beam":
        lp = torch.log_softmax(s["logits"].double(), -1) + s["scores"].double()[..., None]
        lp = torch.where(s["done"].bool()[..., None], torch.full_like(lp, NEG), lp)
        i = torch.arange(c["vocab"], device=DEV) == s["eos"]
        lp = torch.where(s["done"].bool()[..., None] & i, s["scores"].double()[..., None], lp)
        flat = lp.view(c["groups"], -1)
        val = torch.topk(flat, min(c["k"], flat.shape[1])).values
        return dict(scores=val, parents=None, tokens=None, done=None)
    # pages and cache rows are moved, not computed
    return None


def _exact_turn(x, pos, c):
    """Rotation as a product of complex numbers."""
    R, theta, f, m = c["rot"], 1e6, c["factor"], 1.0
    if c["scaling"] == "ntk":
        theta *= f ** (R / (R - 2))
    w = torch.tensor([theta ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64, device=DEV)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "parts":
        g = ((32768 * w / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
        w, m = w * g + w / f * (1 - g), 1 + 0.1 * math.log(f)
    z = torch.polar(torch.full_like(w, m).expand(len(pos), -1), pos.double()[:, None] * w)[:, None]
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if c["inter"] else (slice(0, R // 2), slice(R // 2, R))
    t = torch.complex(x[..., a], x[..., b]) * z
    y[..., a], y[..., b] = t.real, t.imag
    return y
