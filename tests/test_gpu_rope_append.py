"""dec_rope_apply and dec_paged_append against their formulas in 64 bits.

Tolerances.  The angle is off by at most pi 2^-24 (its top 32 bits rounded to
fp32) and sine and cosine by 2 ulp, so a rotated element is off by less than
2^-20 (|a| + |b|) times mscale; RMSNorm adds 2^-21 of the value (sum of 128
squares in fp32, rsqrt).  bf16 results add half a step, 2^-8 of the value;
E4M3 half a step, 2^-4 of the value or 2^-10 of the scale (subnormal codes).
"""
import pytest
import torch

import paged_ref as ref
from decoder_greedy_decode_b200 import capi
from decoder_greedy_decode_b200.paged import PagedKV
from decoder_greedy_decode_b200.rotary import Rope

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -19
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def pair_size(x, R, inter):
    """|a| + |b| of each element's pair (its own size behind R)."""
    y = x.abs().clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    s = x[..., a].abs() + x[..., b].abs()
    y[..., a], y[..., b] = s, s
    return y


SCALED = [("none", dict()), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
          ("parts", dict(factor=4.0, orig_ctx=32768.0)),
          ("parts", dict(factor=8.0, orig_ctx=8192.0, alpha=1.0, beta=4.0, mscale=1.0))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (128, 64), (64, 32), (128, 2), (64, 6),
                                 (128, 10), (128, 126), (64, 62), (128, 4)])
@pytest.mark.parametrize("T,H", [(1, 1), (7, 5), (33, 8)])
def test_rotation(T, H, D, R, inter, dtype):
    g = torch.Generator().manual_seed(T * H + R)
    scaling, kw = SCALED[(T + R + D // 64) % len(SCALED)] if R > 2 else SCALED[0]
    x = torch.randn((T, H, D), generator=g).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).int()
    pos[0] = (1 << 31) - 1 if T > 1 else 0
    r = Rope(R, 1e6, interleaved=inter, scaling=scaling, **kw)
    got = r.apply(x.cuda(), pos.cuda())
    f = ref.inv_freq(R, 1e6, scaling, **{k: v for k, v in kw.items() if k != "mscale"})
    # (the reference's own angle, a product of doubles, is good to 2^-53 of it)
    want = ref.rotate(x.double(), pos, f, inter, r.mscale)
    tol = FP32 * r.mscale * pair_size(x.double(), R, inter) + HALF[dtype] * want.abs()
    tol[..., R:] = 0
    slack = (2.0 ** -52 * pos.double() * 2)[:, None, None] * pair_size(x.double(), R, inter)
    slack[..., R:] = 0
    assert bool(((got.cpu().double() - want).abs() <= tol + slack).all())


def test_in_place_strides_and_padding():
    T, H, D = 9, 4, 128
    buf = torch.randn((T, 3 * H * D)).bfloat16().cuda()
    x = buf[:, H * D: 2 * H * D].unflatten(1, (H, D))
    was = buf.clone()
    pos = torch.tensor([5, -1, 0, 7, -3, 100, 2, 1, 9], dtype=torch.int32).cuda()
    r = Rope(D)
    want = r.apply(x.contiguous(), pos)
    got = r.apply(x, pos, out=x)
    assert torch.equal(got, want)
    assert torch.equal(x[pos < 0], was[:, H * D: 2 * H * D].unflatten(1, (H, D))[pos < 0])
    assert torch.equal(buf[:, : H * D], was[:, : H * D]) and torch.equal(buf[:, 2 * H * D:], was[:, 2 * H * D:])
    assert r.apply(x[:0], pos[:0]).shape == (0, H, D)


def test_passed_elements_keep_infinities():
    x = torch.randn((2, 3, 64)).cuda()
    x[..., 40] = float("inf")
    x[..., 50] = float("nan")
    for inter in (False, True):
        got = Rope(32, interleaved=inter).apply(x, torch.tensor([3, 9], dtype=torch.int32).cuda())
        assert torch.equal(got[..., 32:].nan_to_num(5, 6, 7), x[..., 32:].nan_to_num(5, 6, 7))
        assert torch.isfinite(got[..., :32]).all()


def test_half_layout_is_the_step_kernels():
    """Unscaled half-split rotation = the decoder's own (its angle is an fp32
    product: equal up to that at small positions)."""
    x = torch.randn((50, 2, 128)).cuda()
    pos = torch.arange(50, dtype=torch.int32).cuda()
    got = Rope(128, 1e6).apply(x, pos).cpu()
    inv = torch.tensor([1e6 ** (-2 * i / 128) for i in range(64)], dtype=torch.float64).float()
    a = (pos.cpu().float()[:, None] * inv).double()[:, None]
    xd = x.cpu().double()
    want = torch.cat((xd[..., :64] * a.cos() - xd[..., 64:] * a.sin(),
                      xd[..., 64:] * a.cos() + xd[..., :64] * a.sin()), -1)
    assert bool(((got.double() - want).abs() <= 50 * 2.0 ** -23 * 8).all())


def cache(S, width, kv, D, P, fmt, layers=1, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = S * width + 2
    table = torch.randperm(n, generator=g)[: S * width].view(S, width).int()
    shape = (layers, n, kv, P, D)
    scales = {}
    if fmt == "bf16":
        k, v = (torch.full(shape, 3.0, dtype=torch.bfloat16) for _ in range(2))
    else:
        k, v = (torch.full(shape, 17, dtype=torch.uint8) for _ in range(2))
        scales = {s: torch.full(shape[:4], 9.0).cuda() for s in ("k_scale", "v_scale")}
    return PagedKV(k.cuda(), v.cuda(), table.cuda(), torch.zeros(S, dtype=torch.int32).cuda(),
                   torch.ones(n, dtype=torch.int32).cuda(), **scales)


APPEND = [  # T, S, width, Hq, kv, D, R, inter, P
    (1, 1, 1, 1, 1, 64, 64, False, 8),
    (64, 64, 3, 16, 8, 128, 128, False, 16),
    (37, 3, 5, 6, 2, 128, 64, True, 16),
    (100, 7, 4, 5, 5, 64, 32, False, 32),
    (19, 2, 2, 0, 3, 128, 128, False, 64),
    (21, 4, 1, 9, 3, 64, 10, False, 1024),
    (13, 2, 4, 2, 1, 128, 0, False, 8),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,S,width,Hq,kv,D,R,inter,P", APPEND)
def test_append(T, S, width, Hq, kv, D, R, inter, P, norm, dtype, fmt):
    g = torch.Generator().manual_seed(T + D + R)
    c = cache(S, width, kv, D, P, fmt, layers=2, seed=T)
    before = [x.clone() for x in (c.k, c.v)]
    cells = torch.randperm(S * width * P, generator=g)[:T]
    seq, pos = (cells // (width * P)).int(), (cells % (width * P)).int()
    if T == 64:
        seq, pos = torch.arange(64).int(), torch.randint(0, width * P, (64,), generator=g).int()
    if T > 10:
        pos[[2, T - 1]] = -1
    qkv = torch.randn((T, (Hq + 2 * kv) * D), generator=g).to(dtype)
    q = qkv[:, : Hq * D].unflatten(1, (Hq, D)) if Hq else None
    k = qkv[:, Hq * D: (Hq + kv) * D].unflatten(1, (kv, D))
    v = qkv[:, (Hq + kv) * D:].unflatten(1, (kv, D))
    gq, gk = ((1 + 0.1 * torch.randn(D, generator=g)).bfloat16() for _ in range(2))
    rope = Rope(R, interleaved=inter) if R else None
    f = ref.inv_freq(R) if R else None
    dq = qkv.cuda()
    q_out = torch.full((T, Hq, D), 2.0, dtype=torch.bfloat16, device="cuda") if Hq else None
    got_q = c.append(1, dq[:, Hq * D: (Hq + kv) * D].unflatten(1, (kv, D)),
                     dq[:, (Hq + kv) * D:].unflatten(1, (kv, D)), pos.cuda(),
                     seqs=None if T == 64 else seq.cuda(), rope=rope,
                     q=dq[:, : Hq * D].unflatten(1, (Hq, D)) if Hq else None, q_out=q_out,
                     q_norm=gq.cuda() if norm and Hq else None, k_norm=gk.cuda() if norm else None)
    assert c.check() == 0

    def turned(x, gain):
        x = x.double()
        if norm:
            x = ref.rms_norm(x, gain, 1e-6)
        size = pair_size(x, R, inter) if R else x.abs()
        return (ref.rotate(x, pos, f, inter, 1.0) if R else x), size

    live = pos >= 0
    if Hq:
        want, size = turned(q, gq)
        err = (got_q.cpu().double() - want).abs()
        assert bool((err <= 2.0 ** -8 * want.abs() + FP32 * size)[live].all())
        assert bool((got_q.cpu()[~live] == 2).all())
    at = live.nonzero().flatten()
    page, row = c.table.cpu()[seq[at].long(), (pos[at] // P).long()].long(), (pos[at] % P).long()
    for name, pool, old, scale, (want, size) in (
            ("k", c.k, before[0], c.k_scale, turned(k, gk)),
            ("v", c.v, before[1], c.v_scale, (v.double(), v.double().abs()))):
        got = pool.cpu()
        stored = got[1][page, :, row]
        want, size = want[at], size[at]
        if fmt == "bf16":
            tol = 2.0 ** -8 * want.abs() + FP32 * size
            assert bool(((stored.double() - want).abs() <= tol).all()), name
        else:
            sc = scale.cpu()[1][page, :, row].double()
            am = want.abs().amax(-1)
            assert bool(((sc - am / 448).abs() <= FP32 * size.amax(-1) / 448 + 2.0 ** -23 * am / 448).all())
            val = ref.decode(stored, sc.float())
            tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 * sc[..., None] + FP32 * size + 2.0 ** -22 * want.abs()
            assert bool(((val - want).abs() <= tol).all()), name
            rest = scale.cpu().clone()
            rest[1][page, :, row] = 9.0
            assert bool((rest == 9).all())
        # everything else is as it was
        got[1][page, :, row] = old.cpu()[1][page, :, row]
        assert torch.equal(got, old.cpu()), name


@pytest.mark.parametrize("D", [64, 128])
def test_codes_are_the_row_quantisers(D):
    """Without norm and rotation the E4M3 rows are dec_kv_quantize_e4m3's (IEEE
    divisions), bit for bit: random rows of every size from the smallest
    subnormals to infinity, zeros, NaN, and values on rounding ties."""
    T, kv = 4096, 4
    c = cache(T, 1, kv, D, 8, "fp8")
    g = torch.Generator().manual_seed(D)
    x = torch.randn((T, kv, D), generator=g) * torch.exp2(torch.rand((T, kv, 1), generator=g) * 280 - 150)
    mids = torch.arange(0, 0x7E).to(torch.uint8).view(torch.float8_e4m3fn).float()
    tie = ((mids[1:] + mids[:-1]) / 2)[torch.randint(0, 125, (T // 4, kv, D), generator=g)]
    sign = torch.where(torch.rand(tie.shape, generator=g) < 0.5, -1.0, 1.0)
    x[: T // 4] = sign * tie * torch.exp2(torch.randint(-140, 110, (T // 4, kv, 1), generator=g).float())
    x[: T // 4, :, 0] = 448.0 * x[: T // 4, :, 0].sign() * \
        (x[: T // 4, :, 1:].abs().amax(-1) / 448.0).clamp(min=1e-44)
    x[-1] = 0
    x[-2, 0, 5] = float("nan")
    x[-3, 1, 9] = float("-inf")
    x[-4] = 3e38
    x[-5] = -1e-45
    x = x.cuda()
    c.append(0, x, x, torch.zeros(T, dtype=torch.int32, device="cuda"))
    codes = torch.zeros((T * kv, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(T * kv, device="cuda")
    capi.dec_kv_quantize_e4m3(x.contiguous(), T * kv, D, codes, scales)
    page = c.table[:, 0].long()
    for pool, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert torch.equal(sc[0][page, :, 0].reshape(-1).view(torch.int32), scales.view(torch.int32))
        assert torch.equal(pool[0][page, :, 0].reshape(T * kv, D), codes)


def test_bad_tokens_are_skipped_whole():
    c = cache(2, 2, 1, 64, 8, "bf16")
    c.table[1, 1] = -1
    old = (c.k.clone(), c.v.clone())
    k = torch.randn((5, 1, 64)).bfloat16().cuda()
    q = torch.randn((5, 2, 64)).bfloat16().cuda()
    q_out = torch.full((5, 2, 64), 2.0, dtype=torch.bfloat16, device="cuda")

    def go(seqs, pos):
        c.append(0, k[: len(pos)], k[: len(pos)], torch.tensor(pos, dtype=torch.int32).cuda(),
                 seqs=torch.tensor(seqs, dtype=torch.int32).cuda(), q=q[: len(pos)], q_out=q_out[: len(pos)])
        return c.check()

    assert go([1], [8]) == capi.DEC_DEV_BAD_PAGE            # not assigned
    assert go([2, -1], [0, 0]) == capi.DEC_DEV_BAD_PAGE     # no such sequence
    assert go([0], [16]) == capi.DEC_DEV_BAD_POSITION       # behind the table
    assert go([0], [2 ** 31 - 1]) == capi.DEC_DEV_BAD_POSITION
    c.table[0, 0] = c.n_pages
    assert go([0], [0]) == capi.DEC_DEV_BAD_PAGE            # no such page
    assert torch.equal(c.k, old[0]) and torch.equal(c.v, old[1]) and bool((q_out == 2).all())
    assert go([0, 0, 1], [3, 9, 2]) == capi.DEC_DEV_BAD_PAGE
    assert bool((q_out[0] == 2).all()) and bool((q_out[1:3] != 2).any(-1).all())


def test_append_replays_in_a_graph():
    c = cache(4, 2, 2, 128, 16, "bf16")
    rope = Rope(128)
    k, v = (torch.randn((4, 2, 128)).bfloat16().cuda() for _ in range(2))
    q = torch.randn((4, 4, 128)).bfloat16().cuda()
    pos = torch.tensor([0, 5, 16, 31], dtype=torch.int32).cuda()
    q_out = torch.zeros((4, 4, 128), dtype=torch.bfloat16, device="cuda")
    c.append(0, k, v, pos, rope=rope, q=q, q_out=q_out)
    want = (c.k.clone(), q_out.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(0, k, v, pos, rope=rope, q=q, q_out=q_out)
    c.k.fill_(3.0), q_out.zero_()
    g.replay()
    assert torch.equal(c.k, want[0]) and torch.equal(q_out, want[1])
    pos.copy_(torch.tensor([1, 2, 3, 4], dtype=torch.int32))
    g.replay()
    assert torch.equal(q_out, c.append(0, k, v, pos, rope=rope, q=q))



@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (128, 20)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_new_q_out_is_zero_where_tokens_are_skipped(D, R, fmt):
    c = PagedKV.create(1, 4, 8, 2, D, 2, 16, dtype=fmt)
    c.resize(torch.tensor([8, 3], dtype=torch.int32).cuda())
    g = torch.Generator().manual_seed(D + R)
    q = torch.randn((70, 5, D), generator=g).bfloat16().cuda()
    k = torch.randn((70, 2, D), generator=g).bfloat16().cuda()
    pos, seqs = torch.full((70,), -1, dtype=torch.int32), torch.zeros(70, dtype=torch.int32)
    pos[3], pos[40], pos[41], pos[69] = 2, 15, 1, 4      # row 15 has no page
    seqs[41], seqs[69] = 1, 7                            # there is no sequence 7
    rope = Rope(R, theta=1e4)
    torch.empty((70, 5, D), dtype=torch.bfloat16, device="cuda").fill_(9.0)   # (its memory may come back)
    out = c.append(0, k, k, pos.cuda(), seqs=seqs.cuda(), rope=rope, q=q)
    assert c.check() == capi.DEC_DEV_BAD_PAGE
    done = torch.zeros(70, dtype=torch.bool)
    done[[3, 41]] = True
    assert bool((out[~done] == 0).all()) and bool((out[done] != 0).any(-1).all())
    kept = torch.full_like(out, 9.0)
    c.append(0, k, k, pos.cuda(), seqs=seqs.cuda(), rope=rope, q=q, q_out=kept)
    assert torch.equal(kept[done], out[done]) and bool((kept[~done] == 9).all())
    c.check()
