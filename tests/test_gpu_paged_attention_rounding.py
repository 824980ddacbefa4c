"""The roundings of dec_paged_attention that a bound over all scores hides.

P enters the second product exactly (bf16 pages: its 24 bits in three planes) or
to 2^-23 (E4M3: two f16 planes of p * scale).  Rows that all hold the same V
return it whatever the scores are, up to fp32 roundings of the two sums: with
at most four rows and V powers of two, the first two planes' sums are exact, the
last one's at most four addends are cut at 2^-23 of the sum, and the sum of p,
its reciprocal and the product round six times by 2^-24: 7 * 2^-23 < 2^-20.
E4M3 adds 2^-23 of the planes and 2^-24 of p * scale: 2^-19."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref
from decoder_greedy_decode_b200.paged import PagedKV
from test_gpu_paged_attention import CASES, attend, build, rows_of

BF16_BOUND, E4M3_BOUND = 2.0 ** -20, 2.0 ** -19


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def cut(x):
    """The top half of fp32 values, as a bf16 plane."""
    return (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)


def nearest(x):
    return torch.from_numpy(x).bfloat16().float().numpy()


@pytest.mark.parametrize("rounding", ["cut", "nearest"])
def test_two_planes_would_exceed_the_bound(rounding):
    """The bound tells three planes of P from two (on the host)."""
    g = np.random.default_rng(1)
    p = np.exp2(-3 * g.random((256, 3))).astype(np.float32)
    p[:, 0] = 1
    first = cut(p)
    rest = p - first
    second = cut(rest) if rounding == "cut" else nearest(rest)
    total = p.astype(np.float64).sum(1)

    def error(planes):
        return np.abs(sum(x.astype(np.float64) for x in planes).sum(1) / total - 1).max()

    assert error([first, second]) > 2 * BF16_BOUND
    if rounding == "cut":
        third = cut(rest - second)
        assert error([first, second, third]) < BF16_BOUND / 8


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_equal_values_return_themselves(fmt, D):
    need_gpu()
    lens = [2 + i % 3 for i in range(64)]
    c = build(lens, 2, D, 8, fmt, seed=50 + D)
    g = torch.Generator().manual_seed(D)
    t = c.table[:, 0].long()       # (4 rows at most: one page)
    v = torch.exp2(torch.randint(-2, 3, (64, 2, 1, D), generator=g).float()) \
        * torch.where(torch.rand((64, 2, 1, D), generator=g) < 0.5, -1.0, 1.0)
    if fmt == "bf16":
        c.v[0, t] = v.bfloat16().cuda().expand(-1, -1, 8, -1)
        want = v[:, :, 0].double()
    else:
        scale = 0.01 + 0.05 * torch.rand((64, 2, 1), generator=g)
        c.v[0, t] = v.to(torch.float8_e4m3fn).view(torch.uint8).cuda().expand(-1, -1, 8, -1)
        c.v_scale[0, t] = scale.cuda().expand(-1, -1, 8)
        want = v[:, :, 0].double() * scale.double()
    # scores apart by a few units at most
    q = (0.5 * torch.randn((64, 6, D), generator=g)).bfloat16().cuda()
    out, _ = attend(c, q, lens)
    want = want.repeat_interleave(3, 1)
    off = ((out.cpu().double() - want) / want).abs().max()
    assert float(off) <= (BF16_BOUND if fmt == "bf16" else E4M3_BOUND)


@pytest.mark.gpu
def test_a_single_row_is_returned_as_it_is():
    """bf16: p = 1 is one plane, and the other two add 2^-126 of V.  E4M3: the
    planes of the scale 2^-23, the cut of two addends 2^-22."""
    need_gpu()
    for fmt in ("bf16", "fp8"):
        c = build([1, 1], 2, 128, 16, fmt, seed=4)
        q = torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        out, _ = attend(c, q, [1, 1])
        for b in range(2):
            v = rows_of(c, 0, b, 1)[1][:, 0].repeat_interleave(2, 0)
            if fmt == "bf16":
                assert torch.equal(out[b].cpu().double(), v)
            else:
                assert bool(((out[b].cpu().double() - v).abs() <= 2.0 ** -21 * v.abs()).all())


def eps(D, n, mag, fmt):
    """Error of out relative to sum p |v|: each score a sum of D exact products
    in fp32 and three more roundings, in numerator and denominator; fp32 sums
    over tiles of 16 rows; the exponentials 2^-21; E4M3 planes 2^-22, and what is
    lost below 2^-39 of the largest p * scale."""
    e = 2 * (D + 3) * 2.0 ** -24 * mag + (n / 16 + 32) * 2.0 ** -23 + 2.0 ** -20
    return e + (2.0 ** -22 if fmt == "fp8" else 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P,window", CASES[3:12])
def test_attention_without_a_term_for_p(lens, Hq, Hkv, D, P, window, fmt):
    """Small queries: scores, and with them their roundings, are near 0."""
    need_gpu()
    c = build(lens, Hkv, D, P, fmt, seed=60 + len(lens) + D)
    q = (torch.randn((len(lens), Hq, D), generator=torch.Generator().manual_seed(3)) / 64).bfloat16().cuda()
    out, lse = attend(c, q, lens, window=window)
    for b, n in enumerate(lens):
        k, v = rows_of(c, 0, b, n)
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        o, l, pv, mag = ref.attention(q[b].double().cpu(), k, v, lo, n)
        e = eps(D, n, mag, fmt)
        tail = 2.0 ** -39 * (n - lo) * v[:, lo:n].abs().amax() if fmt == "fp8" else 0.0
        assert bool(((out[b].double().cpu() - o).abs() <= e * pv + tail).all()), (b, n)
        assert bool(((lse[b].double().cpu() - l).abs() <= e + 2.0 ** -22 * l.abs()).all()), (b, n)
