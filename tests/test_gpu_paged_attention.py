"""dec_paged_attention against a 64-bit softmax over the same rows."""
import math

import pytest
import torch

import paged_ref as ref
from decoder_greedy_decode_b200 import capi
from decoder_greedy_decode_b200.paged import PagedKV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def build(lens, kv, D, P, fmt, seed, layers=1, spare=3, max_rows=None, poison=True):
    """A cache whose sequences hold `lens` random rows on shuffled pages; every
    other row of the pool is NaN (NaN codes and scales) when `poison`."""
    g = torch.Generator().manual_seed(seed)
    width = max(1, -(-(max_rows or max(max(lens), 1)) // P))
    need = [-(-n // P) for n in lens]
    n = sum(need) + spare
    order = torch.randperm(n, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    held = torch.zeros((n, P), dtype=torch.bool)
    for b, rows in enumerate(lens):
        for j in range(need[b]):
            p = order.pop()
            table[b, j] = p
            held[p, : min(P, rows - j * P)] = True
    shape = (layers, n, kv, P, D)
    if fmt == "bf16":
        k, v = (torch.randn(shape, generator=g).bfloat16() for _ in range(2))
        scales = {}
        if poison:
            for x in (k, v):
                x.masked_fill_(~held[None, :, None, :, None], float("nan"))
    else:
        k, v = ((torch.randn(shape, generator=g) * 32).to(torch.float8_e4m3fn).view(torch.uint8)
                for _ in range(2))
        ks, vs = (0.01 + 0.06 * torch.rand(shape[:4], generator=g) for _ in range(2))
        if poison:
            for x in (k, v):
                x.masked_fill_(~held[None, :, None, :, None], 0x7F)
            for x in (ks, vs):
                x.masked_fill_(~held[None, :, None, :], float("nan"))
        scales = dict(k_scale=ks.cuda(), v_scale=vs.cuda())
    refs = torch.bincount(table[table >= 0].long(), minlength=n).int()
    return PagedKV(k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                   refs.cuda(), **scales)


def rows_of(c, layer, b, n):
    """Keys and values [kv, n, D] float64 of sequence b."""
    P = c.page_rows
    t = c.table[b].long().cpu()[: -(-n // P)]
    out = []
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        r = x[layer].cpu()[t]
        r = r.double() if s is None else ref.decode(r, s[layer].cpu()[t])
        out.append(r.permute(1, 0, 2, 3).reshape(c.n_kv_heads, -1, c.head_dim)[:, :n])
    return out


def check(c, layer, q, lens, out, lse, window=0):
    qd = q.double().cpu()
    for b, n in enumerate(lens):
        k, v = rows_of(c, layer, b, n)
        lo = max(0, n - window) if window else 0
        o, l, pv, mag = ref.attention(qd[b], k, v, lo, n)
        got, gl = out[b].double().cpu(), lse[b].double().cpu()
        if n <= lo:
            assert torch.count_nonzero(got) == 0 and bool((gl == -math.inf).all())
            continue
        eps = ref.attention_eps(c.head_dim, n, mag)
        assert bool(((got - o).abs() <= eps * pv + 1e-30).all()), (b, n, float(((got - o).abs() / pv).max()), eps)
        assert bool(((gl - l).abs() <= eps + 2.0 ** -22 * l.abs()).all()), (b, n)


def attend(c, q, lens, layer=0, window=0):
    rows = torch.tensor(lens, dtype=torch.int32).cuda()
    r = c.attend(layer, q, rows, window=window, return_lse=True)
    assert c.check() == 0
    return r


CASES = [
    # lens, q heads, kv heads, D, page, window
    ([1], 1, 1, 64, 8, 0),
    ([1], 16, 8, 128, 16, 0),
    ([7, 8, 9], 4, 2, 64, 8, 0),
    ([15, 16, 17, 0, 31, 33], 8, 8, 128, 8, 0),
    ([0, 0, 5, 0, 1, 0], 6, 2, 128, 16, 0),
    ([795], 16, 8, 128, 16, 0),
    ([200, 420, 333, 1, 64, 65, 63], 24, 8, 128, 16, 0),
    ([1025, 77, 4096], 8, 1, 128, 32, 0),
    ([1023, 5, 640], 7, 1, 64, 1024, 0),
    ([999, 130], 15, 5, 128, 128, 0),
    ([2500, 40, 17, 16, 0], 10, 2, 64, 64, 33),
    ([300, 16, 15, 17, 1], 4, 4, 128, 8, 16),
    ([300, 299, 298, 297, 296, 295, 294, 293], 5, 1, 128, 8, 1),
    ([5000], 16, 2, 128, 16, 4096),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P,window", CASES)
def test_attention_matches_64_bits(lens, Hq, Hkv, D, P, window, fmt):
    c = build(lens, Hkv, D, P, fmt, seed=sum(lens) + Hq + D, layers=2)
    if window:   # pages wholly before the window may be gone
        t = c.table.cpu()
        for b, n in enumerate(lens):
            t[b, : max(0, n - window) // P] = -1
    q = torch.randn((len(lens), Hq, D), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    keep = c.table.clone()
    if window:
        c.table.copy_(t)
    out, lse = attend(c, q, lens, layer=1, window=window)
    again, _ = attend(c, q, lens, layer=1, window=window)
    c.table.copy_(keep)
    assert torch.equal(out, again)
    check(c, 1, q, lens, out, lse, window)


def test_a_single_row_returns_its_value():
    for fmt in ("bf16", "fp8"):
        c = build([1, 1], 2, 128, 16, fmt, seed=4)
        q = torch.randn((2, 4, 128)).bfloat16().cuda()
        out, _ = attend(c, q, [1, 1])
        for b in range(2):
            v = rows_of(c, 0, b, 1)[1][:, 0].float().repeat_interleave(2, 0)
            assert torch.allclose(out[b].cpu(), v, rtol=2.0 ** -17, atol=0)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_ragged_batch_of_many_sequences(fmt):
    lens = [(37 * i * i) % 421 for i in range(150)]
    c = build(lens, 2, 128, 16, fmt, seed=8)
    q = torch.randn((150, 8, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out, lse = attend(c, q, lens)
    check(c, 0, q, lens, out, lse)


def test_agrees_with_the_contiguous_attention():
    B, Hq, Hkv, D, n = 3, 16, 8, 128, 795
    lens = [795, 400, 1]
    c = build(lens, Hkv, D, 16, "bf16", seed=5)
    q = torch.randn((B, Hq, D), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    out, _ = attend(c, q, lens)
    k, v = (torch.zeros((B, Hkv, n, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for b, m in enumerate(lens):
        kk, vv = rows_of(c, 0, b, m)
        k[b, :, :m], v[b, :, :m] = kk.bfloat16().cuda(), vv.bfloat16().cuda()
    nb = capi.dec_attention_workspace_bytes(B, Hq, Hkv, D, n)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    ref_out = torch.zeros((B, Hq, D), device="cuda")
    capi.dec_attention(B, Hq, Hkv, D, q, k, v, n, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       ref_out, ws, nb)
    assert torch.allclose(out, ref_out, rtol=0, atol=2e-5)


def test_strided_queries_and_nested_layouts():
    # pages outermost, K and V of a layer in one buffer; q a slice of qkv
    L, n, H, P, D = 3, 9, 2, 16, 64
    g = torch.Generator().manual_seed(9)
    buf = torch.randn((n, L, 2, H, P, D), generator=g).bfloat16().cuda()
    k, v = buf[:, :, 0].transpose(0, 1), buf[:, :, 1].transpose(0, 1)
    table = torch.tensor([[4, 0, 7], [8, 2, -1]], dtype=torch.int32).cuda()
    lens = [40, 32]
    refs = torch.zeros(n, dtype=torch.int32).cuda()
    c = PagedKV(k, v, table, torch.tensor(lens, dtype=torch.int32).cuda(), refs)
    qkv = torch.randn((2, 8 * D), generator=g).bfloat16().cuda()
    q = qkv[:, : 4 * D].unflatten(1, (4, D))
    for layer in range(L):
        out, lse = c.attend(layer, q, return_lse=True)   # rows: the map's own
        check(c, layer, q, lens, out, lse)
    assert c.check() == 0


def test_element_offsets_beyond_32_bits():
    # pages 2^28 elements apart: the last one starts past 2^31 elements
    H, P, D, n = 1, 16, 128, 12
    stride = 1 << 28
    big = torch.empty((n - 1) * stride + H * P * D, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((1, n, H, P, D), (stride * n, stride, P * D, D, 1))
    vbuf = torch.empty(n * H * P * D, dtype=torch.bfloat16, device="cuda")
    for p in range(n):
        k[0, p] = torch.randn((H, P, D), device="cuda")
    # V shares K's strides: the same pages, one page row further in the buffer
    v = big[P * D:].as_strided((1, n - 1, H, P, D), (stride * n, stride, P * D, D, 1))
    k = big.as_strided((1, n - 1, H, P, D), (stride * n, stride, P * D, D, 1))
    for p in range(n - 1):
        v[0, p] = torch.randn((H, P, D), device="cuda")
    table = torch.tensor([[10, 3, 9]], dtype=torch.int32, device="cuda")
    c = PagedKV(k, v, table, torch.tensor([48], dtype=torch.int32, device="cuda"),
                torch.zeros(n - 1, dtype=torch.int32, device="cuda"))
    q = torch.randn((1, 2, D), device="cuda").bfloat16()
    out, lse = c.attend(0, q, return_lse=True)
    assert c.check() == 0
    kk = torch.cat([k[0, p] for p in (10, 3, 9)], 1).double().cpu()
    vv = torch.cat([v[0, p] for p in (10, 3, 9)], 1).double().cpu()
    o, l, pv, mag = ref.attention(q[0].double().cpu(), kk, vv, 0, 48)
    assert bool(((out[0].double().cpu() - o).abs() <= ref.attention_eps(D, 48, mag) * pv).all())
    del vbuf


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_large_and_tiny_scores(fmt):
    """Scores of +-1e4 (one row takes all), rows of very different size, all
    equal rows."""
    lens = [333, 100, 64]
    c = build(lens, 2, 128, 16, fmt, seed=21)
    t = c.table[1].long()
    if fmt == "bf16":
        c.k[:, c.table[0].long()] *= 300
        c.v[:, t[0]] *= 1e20
        c.v[:, t[1]] *= 1e-20
        c.k[:, c.table[2, 0].long()] = c.k[:, c.table[2, 0].long()][:, :, :1]
    else:
        c.k_scale[:, c.table[0].long()] *= 300
        c.v_scale[:, t[0]] *= 1e20
        c.v_scale[:, t[1]] *= 1e-20
    q = torch.randn((3, 4, 128), generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    q[2, 1] *= 1e-30
    q[2, 2] = 0
    out, lse = attend(c, q, lens)
    check(c, 0, q, lens, out, lse)


def test_e4m3_rows_far_apart_in_size():
    """A V row that is 2^40 larger than the others but holds no weight: the
    others keep their precision."""
    c = build([200], 1, 128, 16, "fp8", seed=22)
    t = c.table[0].long()
    q = torch.ones((1, 1, 128)).bfloat16().cuda()
    # row 0: a large V row whose score is far below the others'
    c.k[0, t[0], 0, 0] = (-torch.full((128,), 400.0)).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    c.k_scale[0, t[0], 0, 0] = 0.03
    c.v_scale[0, t[0], 0, 0] *= 2.0 ** 40
    out, lse = attend(c, q, [200])
    check(c, 0, q, [200], out, lse)


def test_infinite_and_nan_rows_follow_the_formula():
    c = build([40, 40, 40], 1, 64, 8, "bf16", seed=23)
    c.k[0, c.table[0, 0].long(), 0, 3] = float("nan")
    c.v[0, c.table[1, 0].long(), 0, 3, 5] = float("inf")
    q = torch.ones((3, 2, 64)).bfloat16().cuda()
    out, lse = c.attend(0, q, return_lse=True)
    assert c.check() == 0
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isinf(out[1, :, 5]).all() and torch.isfinite(out[1, :, :5]).all()
    assert torch.isfinite(out[2]).all()


def test_e4m3_nan_codes_reach_the_output():
    c = build([40, 40], 1, 128, 8, "fp8", seed=24)
    c.v[0, c.table[0, 1].long(), 0, 2, 7] = 0x7F
    out = c.attend(0, torch.ones((2, 2, 128)).bfloat16().cuda())
    assert torch.isnan(out[0, :, 7]).all() and torch.isfinite(out[0, :, :7]).all()
    assert torch.isfinite(out[1]).all()


@pytest.mark.parametrize("long", [40, 9000])
def test_bad_pages_and_lengths_leave_the_output(long):
    """Whole and split sequences: a page out of range leaves that sequence's
    output as it was and raises the bit; so does a length out of range."""
    c = build([long, 50, 60, 10], 2, 128, 16, "bf16", seed=25, poison=False)
    c.table[0, 1] = c.n_pages
    c.table[1, 0] = -1
    q = torch.randn((4, 4, 128)).bfloat16().cuda()
    out = torch.full((4, 4, 128), 7.0, device="cuda")
    rows = torch.tensor([long, 50, 60, c.width * 16 + 1], dtype=torch.int32, device="cuda")
    c.attend(0, q, rows, out=out)
    assert c.check() == capi.DEC_DEV_BAD_PAGE | capi.DEC_DEV_BAD_POSITION
    assert bool((out[[0, 1, 3]] == 7).all())
    assert bool((out[2] != 7).all())
    assert c.check() == 0
    rows[3] = -1
    rows[:2] = 0
    c.attend(0, q, rows, out=out)
    assert c.check() == capi.DEC_DEV_BAD_POSITION
    assert torch.count_nonzero(out[:2]) == 0 and bool((out[3] == 7).all())


def test_rows_behind_the_batch_are_left():
    c = build([30, 20, 10], 2, 64, 8, "bf16", seed=26)
    buf = torch.full((3, 4, 64), 5.0, device="cuda")
    q = torch.randn((2, 4, 64)).bfloat16().cuda()
    c.attend(0, q, c.rows[:2].contiguous(), out=buf[:2])
    assert bool((buf[2] == 5).all()) and bool((buf[:2] != 5).all())


def test_captured_and_overlapping_calls():
    """Two graphs of one cache replayed on two streams at once, with lengths
    changed between replays."""
    lens = [700, 33, 260, 0]
    c = build([1000] * 4, 2, 128, 16, "bf16", seed=27)
    rows = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(i)).bfloat16().cuda()
          for i in range(2)]
    c.attend(0, qs[0], rows)
    graphs, outs, streams = [], [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs.append(c.attend(0, q, rows))
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    for new in (lens, [1, 999, 500, 16]):
        rows.copy_(torch.tensor(new, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for q, o in zip(qs, outs):
            want, lse = c.attend(0, q, rows, return_lse=True)
            assert torch.equal(o, want)
            check(c, 0, q, new, want, lse)


def test_side_stream():
    c = build([500, 20], 2, 64, 16, "fp8", seed=28)
    q = torch.randn((2, 4, 64)).bfloat16().cuda()
    want = c.attend(0, q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = c.attend(0, q, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_windows_longer_than_the_context_and_of_one_row():
    lens = [100, 31, 64, 1]
    c = build(lens, 2, 64, 16, "fp8", seed=31)
    q = torch.randn((4, 6, 64), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    whole = attend(c, q, lens)
    for w in (100, 1 << 30):
        got = attend(c, q, lens, window=w)
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])
    out, lse = attend(c, q, lens, window=1)
    check(c, 0, q, lens, out, lse, 1)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_many_kv_heads_and_long_skewed_batches(fmt):
    """More heads than a worker's CTA holds, and one sequence that all workers
    share beside short ones."""
    c = build([77, 5], 96, 64, 8, fmt, seed=32)
    q = torch.randn((2, 96, 64), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    out, lse = attend(c, q, [77, 5])
    check(c, 0, q, [77, 5], out, lse)
    lens = [30000] + [3] * 9 + [0]
    c = build(lens, 1, 128, 64, fmt, seed=33)
    q = torch.randn((11, 8, 128), generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    out, lse = attend(c, q, lens)
    check(c, 0, q, lens, out, lse)


def test_a_small_sequence_in_a_large_table():
    """The table's width says nothing about the work: lengths do."""
    c = build([50, 20], 2, 64, 16, "bf16", seed=34, max_rows=1 << 20)
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    out, lse = attend(c, q, [50, 20])
    check(c, 0, q, [50, 20], out, lse)
