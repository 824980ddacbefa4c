"""dec_pages_resize, dec_pages_fork and dec_pages_compact against a map of
Python lists that changes one sequence at a time; data moves bit for bit."""
import random

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


def make(n_pages, n_seqs, width, P, fmt="bf16", layers=2, kv=2, D=64, seed=0):
    """An empty map over a pool of random bytes, and its reference."""
    c = PagedKV.create(layers, n_pages, P, kv, D, n_seqs, width * P, dtype=fmt)
    g = torch.Generator().manual_seed(seed)
    for x in (c.k, c.v):
        x.view(torch.uint8).copy_(torch.randint(0, 256, x.view(torch.uint8).shape, generator=g).to(torch.uint8))
    pools = [c.k, c.v]
    if fmt == "fp8":
        for x in (c.k_scale, c.v_scale):
            x.copy_(torch.rand(x.shape, generator=g))
        pools += [c.k_scale, c.v_scale]
    host = [x.cpu().view(torch.int16 if x.dtype == torch.bfloat16 else x.dtype).clone() for x in pools]
    return c, ref.RefMap(n_pages, n_seqs, width, P), pools, host


def same(c, m, pools, host):
    assert c.table.cpu().tolist() == m.table()
    assert c.rows.cpu().tolist() == m.rows
    assert c.refs.cpu().tolist() == m.refs
    for x, y in zip(pools, host):
        z = x.cpu()
        assert torch.equal(z.view(y.dtype), y)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("P,n_seqs,n_pages,width,seed", [
    (8, 1, 5, 4, 0), (8, 6, 30, 6, 1), (16, 40, 300, 11, 2), (64, 3, 7, 3, 3), (32, 16, 20, 5, 4), (8, 70, 9000, 40, 5),
])
def test_random_histories(P, n_seqs, n_pages, width, seed, fmt):
    if n_pages > 1000 and fmt == "fp8":
        pytest.skip("the pool is large enough once")
    rng = random.Random(seed)
    c, m, pools, host = make(n_pages, n_seqs, width, P, fmt, layers=1 if n_pages > 1000 else 2, seed=seed)
    full = 0
    for step in range(25):
        what = rng.random()
        if what < 0.55:
            target = []
            for s in range(n_seqs):
                r = rng.random()
                target.append(-1 if r < 0.2 else 0 if r < 0.25 else rng.randint(0, width * P) if r < 0.4
                              else min(width * P, m.rows[s] + rng.randint(0, 2 * P)) if r < 0.9
                              else max(0, m.rows[s] - rng.randint(0, P)))
            ok = m.resize(target)
            c.resize(i32(target))
            assert c.check() == (0 if ok else capi.DEC_DEV_NO_PAGES)
            if ok:
                m.move(*host)
            full += not ok
        elif what < 0.85:
            parents = [rng.choice([s, rng.randrange(n_seqs), -1 if rng.random() < 0.3 else s]) for s in range(n_seqs)]
            m.fork(parents)
            c.fork(i32(parents))
            assert c.check() == 0
        else:
            n = m.compact()
            live = c.compact()
            assert c.check() == 0 and int(live) == n
            m.move(*host)
        if step % 5 == 4 or n_pages < 1000:
            same(c, m, pools, host)
    same(c, m, pools, host)


def test_shared_last_page_leaves_one_holder():
    """Four copies of one sequence with a partly filled page: three of the four
    that grow get pages of their own, and only the filled rows move."""
    c, m, pools, host = make(12, 5, 4, 8, seed=6)
    m.resize([11, -1, -1, -1, -1]), c.resize(i32([11, -1, -1, -1, -1]))
    m.fork([0, 0, 0, 0, -1]), c.fork(i32([0, 0, 0, 0, -1]))
    m.resize([12, 12, 12, 12, 0]), c.resize(i32([12, 12, 12, 12, 0]))
    assert len(m.copies) == 3 and all(r == 3 for _, _, r in m.copies)
    m.move(*host)
    same(c, m, pools, host)
    # one of the holders stays: both others that grow are copied
    c, m, pools, host = make(12, 3, 4, 8, seed=7)
    for x in (m, c):
        f = (lambda v: v) if x is m else i32
        x.resize(f([11, -1, -1])), x.fork(f([0, 0, 0])), x.resize(f([-1, 12, 13]))
    assert len(m.copies) == 2
    m.move(*host)
    same(c, m, pools, host)


def test_crop_into_a_shared_page_copies_before_it_grows():
    c, m, pools, host = make(10, 2, 4, 8, seed=8)
    for x in (m, c):
        f = (lambda v: v) if x is m else i32
        x.resize(f([24, 0])), x.fork(f([0, 0])), x.resize(f([-1, 10])), x.resize(f([-1, 11]))
    assert m.copies == [(1, 2, 2)] or len(m.copies) == 1
    m.move(*host)
    same(c, m, pools, host)


def test_pages_released_in_a_call_serve_it():
    c, m, pools, host = make(4, 2, 4, 8)
    for x in (m, c):
        f = (lambda v: v) if x is m else i32
        x.resize(f([32, 0])), x.resize(f([0, 32]))
    assert c.check() == 0
    same(c, m, pools, host)


def test_errors_change_nothing():
    c, m, pools, host = make(6, 3, 4, 8, seed=9)
    m.resize([9, 20, 0]), c.resize(i32([9, 20, 0]))
    c.resize(i32([0, 32, 32]))                       # 8 pages of 6
    assert c.check() == capi.DEC_DEV_NO_PAGES
    same(c, m, pools, host)
    c.resize(i32([33, 0, 0]))                        # behind the table
    assert c.check() == capi.DEC_DEV_BAD_POSITION
    same(c, m, pools, host)
    c.fork(i32([0, 3, 1]))
    assert c.check() == capi.DEC_DEV_BAD_PAGE
    same(c, m, pools, host)
    keep = c.table.clone()
    c.table[1, 2] = 6                                # a page that is not there
    c.resize(i32([-1, 8, -1]))
    assert c.check() == capi.DEC_DEV_BAD_PAGE
    c.resize(i32([-1, 21, -1]))
    assert c.check() == capi.DEC_DEV_BAD_PAGE
    c.table.copy_(keep)
    c.rows[0] = -5
    c.resize(i32([-1, 8, -1]))
    assert c.check() == capi.DEC_DEV_BAD_POSITION
    c.rows[0] = 9
    same(c, m, pools, host)


def test_compaction_of_empty_full_and_packed_pools():
    c, m, pools, host = make(9, 2, 4, 8, seed=10)
    assert int(c.compact()) == m.compact() == 0
    m.resize([30, 0]), c.resize(i32([30, 0]))
    assert int(c.compact()) == m.compact() == 4      # already in front
    same(c, m, pools, host)
    m.resize([30, 32]), c.resize(i32([30, 32]))
    m.resize([0, 32]), c.resize(i32([0, 32]))
    assert int(c.compact()) == m.compact() == 4
    m.move(*host)
    same(c, m, pools, host)
    c.table[0, 3] = -7
    c.compact()
    assert c.check() == capi.DEC_DEV_BAD_PAGE and int(c.table[0, 3]) == -7


def test_many_sequences():
    n = 4096
    c, m, pools, host = make(6000, n, 3, 8, layers=1, kv=1, seed=11)
    t = [(7 * s) % 12 for s in range(n)]
    m.resize(t), c.resize(i32(t))
    par = [s if s % 3 else (5 * s) % n for s in range(n)]
    assert c.check() == 0
    m.fork(par), c.fork(i32(par))
    same(c, m, pools, host)
    t = [min(24, r + 1) if s % 5 == 0 else -1 for s, r in enumerate(m.rows)]
    ok = m.resize(t)
    c.resize(i32(t))
    assert c.check() == (0 if ok else capi.DEC_DEV_NO_PAGES)
    if ok:
        m.move(*host)
    same(c, m, pools, host)


@pytest.mark.parametrize("n", [300, 1025, 2500])
def test_sequences_shrink_and_grow_by_many_pages_at_once(n):
    """Every kind of change in one call: freed, cropped, kept, grown by a row (a
    copy where the page is shared), by a few pages and by many."""
    width = 9
    c, m, pools, host = make(n * 6, n, width, 8, layers=1, kv=1, seed=n)
    rng = random.Random(n)
    t = [rng.choice([0, 3, 8, 20, 41]) for _ in range(n)]
    assert m.resize(t)
    c.resize(i32(t))
    par = [s // 2 * 2 if s % 3 else s for s in range(n)]
    m.fork(par), c.fork(i32(par))
    for _ in range(3):
        t = [rng.choice([0, r // 2, -1, r, min(72, r + 1), min(72, r + 30), 72]) for r in m.rows]
        if not m.resize(t):
            c.resize(i32(t))
            assert c.check() == capi.DEC_DEV_NO_PAGES
        else:
            c.resize(i32(t))
            assert c.check() == 0
            m.move(*host)
        same(c, m, pools, host)


def test_nested_layout_moves_only_its_pages():
    """Pages outermost, K and V of all layers in one buffer."""
    g = torch.Generator().manual_seed(12)
    n, L, H, P, D = 8, 3, 2, 8, 64
    buf = torch.randint(-30000, 30000, (n, L, 2, H, P, D), generator=g, dtype=torch.int16)
    dev = buf.cuda()
    k, v = (dev[:, :, i].transpose(0, 1).view(torch.bfloat16) for i in range(2))
    table = torch.tensor([[7, 5, -1], [2, -1, -1]], dtype=torch.int32).cuda()
    refs = torch.zeros(n, dtype=torch.int32).cuda()
    refs[[7, 5, 2]] = 1
    c = PagedKV(k, v, table, i32([12, 3]), refs)
    assert int(c.compact()) == 3 and c.check() == 0
    want = buf.clone()
    want[0], want[1] = buf[5], buf[7]
    assert torch.equal(dev.cpu(), want)
    assert c.table.cpu().tolist() == [[1, 0, -1], [2, -1, -1]]
    assert c.refs.cpu().tolist() == [1, 1, 1, 0, 0, 0, 0, 0]


def test_captured_fork_and_resize():
    c, m, pools, host = make(20, 4, 5, 8, seed=13)
    m.resize([11, 0, 0, 0]), c.resize(i32([11, 0, 0, 0]))
    par, tgt = i32([0, 0, 0, -1]), i32([12, 13, 14, 0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.fork(par)
        c.resize(tgt)
    for p, t in (([0, 0, 0, -1], [12, 13, 14, 0]), ([2, 1, 2, 0], [15, 14, 20, 13])):
        par.copy_(i32(p)), tgt.copy_(i32(t))
        g.replay()
        m.fork(p), m.resize(t)
        m.move(*host)
        assert c.check() == 0
        same(c, m, pools, host)
