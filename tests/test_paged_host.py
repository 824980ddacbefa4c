"""The paged-cache and beam entry points without a GPU: what they refuse on
the host (the pointers are fake and never read), and the rotation's table."""
import ctypes

import numpy as np
import pytest

import paged_ref as ref
from decoder_greedy_decode_b200 import capi

P = 1 << 20   # a fake device address


def pool(**kw):
    d = dict(k=P, v=P, k_scale=None, v_scale=None, n_layers=2, n_pages=10, page_rows=16, n_kv_heads=8,
             head_dim=128, dtype=0, layer_stride=10 * 8 * 16 * 128, page_stride=8 * 16 * 128)
    d.update(kw)
    return capi.dec_pages(*d.values())


def pmap(**kw):
    d = dict(table=P, rows=P, refs=P, n_seqs=4, width=8)
    d.update(kw)
    return capi.dec_page_map(*d.values())


BAD_POOLS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(dtype=2), -5), (dict(dtype=1), -1),
    (dict(head_dim=96), -2), (dict(page_rows=12), -2), (dict(page_rows=4), -2), (dict(page_rows=2048), -2),
    (dict(page_rows=0), -2), (dict(n_layers=0), -2), (dict(n_pages=0), -2), (dict(n_kv_heads=0), -2),
    (dict(page_stride=8 * 16 * 128 - 128), -2), (dict(layer_stride=0), -2),
    (dict(page_stride=8 * 16 * 128 + 8), -2), (dict(k=P + 8), -6),
    (dict(dtype=1, k_scale=P, v_scale=P + 8), -6),
    (dict(dtype=1, k_scale=P, v_scale=P, page_stride=8 * 16 * 128 + 128), -6), (dict(n_kv_heads=257), -2),
]
BAD_MAPS = [(dict(table=None), -1), (dict(rows=None), -1), (dict(refs=None), -1), (dict(n_seqs=0), -3),
            (dict(n_seqs=4097), -3), (dict(width=0), -2), (dict(width=1 << 28), -2), (dict(table=P + 2), -6)]


def calls(pg, pm):
    L = capi.lib()
    a, b = ctypes.byref(pg), ctypes.byref(pm)
    io = append_io()
    return [L.dec_pages_resize(a, b, P, P, 1 << 30, None, None), L.dec_pages_fork(a, b, P, None, None),
            L.dec_pages_compact(a, b, P, P, 1 << 30, None, None),
            L.dec_paged_append(a, b, 0, ctypes.byref(io), None, None),
            L.dec_paged_attention(a, b, 0, 1, 8, P, 0, None, 0, P, None, P, 1 << 30, None, None)]


def append_io(**kw):
    d = dict(n_tokens=4, dtype=0, n_q_heads=16, q=P, k=P, v=P, q_stride=4096, k_stride=4096, v_stride=4096,
             q_out=P, positions=P, seqs=P, q_norm=None, k_norm=None, eps=1e-6, rope=None)
    d.update(kw)
    return capi.dec_append(*d.values())


@pytest.mark.parametrize("kw,code", BAD_POOLS)
def test_pools_that_every_call_refuses(kw, code):
    assert calls(pool(**kw), pmap()) == [code] * 5
    assert capi.dec_pages_workspace_bytes(pool(**kw), pmap()) == 0
    assert capi.dec_paged_attention_workspace_bytes(pool(**kw), 1, 8) == 0


@pytest.mark.parametrize("kw,code", BAD_MAPS)
def test_maps_that_every_call_refuses(kw, code):
    assert calls(pool(), pmap(**kw)) == [code] * 5
    assert capi.dec_pages_workspace_bytes(pool(), pmap(**kw)) == 0


def test_a_table_of_more_than_int32_cells_is_refused():
    big = pmap(n_seqs=4096, width=1 << 19)    # 2^31 cells
    assert calls(pool(), big) == [-2] * 5
    assert capi.dec_pages_workspace_bytes(pool(), big) == 0
    assert capi.dec_pages_workspace_bytes(pool(), pmap(n_seqs=4095, width=1 << 19)) > 0


def test_page_calls_refuse_bad_arguments():
    L = capi.lib()
    a, b = ctypes.byref(pool()), ctypes.byref(pmap())
    need = capi.dec_pages_workspace_bytes(pool(), pmap())
    assert need > 0
    for f in (L.dec_pages_resize, L.dec_pages_compact):
        assert f(None, b, P, P, need, None, None) == -1
        assert f(a, None, P, P, need, None, None) == -1
        assert f(a, b, None, P, need, None, None) == -1
        assert f(a, b, P, None, need, None, None) == -1
        assert f(a, b, P, P + 16, need, None, None) == -6
        assert f(a, b, P + 1, P, need, None, None) == -6
        assert f(a, b, P, P, need - 1, None, None) == -4
    assert L.dec_pages_fork(a, b, None, None, None) == -1
    assert L.dec_pages_fork(a, b, P + 2, None, None) == -6 and L.dec_pages_fork(a, b, P, P + 2, None) == -6
    assert L.dec_pages_resize(a, b, P, P, need, P + 1, None) == -6
    assert L.dec_pages_compact(a, b, P, P, need, P + 1, None) == -6


def test_attention_refuses_bad_arguments():
    L = capi.lib()
    a, b = ctypes.byref(pool()), ctypes.byref(pmap())
    need = capi.dec_paged_attention_workspace_bytes(pool(), 4, 16)
    assert need > 0

    def go(layer=0, batch=4, hq=16, q=P, stride=2048, window=0, out=P, ws=P, nb=need):
        return L.dec_paged_attention(a, b, layer, batch, hq, q, stride, None, window, out, None, ws, nb, None, None)

    assert go(q=None) == -1 and go(out=None) == -1 and go(ws=None) == -1
    assert go(batch=0) == -3 and go(batch=5) == -3
    assert go(layer=-1) == -9 and go(layer=2) == -9 and go(window=-1) == -9
    assert go(hq=0) == -2 and go(hq=12) == -2 and go(hq=72) == -2 and go(hq=-8) == -2
    assert go(stride=2040) == -2 and go(stride=2052) == -6
    assert go(q=P + 8) == -6 and go(ws=P + 16) == -6 and go(out=P + 4) == -6
    assert go(nb=need - 1) == -4
    for rows, lse, status in ((P + 2, None, None), (P, P + 2, None), (P, None, P + 1)):
        assert L.dec_paged_attention(a, b, 0, 4, 16, P, 2048, rows, 0, P, lse, P, need, status, None) == -6


def test_append_refuses_bad_arguments():
    L = capi.lib()
    a, b = ctypes.byref(pool()), ctypes.byref(pmap())

    def go(layer=0, **kw):
        return L.dec_paged_append(a, b, layer, ctypes.byref(append_io(**kw)), None, None)

    assert L.dec_paged_append(a, b, 0, None, None, None) == -1
    assert go(layer=2) == -9 and go(layer=-1) == -9
    assert go(n_tokens=-1) == -3 and go(n_tokens=5, seqs=None) == -3
    assert go(dtype=2) == -5 and go(n_q_heads=-1) == -2
    assert go(k=None) == -1 and go(v=None) == -1 and go(positions=None) == -1
    assert go(q=None) == -1 and go(q_out=None) == -1 and go(n_q_heads=0) == -1
    assert go(eps=-1.0) == -9 and go(eps=float("nan")) == -9
    assert go(k=P + 4) == -6 and go(q=P + 2) == -6 and go(q_out=P + 4) == -6
    assert go(dtype=1, v=P + 8) == -6 and go(q_norm=P + 8) == -6
    assert go(k_stride=4100) == -6 and go(k_stride=512) == -2 and go(q_stride=2040) == -2
    for rope, code in ((capi.dec_rope(None, 128, 0, 1.0), -1), (capi.dec_rope(P, 0, 0, 1.0), -2),
                       (capi.dec_rope(P, 130, 0, 1.0), -2), (capi.dec_rope(P, 7, 0, 1.0), -2),
                       (capi.dec_rope(P + 4, 64, 0, 1.0), -6)):
        assert go(rope=ctypes.pointer(rope)) == code
    assert go(positions=P + 2) == -6 and go(seqs=P + 1) == -6
    assert L.dec_paged_append(a, b, 0, ctypes.byref(append_io()), P + 2, None) == -6
    assert go(n_tokens=0) == 0      # nothing to do


def test_rotation_refuses_bad_arguments():
    L = capi.lib()
    r = capi.dec_rope(P, 64, 0, 1.0)

    def go(n=4, H=2, D=64, dt=0, x=P, xs=128, out=1 << 24, os=128, pos=P, rope=r):
        return L.dec_rope_apply(n, H, D, dt, x, xs, out, os, pos, ctypes.byref(rope) if rope else None, None)

    assert go(rope=None) == -1 and go(n=-1) == -3 and go(dt=3) == -5
    assert go(D=96) == -2 and go(H=0) == -2 and go(rope=capi.dec_rope(P, 66, 0, 1.0)) == -2
    assert go(x=None) == -1 and go(out=None) == -1 and go(pos=None) == -1
    assert go(x=P + 4) == -6 and go(dt=1, x=P + 8) == -6 and go(xs=132) == -6 and go(os=64) == -2
    assert go(pos=P + 2) == -6
    assert go(out=P, os=256) == -9   # in place with another stride
    assert go(n=0, x=None) == 0


def test_beam_calls_refuse_bad_arguments():
    L = capi.lib()
    need = capi.dec_beam_workspace_bytes(2, 4, 1000, 8)
    assert need > 0
    for bad in ((0, 4, 1000, 8), (2, 0, 1000, 8), (2, 33, 1000, 8), (2, 4, 1000, 0), (2, 4, 1000, 33),
                (2, 4, 7, 8), (2, 4, 1 << 20, 8), (1 << 16, 4, 1000, 8)):
        assert capi.dec_beam_workspace_bytes(*bad) == 0
        assert L.dec_beam_select(*bad, 0, P, 1000, P, None, -1, P, P, P, P, P, 1 << 40, None) == -9

    def go(dt=1, x=P, stride=1000, sc=P, done=None, eos=-1, o=(P + 4, P, P, None), ws=P, nb=need, k=8):
        return L.dec_beam_select(2, 4, 1000, k, dt, x, stride, sc, done, eos, *o, ws, nb, None)

    assert go(x=None) == -1 and go(sc=None) == -1 and go(ws=None) == -1
    for i in range(3):
        o = [P + 4, P, P, None]
        o[i] = None
        assert go(o=o) == -1
    assert go(dt=2) == -5 and go(eos=-2) == -9 and go(eos=1000) == -9 and go(done=P) == -9
    assert go(stride=999) == -2 and go(x=P + 2) == -6 and go(ws=P + 64) == -6 and go(nb=need - 1) == -4
    assert go(o=(P, P, P, None)) == -9                        # in place with k != beams
    assert go(done=P, eos=1, o=(P + 4, P, P, P)) == -9

    def re(L_=2, H=2, D=64, dt=0, kvb=4, ctx=64, val=P, sc=None, b=4, par=P, rows=P):
        return L.dec_kv_reorder(L_, H, D, dt, kvb, ctx, val, sc, b, par, rows, None, None)

    assert re(val=None) == -1 and re(par=None) == -1 and re(rows=None) == -1 and re(dt=1) == -1
    assert re(D=32) == -2 and re(L_=0) == -2 and re(H=0) == -2 and re(dt=2) == -5
    assert re(b=0) == -3 and re(b=5) == -3 and re(b=65, kvb=100) == -3
    assert L.dec_kv_reorder(2, 2, 64, 0, 4, 64, P, None, 4, P, P, P + 2, None) == -6
    assert re(ctx=24) == -9 and re(ctx=0) == -9 and re(val=P + 8) == -6 and re(par=P + 1) == -6
    assert L.dec_beam_backtrace(-1, 1, 1, P, P, P, None) == -9
    assert L.dec_beam_backtrace(1, 0, 1, P, P, P, None) == -9
    assert L.dec_beam_backtrace(1, 1, 1, None, P, P, None) == -1
    assert L.dec_beam_backtrace(0, 1, 1, None, None, None, None) == 0


def phases(R, theta=1e6, scaling=0, factor=1.0, orig=0.0, alpha=1.0, beta=32.0):
    out = (ctypes.c_uint64 * 64)()
    capi.dec_rope_phases(R, theta, scaling, factor, orig, alpha, beta, out)
    return list(out)[: R // 2]


@pytest.mark.parametrize("name,code,kw", [("none", 0, {}), ("linear", 1, dict(factor=4.0)),
                                          ("ntk", 2, dict(factor=8.0)),
                                          ("parts", 3, dict(factor=4.0, orig=32768.0)),
                                          ("linear", 1, dict(factor=0.05))])
@pytest.mark.parametrize("R", [4, 64, 126, 128])
def test_phases_match_the_formula(R, name, code, kw):
    got = phases(R, scaling=code, **kw)
    f = ref.inv_freq(R, 1e6, name, kw.get("factor", 1.0), kw.get("orig", 0.0))
    for g, x in zip(got, f):
        turns = x / (2 * np.pi)
        want = int(round((turns % 1.0) * 2.0 ** 64))
        off = abs(g - want)
        off = min(off, 2 ** 64 - off)     # modulo one turn
        # the reference: six double roundings (2^-53 each, of all turns), and
        # both sides rounded to a whole number (half each)
        assert off <= turns * 2.0 ** 64 * 2.0 ** -50 + 1, (R, name)


def test_phases_refuse_bad_arguments():
    L = capi.lib()
    out = ctypes.cast((ctypes.c_uint64 * 64)(), ctypes.c_void_p)

    def go(R=64, theta=1e6, sc=0, f=1.0, orig=0.0, al=1.0, be=32.0, o=out):
        return L.dec_rope_phases(R, theta, sc, f, orig, al, be, o)

    assert go() == 0 and go(o=None) == -1
    assert go(R=0) == -2 and go(R=63) == -2 and go(R=130) == -2 and go(R=-2) == -2
    assert go(theta=1.0) == -9 and go(theta=float("nan")) == -9 and go(theta=float("inf")) == -9
    assert go(sc=4) == -9 and go(sc=-1) == -9 and go(sc=1, f=0.0) == -9 and go(sc=1, f=float("nan")) == -9
    assert go(R=2, sc=2, f=2.0) == -9
    assert go(sc=3, f=2.0) == -9 and go(sc=3, f=2.0, orig=100.0, al=3.0, be=3.0) == -9
    assert go(sc=3, f=2.0, orig=100.0) == 0


def test_messages_of_the_device_bits():
    s = capi.error_string(capi.DEC_DEV_BAD_PAGE | capi.DEC_DEV_NO_PAGES | capi.DEC_DEV_BAD_POSITION |
                          capi.DEC_DEV_BAD_TOKEN | capi.DEC_DEV_TIMEOUT)
    assert "page" in s and "free" in s and "position" in s and "token" in s and "wait" in s
