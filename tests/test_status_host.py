"""dec_status_take without a GPU: what it refuses on the host (the pointers are
fake and never read)."""
from decoder_greedy_decode_b200 import capi


def test_bad_pointers_are_refused():
    L, p = capi.lib(), 1 << 20
    assert L.dec_status_take(None, p, None) == -1 and L.dec_status_take(p, None, None) == -1
    assert L.dec_status_take(p + 2, p, None) == -6 and L.dec_status_take(p, p + 1, None) == -6
