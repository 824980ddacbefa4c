"""PagedKV.check: the status word is read and cleared in one step."""
import pytest
import torch

from decoder_greedy_decode_b200 import capi
from decoder_greedy_decode_b200.paged import PagedKV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_a_bit_raised_while_the_word_is_read_is_kept(monkeypatch):
    """Another stream's call raises a bit just after the host has read the
    word: the next check reports it."""
    c = PagedKV.create(1, 4, 8, 1, 64, 2, 16)
    item, late = torch.Tensor.item, []

    def read(t):
        v = item(t)
        if not late:
            late.append(c.status.bitwise_or_(capi.DEC_DEV_BAD_PAGE))
        return v

    c.status.fill_(capi.DEC_DEV_NO_PAGES)
    monkeypatch.setattr(torch.Tensor, "item", read)
    assert c.check() == capi.DEC_DEV_NO_PAGES
    assert late and c.check() == capi.DEC_DEV_BAD_PAGE
    assert c.check() == 0


def test_check_on_a_side_stream():
    c = PagedKV.create(1, 2, 8, 1, 64, 2, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.resize(torch.tensor([16, 16], dtype=torch.int32).cuda())
        assert c.check() == capi.DEC_DEV_NO_PAGES and c.check() == 0
