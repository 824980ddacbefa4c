"""What Decoder.beam_search refuses, it refuses before it touches the cache."""
import pytest
import torch

from decoder_greedy_decode_b200 import capi, synth
from decoder_greedy_decode_b200.decoder import Decoder, to_device

pytestmark = pytest.mark.gpu


def test_a_refused_search_leaves_the_cache():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s = synth.TINY
    dec = Decoder(s, to_device(synth.model_weights(s, seed=3)), 64)
    kv = dec.kv_cache(64, 64)
    host, _ = synth.kv_prefill(s, 64, 64, [20] * 64, seed=4)
    kv.values.copy_(host.cuda())
    tok, pos = synth.tokens(s.vocab, 1, seed=5).cuda(), torch.tensor([20], dtype=torch.int32).cuda()
    for beams, eos in ((33, -1), (0, -1), (-1, -1), (4, s.vocab), (4, -2), (65, -1)):
        with pytest.raises((ValueError, capi.DecError)):
            dec.beam_search(kv, tok, pos, 3, beams, eos=eos)
        same = torch.equal(kv.values, host.cuda())
        assert same, (beams, eos)
    dec.beam_search(kv, tok, pos, 3, 32, eos=s.vocab - 1)
    assert dec.check() == 0
    dec.close()
