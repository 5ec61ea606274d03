"""The generating example: its graph gives what its eager steps give, greedy
tokens are the head's argmax, and each layer's attention is that of all the
keys so far."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def decoder(request):
    import int4_q4_weight_gb300 as q4w
    q4w.load()
    import generate
    return generate.Decoder(layers=4, H=256, mlp=512, V=1024, max_len=700, seed=3)


def test_graph_and_eager_steps_agree(cuda_lib, decoder):
    u = torch.rand(40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    decoder.capture()
    a, la = decoder.generate(5, 40, u, graph=True)
    b, lb = decoder.generate(5, 40, u, graph=False)
    cuda_lib.q4_device_status()
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert len(set(a.tolist())) > 5 and int(decoder.kv_lens) == 40
    assert torch.all(torch.isfinite(la)) and torch.all(la <= 0)


def test_greedy_tokens_are_the_argmax(cuda_lib, decoder):
    decoder.settings["temperature"].zero_()
    try:
        decoder.token.fill_(7)
        decoder.kv_lens.zero_()
        for _ in range(10):
            decoder.step()
            assert int(decoder.token) == int(decoder.idx) and float(decoder.logprob) == 0.0
    finally:
        decoder.settings["temperature"].fill_(1.0)


def test_attention_of_the_last_step(cuda_lib, decoder):
    """The last layer's (head size 512, no window) and the first's (window 512) attention
    after 600 tokens, from the caches and the rotated query, in fp64."""
    u = torch.rand(600, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    decoder.generate(3, 600, u, graph=False)
    cuda_lib.q4_device_status()
    pages = decoder.block_table[0].cpu().numpy()
    for L, window in ((decoder.layers[0], 512), (decoder.layers[3], 600)):
        D = L["D"]
        k = L["kc"].double().cpu().numpy()[pages, 0].reshape(-1, D)[:600][-window:]
        v = L["vc"].double().cpu().numpy()[pages, 0].reshape(-1, D)[:600][-window:]
        q = L["q16"][0].double().cpu().numpy()
        s = q @ k.T / np.sqrt(D)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        ref, a = w @ v, w @ np.abs(v)
        got = L["att"][0].double().cpu().numpy()
        # one rounding of the probabilities and one of the output (2^-11 each), fp32 scores
        assert np.all(np.abs(got - ref) <= 2.0 ** -11 * (a + np.abs(ref)) * 1.01 + 1e-5 * a + 1e-6)
