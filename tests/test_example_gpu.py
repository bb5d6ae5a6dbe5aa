"""examples/speculative_decode.py: with temperature 0 the speculative tokens
are those of decoding one at a time, in fewer steps; at a temperature it runs
and accepts."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("fmt", ["F16", "Q8", "Q4"])
def test_speculative_decoding_gives_the_same_tokens(fmt):
    import quant_quantized_matvec_gb300 as kq
    import speculative_decode as S
    prompt = [(7 * i * i + 3) % 1003 for i in range(40)] * 2
    model = S.Model(fmt=getattr(kq, "KV_" + fmt))
    plain, one = S.generate(model, prompt, 128, depth=0)
    model = S.Model(fmt=getattr(kq, "KV_" + fmt))
    text, steps = S.generate(model, prompt, 128)
    assert text == plain
    assert all(s == 1 for s in one) and len(steps) < len(one)
    _, steps = S.generate(model, prompt, 16, temperature=0.5)
    assert sum(steps) >= len(steps)
    assert not kq.device_error()


@pytest.mark.parametrize("fmt", ["F16", "Q8", "Q4"])
def test_speculative_decoding_at_a_temperature_accepts(fmt):
    """Drafts are accepted at a temperature too (steps that give more than
    one token), and the same seed gives the same text."""
    import quant_quantized_matvec_gb300 as kq
    import speculative_decode as S
    prompt = [(7 * i * i + 3) % 1003 for i in range(40)] * 2
    model = S.Model(fmt=getattr(kq, "KV_" + fmt))
    text, steps = S.generate(model, prompt, 128, temperature=0.5)
    assert len(text) == 128 and all(0 <= t < model.vocab for t in text)
    assert sum(steps) > len(steps)
    assert S.generate(S.Model(fmt=getattr(kq, "KV_" + fmt)), prompt, 128, temperature=0.5) == (text, steps)
    assert not kq.device_error()
