"""Scales of the prompt's attention at both ends of f32."""
import pytest

import prompt_ref as R
from quant_quantized_matvec_gb300 import _binding
from quant_quantized_matvec_gb300 import build as kbuild

torch = pytest.importorskip("torch")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
SHAPE, ALIGN = 2, 5
A = [0x7f0000000000 + (i << 36) for i in range(8)]  # (never dereferenced)


@pytest.mark.parametrize("code", [0, 1, 30])
def test_refusals(code):
    kbuild.build()
    lib = _binding.load()

    def call(scale):  # (refused for its address, at the latest)
        return lib.kq_prompt_attention(code, 1, 9, 9, A[0], None, A[1], 512, 4, A[2], 256, A[3], 256, 2,
                                       128, scale, A[4] + 4, None, 0, None)

    for scale in (2.35e38, -2.35e38, 1.2e-38, 1e-45, 0.0):
        assert call(scale) == ALIGN
    for scale in (2.4e38, 3.4e38, -3.4e38):
        assert call(scale) == (ALIGN if code == 0 else SHAPE)
    for scale in (float("inf"), float("nan")):
        assert call(scale) == SHAPE


def inputs(dim, kind, qsize, ksize):
    g = torch.Generator(device="cuda").manual_seed(dim)
    q = (qsize * torch.randn(90, 4, dim, generator=g, device="cuda")).to(kind)
    k = (ksize * torch.randn(120, 2, dim, generator=g, device="cuda")).to(kind)
    v = torch.randn(120, 2, dim, generator=g, device="cuda").to(kind)
    return q, k, v


# scale, and sizes of queries and keys that make logits of a few units
ENDS = [(F32, 3.4e38, 3e-30, 1e-9), (F32, -2.5e38, 1e-36, 4e-3), (F32, 1.1e-38, 1e28, 1e10),
        (F32, 1e-41, 1e30, 1e11), (F32, 2.0 ** -149, 3e35, 2e9), (F32, 3.4e38, 2e-38, 0.2),
        (BF16, 2.3e38, 1e-20, 5e-19), (BF16, 3e-39, 1e18, 3e18), (BF16, -1e-40, 1e18, 3e18),
        (F16, 2.3e38, 0.0, 1.0), (F16, 1e-45, 100.0, 100.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind,scale,qsize,ksize", ENDS)
def test_scales_at_both_ends(kind, scale, qsize, ksize, dim):
    import quant_quantized_matvec_gb300 as kq
    q, k, v = inputs(dim, kind, qsize, ksize)
    s, ks = [0, 90], [0, 120]
    scale = torch.tensor(scale, dtype=F32).item()
    sd, kd = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (s, ks))
    got = kq.prompt_attention(q, k, v, sd, kd, scale=scale)
    want, bound, _ = R.attention(q, k, v, s, ks, scale)
    # Queries, and their products with the scale's fraction, below 2^-126 are held
    # to 2^-150; a tiny scale's product with log2(e) to 2^-150 (16 bits).
    low = 2.0 ** -150 * 2 * (abs(scale) * k.double().abs().sum(-1).max() if kind is F32
                             else (q.double().abs().amax() * k.double().abs().sum(-1).max()))
    d = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (d <= bound + 4 * low * v.double().abs().max()).all(), (d / bound).max().item()


@pytest.mark.gpu
def test_refused_by_the_call():
    import quant_quantized_matvec_gb300 as kq
    q, k, v = inputs(64, BF16, 1e-20, 1e-19)
    s, ks = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 90], [0, 120]))
    with pytest.raises(kq.KQError, match="SHAPE"):
        kq.prompt_attention(q, k, v, s, ks, scale=3e38)
