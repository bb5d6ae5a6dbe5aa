"""Prompts of lengths three decades apart in one call, few enough that their keys
are cut into parts."""
import pytest

import prompt_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402

KINDS = [torch.float32, torch.float16, torch.bfloat16]


def starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return s


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,ctx", [
    ([300] + [16] * 7, [12001] + [0] * 7), ([16] * 7 + [300], [0] * 7 + [12001]),
    ([1, 200, 1, 1], [5, 9001, 0, 4000]), ([3, 2, 5], [20000, 1, 30]), ([0, 130, 0, 7], [700, 6000, 0, 0])])
def test_lengths_far_apart(new, ctx, dim, kind):
    g = torch.Generator(device="cuda").manual_seed(len(new) + dim)
    held = [a + b for a, b in zip(new, ctx)]

    def normal(n, h):
        return torch.randn(n, h, dim, generator=g, device="cuda")

    q, k, v = (x.to(kind) for x in (2 * normal(sum(new), 4), normal(sum(held), 2), normal(sum(held), 2)))
    s, ks = starts(new), starts(held)
    sd, kd = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (s, ks))
    need = kq.prompt_workspace_bytes(q, k, len(new))
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    got = kq.prompt_attention(q, k, v, sd, kd, workspace=ws)
    want, bound, _ = R.attention(q, k, v, s, ks, dim ** -0.5)
    assert torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= bound).all()
    assert (ws[need:] == 255).all()
    for _ in range(3):
        assert torch.equal(kq.prompt_attention(q, k, v, sd, kd), got)
    # each by itself: other parts, the same within both bounds
    for b in range(len(new)):
        if new[b]:
            one = kq.prompt_attention(q[s[b]:s[b + 1]], k[ks[b]:ks[b + 1]], v[ks[b]:ks[b + 1]],
                                      torch.tensor([0, new[b]], dtype=torch.int32, device="cuda"),
                                      torch.tensor([0, held[b]], dtype=torch.int32, device="cuda"))
            assert ((one.double() - got[s[b]:s[b + 1]].double()).abs() <= 2 * bound[s[b]:s[b + 1]]).all()
    assert not kq.device_error()
