"""How far f32 attention of prompts is off as a rule.  Bounds of the worst case
(prompt_ref.py) are far wider than that at some sizes; these limits tell two f16
terms of each operand from one."""
import math

import pytest

import prompt_ref as R

torch = pytest.importorskip("torch")

# Inputs are normal, queries twice that, so logits are about 2 in size, values 1.
# A row's error goes by the row's own size.  Operands of two terms are off by
# 2^-24 or so, and so are what the sums are rounded by; the largest part is logits'
# sums, which the tensor core may cut off at each of d / 16 steps of the large
# products: at d = 256 half of 16 * 2^-23 of partial sums of about 1.3, 1.2e-6, which
# two logits in size make 2.5e-6 of a row.  Taken as 4e-6; ten times that for the
# largest of 10^5 values or so (five times the rule, and rows of one size another
# half).  An operand of one f16 term is off by 2^-12 / 3^(1/2), about 1e-4.
RULE, LARGEST = 4e-6, 4e-5

SHAPES = [([77], [0]), ([5, 1, 130, 64, 33], [0, 3, 0, 100, 7]), ([2100, 700], [0, 1500]), ([9], [3000])]


def off(got, want):
    """(root of the mean square, largest) error of rows [.., d], by a row's size."""
    size = want.square().mean(-1, keepdim=True).sqrt()
    e = (got.double() - want).abs() / size
    return e.square().mean().sqrt().item(), e.max().item()


def inputs(new, ctx, dim, seed, device):
    g = torch.Generator().manual_seed(seed)

    def normal(n, h):
        return torch.randn(n, h, dim, generator=g)

    held = sum(new) + sum(ctx)
    q, k, v = 2 * normal(sum(new), 4), normal(held, 2), normal(held, 2)
    s, ks = [0], [0]
    for a, b in zip(new, ctx):
        s.append(s[-1] + a), ks.append(ks[-1] + a + b)
    return q.to(device), k.to(device), v.to(device), s, ks


def terms(x):
    """Two f16 terms of x (64 bits), after a scaling that brings its largest to 2^15."""
    up = 2.0 ** (14 - math.floor(math.log2(x.abs().max().item())))
    hi = (x * up).half().double()
    return hi / up, (x * up - hi).half().double() / up


def with_terms(q, k, v, s, ks, drop):
    """Attention in 64 bits of operands in two f16 terms, without the products of
    one low term."""
    n, hq, d = q.shape
    out = torch.zeros(n, hq, d, dtype=torch.float64)
    for b in range(len(s) - 1):
        m, c = ks[b + 1] - ks[b], s[b + 1] - s[b]
        seen = torch.ones(c, m, dtype=torch.bool).tril(m - c)
        for h in range(hq):
            (q1, q0), (k1, k0), (v1, v0) = (terms(x.double()) for x in (
                q[s[b]:s[b + 1], h] * d ** -0.5, k[ks[b]:ks[b + 1], h // 2], v[ks[b]:ks[b + 1], h // 2]))
            x = q1 @ k1.T
            if drop != "q":
                x = x + q0 @ k1.T
            if drop != "k":
                x = x + q1 @ k0.T
            x = x.masked_fill(~seen, -math.inf)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p1, p0 = terms(p)
            y = p1 @ v1
            if drop != "p":
                y = y + p0 @ v1
            if drop != "v":
                y = y + p1 @ v0
            out[s[b]:s[b + 1], h] = y / p.sum(-1, keepdim=True)
    return out


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,ctx", SHAPES[:2] + [([400, 100], [0, 300])])
def test_limits_tell_two_terms_from_one(new, ctx, dim):
    q, k, v, s, ks = inputs(new, ctx, dim, dim, "cpu")
    want = R.attention(q, k, v, s, ks, dim ** -0.5)[0]
    rule, largest = off(with_terms(q, k, v, s, ks, None), want)
    assert rule <= RULE / 4 and largest <= LARGEST / 4
    for drop in "qkvp":
        rule, largest = off(with_terms(q, k, v, s, ks, drop), want)
        assert rule > 4 * RULE, drop
        assert largest > LARGEST, drop


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,ctx", SHAPES)
def test_f32_as_a_rule(new, ctx, dim):
    import quant_quantized_matvec_gb300 as kq
    q, k, v, s, ks = inputs(new, ctx, dim, dim + 1, "cuda")
    want = R.attention(q, k, v, s, ks, dim ** -0.5)[0]
    sd, kd = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (s, ks))
    rule, largest = off(kq.prompt_attention(q, k, v, sd, kd), want)
    assert rule <= RULE and largest <= LARGEST
    # tokens of sizes up to 2^20 apart, which have powers of two of their own
    g = torch.Generator().manual_seed(dim)
    by = (2.0 ** (20 * torch.rand(k.shape[0], 1, 1, generator=g) - 20)).cuda()
    v = v * by
    want = R.attention(q, k, v, s, ks, dim ** -0.5)[0]
    rule, largest = off(kq.prompt_attention(q, k, v, sd, kd), want)
    assert rule <= RULE and largest <= LARGEST
