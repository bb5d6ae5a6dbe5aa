"""f32 attention of prompts whose tokens' sizes lie far apart: what a row does
not attend, or attends with no weight, takes no bits from what it does."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402

DIMS = [64, 128, 256]


def dev(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def row(q, k, v, scale):
    """(out, bound) of one token's heads q [hq, d] over the keys that it attends,
    in 64 bits.

    A logit's operands are held to 2^-22 each and the product of their low terms
    is left out, 3 * 2^-22 < 2^-20 of the products' sizes, and so is what lies
    below 2^-27 of the key's largest value; a sum of d products in three terms
    may be cut off at each of 3 d / 16 steps, 2^-23, fewer than d.  A probability
    is off by twice that, by exp2 (2^-22) in numerator and sum, and by the sum's
    roundings: a thread adds at most 16 values four ways and 2, and one a tile, 16
    at most here, 34 half steps of 2^-24.  O: three terms of 4 products' steps and
    a rounding, and one a tile, 2^-23 each: 29.  Values and probabilities are held
    to 2^-22, without the low terms' product: 3 * 2^-22.  Of a value, what is below
    2^-27 of its token's largest is dropped, and of a probability's share in the
    sum 2^-39 of the largest share there is (its own tile's or a larger one's)."""
    hq, d = q.shape
    g = hq // k.shape[1]
    qq, kk, vv = q.double().view(-1, g, d), k.double(), v.double()
    x = torch.einsum("hgd,jhd->hgj", qq, kk) * scale
    size = torch.einsum("hgd,jhd->hgj", qq.abs(), kk.abs()) * abs(scale)
    low = qq.abs().sum(-1)[..., None] * kk.abs().amax(-1).T[:, None] * abs(scale)
    es = (((d + 8) * 2.0 ** -23 + 2.0 ** -20) * size + 2.0 ** -27 * low).amax(-1, keepdim=True)
    p = torch.softmax(x, -1)
    each = 2 * (2 * es + 2.0 ** -22) + (34 / 2 + 29 + 6) * 2.0 ** -23
    top = vv.abs().amax(-1).T[:, None]  # [h, 1, j]
    out = torch.einsum("hgj,jhd->hgd", p, vv)
    bound = torch.einsum("hgj,jhd->hgd", p * each, vv.abs())
    bound = bound + ((p * top).sum(-1) * 2.0 ** -27 + len(k) * 2.0 ** -38 * (p * top).amax(-1))[..., None]
    return out.view(hq, d), bound.view(hq, d) + 2.0 ** -140


def check(got, q, k, v, ctx, rows, scale):
    for t in rows:
        want, bound = row(q[t], k[:ctx + t + 1], v[:ctx + t + 1], scale)
        assert torch.isfinite(got[t]).all(), t
        d = (got[t].double() - want).abs()
        assert (d <= bound).all(), (t, (d / bound).max().item())


def inputs(n, ctx, dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(n, h):
        return torch.randn(n, h, dim, generator=g, device="cuda")

    return normal(n, 4), normal(n + ctx, 2), normal(n + ctx, 2), dev([0, n]), dev([0, n + ctx])


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("big", [1e3, 1e5, 1e8, 1e20, 3e37])
@pytest.mark.parametrize("n,ctx,at", [(100, 0, 50), (150, 40, 130), (20, 3000, 3010)])
def test_later_token_of_another_size(n, ctx, at, big, dim):
    """A key and a value that rows before it do not attend, far larger than
    theirs, in the same tile."""
    q, k, v, s, ks = inputs(n, ctx, dim, 1)
    t = at - ctx
    before = range(0, t, 7) if n > 20 else range(t)
    k2, v2 = k.clone(), v.clone()
    k2[at], v2[at] = big, big
    got = kq.prompt_attention(q, k, v2, s, ks)
    check(got, q, k, v2, ctx, list(before) + [t - 1, t, n - 1], dim ** -0.5)
    got = kq.prompt_attention(q, k2, v, s, ks)
    check(got, q, k2, v, ctx, list(before) + [t - 1], dim ** -0.5)
    got = kq.prompt_attention(q, k2, v2, s, ks)
    check(got, q, k2, v2, ctx, list(before) + [t - 1], dim ** -0.5)
    assert not kq.device_error()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("step", [2.0, 3.0, 0.4])
def test_values_that_grow_or_shrink_from_token_to_token(step, dim):
    n = 70
    q, k, v, s, ks = inputs(n, 0, dim, 2)
    v *= (step ** (torch.arange(n, device="cuda") - n / 2))[:, None, None]
    check(kq.prompt_attention(q, k, v, s, ks), q, k, v, 0, range(n), dim ** -0.5)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("step", [2.0, 3.0])
def test_keys_that_grow_from_token_to_token(step, dim):
    """Queries as small as the largest key they see is large: logits near one."""
    n = 70
    q, k, v, s, ks = inputs(n, 0, dim, 3)
    by = (step ** (torch.arange(n, device="cuda") - n / 2))[:, None, None]
    k, q = k * by, q / by
    check(kq.prompt_attention(q, k, v, s, ks), q, k, v, 0, range(n), dim ** -0.5)


@pytest.mark.parametrize("dim", DIMS)
def test_large_value_without_weight(dim):
    """A value of 1e30 that a row attends with a probability of about 1e-60, and
    smaller ones whose products with their probabilities are alike."""
    n = 90
    q, k, v, s, ks = inputs(n, 0, dim, 4)
    q[..., 0] = 4.0
    k[:, :, 0] = 0.0
    for j, logit, size in ((5, -138.0, 1e30), (9, -69.0, 1e25), (70, -30.0, 1e13)):
        k[j, :, 0] = logit * dim ** 0.5 / 4.0
        v[j] *= size
    check(kq.prompt_attention(q, k, v, s, ks), q, k, v, 0, range(n), dim ** -0.5)


@pytest.mark.parametrize("dim", DIMS)
def test_sizes_apart_beside_what_is_not_finite(dim):
    """NaN and infinities in later tokens of a tile whose sizes lie far apart,
    and tokens of zeros."""
    n = 64
    q, k, v, s, ks = inputs(n, 0, dim, 5)
    v[3], k[7] = 0.0, 0.0
    k[40], v[41], k[45] = 1e15, 1e20, 0.0
    k[50, 0, 3], v[52, 1, 5], v[53] = float("nan"), float("inf"), float("nan")
    got = kq.prompt_attention(q, k, v, s, ks)
    check(got, q, k, v, 0, range(40), dim ** -0.5)
    assert got[53:, 2:].isnan().all() and got[50:, :2].isnan().all()
    # (values alone: the column of an infinity, and no other)
    k[40], k[50, 0, 3], v[53] = 0.5, 0.25, 1.0
    got = kq.prompt_attention(q, k, v, s, ks)
    assert (got[52:, 2:, 5] == float("inf")).all() and torch.isfinite(got[:, :2]).all()
    v[52, 1, 5] = 0.0
    check(got[:, :2], q[:, :2], k[:, :1], v[:, :1], 0, range(n), dim ** -0.5)
