"""Plain 64-bit forms of a prompt's operators, and how far the library's
arithmetic may be from them."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24  # half a step of f32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm_rope(x, weight, pos, table, inter, eps):
    """(y, size) in 64 bits: size is |a c| + |b s| of each value's rotation (or
    |y|), which its rounding errors go by."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    if table is None:
        return y, y.abs()
    cs = table.double()[pos.long()][:, None]
    c, s = cs[..., 0], cs[..., 1]
    half = c.shape[-1]
    i = torch.arange(half, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + half)
    z, size = y.clone(), y.abs()
    a, b = y[..., ia], y[..., ib]
    z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = (a * c).abs() + (b * s).abs()
    size[..., ib] = (b * c).abs() + (a * s).abs()
    return z, size


def norm_bound(y, size, dtype):
    """The squares' sum is at most 32 fused steps of a lane and five of the
    lanes, all of one sign: 37 half steps of it, of which the root keeps half;
    a division, a sum, a root, a division, two products, and of a rotation two
    products and a sum: 18.5 + 9 half steps of f32, taken as 32.  Then half a
    step of the output's type, or of its smallest numbers."""
    b = size * (32 * U)
    if dtype is not torch.float32:
        b = b + (y.abs() + b) * half_step(dtype)
    return b + torch.finfo(dtype).smallest_normal * half_step(dtype)


def attention(q, k, v, start, key_start, scale):
    """(out, bound, seen): packed causal attention in 64 bits; seen [ntok] is
    the number of keys that a token attends, -1 for tokens of no sequence.

    16-bit types: a logit is a sum of D exact products in additions that may
    truncate, 2^-23 a step, and a product with the scale.  A probability is off
    by twice that (numerator and sum), exp2 (2^-22) and half a step of its type;
    values' sums take a step (2^-23 at most) for each 16 tokens and a few for
    each tile and part.  f32: queries, keys, values and probabilities are held
    to 2^-22 each, and the product of the two low terms is left out (2^-22);
    parts below 2^-39 of a row's or tile's largest are dropped."""
    f32 = q.dtype is torch.float32
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    seen = torch.full((n,), -1, device=q.device)
    for b in range(len(start) - 1):
        s0, s1, k0, k1 = start[b], start[b + 1], key_start[b], key_start[b + 1]
        if s1 <= s0:
            continue
        limit = torch.arange(s1 - s0, device=q.device) + (k1 - k0) - (s1 - s0) + 1
        seen[s0:s1] = limit.clamp(min=0)
        if k1 <= k0:
            continue
        at = torch.arange(k1 - k0, device=q.device) < limit[:, None]
        qq = q[s0:s1].double().reshape(s1 - s0, -1, g, d)
        kk, vv = k[k0:k1].double(), v[k0:k1].double()
        # (values that no row attends do not count, whatever they are)
        most = vv[:int(limit.max().clamp(min=0))]
        vv = torch.where(torch.isfinite(vv), vv, 0.0)
        kk = torch.where(torch.isfinite(kk), kk, 0.0)
        x = torch.einsum("thgd,jhd->hgtj", qq, kk) * scale
        size = (torch.einsum("thgd,jhd->hgtj", qq.abs(), kk.abs()) * abs(scale)).masked_fill(~at, 0).amax(-1)
        x = x.masked_fill(~at, -math.inf)
        p = torch.softmax(x, -1)
        p = torch.where(at.any(-1)[:, None], p, 0.0)
        out[s0:s1] = torch.einsum("hgtj,jhd->thgd", p, vv).reshape(s1 - s0, hq, d)
        es = ((d + 8) * 2.0 ** -23 + (2.0 ** -20 if f32 else 0)) * size
        steps = 64 + (k1 - k0) / 8 + 304
        each = 2 * (2 * es + 2.0 ** -21) + steps * 2.0 ** -22
        each = each + (3 * 2.0 ** -22 if f32 else half_step(q.dtype))
        top = torch.where(torch.isfinite(most), most, 0.0).abs().amax() if most.numel() else 0.0
        bb = torch.einsum("hgtj,jhd->thgd", p * each[..., None], vv.abs())
        bound[s0:s1] = bb.reshape(s1 - s0, hq, d) + (k1 - k0) * 2.0 ** -38 * top
    if not f32:
        bound = bound + (out.abs() + bound) * half_step(q.dtype) \
            + torch.finfo(q.dtype).smallest_normal * half_step(q.dtype)
    return out, bound, seen


def logprobs(logits, tokens, top):
    """(logp, entropy, top_logp, top_tokens) in 64 bits."""
    x = logits.double()
    n, v = x.shape
    lp = torch.log_softmax(x, -1)
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    ent = torch.where(torch.isnan(lp).any(-1), math.nan, ent)
    logp = torch.full((n,), math.nan, dtype=torch.float64, device=x.device)
    ok = (tokens >= 0) & (tokens < v)
    logp[ok] = lp[ok].gather(-1, tokens[ok].long()[:, None])[:, 0]
    key = torch.where(torch.isnan(x), math.inf, x)
    order = torch.sort(key, stable=True, dim=-1, descending=True).indices[:, :top]
    return logp, ent, lp.gather(-1, order), order.int()


def logprob_bound(value, spread, vocab):
    """The distance to the maximum is one rounding, times log2(e) another, and
    ex2 2^-22: a weight is off by 2^-22 and (distance) 2^-23, which sums keep
    (weights of distance above 30 do not count), and a thread's sum takes a
    rounding a batch and value (vocab / 512 at most) and 30 in the joins.  The
    logarithm adds two steps of its value, the differences one of theirs."""
    rel = 2.0 ** -22 + 30 * 2.0 ** -23 + (min(vocab / 512, 1024) + 40) * U
    return rel * (1 + spread) + 4 * U * value.abs()
