"""Plain references for the decode-step operators, written from their
formulas: the cache's f32 quantisation step by step and its byte layout
(numpy), attention in 64 bits, and the verification in whole numbers."""
from __future__ import annotations

import numpy as np

PAGE, GROUP = 64, 32
F16, Q4, Q8 = 1, 2, 8
BITS = {F16: 16, Q8: 8, Q4: 4}
NAMES = {F16: "f16", Q8: "q8", Q4: "q4"}


def rotate(x, pos, table, inter, inverse=False, dtype=np.float64):
    """x [n, heads, dim] turned by table [positions, rot/2, 2]; with dtype
    float32 every product and sum is rounded, as the library defines it."""
    x, y = x.astype(dtype), x.astype(dtype).copy()
    half = table.shape[1]
    c = table[pos][:, None, :, 0].astype(dtype)
    s = table[pos][:, None, :, 1].astype(dtype) * (-1 if inverse else 1)
    ia = np.arange(half) * 2 if inter else np.arange(half)
    ib = ia + (1 if inter else half)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def quantise(x, fmt):
    """(codes, scales) of f32 x [..., dim] in the library's f32 steps."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if fmt == F16:
            return x.astype(np.float16), None
        g = x.reshape(*x.shape[:-1], -1, GROUP)
        hi, lo = g.max(-1), g.min(-1)
        if fmt == Q8:
            d = np.maximum(hi, -lo) / np.float32(127)
        else:
            d = np.where(hi >= -lo, hi, lo) / np.float32(-8)
        d = np.clip(d, -65504, 65504).astype(np.float16)
        d = np.where(np.isfinite(g).all(-1), d, np.float16(np.nan))
        c = np.rint(g / d[..., None].astype(np.float32))
        c = np.where((d == 0)[..., None] | np.isnan(d)[..., None], 0, c)
        c = np.clip(c, -127, 127) if fmt == Q8 else np.clip(c, -8, 7)
    return c.astype(np.int8).reshape(x.shape), d


def values(code, scale):
    """f32 values of codes and scales."""
    if scale is None:
        return code.astype(np.float32)
    g = code.reshape(*code.shape[:-1], -1, GROUP).astype(np.float32)
    with np.errstate(invalid="ignore"):
        return (g * scale[..., None].astype(np.float32)).reshape(code.shape)


def _code_bytes(code, fmt):
    if fmt == F16:
        return np.ascontiguousarray(code).view(np.uint8).ravel()
    if fmt == Q8:
        return code.astype(np.int8).view(np.uint8).ravel()
    u = (code.astype(np.int64) & 15).astype(np.uint8).ravel()
    return u[0::2] | (u[1::2] << 4)


def pack_block(kc, ks, vc, vs, fmt):
    """Bytes of one page and head from codes [64, dim] and scales [64, groups],
    one token and octet after another as the header describes."""
    dim = kc.shape[1]
    groups = dim // GROUP
    per = {F16: 1, Q8: 2, Q4: min(4, groups)}[fmt]
    ob = BITS[fmt]  # bytes of an octet
    slab_bytes = per * 4 * ob
    codes = PAGE * dim * BITS[fmt] // 8
    k = np.zeros(codes, np.uint8)
    for t in range(PAGE):
        for o in range(dim // 8):
            g, c = divmod(o, 4)
            slab, gl = divmod(g, per)
            at = slab * PAGE * slab_bytes + t * slab_bytes + (c * per + gl) * ob
            k[at:at + ob] = _code_bytes(kc[t, 8 * o:8 * o + 8], fmt)
    vt = 32 if fmt == F16 else 64
    v = []
    for slab in range(PAGE // vt):
        for e in range(dim):
            v.append(_code_bytes(vc[slab * vt:(slab + 1) * vt, e], fmt))
    parts = [k]
    if ks is not None:
        parts.append(np.ascontiguousarray(ks).view(np.uint8).ravel())
    parts += v
    if vs is not None:
        parts.append(np.ascontiguousarray(vs.T).view(np.uint8).ravel())
    return np.concatenate(parts)


def pack(kc, ks, vc, vs, fmt):
    """Cache bytes from codes [pages, 64, heads, dim], scales [..., groups]."""
    out = []
    for p in range(kc.shape[0]):
        for h in range(kc.shape[2]):
            out.append(pack_block(kc[p, :, h], None if ks is None else ks[p, :, h],
                                  vc[p, :, h], None if vs is None else vs[p, :, h], fmt))
    return np.concatenate(out)


def attention(q, k, v, seen, scale):
    """One sequence in 64 bits: q [n, hq, d], k and v [len, hkv, d] f32 values,
    seen [n, len].  Returns (out, bound): bound is a worst-case error of the
    library's arithmetic, derived as follows.

    A logit is a sum of D products of an exact code with a query held to
    2^-22, in f32 additions that may truncate (2^-23 a step) with a scale
    multiplied in: off by at most e_s = (2^-22 + (D + 8) 2^-23) sum |q k|
    scale (times log2 e / log2 e).  A probability is then off by a factor of
    1 +- (2 max e_s + 2^-21) with exp2 (2^-22) and its two-term form (2^-22),
    in the numerator and the sum alike (hence twice), and the sums over
    tokens round at most once a token pair of a tile, once a tile and once a
    part: 64 + tiles + 304 steps of 2^-23.  Small probabilities are held in
    steps of 2^-39 of the row's largest at worst (f16 subnormals, scaled):
    2^-38 max |v| a token."""
    n, hq, d = q.shape
    length, hkv = k.shape[:2]
    out, bound = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        at = np.flatnonzero(seen[i])
        if at.size == 0:
            continue
        for h in range(hq):
            kk, vv = (x[at, h // (hq // hkv)].astype(np.float64) for x in (k, v))
            qq = q[i, h].astype(np.float64) * scale
            with np.errstate(invalid="ignore", over="ignore"):
                s = kk @ qq
                p = np.exp(s - s.max())
                p /= p.sum()
                out[i, h] = p @ vv
                es = (2.0 ** -22 + (d + 8) * 2.0 ** -23) * (np.abs(kk) @ np.abs(qq)).max()
                steps = 64 + length / PAGE + 304
                bound[i, h] = (p @ np.abs(vv)) * (2 * (2 * es + 2.0 ** -21) + steps * 2.0 ** -22) \
                    + length * 2.0 ** -38 * np.abs(vv).max()
    return out, bound


def verify(n, token, parent, p, q, u, u_next):
    """One sequence's tree: p and q f32 [n, vocab].  Returns (path, next)."""
    f = np.float32

    def fixed(r):
        return [int(float(x) * 2 ** 44) for x in np.clip(r, 0, 1)]

    cur, path, r, z = 0, [0], np.clip(np.nan_to_num(p[0]), 0, 1), f(1)
    for x in range(1, n):
        if parent[x] != cur or not 0 <= token[x] < p.shape[1]:
            continue
        t = token[x]
        d = z if q is None else f(np.clip(q[cur][t], 0, 1) * z)
        if f(u[x] * d) < r[t]:
            cur, r, z = x, np.clip(np.nan_to_num(p[x]), 0, 1), f(1)
            path.append(x)
            continue
        if q is None:
            left = r.copy()
            left[t] = 0
        else:
            left = np.maximum(r - z * np.clip(q[cur], 0, 1), f(0))
        total = sum(fixed(left))
        if total:
            r, z = left, f(float(total) * 2.0 ** -44)
    w = fixed(r)
    goal = sum(w) * int(float(u_next) * 2 ** 31) >> 31
    run = np.cumsum(np.array(w, dtype=object))
    nxt = next((i for i, c in enumerate(run) if c > goal), len(w) - 1)
    return path, nxt
