"""Measured cases of the decode-step operators: rotary positions, the quantised
key/value cache (written and read back), attention of drafted tokens over that
cache, and the verification of the drafts.

`run` computes a case either in plain torch (own = False: elementary f32
operations) or with the library's kernels (own = True).  `prepare` makes what a
decoding program holds before the call.  Sizes follow the repository's own
model geometry (32 query heads, 2 key/value heads, head width 128, a 202048-word
vocabulary, up to 16 token columns) and generic decoder geometries around it.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64          # tokens of a cache page
GROUP = 32         # values that share one scale
BITS = {"f16": 16, "q8": 8, "q4": 4}
VOCAB = 202048


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of one sequence: the query heads of one token
        dict(name="rope_token", op="rope", ntok=1, heads=32, dim=128, rot=128, inter=False,
             inverse=False, scaling="none", far=4000),
        # a long prompt, half of each head rotated, positions scaled for a long context
        dict(name="rope_prompt", op="rope", ntok=8191, heads=32, dim=128, rot=64, inter=True,
             inverse=False, scaling="ramp", far=131072),
        # 16 drafted tokens of one sequence enter an 8-bit cache and are read back
        dict(name="cache_draft_q8", op="cache", fmt="q8", nseq=1, new=16, ctx=1003, hkv=2, hq=32,
             dim=128, rot=128, inter=False, ragged=1),
        # prompts of three users enter a 4-bit cache
        dict(name="cache_prompt_q4", op="cache", fmt="q4", nseq=3, new=6001, ctx=77, hkv=8, hq=32,
             dim=128, rot=128, inter=True, ragged=2),
        # prompt pieces of a batch, unquantised, narrow heads
        dict(name="cache_batch_f16", op="cache", fmt="f16", nseq=16, new=300, ctx=5000, hkv=8,
             hq=8, dim=64, rot=32, inter=False, ragged=3),
        # the smallest step: one token of one sequence after a short prompt
        dict(name="attend_token_f16", op="attend", fmt="f16", nseq=1, new=1, ctx=777, hkv=2, hq=32,
             dim=128, tree="chain", ragged=4),
        # a tree of 16 drafts over a long 8-bit cache, the repository's head geometry
        dict(name="attend_tree_q8", op="attend", fmt="q8", nseq=1, new=16, ctx=32001, hkv=2, hq=32,
             dim=128, tree="tree", ragged=5),
        # a serving batch, one token a sequence, ragged lengths, 4-bit cache
        dict(name="attend_batch_q4", op="attend", fmt="q4", nseq=32, new=1, ctx=16384, hkv=8,
             hq=32, dim=128, tree="chain", ragged=6),
        # very long contexts, chains of 8 drafts, unquantised cache
        dict(name="attend_long_f16", op="attend", fmt="f16", nseq=4, new=8, ctx=131071, hkv=8,
             hq=32, dim=128, tree="chain", ragged=7),
        # wide heads, a batch of small trees, 8-bit cache
        dict(name="attend_wide_q8", op="attend", fmt="q8", nseq=8, new=5, ctx=4100, hkv=4, hq=16,
             dim=256, tree="tree", ragged=8),
        # one sequence's chain of five drafts
        dict(name="verify_chain", op="verify", nseq=1, new=6, vocab=VOCAB, tree="chain",
             draft="probs", ragged=9),
        # trees of 16 nodes for a batch
        dict(name="verify_trees", op="verify", nseq=16, new=16, vocab=VOCAB, tree="tree",
             draft="probs", ragged=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "cache", "attend", "attend", "attend", "verify"])
    ragged = rng.randrange(1000, 1 << 30)
    if op == "rope":
        dim = rng.choice([64, 96, 128, 256])
        return dict(op=op, ntok=_log(rng, 1, 8191), heads=rng.choice([1, 2, 8, 32, 40]), dim=dim,
                    rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ramp"]),
                    far=_log(rng, 8192, 131072))
    if op == "cache":
        dim = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        nseq = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 16000 * 1024 // (nseq * hkv * dim)))
        return dict(op=op, fmt=rng.choice(["f16", "q8", "q4"]), nseq=nseq, new=min(new, 8192),
                    ctx=_log(rng, 1, 8192) - 1, hkv=hkv, hq=hkv * rng.choice([1, 4, 8]), dim=dim,
                    rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5, ragged=ragged)
    if op == "attend":
        dim = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 4, 5, 8, 16])
        nseq = _log(rng, 1, 64)
        new = _log(rng, 1, 32)
        # at most the largest listed case's cache, and its scores
        most = min(400e6 / (nseq * hkv * dim), 500e6 / (4 * nseq * new * hkv * g), 131071)
        return dict(op=op, fmt=rng.choice(["f16", "q8", "q4"]), nseq=nseq, new=new,
                    ctx=_log(rng, 1, max(2, most)) - 1, hkv=hkv, hq=hkv * g, dim=dim,
                    tree=rng.choice(["chain", "tree"]), ragged=ragged)
    return dict(op=op, nseq=_log(rng, 1, 16), new=_log(rng, 1, 16), vocab=_log(rng, 1001, VOCAB),
                tree=rng.choice(["chain", "tree"]), draft=rng.choice(["probs", "tokens"]),
                ragged=ragged)


def _lens(case):
    """(new tokens, tokens held) of each sequence: the first has the case's own."""
    r = random.Random(case["ragged"])
    new, ctx = [case["new"]], [case.get("ctx", 0)]
    for _ in range(case["nseq"] - 1):
        new.append(r.randint(max(1, case["new"] // 2), case["new"]))
        ctx.append(r.randint(case.get("ctx", 0) // 3, case.get("ctx", 0)))
    return new, ctx


def _parents(case):
    """Each sequence's tree: node 0 is the last committed token, the others are drafts."""
    r = random.Random(case["ragged"] + 1)
    every = []
    for n in _lens(case)[0]:
        every.append([-1] + [j - 1 if case["tree"] == "chain" else r.randrange(max(0, j - 5), j)
                             for j in range(1, n)])
    return every


def _masks(parents):
    """Bit j of node i: node j is i or an ancestor of it (as a signed 64-bit number)."""
    out = []
    for tree in parents:
        m = []
        for i, p in enumerate(tree):
            m.append((m[p] if p >= 0 else 0) | (1 << i))
        out += [x - (1 << 64) if x >> 63 else x for x in m]
    return out


def work(case):
    if case["op"] == "rope":
        n = case["ntok"] * case["heads"]
        return {"bytes": 8 * n * case["dim"] + 4 * case["ntok"] * (case["rot"] + 1),
                "flops": 3 * n * case["rot"]}
    new, ctx = _lens(case)
    if case["op"] == "verify":
        # the row that gives the next token and the draft's row that corrects it
        rows = 2 if case["draft"] == "probs" else 1
        return {"bytes": 4 * case["nseq"] * case["vocab"] * rows + 12 * sum(new),
                "flops": 3 * case["nseq"] * case["vocab"]}
    each = case["dim"] * BITS[case["fmt"]] // 8
    each += 0 if case["fmt"] == "f16" else case["dim"] // GROUP * 2
    if case["op"] == "cache":
        n = sum(new) * case["hkv"]
        return {"bytes": n * (4 * case["dim"] * 4 + 4 * each) + 4 * sum(new) * case["rot"],
                "flops": n * case["dim"] * 8}
    held = [a + b for a, b in zip(new, ctx)]
    return {"bytes": 2 * sum(held) * case["hkv"] * each + 8 * sum(new) * case["hq"] * case["dim"],
            "flops": 4 * sum(a * b for a, b in zip(new, held)) * case["hq"] * case["dim"]}


# ---------------------------------------------------------------- inputs
def _table(n, rot, scaling):
    """(cos, sin) of every position and pair, formed in 64 bits and rounded once."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    f = 500000.0 ** (-i / rot)
    mag = 1.0
    if scaling == "linear":
        f = f / 8
    elif scaling == "ramp":
        # pairs that turn over 32 times within 8192 positions keep their speed, those that
        # turn less than once are slowed eight times, those between are blended
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f / 8 * (1 - keep) + f * keep
        mag = 0.1 * math.log(8) + 1
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos() * mag, a.sin() * mag], -1).float()


def _quantise(x, fmt):
    """Codes and scales of groups of 32: x ~ code * scale."""
    if fmt == "f16":
        return x.half(), None
    g = x.unflatten(-1, (-1, GROUP))
    hi, lo = g.amax(-1, keepdim=True), g.amin(-1, keepdim=True)
    if fmt == "q8":
        d = torch.maximum(hi, -lo) / torch.full_like(hi, 127)  # (a division, not a product with 1/127)
    else:
        d = torch.where(hi >= -lo, hi, lo) / -8
    d = d.clamp(-65504, 65504).half()
    c = torch.where(d == 0, 0.0, torch.round(g / d.float()))
    c = c.clamp(-127, 127) if fmt == "q8" else c.clamp(-8, 7)
    return c.to(torch.int8).flatten(-2), d[..., 0]


def _values(code, scale):
    """The f32 values that codes [..., dim] and scales [..., dim / 32] stand for."""
    if scale is None:
        return code.float()
    return (code.unflatten(-1, (-1, GROUP)).float() * scale[..., None].float()).flatten(-2)


def _bytes(code, fmt):
    """Codes [..., n] as the bytes [..., n * bits / 8] that hold them; 4-bit codes low first."""
    if fmt == "f16":
        return code.contiguous().view(torch.uint8)
    if fmt == "q8":
        return code.contiguous().view(torch.uint8)
    u = (code & 15).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _pack(kc, ks, vc, vs, fmt):
    """The library's cache pages from codes [pages * 64, heads, dim] in plain order.

    Of each page and head: the keys' codes as slabs [slab][token][64 bytes] (octets of a slab's
    groups interleaved: octet c of group g at place c * groups + g), the keys' scales
    [token][group], the values' codes as [slab of tokens][dim][tokens], their scales
    [group][token]."""
    slots, h, d = kc.shape
    pages = slots // PAGE
    gs = min({"f16": 1, "q8": 2, "q4": 4}[fmt], d // GROUP)
    k = kc.view(pages, PAGE, h, d // (gs * GROUP), gs, 4, 8).permute(0, 2, 3, 1, 5, 4, 6)
    parts = [_bytes(k.reshape(pages, h, -1, gs * GROUP), fmt).reshape(pages, h, -1)]
    if ks is not None:
        s = ks.view(pages, PAGE, h, -1).permute(0, 2, 1, 3).contiguous()
        parts.append(s.view(torch.uint8).reshape(pages, h, -1))
    t = 32 if fmt == "f16" else 64
    v = vc.view(pages, PAGE // t, t, h, d).permute(0, 3, 1, 4, 2)
    parts.append(_bytes(v.reshape(pages, h, -1, t), fmt).reshape(pages, h, -1))
    if vs is not None:
        s = vs.view(pages, PAGE, h, -1).permute(0, 2, 3, 1).contiguous()
        parts.append(s.view(torch.uint8).reshape(pages, h, -1))
    return torch.cat(parts, -1).flatten()


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _batch(case, gen):
    """Lengths, starts and a page table whose pages lie scattered in the pool."""
    new, ctx = _lens(case)
    start = np.concatenate([[0], np.cumsum(new)])
    need = [-(-(a + b) // PAGE) for a, b in zip(new, ctx)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((case["nseq"], max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return dict(start=_int(start.tolist()), ctx=_int(ctx), table=table, pages=pages,
                ntok=int(start[-1]), new=max(new), most=max(a + b for a, b in zip(new, ctx)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case=case)
    if case["op"] == "rope":
        s["x"] = normal(case["ntok"], case["heads"], case["dim"])
        n = case["far"]
        first = int(torch.randint(0, n - case["ntok"] + 1, (1,), generator=gen, device="cuda"))
        s["pos"] = torch.arange(first, first + case["ntok"], dtype=torch.int32, device="cuda")
        s["cs"] = _table(n, case["rot"], case["scaling"])
        return s
    if case["op"] == "verify":
        new, _ = _lens(case)
        n, v = sum(new), case["vocab"]
        start = [0] + np.cumsum(new).tolist()
        par = sum(_parents(case), [])
        up = torch.tensor([start[b] + max(p, 0) for b, t in enumerate(_parents(case)) for p in t],
                          device="cuda")
        logits = 2.5 * normal(n, v)
        s["p"] = torch.softmax(logits, -1)
        draft = torch.softmax(logits + 0.7 * normal(n, v), -1)
        s["tok"] = torch.multinomial(draft[up], 1, generator=gen)[:, 0].int()
        s["q"] = draft if case["draft"] == "probs" else None
        s["start"], s["parent"], s["nseq"], s["new"] = _int(start), _int(par), case["nseq"], max(new)
        s["ua"] = torch.rand(n, generator=gen, device="cuda")
        s["us"] = torch.rand(case["nseq"], generator=gen, device="cuda")
        return s
    b = _batch(case, gen)
    s.update(b)
    fmt, h, d = case["fmt"], case["hkv"], case["dim"]
    slots = b["pages"] * PAGE
    if case["op"] == "cache":
        # what a fused projection wrote: query, key and value heads of a token side by side
        hq = case["hq"]
        qkv = normal(b["ntok"], hq + 2 * h, d)
        s["k"], s["v"] = qkv[:, hq:hq + h], qkv[:, hq + h:]
        at = [c + j for n, c in zip(*_lens(case)) for j in range(n)]
        s["pos"] = _int(at)
        s["cs"] = _table(b["most"], case["rot"], "none")
        kind = torch.float16 if fmt == "f16" else torch.int8
        s["kc"] = torch.zeros(slots, h, d, dtype=kind, device="cuda")
        s["vc"] = torch.zeros_like(s["kc"])
        s["ks"] = s["vs"] = None
        if fmt != "f16":
            s["ks"] = torch.zeros(slots, h, d // GROUP, dtype=torch.float16, device="cuda")
            s["vs"] = torch.zeros_like(s["ks"])
        s["data"] = _pack(s["kc"], s["ks"], s["vc"], s["vs"], fmt)
    else:
        s["q"] = 3 * normal(b["ntok"], case["hq"], d)
        s["kc"], s["ks"] = _quantise(normal(slots, h, d), fmt)
        s["vc"], s["vs"] = _quantise(normal(slots, h, d), fmt)
        s["data"] = _pack(s["kc"], s["ks"], s["vc"], s["vs"], fmt)
        s["mask"] = torch.tensor(_masks(_parents(case)), dtype=torch.int64, device="cuda")
    if own:  # the handles that a decoding program keeps from step to step
        import quant_quantized_matvec_gb300 as kq
        s["cache"] = kq.KVCache(getattr(kq, "KV_" + fmt.upper()), h, d, b["pages"],
                                data=s["data"])
        s["batch"] = kq.KVBatch(b["start"], b["ctx"], b["table"], b["ntok"], b["new"])
    return s


# ------------------------------------------------------------ plain forms
def _rotate(x, pos, cs, inter, inverse):
    t = cs[pos.long()][:, None]
    c, n = t[..., 0], t[..., 1]
    if inverse:
        n = -n
    rot = 2 * c.shape[-1]
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * n, b * c + a * n
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * n, b * c + a * n
    return y


def _tokens(s):
    """Sequence and place within it of every new token."""
    i = torch.arange(s["ntok"], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(s["start"][1:], i, right=True)
    return seq, i - s["start"][seq]


def _slots(s, seq, at):
    return s["table"][seq, at // PAGE].long() * PAGE + at % PAGE


def _plain_cache(s):
    case = s["case"]
    seq, j = _tokens(s)
    slot = _slots(s, seq, s["ctx"][seq] + j)
    k = _rotate(s["k"], s["pos"], s["cs"], case["inter"], False)
    for x, code, scale in ((k, s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        c, d = _quantise(x, case["fmt"])
        code[slot] = c
        if d is not None:
            scale[slot] = d
    return [_values(code[slot], None if scale is None else scale[slot])
            for code, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]


def _plain_attend(s):
    case = s["case"]
    n, h, d, new, most = case["nseq"], case["hkv"], case["dim"], s["new"], s["most"]
    seq, j = _tokens(s)
    q = torch.zeros(n, new, case["hq"], d, device="cuda")
    q[seq, j] = s["q"]
    m = torch.zeros(n, new, dtype=torch.int64, device="cuda")
    m[seq, j] = s["mask"]
    # every sequence's tokens, padded to the longest
    at = torch.arange(most, dtype=torch.int32, device="cuda").expand(n, -1)
    slot = _slots(s, torch.arange(n, device="cuda")[:, None].expand(-1, most), at).clamp(min=0)
    k = _values(s["kc"][slot], None if s["ks"] is None else s["ks"][slot])
    v = _values(s["vc"][slot], None if s["vs"] is None else s["vs"][slot])
    draft = at - s["ctx"][:, None]
    count = (s["start"][1:] - s["start"][:-1])[:, None]
    bit = (m[:, :, None] >> draft.clamp(0, 63)[:, None]) & 1
    seen = (draft < 0)[:, None] | ((draft < count)[:, None] & (draft >= 0)[:, None] & (bit == 1))
    g = case["hq"] // h
    q = q.view(n, new, h, g, d).permute(0, 2, 1, 3, 4).reshape(n, h, new * g, d)
    x = (q * d ** -0.5) @ k.permute(0, 2, 3, 1)
    x = x.view(n, h, new, g, most).masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    y = x.view(n, h, new * g, most) @ v.permute(0, 2, 1, 3)
    y = y.view(n, h, new, g, d) / torch.where(total == 0, 1.0, total)
    return y.permute(0, 2, 1, 3, 4).reshape(n, new, case["hq"], d)[seq, j]


def _fixed(r):
    """Probabilities in whole multiples of 2^-44."""
    return (r.clamp(0, 1).double() * 2.0 ** 44).long()


def _plain_verify(s):
    n, new, p, q, tok, parent = s["nseq"], s["new"], s["p"], s["q"], s["tok"], s["parent"]
    seqs = torch.arange(n, device="cuda")
    first, count = s["start"][:-1].long(), (s["start"][1:] - s["start"][:-1]).long()
    path = torch.full((p.shape[0],), -1, dtype=torch.int32, device="cuda")
    path[first] = 0
    got = torch.ones(n, dtype=torch.int64, device="cuda")
    cur = torch.zeros(n, dtype=torch.int64, device="cuda")
    r, z = p[first], torch.ones(n, device="cuda")
    # the nodes one after another: whether a node is looked at depends on those before it
    for j in range(1, new):
        at = (first + j).clamp(max=p.shape[0] - 1)
        t = tok[at].long()
        look = (j < count) & (parent[at] == cur)
        have = r[seqs, t]
        d = z if q is None else q[first + cur, t] * z
        yes = look & (s["ua"][at] * d < have)
        no = look & ~yes
        if q is None:
            left = r.clone()
            left[seqs, t] = 0
        else:
            left = (r - z[:, None] * q[first + cur]).clamp(min=0)
        total = _fixed(left).sum(-1)
        keep = no & (total > 0)
        r = torch.where(yes[:, None], p[at], torch.where(keep[:, None], left, r))
        z = torch.where(yes, 1.0, torch.where(keep, (total.double() * 2.0 ** -44).float(), z))
        cur = torch.where(yes, j, cur)
        where = torch.where(yes, first + got, path.numel())
        path = torch.cat([path, path[:1]]).index_put((where,), cur.int())[:-1]
        got = got + yes
    w = _fixed(r)
    total = w.sum(-1)
    u = (s["us"].double() * 2.0 ** 31).long()
    goal = (total >> 31) * u + (((total & (2 ** 31 - 1)) * u) >> 31)
    nxt = (w.cumsum(-1) <= goal[:, None]).sum(-1).clamp(max=p.shape[1] - 1)
    return [path, got.int(), nxt.int()]


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "rope":
            return _rotate(s["x"], s["pos"], s["cs"], case["inter"], case["inverse"])
        return {"cache": _plain_cache, "attend": _plain_attend, "verify": _plain_verify}[case["op"]](s)
    import quant_quantized_matvec_gb300 as kq
    if case["op"] == "rope":
        return kq.rope(s["x"], s["pos"], s["cs"], interleaved=case["inter"],
                       inverse=case["inverse"])
    if case["op"] == "cache":
        kq.kv_append(s["cache"], s["batch"], s["k"], s["v"], positions=s["pos"], table=s["cs"],
                     interleaved=case["inter"])
        return list(kq.kv_read(s["cache"], s["batch"]))
    if case["op"] == "attend":
        return kq.tree_attention(s["cache"], s["batch"], s["q"], mask=s["mask"])
    return list(kq.verify_tree(s["start"], s["tok"], s["parent"], s["p"], s["q"], s["ua"], s["us"],
                               s["new"]))


# ------------------------------------------------------------- in 64 bits
def _exact_rotate(x, pos, cs, inter, sign):
    x = x.double()
    z = torch.view_as_complex(cs.double())[pos.long()][:, None]
    z = torch.complex(z.real, sign * z.imag)
    half = z.shape[-1]
    if inter:
        w = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z
        turned = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(x[..., :half], x[..., half:2 * half]) * z
        turned = torch.cat([w.real, w.imag], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _exact_stored(x, fmt):
    x = x.double()
    if fmt == "f16":
        return x.half().double()
    y = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    big = y.abs().max(-1, keepdim=True)
    lead = torch.gather(y, -1, big.indices)
    step = (big.values / 127 if fmt == "q8" else lead / -8).half().double()
    low, high = (-127, 127) if fmt == "q8" else (-8, 7)
    code = (y / step).round().nan_to_num(0).clamp(low, high)
    return (code * step).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotate(s["x"], s["pos"], s["cs"], case["inter"], -1 if case["inverse"] else 1)
    if case["op"] == "cache":
        k = _exact_rotate(s["k"], s["pos"], s["cs"], case["inter"], 1)
        return [_exact_stored(k, case["fmt"]), _exact_stored(s["v"], case["fmt"])]
    new, ctx = _lens(case)
    h, g = case["hkv"], case["hq"] // case["hkv"]
    rows, table, mask, at = [], s["table"].tolist(), s["mask"].tolist(), 0
    for b in range(case["nseq"]):
        held = new[b] + ctx[b]
        pages = torch.tensor(table[b][:-(-held // PAGE)], device="cuda").long()
        kv = []
        for code, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
            x = code.unflatten(0, (-1, PAGE))[pages].flatten(0, 1)[:held].double()
            if scale is not None:
                f = scale.unflatten(0, (-1, PAGE))[pages].flatten(0, 1)[:held].double()
                x = x * f.repeat_interleave(GROUP, -1)
            kv.append(x.transpose(0, 1))
        bits = [[c < ctx[b] or (mask[at + i] >> (c - ctx[b])) & 1 for c in
                 range(max(0, held - 64), held)] for i in range(new[b])]
        seen = torch.ones(new[b], held, dtype=torch.bool, device="cuda")
        tail = torch.tensor(bits, device="cuda").bool()
        seen[:, held - tail.shape[1]:] = tail
        q = s["q"][at:at + new[b]].double().reshape(new[b], h, g, -1)
        x = torch.einsum("nhgd,hld->hgnl", q, kv[0]) / math.sqrt(case["dim"])
        x = torch.where(seen, x, -math.inf).softmax(-1)
        rows.append(torch.einsum("hgnl,hld->nhgd", x, kv[1]).reshape(new[b], case["hq"], -1))
        at += new[b]
    return torch.cat(rows)
