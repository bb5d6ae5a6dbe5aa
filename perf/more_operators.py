"""Measured cases of a prompt's operators: the norms of query and key heads with
their rotary positions, the prompt's causal attention over packed sequences,
and the log probabilities of given tokens.

`run` computes a case either in plain torch (own = False: elementary f32
operations) or with the library's kernels (own = True).  `prepare` makes what a
program holds before the call.  Sizes follow the repository's own model geometry
(32 query heads, 2 key/value heads, head width 128, a 202048-word vocabulary)
and generic decoder geometries around it.
"""
import math
import random

import torch

own = False

VOCAB = 202048
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's one token, the repository's head geometry
        dict(name="norm_token", op="norm", ntok=1, hq=32, hkv=2, dim=128, rot=128, inter=False,
             out="f32", far=4000),
        # a long prompt, half of each head rotated, rounded for attention in 16 bits
        dict(name="norm_prompt", op="norm", ntok=8191, hq=32, hkv=8, dim=128, rot=64, inter=True,
             out="bf16", far=131072),
        # the smallest prompt: a question of one user, in the library's own f32
        dict(name="prompt_short_f32", op="prompt", kind="f32", nseq=1, new=77, ctx=0, hkv=2, hq=32,
             dim=128, ragged=1),
        # a document of one user, in f32
        dict(name="prompt_f32", op="prompt", kind="f32", nseq=1, new=4097, ctx=0, hkv=2, hq=32,
             dim=128, ragged=2),
        # prompts of nine users packed into one call, ragged
        dict(name="prompt_packed_bf16", op="prompt", kind="bf16", nseq=9, new=2049, ctx=0, hkv=8,
             hq=32, dim=128, ragged=3),
        # one long document
        dict(name="prompt_long_bf16", op="prompt", kind="bf16", nseq=1, new=12001, ctx=0, hkv=8,
             hq=32, dim=128, ragged=4),
        # the next turn of a long conversation: few new tokens behind many held ones
        dict(name="prompt_turn_f16", op="prompt", kind="f16", nseq=1, new=300, ctx=32001, hkv=8,
             hq=32, dim=128, ragged=5),
        # wide heads, three prompts that continue shorter ones
        dict(name="prompt_wide_bf16", op="prompt", kind="bf16", nseq=3, new=3001, ctx=500, hkv=4,
             hq=16, dim=256, ragged=6),
        # narrow heads without sharing, a batch of short prompts
        dict(name="prompt_narrow_f16", op="prompt", kind="f16", nseq=16, new=1001, ctx=0, hkv=8,
             hq=8, dim=64, ragged=7),
        # the word that a decode step drew, with its 20 best alternatives
        dict(name="score_token", op="score", n=1, vocab=VOCAB, kind="f32", top=20, banned=0.0),
        # a prompt's own words under the model
        dict(name="score_prompt", op="score", n=1999, vocab=VOCAB, kind="f32", top=5, banned=0.0),
        # a serving batch, 16-bit logits (many equal), a grammar's forbidden words
        dict(name="score_batch_bf16", op="score", n=64, vocab=32000, kind="bf16", top=20,
             banned=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "prompt", "prompt", "prompt", "score"])
    if op == "norm":
        dim = rng.choice([64, 96, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5])
        # at most the largest listed case's values
        most = min(8191, 8191 * 40 * 128 // ((hq + hkv) * dim))
        return dict(op=op, ntok=_log(rng, 1, most), hq=hq, hkv=hkv, dim=dim, rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5,
                    out=rng.choice(["f32", "f16", "bf16"]), far=_log(rng, 16384, 131072))
    if op == "score":
        n = _log(rng, 1, 1999)
        return dict(op=op, n=n, vocab=_log(rng, 1001, VOCAB), kind=rng.choice(list(TYPES)),
                    top=rng.choice([0, 1, 5, 20]), banned=rng.choice([0.0, 0.0, 0.5]))
    kind = rng.choice(list(TYPES))
    dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    nseq = _log(rng, 1, 16)
    # scores that the plain form holds for all sequences, and the products: at
    # most those of the largest listed case
    cap = 32 * 12001 * 12001 * min(1.0, 128 / dim) / (nseq * hq)
    new = _log(rng, 1, min(12001, math.sqrt(cap)))
    ctx = _log(rng, 1, max(1, min(32768, cap / new - new))) - 1 if rng.random() < 0.6 else 0
    return dict(op=op, kind=kind, nseq=nseq, new=new, ctx=ctx, hkv=hkv, hq=hq, dim=dim,
                ragged=rng.randrange(1000, 1 << 30))


def _lens(case):
    """(new tokens, tokens before them) of each sequence: the first has the case's own."""
    r = random.Random(case["ragged"])
    new, ctx = [case["new"]], [case["ctx"]]
    for _ in range(case["nseq"] - 1):
        new.append(r.randint(max(1, case["new"] // 3), case["new"]))
        ctx.append(r.randint(case["ctx"] // 3, case["ctx"]))
    return new, ctx


def _size(kind):
    return 4 if kind == "f32" else 2


def work(case):
    if case["op"] == "norm":
        n = case["ntok"] * (case["hq"] + case["hkv"]) * case["dim"]
        return {"bytes": n * (4 + _size(case["out"])) + 4 * case["ntok"] * (case["rot"] + 1),
                "flops": 7 * n}
    if case["op"] == "score":
        n = case["n"]
        return {"bytes": n * (case["vocab"] * _size(case["kind"]) + 12 + 8 * case["top"]),
                "flops": 5 * n * case["vocab"]}
    new, ctx = _lens(case)
    held = sum(new) + sum(ctx)
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    values = (2 * sum(new) * case["hq"] + 2 * held * case["hkv"]) * case["dim"]
    return {"bytes": values * _size(case["kind"]), "flops": 4 * pairs * case["hq"] * case["dim"]}


# ---------------------------------------------------------------- inputs
def _table(n, rot):
    """(cos, sin) of every position and pair, formed in 64 bits and rounded once."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case=case)
    if case["op"] == "norm":
        hq, hkv, dim, n = case["hq"], case["hkv"], case["dim"], case["ntok"]
        # what a fused projection wrote: query, key and value heads of a token side by
        # side, of another size in each token
        qkv = normal(n, hq + 2 * hkv, dim) * (0.2 + 3 * torch.rand(n, 1, 1, generator=gen, device="cuda"))
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["wq"], s["wk"] = 1 + 0.2 * normal(dim), 1 + 0.2 * normal(dim)
        first = int(torch.randint(0, case["far"] - n + 1, (1,), generator=gen, device="cuda"))
        s["pos"] = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
        s["cs"] = _table(case["far"], case["rot"])
        return s
    if case["op"] == "score":
        logits = 2.5 * normal(case["n"], case["vocab"])
        if case["banned"]:
            off = torch.rand(case["vocab"], generator=gen, device="cuda") < case["banned"]
            off[0] = False
            logits.masked_fill_(off, -math.inf)
        # the tokens: drawn from the distribution, by the largest of logit plus noise
        noise = torch.rand(case["vocab"], generator=gen, device="cuda").clamp(min=1e-9).log().neg().log().neg()
        s["tokens"] = (logits + noise).argmax(-1).int()
        s["logits"] = logits.to(TYPES[case["kind"]])
        return s
    kind = TYPES[case["kind"]]
    new, ctx = _lens(case)
    held = [a + b for a, b in zip(new, ctx)]
    # heads after their norms: of like size, with a direction that all keys share
    s["q"] = (1.5 * normal(sum(new), case["hq"], case["dim"])).to(kind)
    s["k"] = (normal(sum(held), case["hkv"], case["dim"]) + 0.5 * normal(1, case["hkv"], case["dim"])).to(kind)
    s["v"] = normal(sum(held), case["hkv"], case["dim"]).to(kind)
    s["start"], s["kstart"] = _starts(new), _starts(held)
    s["new"], s["most"] = max(new), max(held)
    return s


# ------------------------------------------------------------ plain forms
def _plain_norm_one(x, w, s):
    case = s["case"]
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    t = s["cs"][s["pos"].long()][:, None]
    c, n = t[..., 0], t[..., 1]
    rot = case["rot"]
    z = y.clone()
    if case["inter"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z[..., 0:rot:2], z[..., 1:rot:2] = a * c - b * n, b * c + a * n
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z[..., :rot // 2], z[..., rot // 2:rot] = a * c - b * n, b * c + a * n
    return z.to(TYPES[case["out"]])


def _rows_of(start, ntok):
    """Sequence and place within it of every token."""
    i = torch.arange(ntok, device="cuda")
    seq = torch.searchsorted(start[1:].long(), i, right=True)
    return seq, i - start[seq]


def _plain_prompt(s):
    case = s["case"]
    n, h, d, new, most = case["nseq"], case["hkv"], case["dim"], s["new"], s["most"]
    g = case["hq"] // h
    # every sequence's tokens, padded to the longest
    sq, jq = _rows_of(s["start"], s["q"].shape[0])
    sk, jk = _rows_of(s["kstart"], s["k"].shape[0])
    q = torch.zeros(n, new, case["hq"], d, device="cuda")
    q[sq, jq] = s["q"].float()
    k = torch.zeros(n, most, h, d, device="cuda")
    k[sk, jk] = s["k"].float()
    v = torch.zeros(n, most, h, d, device="cuda")
    v[sk, jk] = s["v"].float()
    count = s["start"][1:] - s["start"][:-1]
    held = s["kstart"][1:] - s["kstart"][:-1]
    last = (held - count)[:, None] + torch.arange(new, device="cuda")
    hidden = torch.arange(most, device="cuda") > last[..., None]
    x = (q * d ** -0.5).view(n, new, h, g, d).permute(0, 2, 3, 1, 4).reshape(n, h, g * new, d)
    x = (x @ k.permute(0, 2, 3, 1)).view(n, h, g, new, most)
    x.masked_fill_(hidden[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    y = (x.view(n, h, g * new, most) @ v.permute(0, 2, 1, 3)).view(n, h, g, new, d) / total
    return y.permute(0, 3, 1, 2, 4).reshape(n, new, case["hq"], d)[sq, jq].to(TYPES[case["kind"]])


def _plain_score(s):
    top = s["case"]["top"]
    x = s["logits"].float()
    y = x - x.amax(-1, keepdim=True)
    e = y.exp()
    total = e.sum(-1, keepdim=True)
    lse = total.log()
    entropy = lse[:, 0] - torch.where(e > 0, e * y, 0.0).sum(-1) / total[:, 0]
    out = [y.gather(-1, s["tokens"].long()[:, None])[:, 0] - lse[:, 0], entropy]
    if not top:
        return out
    # whole numbers that order like the values, and of equal values the lower index first
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) << 20
    key += torch.arange(x.shape[1] - 1, -1, -1, device="cuda")
    best = torch.topk(key, top, -1).values
    token = x.shape[1] - 1 - (best & 0xFFFFF)
    return out + [y.gather(-1, token) - lse, token.int()]


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "norm":
            return [_plain_norm_one(s["q"], s["wq"], s), _plain_norm_one(s["k"], s["wk"], s)]
        return _plain_prompt(s) if case["op"] == "prompt" else _plain_score(s)
    import quant_quantized_matvec_gb300 as kq
    if case["op"] == "norm":
        return list(kq.norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["cs"], eps=1e-6,
                                 interleaved=case["inter"], dtype=TYPES[case["out"]]))
    if case["op"] == "prompt":
        return kq.prompt_attention(s["q"], s["k"], s["v"], s["start"], s["kstart"])
    got = kq.token_logprobs(s["logits"], s["tokens"], top=case["top"])
    return list(got) if case["top"] else list(got[:2])


# ------------------------------------------------------------- in 64 bits
def _exact_norm(x, w, s):
    case = s["case"]
    x = x.double()
    y = w.double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6)
    z = torch.view_as_complex(s["cs"].double())[s["pos"].long()][:, None]
    half = case["rot"] // 2
    if case["inter"]:
        turned = torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z
        turned = torch.view_as_real(turned).flatten(-2)
    else:
        turned = torch.complex(y[..., :half], y[..., half:2 * half]) * z
        turned = torch.cat([turned.real, turned.imag], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _exact_prompt(s):
    case = s["case"]
    g = case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    a, b = s["start"].tolist(), s["kstart"].tolist()
    for i in range(case["nseq"]):
        n, m = a[i + 1] - a[i], b[i + 1] - b[i]
        for h in range(case["hkv"]):
            k, v = (s[x][b[i]:b[i + 1], h].double() for x in ("k", "v"))
            for at in range(0, n, 1024):  # rows by the thousand, over the keys they can see
                to = min(n, at + 1024)
                end = m - n + to
                q = s["q"][a[i] + at:a[i] + to, h * g:(h + 1) * g].double()
                x = torch.einsum("tgd,kd->gtk", q, k[:end]) / math.sqrt(case["dim"])
                seen = torch.ones(to - at, end, dtype=torch.bool, device="cuda").tril(end - (to - at))
                p = torch.softmax(torch.where(seen, x, -math.inf), -1)
                out[a[i] + at:a[i] + to, h * g:(h + 1) * g] = torch.einsum("gtk,kd->tgd", p, v[:end])
    return out


def _exact_score(s):
    case, parts = s["case"], []
    for at in range(0, case["n"], 256):
        x, t = s["logits"][at:at + 256], s["tokens"][at:at + 256]
        logp = torch.log_softmax(x.double(), -1)
        p = logp.exp()
        row = [logp[torch.arange(t.numel(), device="cuda"), t.long()],
               -(p * logp.clamp(min=-1e300)).sum(-1)]
        if case["top"]:
            row.append(torch.sort(logp, stable=True, dim=-1, descending=True).values[:, :case["top"]])
        parts.append(row)
    out = [torch.cat(x) for x in zip(*parts)]
    return out + [None] if case["top"] else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return [_exact_norm(s["q"], s["wq"], s), _exact_norm(s["k"], s["wk"], s)]
    return _exact_prompt(s) if case["op"] == "prompt" else _exact_score(s)
