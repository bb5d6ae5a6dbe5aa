"""A prompt's operators: norms of query and key heads with their rotary
positions, causal attention of whole prompts packed one behind the other, and
the log probabilities of given tokens.

Thin layer over include/kq_prompt.h: arguments are checked here (types,
shapes, devices) and in the library (ranges, alignment, overlaps, memory).

    q, k = kq.norm_rope(q, k, q_weight, k_weight, positions, table)   # [ntok, heads, dim]
    y = kq.prompt_attention(q, k, v, start)                           # start: int32 [nseq + 1]
    logp, entropy, top_logp, top_tokens = kq.token_logprobs(logits, tokens, top=5)

A prompt that continues a cached sequence attends the sequence's keys and
values, read back in order (kv_read with ctx 0), with their own starts:

    y = kq.prompt_attention(q, k_all, v_all, start, key_start)
"""
from __future__ import annotations

import ctypes

import torch

from . import KQError, _binding
from .decode import _call, _empty, _on, _out, _table, _tensor

MAX_TOP = 32
TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 30}


def _type(dtype, name):
    code = TYPES.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return code


def _strided(t, name, dtype, shape):
    """Address and token stride of [ntok, heads, dim] whose tokens may lie
    apart (a slice of a fused projection's output)."""
    p = _tensor(t, name, dtype, shape, dense=False)
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        if n == 0:
            return p, h * d
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return p, s0 if n > 1 else h * d


def norm_rope(q, k=None, q_weight=None, k_weight=None, positions=None, table=None, eps=1e-6,
              interleaved=False, dtype=None, q_out=None, k_out=None, stream=None):
    """Each head of q and k [ntok, heads, dim] divided by the root of its mean
    square (plus eps) and multiplied by its weight (f32 [dim]; None: ones), then,
    with a table, turned by its token's position as rope does: one launch.  k
    may be None.  dtype: of the outputs, which may be float16 or bfloat16 where
    the inputs are float32 (it is the inputs' unless given).  q_out and k_out may
    be q and k.  Returns (q, k)."""
    xs = [(q, q_weight, q_out, "q")]
    if k is not None:
        xs.append((k, k_weight, k_out, "k"))
    if q.dim() != 3:
        raise ValueError("q must be [ntok, heads, dim]")
    n, _, d = q.shape
    kind = _type(q.dtype, "q")
    dtype = q.dtype if dtype is None else dtype
    out_kind = _type(dtype, "dtype")
    pp = tp = None
    npos = rot = 0
    if table is not None:
        tp, npos, rot = _table(table)
        if positions is None:
            raise ValueError("a table needs positions")
        pp = _tensor(positions, "positions", torch.int32, (n,))
    st, on = _on(stream)
    parts = (_binding.KqNormPart * len(xs))()
    outs = []
    for part, (x, weight, out, name) in zip(parts, xs):
        if x.dim() != 3 or x.shape[0] != n or x.shape[2] != d:
            raise ValueError(f"{name} must be [{n}, heads, {d}], got {tuple(x.shape)}")
        part.x, part.stride = _strided(x, name, q.dtype, x.shape)
        part.weight = None if weight is None else _tensor(weight, name + "_weight", torch.float32, (d,))
        if out is None:
            out = _empty(x.shape, dtype, x.device, on)
            part.out, part.out_stride = out.data_ptr(), x.shape[1] * d
        else:
            part.out, part.out_stride = _strided(out, name + "_out", dtype, x.shape)
        part.heads = x.shape[1]
        outs.append(out)
    _call("kq_norm_rope", parts, len(xs), kind, out_kind, n, d, float(eps), pp, tp, npos, rot,
          bool(interleaved), st)
    return outs[0], outs[1] if k is not None else None


def prompt_workspace_bytes(q, k, nseq):
    """Bytes of prompt_attention's workspace for q [ntok, q_heads, dim] and k
    [nkeys, kv_heads, dim] of nseq sequences (it depends on sizes and type
    alone)."""
    n = int(_binding.load().kq_prompt_workspace_bytes(
        _type(q.dtype, "q"), int(nseq), q.shape[0], k.shape[0], q.shape[1], k.shape[1], q.shape[2]))
    if n < 0:
        raise KQError(-n, "kq_prompt_workspace_bytes")
    return n


def prompt_attention(q, k, v, start, key_start=None, scale=None, out=None, workspace=None,
                     stream=None):
    """Causal attention of packed prompts: q [ntok, q_heads, dim], k and v
    [nkeys, kv_heads, dim], all float32, float16 or bfloat16; sequence b has the
    queries start[b]..start[b+1]-1 and the keys key_start[b]..key_start[b+1]-1
    (int32 [nseq + 1]; None: start), of whose tokens its queries are the last.
    scale: 1 / sqrt(dim) unless given.  workspace: a CUDA uint8 tensor of
    prompt_workspace_bytes(...) or more; otherwise torch's allocator gives one
    for the call.  Returns [ntok, q_heads, dim] of q's type."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, dim]")
    kind = _type(q.dtype, "q")
    (n, h, d), (m, g, _) = q.shape, k.shape
    qp, qs = _strided(q, "q", q.dtype, (n, h, d))
    kp, ks = _strided(k, "k", q.dtype, (m, g, d))
    vp, vs = _strided(v, "v", q.dtype, (m, g, d))
    nseq = start.numel() - 1
    sp = _tensor(start, "start", torch.int32, (nseq + 1,))
    cp = None if key_start is None else _tensor(key_start, "key_start", torch.int32, (nseq + 1,))
    st, on = _on(stream)
    out, op = _out(out, "out", q.dtype, (n, h, d), q.device, on)
    wp, wn = None, 0
    if workspace is not None:
        wp, wn = _tensor(workspace, "workspace", torch.uint8), workspace.numel()
    else:
        wn = prompt_workspace_bytes(q, k, nseq)
        if wn:
            workspace = _empty(wn, torch.uint8, q.device, on)
            wp = workspace.data_ptr()
    _call("kq_prompt_attention", kind, nseq, n, m, sp, cp, qp, qs, h, kp, ks, vp, vs, g, d,
          d ** -0.5 if scale is None else float(scale), op, wp, wn, st)
    return out


def token_logprobs(logits, tokens=None, top=0, entropy=True, stream=None):
    """Log probabilities from rows of logits [n, vocab] (float32, float16 or
    bfloat16; rows may lie apart): of the given tokens (int32 [n]; None: left
    out), the rows' entropies, and the `top` best alternatives (at most 32),
    best first, of equal ones the lower token first.  Returns (logp [n], entropy
    [n], top_logp [n, top], top_tokens int32 [n, top]), None for what was left
    out."""
    if logits.dim() != 2:
        raise ValueError("logits must be [n, vocab]")
    n, vocab = logits.shape
    kind = _type(logits.dtype, "logits")
    xp = _tensor(logits, "logits", logits.dtype, dense=False)
    if n and vocab > 1 and logits.stride(1) != 1:
        raise ValueError("logits: a row must be contiguous")
    stride = logits.stride(0) if n > 1 else vocab
    tp = None if tokens is None else _tensor(tokens, "tokens", torch.int32, (n,))
    st, on = _on(stream)
    dev = logits.device

    def new(want, dtype, *shape):
        if not want:
            return None, None
        t = _empty(shape, dtype, dev, on)
        return t, t.data_ptr()

    logp, lp = new(tokens is not None, torch.float32, n)
    ent, ep = new(entropy, torch.float32, n)
    top_logp, tlp = new(top > 0, torch.float32, n, max(top, 0))
    top_token, ttp = new(top > 0, torch.int32, n, max(top, 0))
    _call("kq_token_logprobs", kind, n, vocab, xp, stride, tp, int(top), lp, ep, tlp, ttp, st)
    return logp, ent, top_logp, top_token
