"""A prompt's operators: norms of query and key heads with their rotary
positions, causal attention of whole prompts packed one behind the other, and
the log probabilities of given tokens.

Thin layer over include/kq_prompt.h: arguments are checked here (types,
shapes, devices) and in the library (ranges, alignment, overlaps, memory).

    q, k = kq.norm_rope(q, k, q_weight, k_weight, positions, table)   # [ntok, heads, dim]
    y = kq.prompt_attention(q, k, v, start)                           # start: int32 [nseq + 1]
    logp, entropy, top_logp, top_tokens = kq.token_logprobs(logits, tokens, top=5)

A prompt that continues a cached sequence attends the sequence's keys and
values, read back in order (kv_read with ctx 0, which gives float32: cast them
for 16-bit queries), with their own starts:

    y = kq.prompt_attention(q, k_all, v_all, start, key_start)
"""
from __future__ import annotations

import struct

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


# The wrappers run between kernels of a few microseconds: each looks at a
# tensor's shape and strides once.
def _strided(t, name, dtype, shape):
    """Address and token stride of [ntok, heads, dim] (of this shape) whose
    tokens may lie apart (a slice of a fused projection's output)."""
    if not (t.is_cuda and t.dtype is dtype):
        _tensor(t, name, dtype, dense=False)  # (says what is wrong)
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        if n == 0:
            return t.data_ptr(), h * d
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return t.data_ptr(), s0 if n > 1 else h * d


def _part(x, weight, out, name, n, d, kind, dtype, on):
    """One tensor of norm_rope: its descriptor and its output."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != n or shape[2] != d:
        raise ValueError(f"{name} must be [{n}, heads, {d}], got {tuple(shape)}")
    xp, xs = _strided(x, name, kind, shape)
    wp = 0 if weight is None else _tensor(weight, name + "_weight", torch.float32, (d,))
    h = shape[1]
    if out is None:
        out = _empty(shape, dtype, x.device, on)
        op, os_ = out.data_ptr(), h * d
    else:
        if out.shape != shape:
            raise ValueError(f"{name}_out must have shape {tuple(shape)}, got {tuple(out.shape)}")
        op, os_ = _strided(out, name + "_out", dtype, shape)
    return _pack_part(xp, xs, wp, op, os_, h, 0), out


_pack_part = struct.Struct("@PqPPqii").pack  # kq_norm_part, without padding


def norm_rope(q, k=None, q_weight=None, k_weight=None, positions=None, table=None, eps=1e-6,
              interleaved=False, dtype=None, q_out=None, k_out=None, stream=None):
    """Each head of q and k [ntok, heads, dim] divided by the root of its mean
    square (plus eps) and multiplied by its weight (f32 [dim]; None: ones), then,
    with a table, turned by its token's position as rope does: one launch.  k
    may be None.  dtype: of the outputs, which may be float16 or bfloat16 where
    the inputs are float32 (it is the inputs' unless given).  q_out and k_out may
    be q and k.  Returns (q, k)."""
    shape, kind = q.shape, q.dtype
    if len(shape) != 3:
        raise ValueError("q must be [ntok, heads, dim]")
    n, _, d = shape
    code = _type(kind, "q")
    if dtype is None:
        dtype, out_code = kind, code
    else:
        out_code = _type(dtype, "dtype")
    pp = tp = None
    npos = rot = 0
    if table is not None:
        tp, npos, rot = _table(table)
        if positions is None:
            raise ValueError("a table needs positions")
        pp = _tensor(positions, "positions", torch.int32, (n,))
    st, on = _on(stream)
    first, q_out = _part(q, q_weight, q_out, "q", n, d, kind, dtype, on)
    if k is None:
        parts, count, k_out = first, 1, None
    else:
        second, k_out = _part(k, k_weight, k_out, "k", n, d, kind, dtype, on)
        parts, count = first + second, 2
    _call("kq_norm_rope", parts, count, code, out_code, n, d, eps, pp, tp, npos, rot, interleaved, st)
    return q_out, k_out


_space = {}  # workspace bytes by device and sizes, which they depend on alone


def _workspace(code, nseq, n, m, h, g, d):
    key = (torch._C._cuda_getDevice(), code, nseq, n, m, h, g, d)
    got = _space.get(key)
    if got is None:
        got = int(_binding.load().kq_prompt_workspace_bytes(code, nseq, n, m, h, g, d))
        if got < 0:
            raise KQError(-got, "kq_prompt_workspace_bytes")
        if len(_space) >= 4096:
            _space.clear()
        _space[key] = got
    return got


def prompt_workspace_bytes(q, k, nseq):
    """Bytes of prompt_attention's workspace for q [ntok, q_heads, dim] and k
    [nkeys, kv_heads, dim] of nseq sequences (it depends on sizes and type
    alone)."""
    return _workspace(_type(q.dtype, "q"), int(nseq), q.shape[0], k.shape[0], q.shape[1], k.shape[1],
                      q.shape[2])


def prompt_attention(q, k, v, start, key_start=None, scale=None, out=None, workspace=None,
                     stream=None):
    """Causal attention of packed prompts: q [ntok, q_heads, dim], k and v
    [nkeys, kv_heads, dim], all float32, float16 or bfloat16; sequence b has the
    queries start[b]..start[b+1]-1 and the keys key_start[b]..key_start[b+1]-1
    (int32 [nseq + 1]; None: start), of whose tokens its queries are the last.
    scale: 1 / sqrt(dim) unless given.  workspace: a CUDA uint8 tensor of
    prompt_workspace_bytes(...) or more; otherwise torch's allocator gives one
    for the call.  Returns [ntok, q_heads, dim] of q's type."""
    shape, held, kind = q.shape, k.shape, q.dtype
    if len(shape) != 3 or len(held) != 3:
        raise ValueError("q and k must be [tokens, heads, dim]")
    code = _type(kind, "q")
    (n, h, d), (m, g, kd) = shape, held
    if kd != d or v.shape != held:
        raise ValueError(f"k and v must be [nkeys, kv_heads, {d}], got {tuple(held)} and {tuple(v.shape)}")
    qp, qs = _strided(q, "q", kind, shape)
    kp, ks = _strided(k, "k", kind, held)
    vp, vs = _strided(v, "v", kind, held)
    nseq = start.numel() - 1
    sp = _tensor(start, "start", torch.int32, (nseq + 1,))
    cp = None if key_start is None else _tensor(key_start, "key_start", torch.int32, (nseq + 1,))
    st, on = _on(stream)
    out, op = _out(out, "out", kind, shape, q.device, on)
    if workspace is not None:
        wp, wn = _tensor(workspace, "workspace", torch.uint8), workspace.numel()
    else:
        wp, wn = None, _workspace(code, nseq, n, m, h, g, d)
        if wn:
            workspace = _empty(wn, torch.uint8, q.device, on)
            wp = workspace.data_ptr()
    _call("kq_prompt_attention", code, nseq, n, m, sp, cp, qp, qs, h, kp, ks, vp, vs, g, d,
          d ** -0.5 if scale is None else scale, op, wp, wn, st)
    return out


def token_logprobs(logits, tokens=None, top=0, entropy=True, stream=None):
    """Log probabilities from rows of logits [n, vocab] (float32, float16 or
    bfloat16; rows may lie apart): of the given tokens (int32 [n]; None: left
    out), the rows' entropies, and the `top` best alternatives (at most 32),
    best first, of equal ones the lower token first.  Returns (logp [n], entropy
    [n], top_logp [n, top], top_tokens int32 [n, top]), None for what was left
    out."""
    shape, kind = logits.shape, logits.dtype
    if len(shape) != 2:
        raise ValueError("logits must be [n, vocab]")
    n, vocab = shape
    code = _type(kind, "logits")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    s0, s1 = logits.stride()
    if n and vocab > 1 and s1 != 1:
        raise ValueError("logits: a row must be contiguous")
    st, on = _on(stream)
    dev = logits.device
    logp = ent = top_logp = top_token = tp = lp = ep = tlp = ttp = None
    if tokens is not None:
        tp = _tensor(tokens, "tokens", torch.int32, (n,))
        logp = _empty((n,), torch.float32, dev, on)
        lp = logp.data_ptr()
    if entropy:
        ent = _empty((n,), torch.float32, dev, on)
        ep = ent.data_ptr()
    if top > 0:
        top_logp = _empty((n, top), torch.float32, dev, on)
        top_token = _empty((n, top), torch.int32, dev, on)
        tlp, ttp = top_logp.data_ptr(), top_token.data_ptr()
    _call("kq_token_logprobs", code, n, vocab, logits.data_ptr(), s0 if n > 1 else vocab, tp, top, lp,
          ep, tlp, ttp, st)
    return logp, ent, top_logp, top_token
