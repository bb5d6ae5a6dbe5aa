"""A decode step around its matvecs: rotary positions, the quantised key/value
cache, attention of the new tokens over it, and the verification of drafts.

Thin layer over include/kq_decode.h: arguments are checked here (types,
shapes, devices) and in the library (ranges, alignment, overlaps, memory).

    cache = kq.KVCache(kq.KV_Q8, kv_heads=2, head_dim=128, pages=4096)
    batch = kq.KVBatch(start, ctx, pages, ntok, max_new)    # device tensors
    q = kq.rope(q, positions, table)                        # [ntok, heads, dim] f32
    kq.kv_append(cache, batch, k, v, positions, table)      # keys are rotated on the way
    y = kq.tree_attention(cache, batch, q, mask)
    path, count, token = kq.verify_tree(start, tokens, parents, p, q, u, u_next, max_new)
    kq.kv_move(cache, batch, path, count)                   # keep the accepted ones

Descriptors (KVCache, KVBatch) are made once and kept; their tensors may
change in value from step to step, so a captured CUDA graph stays valid.
Their attributes cannot be set again: other tensors or sizes need another
descriptor.
"""
from __future__ import annotations

import ctypes

import torch

from . import KQError, _binding

KV_F16, KV_Q4, KV_Q8 = 1, 2, 8
KV_PAGE = 64
MAX_DRAFT = 64
SCALINGS = {None: 0, "linear": 1, "base": 2, "ramp": 3}


# The library's functions, looked up once: the wrappers below run between
# kernels of a few microseconds.
_fn = {}


def _call(name, *args):
    f = _fn.get(name)
    if f is None:
        f = _fn[name] = getattr(_binding.load(), name)
    st = f(*args)
    if st != 0:
        raise KQError(st, name)


def _on(stream):
    """The stream's pointer, and a context in which new tensors belong to it
    (None: they do already)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()), None
    return stream.cuda_stream, torch.cuda.stream(stream)


def _empty(shape, dtype, device, on):
    if on is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with on:
        return torch.empty(shape, dtype=dtype, device=device)


def _tensor(t, name, dtype, shape=None, dense=True):
    """The address of a CUDA tensor after the checks."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype
            and (shape is None or t.shape == shape) and (not dense or t.is_contiguous())):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _out(t, name, dtype, shape, device, on):
    """An output that was given, checked, or a new one; and its address."""
    if t is None:
        t = _empty(shape, dtype, device, on)
        return t, t.data_ptr()
    return t, _tensor(t, name, dtype, shape)


def _heads(t, name, shape):
    """Address and token stride of f32 [ntok, heads, dim] whose tokens may lie
    apart (a slice of a fused projection's output)."""
    p = _tensor(t, name, torch.float32, shape, dense=False)
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        if n == 0:
            return p, h * d
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return p, s0 if n > 1 else h * d


class _Fixed:
    """A descriptor: the C struct behind it holds its tensors' addresses and
    its sizes, so no attribute is set again after it was made."""

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__}.{name} is fixed: make another "
                             f"{type(self).__name__}, or change the tensor's values in place")

    def __delattr__(self, name):
        raise AttributeError(f"{type(self).__name__}.{name} is fixed")


class KVCache(_Fixed):
    """A paged key/value cache of one layer: `pages` pages of 64 tokens, in
    KV_F16, KV_Q8 or KV_Q4 (layout: include/kq_decode.h).  data: its bytes,
    a CUDA uint8 tensor (made, zeroed, if not given)."""

    def __init__(self, fmt, kv_heads, head_dim, pages, data=None, device="cuda"):
        each = int(_binding.load().kq_kv_page_bytes(int(fmt), int(kv_heads), int(head_dim)))
        if each < 0:
            raise ValueError("fmt must be KV_F16, KV_Q8 or KV_Q4, kv_heads 1..1024, "
                             "head_dim 64, 128 or 256")
        if pages < 1:
            raise ValueError("pages must be positive")
        if data is None:
            data = torch.zeros(each * pages, dtype=torch.uint8, device=device)
        _tensor(data, "data", torch.uint8, (each * pages,))
        c = _binding.KqKv(int(fmt), int(kv_heads), int(head_dim), 0, data.data_ptr(), int(pages))
        self.__dict__.update(fmt=int(fmt), kv_heads=int(kv_heads), head_dim=int(head_dim),
                             pages=int(pages), page_bytes=each, data=data, _c=c,
                             _p=ctypes.byref(c))


class KVBatch(_Fixed):
    """The sequences of a step (kq_batch): start [nseq + 1], ctx [nseq] and
    pages [nseq, max_pages], int32 CUDA tensors; ntok new tokens in all, at
    most max_new of one sequence."""

    def __init__(self, start, ctx, pages, ntok, max_new):
        nseq = ctx.numel()
        if pages.dim() != 2:
            raise ValueError("pages must be [nseq, max_pages]")
        _tensor(start, "start", torch.int32, (nseq + 1,))
        _tensor(ctx, "ctx", torch.int32, (nseq,))
        _tensor(pages, "pages", torch.int32, (nseq, pages.shape[1]))
        c = _binding.KqBatch(nseq, int(max_new), int(ntok), start.data_ptr(), ctx.data_ptr(),
                             pages.data_ptr(), pages.shape[1])
        self.__dict__.update(start=start, ctx=ctx, pages=pages, nseq=nseq, ntok=int(ntok),
                             max_new=int(max_new), _c=c, _p=ctypes.byref(c),
                             _ws={})  # workspace bytes of the attention calls made with it


def rope_table(positions, rot, base=10000.0, scaling=None, factor=1.0, orig=1, fast=32.0,
               slow=1.0, magnitude=1.0, device="cuda", stream=None):
    """(cos, sin) of positions 0..positions-1: f32 [positions, rot / 2, 2].
    scaling for long contexts: None, "linear", "base" or "ramp", a blend that
    is linear in a pair's turns (kq_rope_scaling)."""
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(map(str, SCALINGS))}")
    if positions < 1 or rot < 2:
        raise ValueError("positions and rot must be positive")
    st, on = _on(stream)
    table = _empty((positions, rot // 2, 2), torch.float32, device, on)
    sc = _binding.KqRopeScaling(SCALINGS[scaling], int(orig), float(factor), float(fast),
                                float(slow), float(magnitude))
    _call("kq_rope_table", int(positions), int(rot), float(base), ctypes.byref(sc),
          table.data_ptr(), st)
    return table


def _table(table):
    s = table.shape
    if len(s) != 3 or s[2] != 2:
        raise ValueError("table must be [positions, rot / 2, 2]")
    return _tensor(table, "table", torch.float32), s[0], 2 * s[1]


def rope(x, positions, table, interleaved=False, inverse=False, out=None, stream=None):
    """x f32 [ntok, heads, dim] with each head's first rot values turned by its
    token's position (int32 [ntok]); rot is the table's.  inverse turns back,
    and is the gradient.  out may be x."""
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be [ntok, heads, dim]")
    n, h, d = shape
    xp, xs = _heads(x, "x", shape)
    tp, npos, rot = _table(table)
    pp = _tensor(positions, "positions", torch.int32, (n,))
    st, on = _on(stream)
    if out is None:
        out = _empty(shape, torch.float32, x.device, on)
        op, os_ = out.data_ptr(), h * d
    else:
        op, os_ = _heads(out, "out", shape)
    _call("kq_rope", xp, xs, op, os_, n, h, d, pp, tp, npos, rot, bool(interleaved),
          bool(inverse), st)
    return out


def kv_append(cache, batch, k, v, positions=None, table=None, interleaved=False, stream=None):
    """Quantise the new tokens' keys and values, f32 [ntok, kv_heads,
    head_dim], into the cache; with a table the keys are rotated first, by
    positions (which are not looked at without one)."""
    shape = (batch.ntok, cache.kv_heads, cache.head_dim)
    kp, ks = _heads(k, "k", shape)
    vp, vs = _heads(v, "v", shape)
    pp = tp = None
    npos = rot = 0
    if table is not None:
        tp, npos, rot = _table(table)
        if positions is None:
            raise ValueError("a table needs positions")
        pp = _tensor(positions, "positions", torch.int32, (batch.ntok,))
    st, _ = _on(stream)
    _call("kq_kv_append", cache._p, batch._p, kp, ks, vp, vs, pp, tp, npos, rot,
          bool(interleaved), st)


def kv_read(cache, batch, k=None, v=None, stream=None):
    """The batch's places read back: (k, v) f32 [ntok, kv_heads, head_dim]."""
    shape = (batch.ntok, cache.kv_heads, cache.head_dim)
    st, on = _on(stream)
    k, kp = _out(k, "k", torch.float32, shape, cache.data.device, on)
    v, vp = _out(v, "v", torch.float32, shape, cache.data.device, on)
    _call("kq_kv_read", cache._p, batch._p, kp, vp, st)
    return k, v


def kv_move(cache, batch, path, count, stream=None):
    """Move the accepted drafts' keys and values (verify_tree's path and
    count) up behind the committed ones."""
    st, _ = _on(stream)
    _call("kq_kv_move", cache._p, batch._p, _tensor(path, "path", torch.int32, (batch.ntok,)),
          _tensor(count, "count", torch.int32, (batch.nseq,)), st)


def tree_mask(parents):
    """The attention masks of one sequence's tree of new tokens: parents (a
    list; -1 for a root, else an earlier node) -> list of ints for an int64
    tensor: bit j of node i is set where j is i or an ancestor of i."""
    if len(parents) > MAX_DRAFT:
        raise ValueError(f"at most {MAX_DRAFT} new tokens of a sequence")
    bits = []
    for i, p in enumerate(parents):
        if not -1 <= p < i:
            raise ValueError("a node's parent comes before it")
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def attention_workspace_bytes(cache, batch, q_heads):
    """Bytes of tree_attention's workspace (it depends on sizes alone, so the
    batch keeps the answer)."""
    key = (cache.fmt, cache.kv_heads, cache.head_dim, q_heads)
    n = batch._ws.get(key)
    if n is None:
        n = int(_binding.load().kq_attn_workspace_bytes(cache._p, batch._p, int(q_heads)))
        if n < 0:
            raise KQError(-n, "kq_attn_workspace_bytes")
        batch._ws[key] = n
    return n


def tree_attention(cache, batch, q, mask=None, scale=None, out=None, workspace=None,
                   stream=None):
    """Attention of the new tokens' queries, f32 [ntok, q_heads, head_dim],
    over the committed tokens and the new ones whose bit is set in mask
    (int64 [ntok]; None: all up to the token itself).  scale: 1 /
    sqrt(head_dim) unless given.  workspace: a CUDA uint8 tensor of
    attention_workspace_bytes(...) or more; otherwise torch's allocator gives
    one for the call."""
    if q.dim() != 3:
        raise ValueError("q must be [ntok, q_heads, head_dim]")
    heads = q.shape[1]
    shape = (batch.ntok, heads, cache.head_dim)
    qp, qs = _heads(q, "q", shape)
    mp = None if mask is None else _tensor(mask, "mask", torch.int64, (batch.ntok,))
    st, on = _on(stream)
    out, op = _out(out, "out", torch.float32, shape, q.device, on)
    if workspace is None:
        wn = attention_workspace_bytes(cache, batch, heads)
        workspace = _empty(wn, torch.uint8, q.device, on)
        wp = workspace.data_ptr()
    else:
        wp, wn = _tensor(workspace, "workspace", torch.uint8), workspace.numel()
    _call("kq_tree_attention", cache._p, batch._p, qp, qs, heads, mp,
          cache.head_dim ** -0.5 if scale is None else float(scale), op, wp, wn, st)
    return out


def verify_tree(start, tokens, parents, p, q, u, u_next, max_new, path=None, count=None,
                next_token=None, stream=None):
    """Verify each sequence's tree of drafted tokens (kq_verify_tree): start
    [nseq + 1], tokens and parents [ntok] int32, the target's and the drafts'
    distributions p and q f32 [ntok, vocab] (q None: drafts without one),
    random numbers u [ntok] and u_next [nseq].  Returns (path [ntok], count
    [nseq], next_token [nseq])."""
    ntok, nseq = tokens.numel(), u_next.numel()
    if p.dim() != 2:
        raise ValueError("p must be [ntok, vocab]")
    shape = (ntok, p.shape[1])

    def rows(t, name):
        ptr = _tensor(t, name, torch.float32, shape, dense=False)
        if ntok and shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: a row must be contiguous")
        return ptr, t.stride(0) if ntok > 1 else shape[1]

    pp, ps = rows(p, "p")
    qp, qs = (None, 0) if q is None else rows(q, "q")
    st, on = _on(stream)
    dev = p.device
    path, path_p = _out(path, "path", torch.int32, (ntok,), dev, on)
    count, count_p = _out(count, "count", torch.int32, (nseq,), dev, on)
    next_token, next_p = _out(next_token, "next_token", torch.int32, (nseq,), dev, on)
    _call("kq_verify_tree", nseq, ntok, int(max_new),
          _tensor(start, "start", torch.int32, (nseq + 1,)),
          _tensor(tokens, "tokens", torch.int32, (ntok,)),
          _tensor(parents, "parents", torch.int32, (ntok,)), pp, ps, qp, qs, shape[1],
          _tensor(u, "u", torch.float32, (ntok,)), _tensor(u_next, "u_next", torch.float32, (nseq,)),
          path_p, count_p, next_p, st)
    return path, count, next_token
