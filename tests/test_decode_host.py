"""The decode-step entry points on the host, without a GPU: exports, sizes,
and the refusal of bad arguments before any CUDA call (fake addresses that
are never dereferenced), and the references' own hand-worked values."""
import ctypes
import os
import re

import numpy as np
import pytest

import decode_ref as R
from quant_quantized_matvec_gb300 import _binding
from quant_quantized_matvec_gb300 import build as kbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, FORMAT, SHAPE, NTOK, NULL, ALIGN, ALIAS, CUDA, TIMEOUT, COUNT, LIMIT, MEMORY = range(12)
A = [0x7f0000000000 + (i << 36) for i in range(16)]  # far apart, well aligned


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _binding.load()


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "kq_decode.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(kq_[a-z_]+)\s*\(", src))
    assert names == set(_binding.DECODE_SYMBOLS)
    for n in names:
        assert hasattr(lib, n)


def test_page_bytes(lib):
    for fmt in (R.F16, R.Q8, R.Q4):
        for d in (64, 128, 256):
            scales = 0 if fmt == R.F16 else d // 32 * 2
            assert lib.kq_kv_page_bytes(fmt, 3, d) == 3 * 2 * 64 * (d * R.BITS[fmt] // 8 + scales)
    for bad in ((3, 1, 64), (R.Q8, 0, 64), (R.Q8, 1025, 64), (R.Q8, 1, 96), (R.Q8, 1, 0)):
        assert lib.kq_kv_page_bytes(*bad) == -1


def kv(**kw):
    d = dict(fmt=R.Q8, kv_heads=2, head_dim=128, reserved=0, data=A[0], pages=10)
    d.update(kw)
    return ctypes.byref(_binding.KqKv(**d))


def batch(**kw):
    d = dict(nseq=2, max_new=8, ntok=12, start=A[1], ctx=A[2], pages=A[3], max_pages=5)
    d.update(kw)
    return ctypes.byref(_binding.KqBatch(**d))


BAD_KV = [(dict(fmt=12), FORMAT), (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE),
          (dict(head_dim=96), SHAPE), (dict(reserved=1), SHAPE), (dict(pages=0), SHAPE),
          (dict(pages=1 << 31), SHAPE), (dict(data=None), NULL), (dict(data=A[0] + 8), ALIGN)]
BAD_BATCH = [(dict(nseq=0), COUNT), (dict(nseq=4097), COUNT), (dict(ntok=-1), NTOK),
             (dict(ntok=(1 << 24) + 1), NTOK), (dict(max_new=0), NTOK), (dict(max_pages=0), SHAPE),
             (dict(start=None), NULL), (dict(ctx=None), NULL), (dict(pages=None), NULL),
             (dict(start=A[1] + 2), ALIGN)]


def append(lib, c=None, b=None, k=A[4], ks=256, v=A[5], vs=256, pos=A[6], table=A[7], npos=100,
           rot=128):
    return lib.kq_kv_append(c or kv(), b or batch(), k, ks, v, vs, pos, table, npos, rot, 0, None)


def read(lib, c=None, b=None, k=A[4], v=A[5]):
    return lib.kq_kv_read(c or kv(), b or batch(), k, v, None)


def move(lib, c=None, b=None, path=A[4], count=A[5]):
    return lib.kq_kv_move(c or kv(), b or batch(), path, count, None)


def attend(lib, c=None, b=None, q=A[4], qs=512, hq=4, mask=A[5], scale=0.1, out=A[6], ws=None,
           wn=0):
    return lib.kq_tree_attention(c or kv(), b or batch(), q, qs, hq, mask, scale, out, ws, wn, None)


@pytest.mark.parametrize("fn", [append, read, move, attend])
def test_descriptors_are_checked(lib, fn):
    for kw, status in BAD_KV:
        assert fn(lib, c=kv(**kw)) == status, kw
    for kw, status in BAD_BATCH:
        assert fn(lib, b=batch(**kw)) == status, kw
    assert fn(lib, b=batch(ntok=0)) == OK


def test_refusals(lib):
    for kw, st in [(dict(ks=255), SHAPE), (dict(ks=258), SHAPE), (dict(vs=0), SHAPE),
                   (dict(k=None), NULL), (dict(v=None), NULL), (dict(pos=None), NULL),
                   (dict(k=A[4] + 4), ALIGN), (dict(rot=132), SHAPE), (dict(rot=136), SHAPE),
                   (dict(rot=4), SHAPE), (dict(npos=0), SHAPE), (dict(k=A[0] + 64), ALIAS),
                   (dict(table=A[0] + 64), ALIAS), (dict(pos=A[0] + 4), ALIAS)]:
        assert append(lib, **kw) == st, kw
    for kw, st in [(dict(k=None, v=None), NULL), (dict(k=A[4] + 4), ALIGN),
                   (dict(k=A[0] + 16), ALIAS), (dict(k=A[5] + 16), ALIAS), (dict(v=A[3]), ALIAS)]:
        assert read(lib, **kw) == st, kw
    for kw, st in [(dict(path=None), NULL), (dict(count=None), NULL), (dict(path=A[4] + 1), ALIGN),
                   (dict(path=A[0]), ALIAS), (dict(b=batch(max_new=65)), NTOK)]:
        assert move(lib, **kw) == st, kw
    for kw, st in [(dict(hq=3), SHAPE), (dict(hq=0), SHAPE), (dict(qs=508), SHAPE),
                   (dict(qs=513), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(q=None), NULL),
                   (dict(out=None), NULL), (dict(mask=A[5] + 4), ALIGN), (dict(q=A[4] + 4), ALIGN),
                   (dict(b=batch(max_new=65)), NTOK), (dict(ws=A[8] + 16, wn=1 << 30), ALIGN)]:
        assert attend(lib, **kw) == st, kw


def test_rope_refusals(lib):
    def rope(x=A[0], xs=512, out=A[1], os_=512, n=5, h=4, d=128, pos=A[2], table=A[3], npos=9,
             rot=64):
        return lib.kq_rope(x, xs, out, os_, n, h, d, pos, table, npos, rot, 0, 0, None)

    for kw, st in [(dict(h=0), SHAPE), (dict(d=124), SHAPE), (dict(d=1032), SHAPE),
                   (dict(rot=136), SHAPE), (dict(rot=12), SHAPE), (dict(npos=0), SHAPE),
                   (dict(xs=511), SHAPE), (dict(os_=514), SHAPE), (dict(n=-1), NTOK),
                   (dict(x=None), NULL), (dict(pos=None), NULL), (dict(table=None), NULL),
                   (dict(x=A[0] + 4), ALIGN), (dict(pos=A[2] + 1), ALIGN), (dict(out=A[0] + 16), ALIAS),
                   (dict(out=A[0], os_=1024), ALIAS), (dict(out=A[3]), ALIAS)]:
        assert rope(**kw) == st, kw
    assert rope(n=0, x=None) == OK

    def table(n=10, rot=64, base=1e4, t=A[0], **kw):
        sc = dict(kind=0, orig=1, factor=1.0, fast=32.0, slow=1.0, magnitude=1.0)
        sc.update(kw)
        return lib.kq_rope_table(n, rot, base, ctypes.byref(_binding.KqRopeScaling(**sc)), t, None)

    for kw, st in [(dict(n=0), SHAPE), (dict(rot=12), SHAPE), (dict(base=0.0), SHAPE),
                   (dict(base=float("inf")), SHAPE), (dict(kind=4), SHAPE), (dict(kind=-1), SHAPE),
                   (dict(kind=1, factor=0.0), SHAPE), (dict(kind=3, factor=2.0, orig=0), SHAPE),
                   (dict(kind=3, factor=2.0, fast=1.0), SHAPE),
                   (dict(magnitude=float("nan")), SHAPE), (dict(t=None), NULL),
                   (dict(t=A[0] + 4), ALIGN)]:
        assert table(**kw) == st, kw


def test_verify_refusals(lib):
    def verify(nseq=2, n=9, new=6, start=A[0], tok=A[1], par=A[2], p=A[3], ps=1000, q=A[4],
               qs=1000, v=1000, u=A[5], un=A[6], path=A[7], count=A[8], nxt=A[9]):
        return lib.kq_verify_tree(nseq, n, new, start, tok, par, p, ps, q, qs, v, u, un, path,
                                  count, nxt, None)

    for kw, st in [(dict(nseq=0), COUNT), (dict(nseq=4097), COUNT), (dict(n=-1), NTOK),
                   (dict(new=0), NTOK), (dict(new=65), NTOK), (dict(v=0), SHAPE),
                   (dict(v=(1 << 19) + 1, ps=1 << 20, qs=1 << 20), SHAPE), (dict(ps=999), SHAPE),
                   (dict(qs=999), SHAPE), (dict(p=None), NULL), (dict(u=None), NULL),
                   (dict(nxt=None), NULL), (dict(p=A[3] + 2), ALIGN), (dict(path=A[1]), ALIAS),
                   (dict(nxt=A[8] + 4), ALIAS)]:
        assert verify(**kw) == st, kw
    assert verify(n=0, p=None) == OK


def test_reference_quantisation_by_hand():
    x = np.zeros(32, np.float32)
    x[3], x[7], x[9] = 12.7, -6.35, 0.049
    c, d = R.quantise(x, R.Q8)
    assert d[0] == np.float16(0.1) and (c[3], c[7], c[9]) == (127, -64, 0)
    x[3] = 4.0
    c, d = R.quantise(x, R.Q4)  # largest magnitude: -6.35 -> code -8
    assert d[0] == np.float16(6.35 / 8) and (c[3], c[7], c[9]) == (5, -8, 0)
    assert R.quantise(np.zeros(32), R.Q8)[1][0] == 0
    x[0] = np.inf
    assert np.isnan(R.values(*R.quantise(x, R.Q8))).all()


def test_reference_verification_by_hand():
    # one draft, token 0, drawn with q = 1/2; the target gives it 1/4
    p = np.array([[0.25, 0.75, 0], [0, 0, 1]], np.float32)
    q = np.array([[0.5, 0.5, 0], [1, 0, 0]], np.float32)
    args = (2, [9, 0], [-1, 0], p, q)
    assert R.verify(*args, [0, 0.49], 0.9) == ([0, 1], 2)  # 0.245 < 0.25: accepted
    assert R.verify(*args, [0, 0.5], 0.0) == ([0], 1)      # what is left: (0, 1/4, 0)
    assert R.verify(2, [9, 0], [-1, 0], p, None, [0, 0.25], 0.0) == ([0], 1)
    assert R.verify(1, [9], [-1], p, q, [0], 0.25) == ([0], 1)
    assert R.verify(1, [9], [-1], p, q, [0], 0.2499) == ([0], 0)


def test_tree_mask():
    torch = pytest.importorskip("torch")
    import quant_quantized_matvec_gb300 as kq
    assert kq.tree_mask([-1, 0, 0, 1]) == [1, 3, 5, 11]
    deep = kq.tree_mask(list(range(-1, 63)))
    assert deep[63] == -1
    torch.tensor(deep, dtype=torch.int64)
    for bad in ([0], [-2], [-1, 1], [-1] * 65):
        with pytest.raises(ValueError):
            kq.tree_mask(bad)


def test_descriptors_cannot_be_changed():
    """The C structs hold addresses and sizes: an attribute that could be set
    would leave them with those of tensors that are gone, or let smaller
    tensors through the checks than the kernels read."""
    torch = pytest.importorskip("torch")
    import quant_quantized_matvec_gb300 as kq
    for cls, names in ((kq.KVCache, ("fmt", "kv_heads", "head_dim", "pages", "page_bytes", "data")),
                       (kq.KVBatch, ("start", "ctx", "pages", "nseq", "ntok", "max_new"))):
        made = object.__new__(cls)
        made.__dict__.update({n: torch.zeros(3) for n in names})
        for n in names:
            with pytest.raises(AttributeError, match="fixed"):
                setattr(made, n, torch.zeros(2))
            with pytest.raises(AttributeError, match="fixed"):
                delattr(made, n)
            assert getattr(made, n).shape == (3,)
