"""The prompt's entry points on the host, without a GPU: exports, and the
refusal of bad arguments before any CUDA call (fake addresses that are never
dereferenced)."""
import ctypes
import os
import re

import pytest

from quant_quantized_matvec_gb300 import _binding
from quant_quantized_matvec_gb300 import build as kbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, FORMAT, SHAPE, NTOK, NULL, ALIGN, ALIAS, CUDA, TIMEOUT, COUNT, LIMIT, MEMORY = range(12)
A = [0x7f0000000000 + (i << 36) for i in range(16)]  # far apart, well aligned
F32, F16, BF16 = 0, 1, 30


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _binding.load()


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "kq_prompt.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(kq_[a-z_]+)\s*\(", src))
    assert names == set(_binding.PROMPT_SYMBOLS)
    for n in names:
        assert hasattr(lib, n)


def part(**kw):
    d = dict(x=A[0], stride=512, weight=A[1], out=A[2], out_stride=512, heads=4, reserved=0)
    d.update(kw)
    return _binding.KqNormPart(**d)


def norm(lib, *parts, n=None, kind=F32, out=F32, ntok=5, dim=128, eps=1e-6, pos=A[6], table=A[7],
         npos=9, rot=64):
    parts = parts or (part(),)
    p = (_binding.KqNormPart * len(parts))(*parts)
    return lib.kq_norm_rope(p, len(parts) if n is None else n, kind, out, ntok, dim, eps, pos,
                            table, npos, rot, 0, None)


def test_norm_refusals(lib):
    for kw, st in [(dict(n=0), COUNT), (dict(n=5), COUNT), (dict(kind=2), FORMAT),
                   (dict(out=8), FORMAT), (dict(kind=F16, out=F32), FORMAT),
                   (dict(kind=BF16, out=F16), FORMAT), (dict(dim=124), SHAPE), (dict(dim=0), SHAPE),
                   (dict(dim=1032), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
                   (dict(eps=float("inf")), SHAPE), (dict(rot=4), SHAPE), (dict(rot=132), SHAPE),
                   (dict(rot=136), SHAPE), (dict(npos=0), SHAPE), (dict(ntok=-1), NTOK),
                   (dict(ntok=(1 << 24) + 1), NTOK), (dict(pos=None), NULL),
                   (dict(pos=A[6] + 2), ALIGN), (dict(table=A[7] + 4), ALIGN),
                   (dict(table=A[2]), ALIAS), (dict(pos=A[2] + 64), ALIAS)]:
        assert norm(lib, **kw) == st, kw
    for kw, st in [(dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(reserved=1), SHAPE),
                   (dict(stride=511), SHAPE), (dict(stride=514), SHAPE), (dict(out_stride=508), SHAPE),
                   (dict(x=None), NULL), (dict(out=None), NULL), (dict(x=A[0] + 4), ALIGN),
                   (dict(weight=A[1] + 8), ALIGN), (dict(out=A[2] + 8), ALIGN),
                   (dict(out=A[0] + 16), ALIAS), (dict(out=A[0], out_stride=1024), ALIAS),
                   (dict(out=A[1]), ALIAS)]:
        assert norm(lib, part(**kw)) == st, kw
    # 16-bit types: strides in multiples of eight values
    assert norm(lib, part(stride=516), kind=F16, out=F16) == SHAPE
    assert norm(lib, part(out_stride=516), out=BF16) == SHAPE
    # a smaller type is not in place
    assert norm(lib, part(out=A[0]), out=F16) == ALIAS
    # outputs that meet; one that meets the other's input
    assert norm(lib, part(), part(x=A[3], out=A[2] + 16)) == ALIAS
    assert norm(lib, part(), part(x=A[3], out=A[0])) == ALIAS
    assert norm(lib, ntok=0, pos=None) == OK


def attend(lib, kind=F32, nseq=2, n=9, m=20, start=A[0], ks=A[1], q=A[2], qs=512, hq=4, k=A[3], kst=256,
           v=A[4], vst=256, hkv=2, dim=128, scale=0.1, out=A[5], ws=None, wn=0):
    return lib.kq_prompt_attention(kind, nseq, n, m, start, ks, q, qs, hq, k, kst, v, vst, hkv, dim, scale,
                                   out, ws, wn, None)


def test_attention_refusals(lib):
    for kw, st in [(dict(kind=8), FORMAT), (dict(nseq=0), COUNT), (dict(nseq=4097), COUNT),
                   (dict(n=-1), NTOK), (dict(n=(1 << 24) + 1), NTOK), (dict(m=-1), NTOK),
                   (dict(m=(1 << 24) + 1), NTOK), (dict(ks=None), NTOK), (dict(hq=3), SHAPE),
                   (dict(hq=0), SHAPE), (dict(hkv=0), SHAPE), (dict(hq=1026), SHAPE), (dict(dim=96), SHAPE),
                   (dict(qs=508), SHAPE), (dict(qs=514), SHAPE), (dict(kst=255), SHAPE),
                   (dict(vst=258), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(start=None), NULL),
                   (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL),
                   (dict(start=A[0] + 2), ALIGN), (dict(q=A[2] + 8), ALIGN), (dict(v=A[4] + 4), ALIGN),
                   (dict(out=A[5] + 4), ALIGN), (dict(ws=A[6] + 16, wn=1 << 30), ALIGN),
                   (dict(kind=BF16, qs=516), SHAPE), (dict(kind=F16, kst=260), SHAPE)]:
        assert attend(lib, **kw) == st, kw
    assert attend(lib, n=0, q=None) == OK


def test_workspace_refusals(lib):
    f = lib.kq_prompt_workspace_bytes
    assert f(8, 1, 9, 9, 4, 2, 128) == -FORMAT and f(F32, 0, 9, 9, 4, 2, 128) == -COUNT
    assert f(F32, 1, -1, 9, 4, 2, 128) == -NTOK and f(F32, 1, 9, 9, 3, 2, 128) == -SHAPE
    assert f(F32, 1, 9, 9, 4, 2, 96) == -SHAPE and f(F32, 1, 0, 9, 4, 2, 128) == 0


def test_logprob_refusals(lib):
    def score(kind=F32, n=5, v=1000, x=A[0], xs=1000, tok=A[1], top=3, lp=A[2], ent=A[3], tl=A[4], tt=A[5]):
        return lib.kq_token_logprobs(kind, n, v, x, xs, tok, top, lp, ent, tl, tt, None)

    for kw, st in [(dict(kind=3), FORMAT), (dict(n=-1), NTOK), (dict(n=(1 << 24) + 1), NTOK),
                   (dict(v=0), SHAPE), (dict(v=(1 << 19) + 1, xs=1 << 20), SHAPE), (dict(xs=999), SHAPE),
                   (dict(top=-1), SHAPE), (dict(top=33), SHAPE), (dict(v=2, top=3), SHAPE),
                   (dict(x=None), NULL), (dict(tok=None), NULL), (dict(lp=None), NULL), (dict(tl=None), NULL),
                   (dict(tt=None), NULL), (dict(tok=None, lp=None, ent=None, top=0), NULL),
                   (dict(x=A[0] + 2), ALIGN), (dict(kind=BF16, x=A[0] + 1), ALIGN), (dict(tok=A[1] + 2), ALIGN),
                   (dict(ent=A[3] + 1), ALIGN), (dict(tt=A[5] + 3), ALIGN), (dict(lp=A[0] + 64), ALIAS),
                   (dict(ent=A[1]), ALIAS), (dict(tt=A[4] + 8), ALIAS)]:
        assert score(**kw) == st, kw
    assert score(n=0, x=None, tok=None) == OK


def test_struct_matches_the_header():
    assert ctypes.sizeof(_binding.KqNormPart) == 48
    torch = pytest.importorskip("torch")  # noqa: F841 (the wrapper's packing needs it)
    from quant_quantized_matvec_gb300 import prompt
    packed = prompt._pack_part(1, 2, 3, 4, 5, 6, 0)
    assert packed == bytes(_binding.KqNormPart(1, 2, 3, 4, 5, 6, 0))


def test_python_checks():
    torch = pytest.importorskip("torch")
    import quant_quantized_matvec_gb300 as kq
    x = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        kq.norm_rope(x.double())
    with pytest.raises(ValueError, match="q must be"):
        kq.norm_rope(x[0])
    with pytest.raises(ValueError, match="tokens, heads, dim"):
        kq.prompt_attention(x[0], x, x, None)
    with pytest.raises(ValueError, match="n, vocab"):
        kq.token_logprobs(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kq.token_logprobs(x[0])
