"""Items of numbers in any order: a CTA takes over the numbers of others as
launch control gives them, which promises no order."""
import ctypes
import os
import random
import subprocess

import pytest

from quant_quantized_matvec_gb300 import build as kbuild

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def items(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("items") / "prompt_items.so")
    subprocess.run([kbuild.nvcc(), kbuild.ARCH, "-O1", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
                    "-I", kbuild.INCLUDE, "-I", kbuild.CSRC, os.path.join(HERE, "prompt_items.cu"), "-o", so],
                   check=True)
    return ctypes.CDLL(so).prompt_items


def expected(new, tok, kv_heads, per, hb):
    """Items by number: a sequence's last block of tokens first, then by heads."""
    out, hblocks = [], -(-per // hb)
    for b, n in enumerate(new):
        for at in reversed(range(-(-n // tok))):
            for h in range(kv_heads * hblocks):
                first = at * tok
                out.append((b, first, min(tok, n - first), h // hblocks,
                            h // hblocks * per + h % hblocks * hb, min(n, first + min(tok, n - first))))
    return out


@pytest.mark.parametrize("order", ["rising", "falling", "shuffled", "past the last ones first"])
@pytest.mark.parametrize("nseq,most,splits,per,hb", [(1, 700, 1, 1, 1), (9, 300, 3, 4, 4), (33, 60, 1, 3, 2),
                                                      (150, 40, 2, 1, 1), (700, 5, 1, 1, 1)])
def test_items_in_any_order(items, nseq, most, splits, per, hb, order):
    rng = random.Random(nseq)
    tok, kv_heads = 16, 2
    new = [rng.randrange(most + 1) for _ in range(nseq)]
    want = expected(new, tok, kv_heads, per, hb)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    there = len(want) * splits
    numbers = list(range(there + 40))
    if order == "falling":
        numbers.reverse()
    elif order == "shuffled":
        rng.shuffle(numbers)
    elif order == "past the last ones first":
        numbers = numbers[there:] + numbers[:there]
    sd, nd = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (start, numbers))
    out = torch.full((len(numbers) + 1, 7), -9, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert items(ctypes.c_void_p(sd.data_ptr()), nseq, start[-1], tok, kv_heads, per, hb, splits,
                 ctypes.c_void_p(nd.data_ptr()), len(numbers), ctypes.c_void_p(out.data_ptr())) == 0
    got = out.tolist()
    asked = [u for u in numbers if u < there]
    assert [r[0] for r in got[:there]] == asked and got[there][0] == -1
    assert [tuple(r[1:]) for r in got[:there]] == [want[u // splits] for u in asked]
