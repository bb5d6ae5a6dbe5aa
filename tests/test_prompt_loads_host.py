"""What a kernel of the prompt's attention reads of another that is still at work
when it begins: by plain loads or copies, after the wait for it.  (No run shows the
difference where the wait comes first, so the source is looked at.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "quant_quantized_matvec_gb300", "csrc")
# written by kq_prompt_split and the kernels that write parts
WRITTEN = r"\b(info|powers|part|tiles|p->|kstate|vstate|ek|vf)\b"


def test_no_load_of_constant_memory_from_what_is_written_beside():
    found = 0
    for name in ("kq_prompt_attn.cuh", "kq_prompt_pairs.cuh", "kq_prompt_attn.cu"):
        with open(os.path.join(CSRC, name)) as f:
            src = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"(__ldg|__ldcs|ld\.global\.nc)", src):
            line = src[src.rfind("\n", 0, m.start()) + 1:src.find(";", m.end())]
            assert not re.search(WRITTEN, line), (name, line)
            found += 1
    assert found  # (inputs are read so)


def test_the_wait_comes_before_the_first_load():
    with open(os.path.join(CSRC, "kq_prompt_attn.cuh")) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    rows = src[src.index("kq_prompt_rows("):]
    wait = rows.rindex("kq::wait_prerequisites()")  # (the one before: of CTAs without an item)
    for name in ("a.info", "a.powers", "a.tiles"):
        assert rows.index(name) > wait, name
