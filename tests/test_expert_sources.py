"""What the experts' kernels may not do because they start while the kernel before them runs, checked on their source.

Such a kernel's inputs are ready after griddepcontrol.wait.  An asm statement that is not volatile, a load by the
read-only path and an access through a __restrict__ pointer are all free to move above that wait."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lossless_bf16_compression_gb300", "csrc", "experts")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
            yield name, text


def test_loads_stay_behind_the_wait():
    seen = 0
    for name, text in sources():
        for m in re.finditer(r"\basm\b(\s+volatile)?\s*\((.*?)\)\s*;", text, flags=re.S):
            code = " ".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(2)))
            if re.search(r"\b(ld|st|atom|red|cp|mbarrier|tcgen05)\.", code) or "griddepcontrol" in code:
                assert m.group(1), (name, m.group(0))
                seen += 1
        assert "__restrict__" not in text, name
        assert not re.search(r"\bld\.global\.nc\b|\b__ldg\s*\(", text), name
    assert seen > 10


def test_the_wait_is_a_barrier_to_the_compiler():
    text = dict(sources())["ex_common.cuh"]
    assert re.search(r'asm volatile\("griddepcontrol\.wait;"\s*:::\s*"memory"\)', text)
