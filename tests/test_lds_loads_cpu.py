"""Hazards of hand-written instructions that the compiler cannot see, checked in the sources."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _asm_blocks():
    """(file, instructions) of every asm statement of the device sources."""
    for path in sorted(glob.glob(os.path.join(ROOT, "maxsim_scoring_amd", "csrc", "*.h*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read()).replace("\\\n", "\n")
        # its strings, and the macros' parameters between them
        for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(((?:\s*(?:\"(?:[^\"\\]|\\.)*\"|[A-Z]\w*))+)", text):
            code = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))
            yield os.path.basename(path), [i.strip() for i in re.split(r"\\n\\t|\\n|;", code) if i.strip()]


def _wait_states(instructions):
    return sum(int(i.split()[1]) + 1 if i.startswith("s_nop") else 1 for i in instructions)


def test_loads_to_lds_hold_their_wait_states():
    """A load to LDS takes its address from M0, which a scalar instruction must
    have written one wait state before, and its base from scalar registers, which
    a vector instruction (the last one before the block, for all we know) must
    have written five before."""
    seen = 0
    for name, code in _asm_blocks():
        for i, ins in enumerate(code):
            if not ins.startswith(("global_load_lds", "buffer_load")):
                continue
            seen += 1
            m0 = [j for j in range(i) if re.match(r"s_\w+\s+m0\s*,", code[j])]
            assert m0, f"{name}: M0 is written elsewhere: {code}"
            assert _wait_states(code[m0[-1] + 1:i]) >= 1, f"{name}: {code}"
            assert _wait_states(code[:i]) >= 5, f"{name}: {code}"
    assert seen >= 7
