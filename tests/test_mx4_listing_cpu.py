"""The block-scaled matrix instruction takes its scales from the lanes that EXEC enables,
which the compiler does not know: results of the 4-bit scores are held where all lanes
get to. Checked in the sources, and in the listing of a kernel built here."""

import glob
import os
import re
import subprocess

import pytest

from maxsim_scoring_amd import build

PROBE = """
#include "mx4_common.hpp"
using namespace maxsim;
__global__ void probe(const i32x4* q, const i32x4* d, const int* sq, const int* sd, const float* keep, float* out)
{
    const int l = lane_id();
    f32x16 acc;
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
    acc = mfma32_mx4<0, 0>(d[l], sd[l], q[l], sq[l], acc);
    stay(acc);
    if (keep[l] > 0.0f) {
        float m = acc[0];
        for (int e = 1; e < 16; ++e) m = __builtin_fmaxf(m, acc[e]);
        out[l] = m;
    }
}
"""


def test_scores_hold_their_results():
    """Every chain of products of the score kernels ends in stay()."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "fwd_mx4*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"static_for<0, G>\(\[&\]\(auto g\) \{\s*(\w+) = mfma32_mx4[^}]*\}\);\s*(\w+\(\w+\);)?", text):
            assert m.group(2) == f"stay({m.group(1)});", f"{os.path.basename(path)}: {m.group(0)}"
            seen += m.group(0).count("mfma32_mx4<")
        seen -= text.count("mfma32_mx4<")
    assert seen == 0, "products outside the chains that were looked at"


def test_a_result_that_some_lanes_use_is_computed_by_all(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    src, out = tmp_path / "probe.hip", tmp_path / "probe.s"
    src.write_text(PROBE)
    flags = [f for f in build.FLAGS if f != "-shared"] + build.EXTRA["fwd_mx4.hip"]
    subprocess.run([build.HIPCC, *flags, "-I", build.CSRC, "--cuda-device-only", "-S", "-o", str(out), str(src)],
                   check=True, capture_output=True)
    code = [i.strip() for i in out.read_text().splitlines()]
    product = [k for k, i in enumerate(code) if i.startswith("v_mfma_scale")]
    narrowed = [k for k, i in enumerate(code) if re.match(r"s_\w*saveexec|s_\w+ exec,", i)]
    assert len(product) == 1 and narrowed and product[0] < narrowed[0]


def test_kernels_call_no_functions():
    """The parts of a kernel are inlined into it. In one that is called, what is uniform for
    the kernel arrives in each lane's registers: its branches narrow EXEC, and what it takes
    by reference lies in scratch memory."""
    from maxsim_scoring_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    text = open(binding.LIB_PATH, "rb").read()
    assert re.search(rb"_ZN6maxsim\w*fwd_mx4_kernel\w*", text)
    assert not set(re.findall(rb"_ZZN6maxsim\w*_kernel\w*_cl\w*", text))
