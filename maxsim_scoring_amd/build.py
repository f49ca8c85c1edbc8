"""Build the HIP library ``libmaxsim_amd.so`` for gfx950 with hipcc.

One shared object holds every kernel and the C ABI of include/maxsim.h. The
library is built in-tree (next to this file) so it travels with the source.
"""

from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmaxsim_amd.so")
# (those that take longest to compile first)
SOURCES = ["embed_linear.hip", "fwd_mx4_wide.hip", "fwd_mx4_short.hip", "fwd_mx4.hip",
           "fwd_mx4_packed.hip", "abi.hip", "fwd_dense.hip", "fwd_varlen.hip", "fwd_dim.hip", "bwd.hip", "topk.hip", "chamfer.hip",
           "embed_abi.hip", "embed_rows.hip", "mx4_abi.hip", "mx4_rows.hip", "mx4_linear.hip",
           "logprob_abi.hip", "logprob.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wno-unused-function",
    # packed fp32 VALU ops stay off in every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # device code: scores are finite or -inf, never NaN; with NaNs not honoured
    # and IEEE mode off, a float max is a single v_max_f32/v_max3_f32 with no
    # canonicalisation of its operands
    "-Xarch_device", "-fno-honor-nans", "-Xarch_device", "-mno-amdgpu-ieee",
    "-I", os.path.join(ROOT, "include"),
]


# Per-source additions. The Chamfer kernel's MFMA results feed VALU min
# updates directly, and those of the 4-bit scores max updates, so they go to
# ordinary VGPRs instead of the accumulation registers (no copy back per MFMA);
# the other kernels keep the compiler's default register form. The embedding
# head carries activations and gradients, where an overflow upstream must stay
# visible: NaNs are honoured there (later flags win), as they are where 4-bit
# rows mark a NaN by their scale and in the log probabilities. They are in the
# top-k too, which keeps k candidates whatever the scores hold.
_NANS = ["-Xarch_device", "-fhonor-nans", "-Xarch_device", "-mamdgpu-ieee"]
EXTRA = {"chamfer.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         "topk.hip": _NANS, "embed_rows.hip": _NANS, "embed_linear.hip": _NANS,
         "mx4_rows.hip": _NANS, "mx4_linear.hip": _NANS, "logprob.hip": _NANS,
         **dict.fromkeys(["fwd_mx4.hip", "fwd_mx4_wide.hip", "fwd_mx4_short.hip",
                          "fwd_mx4_packed.hip"],
                         _NANS + ["-mllvm", "-amdgpu-mfma-vgpr-form"])}


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass warns that it does not know the packed-fp32 feature
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (r.stderr or "").splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compile every kernel source (one object each, in parallel) and link
    them into LIB; always recompiles."""
    from concurrent.futures import ThreadPoolExecutor
    import tempfile
    compile_flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="maxsim_build_") as td:
        objs = [os.path.join(td, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [[HIPCC, *compile_flags, *EXTRA.get(s, []), "-c", "-o", o, os.path.join(CSRC, s)]
                for s, o in zip(SOURCES, objs)]
        with ThreadPoolExecutor(max_workers=min(8, len(cmds))) as ex:
            list(ex.map(lambda c: _run(c, verbose), cmds))
        tmp = LIB + ".tmp%d" % os.getpid()
        _run([HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
