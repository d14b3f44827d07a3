"""Build the gfx950 HIP library ``libssm.so`` in-tree with hipcc.

    python -m selective_state_space_35_amd.build

Flags: gfx950 only; packed-FP32 instruction selection is disabled
(``-Xclang -target-feature -Xclang -packed-fp32-ops``) so the compiler emits
only scalar-lane FP32 VALU ops; host symbols are hidden except the C ABI.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libssm.so")
CALIB_SRC = os.path.join(PKG, "calib", "ssm_calib.hip")
CALIB_LIB = os.path.join(PKG, "libssm_calib.so")
SOURCES = ["ssm_kernels.hip", "ssm_fused.hip", "ssm_conv.hip", "ssm_bwd.hip", "ssm_ssd.hip", "ssm_api.hip", "ssm_profile.hip",
           "ssm_noalloc.hip", "ssm_linattn.hip", "ssm_layernorm.hip"]
ARCH = os.environ.get("SSM_OFFLOAD_ARCH", "gfx950")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature: harmless
    noise = [ln for ln in (r.stdout + r.stderr).splitlines() if ln.strip() and "packed-fp32-ops" not in ln]
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(noise))
    if verbose and noise:
        print("\n".join(noise), flush=True)


def build(verbose: bool = False, out: str = LIB, defines=()) -> str:
    """Compile and link libssm.so.  ``defines`` (e.g. ["SSM_KGROUP=4"]) override tuning macros."""
    objdir = os.path.join(PKG, "_build" if not defines else "_build_" + "_".join(d.replace("=", "") for d in defines))
    os.makedirs(objdir, exist_ok=True)
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".hip", ".o"))
        objs.append(obj)
        cmds.append([HIPCC, *COMMON, *[f"-D{d}" for d in defines], "-c", os.path.join(CSRC, src), "-o", obj])
    with ThreadPoolExecutor(max_workers=len(cmds)) as ex:
        list(ex.map(lambda c: _run(c, verbose), cmds))
    tmp = out + ".tmp"
    _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
    os.replace(tmp, out)
    return out


def build_calib(verbose: bool = False, out: str = CALIB_LIB) -> str:
    """Compile libssm_calib.so: the issue-rate calibration kernels (benchmark support), same flags."""
    tmp = out + ".tmp"
    _run([HIPCC, *COMMON, "-shared", CALIB_SRC, "-o", tmp], verbose)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose="-q" not in sys.argv))
    print(build_calib(verbose="-q" not in sys.argv))
