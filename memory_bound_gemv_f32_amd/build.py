"""Build libgemv.so (the HIP kernels and the C ABI) for gfx950 with hipcc.

Run as ``python memory_bound_gemv_f32_amd/build.py`` (a standalone script: it
does not import the package, whose import needs the built library);
``__graft_entry__.build`` loads this file by path and calls :func:`build`.
The library is written next to this file, in-tree.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from pathlib import Path

PACKAGE = Path(__file__).resolve().parent
ROOT = PACKAGE.parent
CSRC = PACKAGE / "csrc"
SOURCES = [CSRC / "gemv_api.hip", CSRC / "fp8_api.hip", CSRC / "kv_api.hip", CSRC / "q4_api.hip",
           CSRC / "rotary_api.hip"]
HEADERS = [CSRC / "gemv_plan.hpp", CSRC / "gemv_device.hpp",
           CSRC / "gemv_kernels.hpp", CSRC / "gemv_launch.hpp",
           CSRC / "fp8_device.hpp", CSRC / "fp8_kernels.hpp",
           CSRC / "kv_kernels.hpp", CSRC / "kv_plan.hpp", CSRC / "q4_kernels.hpp", CSRC / "q4_plan.hpp",
           CSRC / "rotary_kernels.hpp", ROOT / "include" / "gemv.h"]
LIBRARY = PACKAGE / "libgemv.so"
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # no packed fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # kernel arguments arrive preloaded in SGPRs (gfx950), so a kernel's
    # first loads do not wait on scalar loads of its argument block
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = shutil.which("hipcc") or os.path.join(rocm, "bin", "hipcc")
    return path


def build(verbose: bool = False, extra_flags: list[str] | None = None,
          output: Path = LIBRARY) -> Path:
    """Compile every HIP source into ``libgemv.so`` (always recompiles)."""
    tmp = output.with_name(f"{output.name}.tmp{os.getpid()}")
    flags = [*HIPCC_FLAGS, *(extra_flags or [])]
    with tempfile.TemporaryDirectory(prefix="libgemv_") as folder:
        # the sources side by side, then one link
        objects = [Path(folder) / f"{s.stem}.o" for s in SOURCES]
        cmds = [[hipcc(), *flags, "-c", str(s), "-o", str(o)]
                for s, o in zip(SOURCES, objects)]
        running = []
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append(subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT, text=True))
        texts = [p.communicate()[0] for p in running]
        failed = any(p.returncode != 0 for p in running)
        if not failed:
            cmd = [hipcc(), *flags, "-shared", *[str(o) for o in objects], "-o", str(tmp)]
            if verbose:
                print(" ".join(cmd), flush=True)
            link = subprocess.run(cmd, capture_output=True, text=True)
            texts.append(link.stdout + link.stderr)
            failed = link.returncode != 0
    # hipcc's host pass does not know the packed-fp32 feature; that warning
    # is expected, anything else is shown
    noise = "is not a recognized feature for this target"
    msgs = [ln for text in texts for ln in text.splitlines()
            if noise not in ln and "(ignoring feature)" not in ln and ln.strip()]
    if failed:
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), file=sys.stderr)
    os.replace(tmp, output)
    return output


def is_stale() -> bool:
    if not LIBRARY.exists():
        return True
    t = LIBRARY.stat().st_mtime
    return any(p.stat().st_mtime > t for p in SOURCES + HEADERS)


if __name__ == "__main__":
    build(verbose=True)
    print(LIBRARY)
