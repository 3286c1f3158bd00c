"""Builds libfa_gb300.so in-tree with nvcc for sm_103a.

The library's translation units (``UNITS``) compile side by side; the ptxas
resource report of the last build is kept in ``_build/ptxas.txt`` at the
repository root.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import tempfile

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libfa_gb300.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
# the same sources with the device-side invariant checks (FA_DEBUG = 1)
DEBUG_LIB_PATH = os.path.join(PKG_DIR, "libfa_gb300_debug.so")
DEBUG_FLAGS = ["-DFA_DEBUG=1"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
UNITS = ("fa_api.cu", "fa_kv4.cu")
COMPILE_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa_gb300.so")


def _sources():
    deps = [os.path.join(INCLUDE, "fa_gb300.h")]
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            deps.append(os.path.join(CSRC, name))
    return deps


STAMP_PATH = LIB_PATH + ".sha256"

# The native marshalling of the cache calls (csrc/fa_binding.cpp): a Python
# extension against the installed torch.  Without it (no compiler or headers
# for it) the same calls are marshalled in Python.
BINDING_PATH = os.path.join(PKG_DIR, "fa_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "fa_binding.cpp")


def binding_command() -> list[str]:
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    lib = os.path.join(root, "lib")
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], cuda, INCLUDE]
    return [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for d in include for x in ("-isystem", d)], BINDING_SOURCE, "-o", BINDING_PATH + ".tmp",
            "-L" + lib, "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def binding_stamp() -> str:
    """What a built binding belongs to: its sources, this Python, torch and machine."""
    import hashlib
    import platform
    import sys
    import torch
    h = hashlib.sha256(f"{sys.version}|{torch.__version__}|{platform.machine()}".encode())
    for path in (BINDING_SOURCE, os.path.join(INCLUDE, "fa_gb300.h")):
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def binding_built() -> bool:
    stamp = BINDING_PATH + ".sha256"
    if not (os.path.exists(BINDING_PATH) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        return f.read().strip() == binding_stamp()


def _start_binding():
    """The running compiler, or None (the binding is built, or cannot be)."""
    try:
        if binding_built():
            return None
        os.makedirs(os.path.join(ROOT, "_build"), exist_ok=True)
        log = open(os.path.join(ROOT, "_build", "binding.txt"), "w")
        return subprocess.Popen(binding_command(), stdout=log, stderr=subprocess.STDOUT)
    except (ImportError, OSError, RuntimeError):
        return None


def _finish_binding(run) -> None:
    if run is not None and run.wait() == 0:
        os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
        with open(BINDING_PATH + ".sha256", "w") as f:
            f.write(binding_stamp() + "\n")


def source_hash(debug: bool = False) -> str:
    """SHA-256 over the library's sources (names and contents), the compile
    command's flags and this machine's architecture: the stamp a built
    library must carry to be reused."""
    import hashlib
    import platform
    h = hashlib.sha256()
    h.update(" ".join(ARCH_FLAGS + COMPILE_FLAGS + (DEBUG_FLAGS if debug else [])).encode())
    h.update(platform.machine().encode())
    for path in _sources():
        with open(path, "rb") as f:
            h.update(os.path.basename(path).encode() + b"\0" + f.read())
    return h.hexdigest()


def needs_build(debug: bool = False) -> bool:
    """True unless the library exists and its stamp matches the sources (file
    times are not trusted: a copied tree can carry a library newer than
    sources it was not built from)."""
    lib = DEBUG_LIB_PATH if debug else LIB_PATH
    stamp = lib + ".sha256"
    if not (os.path.exists(lib) and os.path.exists(stamp)):
        return True
    with open(stamp) as f:
        return f.read().strip() != source_hash(debug)


# Registers per thread the attention kernel must launch with, by its last
# template argument (softmax threads per row): its warpgroups re-split this
# budget with setmaxnreg (fa_fwd_kernel.cuh, WarpLayout::kLaunchRegs), and a
# smaller launch budget would leave the increasing warpgroups waiting for
# registers that never come.
KERNEL_LAUNCH_REGS = {1: 168, 2: 96}
# The same for prompt_kernel of the quantised cache, for heads of at most 4
# groups of 32 (kv4_prompt.cuh, Prompt::kLaunchRegs); wider ones do not re-split.
PROMPT_LAUNCH_REGS, PROMPT_RESPLIT_GROUPS = 96, 4


def _expected_regs(mangled: str) -> int:
    m = re.search(r"fa_fwd_kernelILi\d+ELb[01]ELi\d+ELi(\d+)(?:ELb[01]|ELi\d+)?EE", mangled)
    if not m:
        raise RuntimeError(f"cannot read the template arguments of {mangled}")
    return KERNEL_LAUNCH_REGS[int(m.group(1))]


def check_launch_registers(ptxas_log: str) -> None:
    """Raise unless every fa_fwd_kernel and prompt_kernel instantiation
    launches with the register count its setmaxnreg split assumes."""
    current = None
    seen = 0
    for line in ptxas_log.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            current = m.group(1)
            continue
        m = re.search(r"Used (\d+) registers", line)
        if m and current is not None:
            prompt = re.search(r"13prompt_kernelILi(\d+)E", current)
            want = None
            if "fa_fwd_kernel" in current:
                seen += 1
                want = _expected_regs(current)
            elif prompt and int(prompt.group(1)) <= PROMPT_RESPLIT_GROUPS:
                want = PROMPT_LAUNCH_REGS
            if want is not None:
                if int(m.group(1)) != want:
                    raise RuntimeError(
                        f"{current} uses {m.group(1)} registers per thread, not "
                        f"{want}: its setmaxnreg split would not fit")
            current = None
    if seen == 0:
        raise RuntimeError("no fa_fwd_kernel register report in the ptxas output")


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile the library unless it exists with the stamp of the current
    sources; ``debug`` builds libfa_gb300_debug.so, the same sources with the
    device-side invariant checks (FA_DEBUG = 1)."""
    binding = None if debug else _start_binding()
    try:
        return _build_library(force, verbose, debug)
    finally:
        _finish_binding(binding)


def _build_library(force: bool, verbose: bool, debug: bool) -> str:
    lib = DEBUG_LIB_PATH if debug else LIB_PATH
    if not force and not needs_build(debug):
        return lib
    out_dir = os.path.join(ROOT, "_build")
    os.makedirs(out_dir, exist_ok=True)
    tmp = lib + ".tmp"
    stamp = source_hash(debug)
    compile_flags = [f for f in COMPILE_FLAGS if f != "-shared"]
    objs, cmds = [], []
    for unit in UNITS:
        objs.append(os.path.join(out_dir, unit + (".debug.o" if debug else ".o")))
        cmds.append([_nvcc(), *ARCH_FLAGS, *compile_flags, *(DEBUG_FLAGS if debug else []), "-Xptxas", "-v",
                     "-I", INCLUDE, "-c", "-o", objs[-1], os.path.join(CSRC, unit)])
    outs = [tempfile.TemporaryFile("w+") for _ in cmds]
    runs = [subprocess.Popen(cmd, stdout=out, stderr=subprocess.STDOUT) for cmd, out in zip(cmds, outs)]
    logs = []
    for run, out in zip(runs, outs):
        run.wait()
        out.seek(0)
        logs.append(out.read())
        out.close()
    with open(os.path.join(out_dir, "ptxas_debug.txt" if debug else "ptxas.txt"), "w") as f:
        for cmd, log in zip(cmds, logs):
            f.write(" ".join(cmd) + "\n" + log)
    for run, log in zip(runs, logs):
        if run.returncode != 0:
            raise RuntimeError(f"nvcc failed ({run.returncode}):\n{log[-4000:]}")
    link = subprocess.run([_nvcc(), *ARCH_FLAGS, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs],
                          capture_output=True, text=True)
    if link.returncode != 0:
        raise RuntimeError(f"nvcc failed to link ({link.returncode}):\n{link.stderr[-4000:]}")
    try:
        check_launch_registers("".join(logs))
    except RuntimeError:
        os.remove(tmp)
        raise
    os.replace(tmp, lib)
    with open(lib + ".sha256", "w") as f:
        f.write(stamp + "\n")
    if verbose:
        print("".join(logs))
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
