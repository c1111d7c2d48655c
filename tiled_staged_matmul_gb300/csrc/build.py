"""Build ``libtsm_gemm.so`` in-tree with nvcc for sm_103a only, and with the host
compiler, where torch is installed, the extension module that passes torch tensors to
some of its calls.

The translation units compile in parallel: the plain GEMM kernels and the
cluster split-K sums, the fused-epilogue GEMM kernels once per activation
(``gemm_epi.cu`` with ``-DTSM_EPI_ACT``), the row-reduction kernels, the
expert token movement, the choice of experts once per type of the logits, the
8-bit integer and the 4-bit products and the host API.  The kernel units are compiled with ``-Xptxas -v`` and the build
fails if ptxas reports any spill stores or loads (only ptxas's printed
summary is read).
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
REPO = os.path.dirname(PKG)
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libtsm_gemm.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
CALLS_PATH = os.path.join(BUILD_DIR, "tsm_tensor_calls.so")
CALLS_SOURCE = "tensor_calls.cpp"
CALLS_STAMP = os.path.join(BUILD_DIR, "tsm_tensor_calls.abi")
PTXAS_LOG = os.path.join(BUILD_DIR, "ptxas.log")

# (source, object name, extra nvcc flags); the activations are gemm_internal.h's kAct* values
ACTIVATIONS = ["none", "relu", "leaky_relu", "gelu", "gelu_tanh", "silu"]
UNITS = ([("gemm_kernels.cu", "gemm_kernels", [])] +
         [("gemm_epi.cu", f"gemm_epi_{a}", [f"-DTSM_EPI_ACT={i}"]) for i, a in enumerate(ACTIVATIONS)] +
         [("rowsum_kernels.cu", "rowsum_kernels", []), ("moe_kernels.cu", "moe_kernels", []),
          ("s8_kernels.cu", "s8_kernels", [])] +
         [("s8_tiled.cu", f"s8_tiled_{a}", [f"-DTSM_S8_ACT={i}"]) for i, a in enumerate(ACTIVATIONS)] +
         [("choose_kernels.cu", f"choose_{t}", [f"-DTSM_CHOOSE_ELEM={i}"]) for i, t in enumerate(("f32", "f16", "bf16"))] +
         [("fp4_quantize.cu", "fp4_quantize", []), ("fp4_product.cu", "fp4_product", [])] +
         [("gemm_api.cu", "gemm_api", []), ("ops_api.cu", "ops_api", []), ("fp4_api.cu", "fp4_api", [])])
HOST_SOURCES = ("gemm_api.cu", "ops_api.cu", "fp4_api.cu")
SOURCES = sorted({u[0] for u in UNITS})
HEADERS = ["api_checks.h", "api_internal.h", "fp4_internal.h", "fp4_plan.h", "fp4_ptx.cuh", "gemm_internal.h",
           "gemm_kernel.cuh", "launch.cuh", "ops_internal.h", "piece.cuh", "ptx.cuh", "s8_common.cuh", "s8_plan.h", "s8_ptx.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def _inputs() -> list[str]:
    files = [os.path.join(HERE, f) for f in SOURCES + HEADERS + [CALLS_SOURCE]]
    files.append(os.path.join(REPO, "include", "tsm_gemm.h"))
    files.append(os.path.abspath(__file__))
    return files


def calls_abi() -> str | None:
    """What the extension module is compiled against and works with alone: this Python's
    ABI and the installed torch (found, not imported); None where there is no torch."""
    torch = importlib.util.find_spec("torch")
    if torch is None or torch.origin is None:  # (a folder of that name is none)
        return None
    torch_dir = os.path.dirname(torch.origin)
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "\n".join([str(sysconfig.get_config_var("EXT_SUFFIX")), torch_dir, f.read()])


def calls_match() -> bool:
    """Whether the extension module that is there was compiled against these."""
    if not os.path.exists(CALLS_PATH) or not os.path.exists(CALLS_STAMP):
        return False
    with open(CALLS_STAMP) as f:
        return f.read() == calls_abi()


def up_to_date() -> bool:
    outputs = [LIB_PATH]
    if calls_abi() is not None:
        if not calls_match():
            return False
        outputs.append(CALLS_PATH)
    if not os.path.exists(LIB_PATH):
        return False
    t = min(os.path.getmtime(f) for f in outputs)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _compile(src: str, obj: str, verbose_ptxas: bool, flags: list[str]) -> str:
    cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", *flags,
           "-I", os.path.join(REPO, "include"), "-c", os.path.join(HERE, src), "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile_calls(obj: str) -> list[str]:
    """Compile the extension module's unit; the command that links it."""
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for i in inc for x in ("-isystem", i)], "-c", os.path.join(HERE, CALLS_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return ["g++", "-shared", obj, "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-L" + BUILD_DIR, "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN"]


def check_spills(log: str) -> None:
    bad = [ln for ln in log.splitlines()
           if re.search(r"(\d+) bytes spill (stores|loads)", ln)
           and not re.search(r"\b0 bytes spill stores, 0 bytes spill loads", ln)]
    if bad:
        raise RuntimeError("ptxas reports register spills:\n" + "\n".join(bad))


def build(force: bool = False, quiet: bool = True) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = [os.path.join(BUILD_DIR, name + ".o") for _, name, _ in UNITS]
    kernel_unit = [src not in HOST_SOURCES for src, _, _ in UNITS]
    with ThreadPoolExecutor(len(UNITS) + 1) as ex:
        abi = calls_abi()
        calls = abi and ex.submit(_compile_calls, os.path.join(BUILD_DIR, "tensor_calls.o"))
        logs = list(ex.map(lambda a: _compile(*a),
                           [(src, o, k, fl) for (src, _, fl), o, k in zip(UNITS, objs, kernel_unit)]))
    ptxas = "".join(log for log, k in zip(logs, kernel_unit) if k)
    with open(PTXAS_LOG, "w") as f:
        f.write(ptxas)
    check_spills(ptxas)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if calls:
        tmp = CALLS_PATH + f".tmp{os.getpid()}"
        r = subprocess.run(calls.result() + ["-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, CALLS_PATH)
        with open(CALLS_STAMP, "w") as f:
            f.write(abi)
    if not quiet:
        print(logs[0], file=sys.stderr)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, quiet=False))
