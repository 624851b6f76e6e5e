"""Build libmoe_decode.so in-tree with nvcc for sm_103a (no cmake; the decode
layer, the prompt operators and the block operators are one translation unit
each, compiled side by side), and with g++ the extension module _moe_torch.so,
which passes torch tensors to the prompt and block operators.

    python -m sparse_expert_gemv_gb300.build
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", f) for f in ("moe_decode.cu", "moe_prompt.cu", "moe_block.cu")]
OUT = os.path.join(HERE, "libmoe_decode.so")
# the same library with the one-launch kernel's per-CTA timeline compiled in
# (-DMOE_TIMELINE: globaltimer stamps per CTA and phase, written to a
# caller-supplied buffer by moe_decode_layer_timeline); never loaded by the
# package itself
OUT_TIMELINE = os.path.join(HERE, "libmoe_decode_timeline.so")
BINDING_SRC = os.path.join(HERE, "csrc", "moe_torch.cpp")
BINDING_OUT = os.path.join(HERE, "_moe_torch.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def command(out: str = OUT, extra=()) -> list[str]:
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "lib64")
    return [nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
            "-cudart", "shared", f"-I{os.path.join(ROOT, 'include')}",
            f"-Xlinker", f"-rpath,{cuda_lib}", "--threads", "0", *extra, *SRCS, "-o", out]


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def torch_version() -> str:
    """torch.__version__, without importing torch."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)


def built_for(version: str) -> str:
    """What the extension module says of the torch it was built with."""
    return f"built with torch {version}"


def binding_commands(obj: str, out: str) -> tuple[list[str], list[str]]:
    """Compile and link commands of the extension module (linked against the
    library beside it)."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cxx = shutil.which("g++") or "c++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", BINDING_SRC, "-o", obj,
                f'-DMOE_BUILT_FOR="{built_for(torch_version())}"',
                f"-I{os.path.join(ROOT, 'include')}", f"-I{sysconfig.get_paths()['include']}",
                f"-I{os.path.join(torch, 'include')}", f"-I{os.path.join(cuda, 'include')}"]
    link = [cxx, "-shared", obj, "-o", out, f"-L{os.path.join(torch, 'lib')}", "-ltorch_python",
            "-ltorch", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-L{HERE}",
            "-lmoe_decode", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _finish(cmd: list[str], out: str, p: subprocess.Popen | None = None) -> str:
    p = p or subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    text = p.communicate()[0]
    if p.returncode != 0:
        sys.stderr.write(text)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {os.path.basename(out)}")
    return text


def build(verbose: bool = False, timeline: bool = False) -> str:
    out = OUT_TIMELINE if timeline else OUT
    tmp, obj, tmp_binding = out + ".tmp", BINDING_OUT[:-3] + ".o", BINDING_OUT + ".tmp"
    extra = (["-Xptxas", "-v"] if verbose else []) + (["-DMOE_TIMELINE"] if timeline else [])
    compile_, link = binding_commands(obj, tmp_binding)
    cxx = None if timeline else subprocess.Popen(compile_, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT, text=True)
    text = _finish(command(tmp, extra), out)
    if verbose:
        sys.stderr.write(text)
    os.replace(tmp, out)
    if not timeline:
        _finish(compile_, BINDING_OUT, cxx)
        _finish(link, BINDING_OUT)
        os.remove(obj)
        os.replace(tmp_binding, BINDING_OUT)
    return out


def stale(path: str) -> bool:
    """True when `path` is missing or older than a source or header; of the
    extension module, which build() makes with the library, also when it was
    built with another torch; and of the library when its module is."""
    if not os.path.exists(path) or (path == OUT and stale(BINDING_OUT)):
        return True
    if path == BINDING_OUT:
        with open(path, "rb") as f:
            if built_for(torch_version()).encode() + b"\0" not in f.read():
                return True
    srcs = [os.path.join(HERE, "csrc", f) for f in os.listdir(os.path.join(HERE, "csrc"))]
    srcs += [os.path.join(ROOT, "include", f) for f in os.listdir(os.path.join(ROOT, "include"))]
    return os.path.getmtime(path) < max(os.path.getmtime(f) for f in srcs)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, timeline="--timeline" in sys.argv))
