"""Build libpp.so in-tree for sm_103a (nvcc, translation units in parallel),
and pp_bind, the C half of the Python binding's lm module."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpp.so")
BIND = os.path.join(PKG, "pp_bind" + sysconfig.get_config_var("EXT_SUFFIX"))  # of this interpreter
SOURCES = ["pp_api.cu", "pp_parse.cu", "pp_tokenize.cu", "pp_generic.cu", "pp_noalloc.cu",
           "pp_stream.cu", "pp_options.cu", "pp_grammar.cu", "pp_logits.cu", "pp_embed.cu",
           "pp_probs.cu", "pp_verify.cu", "pp_adamw.cu"]
HEADERS = ["pp_device.cuh", "pp_numeric.cuh", "pp_stv16.cuh", "pp_internal.h", "pp_lm.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC",
              "-I" + os.path.join(ROOT, "include"), "-I" + CSRC] + ARCH


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    table = os.path.join(CSRC, "pow5_table.inc")
    gen = os.path.join(CSRC, "gen_pow10.py")
    if force or _stale(table, [gen]):
        subprocess.check_call([sys.executable, gen, table])
    common = [os.path.join(ROOT, "include", "pp.h"), table] + \
        [os.path.join(CSRC, h) for h in HEADERS]
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or _stale(o, [s] + common):
            cmd = [nvcc] + NVCC_FLAGS + ["-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose:
                sys.stderr.write(r.stderr)
        return o

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        subprocess.check_call([nvcc, "-shared"] + ARCH + ["-o", tmp] + objs)
        os.replace(tmp, LIB)
    bind_src, include = os.path.join(CSRC, "pp_bind.c"), sysconfig.get_path("include")
    if not os.path.exists(os.path.join(include, "Python.h")):
        sys.stderr.write(f"no Python.h in {include}: built without pp_bind, which the lm module's calls need\n")
    elif force or _stale(BIND, [bind_src, common[0]]):
        tmp = BIND + ".tmp"
        subprocess.check_call([nvcc, "-shared", "-cudart", "none", "-O2", "-Xcompiler", "-fPIC",
                               "-I" + os.path.join(ROOT, "include"), "-I" + include, "-o", tmp, bind_src])
        os.replace(tmp, BIND)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
