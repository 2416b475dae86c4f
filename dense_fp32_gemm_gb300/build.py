"""Build the CUDA library libsgemm_gb300.so in-tree for sm_103a.

Each .cu file under csrc/ is compiled on its own (in parallel), together with
one generated translation unit per tile configuration of the configuration
list (csrc/configs.inc, written by configgen.py / tune.py), so that the
configurations compile in parallel. The objects are linked into
``_lib/libsgemm_gb300.so`` with the CUDA runtime linked statically, so the
library loads on any machine with the driver installed. Only the functions
declared in include/sgemm_gb300.h are exported.

``build(config_list=..., tuned_table=..., out_dir=...)`` builds a separate
library from another configuration list (the tuner's candidate set) without
touching the product library.

Beside it, csrc_torch/marshal.cpp (the torch conveniences of binding.py) is
compiled with the host compiler against the installed torch, if there is one;
the library needs neither.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB_NAME = "libsgemm_gb300.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
CONFIG_LIST = os.path.join(CSRC, "configs.inc")
TUNED_TABLE = os.path.join(CSRC, "tuned_table.inc")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "--expt-relaxed-constexpr", "-O3", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-Xptxas", "-v"] + ARCH

_CFG_TU = """// Generated by dense_fp32_gemm_gb300/build.py from the configuration list:
// the FFMA kernel instantiated for one tile configuration (one translation
// unit each, so that the configurations compile in parallel).
#include "launch.cuh"

SGEMM_GB300_DEFINE_CONFIG({name})
"""


MARSHAL_SOURCE = os.path.join(HERE, "csrc_torch", "marshal.cpp")


def torch_dir() -> str | None:
    """Where torch is installed (it is not imported); None without it."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None else spec.submodule_search_locations[0]


def marshal_path() -> str:
    """The torch marshalling module built for the installed torch and this
    Python (another version of either needs another build)."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:   # (installed without metadata)
        import torch
        version = torch.__version__
    soabi = sysconfig.get_config_var("SOABI")
    return os.path.join(OUT_DIR, f"_marshal_{version.replace('+', '_')}.{soabi}.so")


def build_marshal() -> str | None:
    """Compile csrc_torch/marshal.cpp against the installed torch, if it or the
    torch or Python version changed; None without torch."""
    torch_at = torch_dir()
    if torch_at is None:
        return None
    path = marshal_path()
    if not _stale(path, [MARSHAL_SOURCE]):
        return path
    os.makedirs(OUT_DIR, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    includes = [sysconfig.get_paths()["include"], os.path.join(torch_at, "include"),
                os.path.join(torch_at, "include", "torch", "csrc", "api", "include"), cuda]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden"]
    cmd += [f"-I{d}" for d in includes]
    cmd += [MARSHAL_SOURCE, "-o", path + ".tmp", "-L" + os.path.join(torch_at, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on marshal.cpp:\n{r.stderr[-4000:]}")
    os.replace(path + ".tmp", path)
    return path


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def fixed_sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h*")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.inc")) + glob.glob(os.path.join(HERE, "..", "include", "*.h"))


def _stale(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(f) > t for f in deps)


def generate_config_units(config_list: str, gen_dir: str):
    """One .cu per configuration of the list (rewritten only when its text
    changes); units of configurations no longer listed are removed."""
    try:
        from . import configgen
    except ImportError:  # run as a script
        import configgen
    entries, _ = configgen.read_configs_inc(config_list)
    os.makedirs(gen_dir, exist_ok=True)
    want = {}
    for t, _ in entries:
        name = configgen.config_name(t)
        want[os.path.join(gen_dir, f"cfg_{name}.cu")] = _CFG_TU.format(name=name)
    for old in glob.glob(os.path.join(gen_dir, "cfg_*.cu")):
        if old not in want:
            os.remove(old)
    for path, text in want.items():
        if not os.path.exists(path) or open(path).read() != text:
            with open(path, "w") as f:
                f.write(text)
    return sorted(want)


def build(verbose: bool = False, jobs: int | None = None, config_list: str | None = None,
          tuned_table: str | None = None, out_dir: str | None = None) -> str:
    """Compile (what changed) and link; returns the library path."""
    out_dir = out_dir or OUT_DIR
    os.makedirs(out_dir, exist_ok=True)
    tool = nvcc()
    extra = ["-I", CSRC]
    deps_extra = []
    if config_list is not None:
        config_list = os.path.abspath(config_list)
        extra.append(f'-DSGEMM_GB300_CONFIG_LIST="{config_list}"')
        deps_extra.append(config_list)
    if tuned_table is not None:
        tuned_table = os.path.abspath(tuned_table)
        extra.append(f'-DSGEMM_GB300_TUNED_TABLE_FILE="{tuned_table}"')
        deps_extra.append(tuned_table)
    gen = generate_config_units(config_list or CONFIG_LIST, os.path.join(out_dir, "gen"))
    srcs = fixed_sources() + gen
    objs = [os.path.join(out_dir, os.path.basename(s)[:-3] + ".o") for s in srcs]
    deps = _headers() + deps_extra
    logs = {}

    def compile_one(pair):
        src, obj = pair
        if not _stale(obj, [src] + deps):
            return
        cmd = [tool] + NVCC_FLAGS + extra + ["-c", src, "-o", obj + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        logs[src] = r.stdout + r.stderr
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr[-4000:]}")
        os.replace(obj + ".tmp", obj)

    # stale objects of configurations that left the list
    keep = set(objs)
    for o in glob.glob(os.path.join(out_dir, "*.o")):
        if o not in keep:
            os.remove(o)
    n = jobs or min(len(srcs), os.cpu_count() or 1)
    with ThreadPoolExecutor(max(1, n + 1)) as ex:
        # (a candidate build of the tuner takes the product's marshalling module)
        marshal = ex.submit(build_marshal) if out_dir == OUT_DIR else None
        list(ex.map(compile_one, zip(srcs, objs)))
    if verbose:
        for src, log in sorted(logs.items()):
            print(f"== {os.path.basename(src)}\n{log}", file=sys.stderr)
    lib_path = os.path.join(out_dir, LIB_NAME)
    lib_stale = not os.path.exists(lib_path) or any(
        os.path.getmtime(o) > os.path.getmtime(lib_path) for o in objs)
    if lib_stale:
        tmp = lib_path + ".tmp"
        subprocess.check_call([tool, "-shared", "-cudart", "static"] + ARCH + objs + ["-o", tmp])
        os.replace(tmp, lib_path)
    if marshal is not None:
        marshal.result()          # its failure leaves the library built
    return lib_path


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
