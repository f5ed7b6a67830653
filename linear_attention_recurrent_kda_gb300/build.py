"""Build the in-tree CUDA libraries for sm_103a.

``libkda_gb300.so``: the translation units of the step and its companions
(the step, split, replay, output-projection, linear-attention, snapshot,
convolution, scan, product and self-test kernels; the C ABI of include/kda.h).
``libkda_probe_gb300.so``: the measurement probe of include/kda_probe.h, a bench
instrument kept out of the product library.
``kda_bind-<python>-torch<version>.so``: the short way from Python to the calls whose
host side is most of their time, against the headers of the installed PyTorch.  The
library does not need it: where it cannot be built the calls take the general way.
Every translation unit is compiled by its own nvcc process (g++ for the binding), in
parallel, with a single ``-gencode arch=compute_103a,code=sm_103a``; each library is
linked by one more nvcc call and sits next to this file.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import tempfile
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libkda_gb300.so")
PROBE_LIB_PATH = os.path.join(HERE, "libkda_probe_gb300.so")
SOURCES = [os.path.join(CSRC, n) for n in ("kda_step.cu", "kda_split.cu",
                                            "kda_recover.cu", "kda_oproj.cu",
                                            "kda_lin.cu", "kda_lin_prompt.cu", "kda_snapshot.cu",
                                            "kda_conv.cu", "kda_ssm.cu", "kda_ssm_prompt.cu",
                                            "kda_linear.cu", "kda_selftest.cu")]
PROBE_SOURCES = [os.path.join(CSRC, "kda_probe.cu")]
HEADERS = [os.path.join(INCLUDE, "kda.h"), os.path.join(INCLUDE, "kda_probe.h"),
           os.path.join(CSRC, "kda_device.cuh"), os.path.join(CSRC, "kda_lin.cuh"),
           os.path.join(CSRC, "kda_rows.cuh"), os.path.join(CSRC, "kda_tc.cuh"),
           os.path.join(CSRC, "kda_ssm.cuh"), os.path.join(CSRC, "kda_linear_tiles.h"),
           os.path.join(CSRC, "kda_host.h")]


def _bind_path():
    """Of the binding for this interpreter and PyTorch; None where PyTorch does not say its
    version (a module for another one's headers must not be loaded)."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None
    return os.path.join(HERE, "kda_bind-%s-torch%s.so" % (sysconfig.get_config_var("SOABI"), version))


BIND_PATH = _bind_path()
BIND_SOURCE = os.path.join(CSRC, "kda_bind.cpp")
LIBS = ((LIB_PATH, SOURCES), (PROBE_LIB_PATH, PROBE_SOURCES))

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _stale(lib: str, sources) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in list(sources) + HEADERS)


def _bind_stale() -> bool:
    return BIND_PATH is not None and _stale(BIND_PATH, [BIND_SOURCE])


def is_stale() -> bool:
    return any(_stale(lib, srcs) for lib, srcs in LIBS) or _bind_stale()


def _bind_command(out: str):
    """The compiler's call for the binding (PyTorch's headers, found without importing it)."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    includes = [os.path.join(torch, "include"),
                os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_path("include"),
                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared"]
            + [a for path in includes for a in ("-isystem", path)]
            + [BIND_SOURCE, "-o", out, "-L" + os.path.join(torch, "lib"),
               "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def _publish(made: str, path: str) -> None:
    """Puts a finished file in place at once (processes may build side by side)."""
    fd, new = tempfile.mkstemp(dir=os.path.dirname(path), prefix=os.path.basename(path) + ".")
    os.close(fd)
    try:
        shutil.copyfile(made, new)
        shutil.copymode(made, new)
        os.replace(new, path)
    except BaseException:
        os.unlink(new)
        raise


def _start(cmd):
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the libraries that are missing or older than their sources.

    Each translation unit compiles in its own nvcc process (all in parallel),
    then one nvcc call per library links it.  A binding that cannot be built is a
    warning.  Returns the product library's path."""
    todo = [(lib, srcs) for lib, srcs in LIBS if force or _stale(lib, srcs)]
    bind = BIND_PATH is not None and (force or _bind_stale())
    if not todo and not bind:
        return LIB_PATH
    with tempfile.TemporaryDirectory() as tmp:
        binding, trouble = None, ""
        if bind:
            try:
                binding = _start(_bind_command(os.path.join(tmp, "kda_bind.so")))
            except (OSError, RuntimeError, AttributeError) as e:     # no compiler, no PyTorch
                trouble = repr(e)
        procs = []
        objs = {lib: [] for lib, _ in todo}
        for lib, srcs in todo:
            for src in srcs:
                obj = os.path.join(tmp, os.path.basename(src) + ".o")
                cmd = [nvcc()] + NVCC_FLAGS + ["-I", INCLUDE, "-c", src, "-o", obj]
                if verbose:
                    cmd.insert(1, "-Xptxas=-v")
                procs.append((src, _start(cmd)))
                objs[lib].append(obj)
        logs = []
        for src, pr in procs:
            out, _ = pr.communicate()
            logs.append(out)
            if pr.returncode != 0:
                raise RuntimeError(f"the compiler failed on {src}:\n{out}")
        for lib, _ in todo:
            out = os.path.join(tmp, os.path.basename(lib))
            link = [nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-shared",
                    "-o", out] + objs[lib]
            res = subprocess.run(link, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError("nvcc link failed:\n" + res.stdout + res.stderr)
            _publish(out, lib)
        if binding is not None:
            out, _ = binding.communicate()
            logs.append(out)
            if binding.returncode == 0:
                _publish(os.path.join(tmp, "kda_bind.so"), BIND_PATH)
            else:
                trouble = out
        if trouble:
            warnings.warn(f"the short way from Python was not built, calls take the general one:\n{trouble}",
                          RuntimeWarning, stacklevel=2)
        if verbose:
            print("".join(logs))
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
