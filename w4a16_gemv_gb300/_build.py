"""Build libnf4.so in-tree with nvcc for sm_103a (one -gencode, sources in parallel), and the compiled
half of the Python binding (_attention.so) with g++."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnf4.so")
BINDING = os.path.join(PKG, "_attention.so")
BINDING_KEY = os.path.join(OBJDIR, "binding.txt")
SOURCES = ("nf4_api.cu", "nf4_dequant.cu", "nf4_gemv.cu", "nf4_gemv_b1.cu", "nf4_gemv_stream.cu",
           "nf4_quantize.cu", "nf4_step.cu", "nf4_gemm_tc.cu", "nf4_attn_api.cu", "nf4_rope.cu",
           "nf4_prefix_attn.cu", "nf4_prefix_attn_tc.cu", "nf4_decoding_api.cu", "nf4_kv_pages.cu", "nf4_adjust_logits.cu",
           "nf4_tree_commit.cu")
BINDINGS = ("attention_binding.cpp", "decoding_binding.cpp")
GENCODE = "arch=compute_103a,code=sm_103a"


def nvcc_path() -> str:
    cand = shutil.which("nvcc")
    if cand:
        return cand
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return os.path.join(home, "bin", "nvcc")


def nvcc_flags(extra: tuple[str, ...] = ()) -> list[str]:
    return ["-gencode", GENCODE, "-lineinfo", "-O3", "-std=c++17", "-ftz=false",
            "-prec-div=true", "-prec-sqrt=true", "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
            "-I", INCLUDE, "-I", CSRC, *extra]


def _binding_key() -> str:
    """What the Python entry points are built against: the interpreter and torch."""
    from importlib import metadata
    try:
        torch = metadata.version("torch")
    except metadata.PackageNotFoundError:
        torch = "none"
    return f"{sys.version} torch {torch}"


def _built_against() -> str | None:
    try:
        with open(BINDING_KEY) as f:
            return f.read()
    except OSError:
        return None


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING) or _built_against() != _binding_key():
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = ([os.path.join(CSRC, f) for f in os.listdir(CSRC)] +
            [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)])
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_commands(out: str) -> tuple[list[list[str]], list[str]]:
    """Compile the Python entry points against the running interpreter, torch and the headers, one command per source;
    link them with libnf4.so."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"),
            INCLUDE]
    libs = os.path.join(root, "lib")
    cxx = os.environ.get("CXX", "g++")
    objs = [os.path.join(OBJDIR, f.replace(".cpp", ".o")) for f in BINDINGS]
    flags = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[a for d in dirs for a in ("-isystem", d)]]
    return ([[cxx, *flags, "-c", os.path.join(CSRC, f), "-o", o] for f, o in zip(BINDINGS, objs)],
            [cxx, "-shared", *objs, "-o", out, "-L", PKG, "-l:libnf4.so", "-L", libs, "-ltorch_python", "-ltorch", "-ltorch_cpu",
             "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"])


def build(force: bool = False, verbose: bool = False, extra: tuple[str, ...] = ()) -> str:
    """Compile every source to an object in parallel, link libnf4.so and the Python entry points."""
    if not force and not _stale():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    nvcc = nvcc_path()
    objs = [os.path.join(OBJDIR, src.replace(".cu", ".o")) for src in SOURCES]
    tmp_binding = BINDING + f".tmp{os.getpid()}"
    compile_binding, link_binding = _binding_commands(tmp_binding)
    procs = []
    for src, cmd in [*((src, [nvcc, *nvcc_flags(extra), "-c", os.path.join(CSRC, src), "-o", obj])
                       for src, obj in zip(SOURCES, objs)), *zip(BINDINGS, compile_binding)]:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"the compiler failed:\n{msg}")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-gencode", GENCODE, "-shared", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    if verbose:
        print(" ".join(link_binding), file=sys.stderr)
    p = subprocess.run(link_binding, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed:\n{p.stdout.decode(errors='replace')}")
    os.replace(tmp_binding, BINDING)
    with open(BINDING_KEY, "w") as f:
        f.write(_binding_key())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
