"""Build the HIP library in-tree (gfx950), and the host extensions of the
drop-in optimizers and of the row operators.  Used by __graft_entry__.build()."""

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(PKG, "csrc", "fo_lib.hip")          # the optimizer step
ROWS_SRC = os.path.join(PKG, "csrc", "fo_rows.hip")     # the row operators
PRODUCTS_SRC = os.path.join(PKG, "csrc", "fo_products.hip")    # linear cross entropy, the gated block
GRADS_SRC = os.path.join(PKG, "csrc", "fo_grads.hip")   # gradient norms and clipping
OUT_DIR = os.path.join(PKG, "lib")
OUT = os.path.join(OUT_DIR, "libfoamd.so")

# -ffp-contract=off: every float operation is rounded once (no FMA formation),
# which the fixed operation order of the update relies on.  Division and square
# root stay IEEE correctly rounded, denormals are preserved.  Packed-FP32
# instruction selection is disabled.
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-variable", "-Wno-unknown-pragmas",
]


def build(verbose: bool = False, extra=()) -> str:
    """Compile the translation units side by side and link them into
    lib/libfoamd.so."""
    os.makedirs(OUT_DIR, exist_ok=True)
    flags = [f for f in FLAGS if f != "-shared"]
    jobs = []
    for src in (SRC, ROWS_SRC, PRODUCTS_SRC, GRADS_SRC):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-4] + ".o")
        cmd = ["/opt/rocm/bin/hipcc", *flags, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    logs = [job.communicate()[0] for _, job in jobs]
    for (_, job), log in zip(jobs, logs):
        if job.returncode != 0:
            sys.stderr.write(log)
            raise RuntimeError("hipcc failed building libfoamd.so")
        if verbose and log.strip():
            print("\n".join(l for l in log.splitlines() if "packed-fp32-ops" not in l)[:4000])
    tmp = OUT + ".tmp"
    res = subprocess.run(["/opt/rocm/bin/hipcc", *FLAGS, *[obj for obj, _ in jobs], "-o", tmp],
                         capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed linking libfoamd.so")
    os.replace(tmp, OUT)
    return OUT


MARSHAL_SRC = os.path.join(PKG, "csrc", "fo_marshal.cpp")
MARSHAL_OUT = os.path.join(OUT_DIR, "fo_marshal.so")


def _build_extension(src, name, out, includes=(), libs=(), verbose=False):
    """Compile one host C++ extension with the flags torch's own C++ extensions use."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ce

    os.makedirs(os.path.dirname(out), exist_ok=True)
    tmp = out + ".tmp"
    libdirs = ce.library_paths()
    # the defines are those torch.utils.cpp_extension.CppExtension passes for
    # this (ROCm) build of torch, so its headers see the configuration they
    # were built with; the sources themselves are host C++ with no GPU code
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-DTORCH_API_INCLUDE_EXTENSION_H", f"-DTORCH_EXTENSION_NAME={name}",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           *[f"-I{d}" for d in ce.include_paths()], f"-I{sysconfig.get_paths()['include']}",
           *[f"-I{d}" for d in includes], src, "-o", tmp,
           *[f"-L{d}" for d in libdirs], *[f"-Wl,-rpath,{d}" for d in libdirs],
           *libs, "-lc10", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"g++ failed building {os.path.basename(out)}")
    os.replace(tmp, out)
    return out


def build_marshal(verbose: bool = False, out: str = MARSHAL_OUT) -> str:
    """Compile csrc/fo_marshal.cpp (host C++, torch headers) into `out`
    (lib/fo_marshal.so)."""
    return _build_extension(MARSHAL_SRC, "fo_marshal", out, verbose=verbose)


ROWS_TORCH_SRC = os.path.join(PKG, "csrc", "fo_rows_torch.cpp")
ROWS_TORCH_OUT = os.path.join(OUT_DIR, "fo_rows_torch.so")


def build_rows_torch(verbose: bool = False) -> str:
    """Compile csrc/fo_rows_torch.cpp (host C++: autograd of the row operators)
    into lib/fo_rows_torch.so, linked to the libfoamd.so beside it."""
    return _build_extension(ROWS_TORCH_SRC, "fo_rows_torch", ROWS_TORCH_OUT, ["/opt/rocm/include"],
                            [f"-L{OUT_DIR}", "-l:libfoamd.so", "-Wl,-rpath,$ORIGIN", "-lc10_hip"], verbose)


STEP_TORCH_SRC = os.path.join(PKG, "csrc", "fo_step_torch.cpp")
STEP_TORCH_OUT = os.path.join(OUT_DIR, "fo_step_torch.so")


def build_step_torch(verbose: bool = False) -> str:
    """Compile csrc/fo_step_torch.cpp (host C++: clipping, linear cross entropy, the
    gated block) into lib/fo_step_torch.so, linked to the libfoamd.so beside it."""
    return _build_extension(STEP_TORCH_SRC, "fo_step_torch", STEP_TORCH_OUT, ["/opt/rocm/include"],
                            [f"-L{OUT_DIR}", "-l:libfoamd.so", "-Wl,-rpath,$ORIGIN", "-lc10_hip"], verbose)


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_marshal(verbose=True))
    print(build_rows_torch(verbose=True))
    print(build_step_torch(verbose=True))
