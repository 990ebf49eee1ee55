"""In-tree build of libringag.so for gfx950 (hipcc cross-compiles; no GPU needed).

    python -m ring_all_gather_amd.build        # or __graft_entry__.build()

Steps:
  1. device code: csrc/device_kernels.hip (the ring GEMMs) and csrc/ops_kernels.hip (the block
     operators) -> one gfx950 code object each (hipcc --genco), compiled with -Xclang
     -target-feature -Xclang -packed-fp32-ops so the compiler forms no packed fp32 VALU
     instructions (v_pk_*_f32);
  2. the code objects are embedded as the symbols ringag_kernels_co and ringag_ops_co (assembler
     .incbin), each with its SHA-256;
  3. host code (csrc/runtime.cpp, launch.cpp, ops_runtime.cpp, ops_launch.cpp) is compiled as plain
     C++ against the HIP runtime API and linked with the blobs into
     ring_all_gather_amd/libringag.so.
The host objects contain no device code, so the library has no HIP registration constructors or
destructors; the kernels are loaded explicitly when a context is created.
"""
import hashlib
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libringag.so")
BUILD_DIR = os.path.join(ROOT, "_build")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.environ.get("HIPCC", os.path.join(ROCM, "bin", "hipcc"))
CXX = os.environ.get("CXX", "g++")
ARCH = "gfx950"
DEVICE_SRCS = {"ringag_kernels": "device_kernels.hip", "ringag_ops": "ops_kernels.hip"}
HOST_SRCS = ["runtime.cpp", "launch.cpp", "ops_runtime.cpp", "ops_launch.cpp"]
DEVICE_FLAGS = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "--genco",
                "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                "-Wno-unused-command-line-argument", f"-I{INCLUDE}", f"-I{CSRC}"]
# the epilogues' blocks have to unroll in full, or the accumulators they index go to memory
DEVICE_EXTRA = {"ringag_ops": ["-mllvm", "-pragma-unroll-threshold=65536"]}
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-unused-function",
              "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{INCLUDE}", f"-I{CSRC}"]


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r


def build_code_object(name: str, extra=()) -> str:
    co = os.path.join(BUILD_DIR, f"{name}.co")
    _run([HIPCC, *DEVICE_FLAGS, *DEVICE_EXTRA.get(name, []), *extra,
          os.path.join(CSRC, DEVICE_SRCS[name]), "-o", co],
         f"device compile of {DEVICE_SRCS[name]}")
    return co


def _blob_object(name: str, co: str) -> str:
    """Embed the code object as <name>_co, and its SHA-256 as the string <name>_sha256 (so that
    measurements taken with one build of the kernels can be told apart from another's)."""
    with open(co, "rb") as f:
        digest = hashlib.sha256(f.read()).hexdigest()
    asm = os.path.join(BUILD_DIR, f"{name}_blob.S")
    with open(asm, "w") as f:
        f.write(f'    .section .rodata.{name},"a"\n'
                "    .balign 4096\n"
                f"    .globl {name}_co\n"
                f"    .type {name}_co, @object\n"
                f"{name}_co:\n"
                f'    .incbin "{co}"\n'
                f"    .size {name}_co, . - {name}_co\n"
                f"    .globl {name}_sha256\n"
                f"    .type {name}_sha256, @object\n"
                f"{name}_sha256:\n"
                f'    .asciz "{digest}"\n'
                f"    .size {name}_sha256, . - {name}_sha256\n"
                '    .section .note.GNU-stack,"",@progbits\n')
    obj = os.path.join(BUILD_DIR, f"{name}_blob.o")
    _run([CXX, "-c", asm, "-o", obj], "blob assembly")
    return obj


def _host_object(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    _run([CXX, *HOST_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj], f"compile of {src}")
    return obj


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=4) as ex:
        cos = {n: ex.submit(build_code_object, n, list(extra)) for n in DEVICE_SRCS}
        hosts = list(ex.map(_host_object, HOST_SRCS))
        blobs = [_blob_object(n, f.result()) for n, f in cos.items()]
    tmp = LIB + ".tmp"
    _run([CXX, "-shared", "-fPIC", *hosts, *blobs, "-o", tmp, f"-L{ROCM}/lib", "-lamdhip64",
          f"-Wl,-rpath,{ROCM}/lib"], "link")
    os.replace(tmp, LIB)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
