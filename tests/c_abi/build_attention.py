"""Sanitizer build for the CPU test of the attention calls' argument validation: the library's
entry points (kvx_attention_api.hip, host code only), stubs of the launches, and the plain C driver
attention_validate.c, with AddressSanitizer and UndefinedBehaviorSanitizer. No device code is
compiled and no GPU is needed. Rebuilds when a source is newer."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(os.path.dirname(HERE)))
from block_table_contiguous_amd import build as B  # noqa: E402

EXE = os.path.join(HERE, "attention_validate")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
SOURCES = [os.path.join(B.CSRC, "kvx_attention_api.hip"), os.path.join(HERE, "attention_stub.cpp"),
           os.path.join(HERE, "attention_validate.c")]
HEADERS = [os.path.join(B.INCLUDE, h) for h in ("kvx.h", "kvx_attention.h")] + \
    [os.path.join(B.CSRC, h) for h in ("kvx_attention_check.h", "kvx_attention_launch.h", "kvx_attention_plan.h")]


def build() -> str:
    if os.path.exists(EXE) and all(os.path.getmtime(p) <= os.path.getmtime(EXE) for p in SOURCES + HEADERS):
        return EXE
    clang = os.path.join(ROCM, "llvm", "bin", "clang")
    flags = ["-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-Wall", "-Wextra",
             "-D__HIP_PLATFORM_AMD__", f"-I{B.INCLUDE}", f"-I{B.CSRC}", f"-I{os.path.join(ROCM, 'include')}"]
    objs = []
    for src, lang in zip(SOURCES, (["-x", "c++", "-std=c++17"], ["-x", "c++", "-std=c++17"], ["-x", "c", "-std=c11", "-Werror"])):
        objs.append(os.path.join(HERE, os.path.basename(src) + ".san.o"))
        subprocess.run([clang, *flags, *lang, "-c", src, "-o", objs[-1]], check=True)
    subprocess.run([clang + "++", "-fsanitize=address,undefined", *objs, "-o", EXE + ".tmp"], check=True)
    for o in objs:
        os.remove(o)
    os.replace(EXE + ".tmp", EXE)
    return EXE


if __name__ == "__main__":
    print(build())
