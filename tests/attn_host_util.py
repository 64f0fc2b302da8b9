"""The host side of the attention operators with launches that are only written down (attn_host.cpp): the
framework's binding calls it in place of the library, so nothing here reaches a GPU."""
import contextlib
import ctypes
import os
import subprocess

from quantized_decoder_decode_gb300 import build as fqbuild
from quantized_decoder_decode_gb300 import fq

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.path.dirname(os.path.dirname(fqbuild.NVCC))
NAMES = ("fq_qk_norm_rope", "fq_attn_prompt", "fq_attn_prompt_workspace", "fq_attn_shared", "fq_attn_shared_workspace",
         "fq_attn_check", "fq_last_error")


def build(folder):
    fqbuild.build()
    out = os.path.join(str(folder), "attn_host.so")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-w", "-fvisibility=default", "-Wl,-Bsymbolic",
                           "-I", fqbuild.INCLUDE, "-I", fqbuild.CSRC, "-I", os.path.join(CUDA, "include"), "-x", "c++",
                           os.path.join(HERE, "attn_host.cpp"), "-o", out])
    L, real = ctypes.CDLL(out), fq.lib()
    for n in NAMES:
        getattr(L, n).argtypes, getattr(L, n).restype = getattr(real, n).argtypes, getattr(real, n).restype
    return L


@contextlib.contextmanager
def recorded(L):
    """fq's calls go to L; yields a function that gives the launches since the last time."""
    real, fq._lib = fq._lib, L

    def launches():
        out = []
        for i in range(L.attn_host_launches(0)):
            n = L.attn_host_launch(i, None, 0)
            a = (ctypes.c_longlong * n)()
            L.attn_host_launch(i, a, n)
            out.append(list(a))
        L.attn_host_launches(1)
        return out
    try:
        launches()
        yield launches
    finally:
        fq._lib = real
