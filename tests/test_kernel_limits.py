"""Kernels that may ask for more LDS than a launch gets by default have to raise their limit, each its own: the flag that
says so is a static variable of a template, so it has to be of the kernel and of no other.  Read from the library's
symbols (CPU only)."""
from __future__ import annotations

import collections
import re
import subprocess

import q4_swiglu_mlp_amd as Z

# every kernel whose dynamic LDS can pass 64 KB (the matvec kernels' is asked for at each call)
KERNELS = {"k_gemm16", "k_gemm16_both", "k_gemm16_beside", "k_fp8_tile", "k_fp8_stream", "k_lora_shrink",
           "k_lora_expand", "k_lora_firsts", "k_lora_seconds"}


def names(pattern, symbols, prefix=""):
    """How often each kernel is named (behind its length, as mangled names are) in the symbols that match."""
    found = collections.Counter()
    for s in symbols:
        if re.search(pattern, s):
            named = [k for k in KERNELS if f"{len(prefix + k)}{prefix}{k}" in s]
            found[named[0] if named else s] += 1
    return found


def test_every_kernel_raises_its_own_limit():
    out = subprocess.run(["nm", Z.LIB_PATH], check=True, stdout=subprocess.PIPE, text=True).stdout
    symbols = {line.split()[-1] for line in out.splitlines()}
    flags = names(r"allow_lds.*5ready$", symbols)
    stubs = names(r"__device_stub__", symbols, "__device_stub__")
    assert set(flags) == KERNELS
    for kernel in KERNELS:
        assert flags[kernel] == stubs[kernel] > 0, kernel
