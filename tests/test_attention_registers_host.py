"""The registers that the compiler gives the kernels whose roles redistribute exactly what the launch has (no GPU): the latent
attention's, and the tiles' for requests that share a prefix.  The library refuses to launch them with another count."""

import os
import re
import subprocess

import pytest

from top_sparse_mla_gb300.build import ARCH_FLAGS, INCLUDE, PKG_DIR, nvcc_path


@pytest.mark.parametrize("source,kernel,variants", [("dsa_mla_prefill.cu", "mla_kernel", 4), ("dsa_kv8_prefix.cu", "tiles_kernel", 4)])
def test_the_compiler_gives_the_registers_that_the_roles_redistribute(source, kernel, variants, tmp_path):
    source = os.path.join(PKG_DIR, "csrc", source)
    want = int(re.search(r"LAUNCH_REGS = ([0-9]+)", open(source).read()).group(1))
    run = subprocess.run([nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-Xptxas",
                          "-v", "-c", "-o", str(tmp_path / "x.o"), source], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    used = re.findall(r"Compiling entry function '(\S*%s\S*)'.*?Used ([0-9]+) registers" % kernel, run.stderr, re.S)
    assert len(used) == variants and all(int(n) == want for _, n in used), used
