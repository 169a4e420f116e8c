"""The registers that the compiler gives the tiles' kernel of the 8-bit attention (no GPU): its roles redistribute exactly what the
launch has, and the library refuses to launch it with another count."""

import os
import re
import subprocess

from top_sparse_mla_gb300.build import ARCH_FLAGS, INCLUDE, PKG_DIR, nvcc_path


def test_the_compiler_gives_the_registers_that_the_roles_redistribute(tmp_path):
    source = os.path.join(PKG_DIR, "csrc", "dsa_kv8_tiles.cu")
    want = int(re.search(r"LAUNCH_REGS = ([0-9]+)", open(source).read()).group(1))
    run = subprocess.run([nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-Xptxas",
                          "-v", "-c", "-o", str(tmp_path / "tiles.o"), source], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    used = re.findall(r"Compiling entry function '(\S*tiles_kernel\S*)'.*?Used ([0-9]+) registers", run.stderr, re.S)
    assert len(used) == 4 and all(int(n) == want for _, n in used), used
