"""What build() hands to nvcc (no GPU, and no nvcc)."""

import importlib
import pathlib

build_module = importlib.import_module("top_sparse_mla_gb300.build")   # the package's `build` is the function


def test_extra_flags_reach_the_compiler_and_the_linker(monkeypatch, tmp_path):
    """A library that a caller adds has to be in the link, behind the objects."""
    calls = []

    def run(cmd, verbose):
        calls.append(cmd)
        pathlib.Path(cmd[cmd.index("-o") + 1]).write_text("")

    monkeypatch.setattr(build_module, "_run", run)
    monkeypatch.setattr(build_module, "nvcc_path", lambda: "nvcc")
    monkeypatch.setattr(build_module, "LIB_PATH", str(tmp_path / "lib.so"))
    assert build_module.build(extra_flags=["-DEXTRA", "-lextra"]) == str(tmp_path / "lib.so")
    compiles, links = [c for c in calls if "-c" in c], [c for c in calls if "-shared" in c]
    assert sorted(c[-1] for c in compiles if "-DEXTRA" in c and "-lextra" in c) == sorted(build_module.SOURCES)
    (link,) = links
    last_object = max(i for i, x in enumerate(link) if x.endswith(".o"))
    assert link.index("-lextra") > last_object
