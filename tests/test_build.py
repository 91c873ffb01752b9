"""build.py compiles what its sources, flags or compiler changed, and nothing else, on
the CPU with a stand-in for nvcc."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("tl_build", os.path.join(ROOT, "tensor_core_gemm_tl_b200", "build.py"))
build_module = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(build_module)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of two sources and a header in place of the library's; `runs` holds the commands since the last look."""
    b = build_module
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("one.cu", "two.cu", "common.cuh"):
        (csrc / name).write_text("x")
    runs = []

    def nvcc(cmd):
        runs.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        if "-c" in cmd:
            with open(cmd[cmd.index("-MF") + 1], "w") as fh:
                fh.write(f"{out} : {cmd[cmd.index('-c') + 1]} \\\n  {csrc / 'common.cuh'}\n")
        open(out, "w").close()

    monkeypatch.setattr(b, "ROOT", str(tmp_path))
    monkeypatch.setattr(b, "CSRC", str(csrc))
    monkeypatch.setattr(b, "INCLUDE", str(tmp_path / "include"))
    monkeypatch.setattr(b.subprocess, "check_call", nvcc)
    lib = str(tmp_path / "lib.so")

    def build(**how):
        runs.clear()
        b.build(out=lib, **how)
        return sorted(os.path.basename(c[c.index("-c") + 1]) for c in runs if "-c" in c)

    def touch(name):
        at = os.path.getmtime(lib) + 10
        os.utime(csrc / name, (at, at))

    build.touch, build.lib = touch, lib
    return build


BOTH = ["one.cu", "two.cu"]


def test_only_what_changed_is_compiled(tree):
    assert tree() == BOTH and tree() == []
    tree.touch("one.cu")
    assert tree() == ["one.cu"]


def test_a_missing_library_is_linked_from_its_objects(tree):
    tree()
    os.remove(tree.lib)
    assert tree() == [] and os.path.exists(tree.lib)


@pytest.mark.parametrize("change", ["flags", "extra", "compiler", "verbose"])
def test_objects_of_another_command_are_compiled_again(tree, change, monkeypatch):
    tree()
    os.remove(tree.lib)
    how = {}
    if change == "flags":
        monkeypatch.setattr(build_module, "NVCC_FLAGS", build_module.NVCC_FLAGS + ["-DOTHER"])
    elif change == "extra":
        how = dict(extra=("-DTL_CHECKED",))
    elif change == "compiler":
        monkeypatch.setattr(build_module, "NVCC", "/another/nvcc")
    else:
        how = dict(ptxas_verbose=True)
    assert tree(**how) == BOTH
    os.remove(tree.lib)
    assert tree(**how) == []


def test_register_counts_are_printed_when_asked_for(tree):
    """-Xptxas -v without --force: the library is up to date, the counts come from compiling it again."""
    tree()
    assert tree(ptxas_verbose=True) == BOTH


def test_flags_stand_in_a_file_the_library_depends_on():
    assert os.path.abspath(build_module.__file__) in [os.path.abspath(f) for f in build_module.inputs()]
