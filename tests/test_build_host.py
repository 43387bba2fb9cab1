"""What build() compiles when, with the compilers replaced: the library and the binding for torch are kept
up to date apart."""
import os
import subprocess
import sys

import pytest

from io_aware_attention_attn_gb300 import build


@pytest.fixture
def steps(tmp_path, monkeypatch):
    """A tree of its own, and the list of what a build ran; a step named in `fail` raises."""
    ran, fail = [], set()
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("a.cu", "b.cu", "c.cuh", "py_binding.cpp"):
        (csrc / name).write_text("")
    inc = tmp_path / "include"
    inc.mkdir()
    (inc / "h.h").write_text("")
    for name, value in (("PKG", tmp_path), ("CSRC", csrc), ("INCLUDE", inc), ("BUILD", tmp_path / "_build"),
                        ("LIB", tmp_path / "lib.so"), ("BINDING", tmp_path / "binding.so"),
                        ("BINDING_SRC", csrc / "py_binding.cpp"), ("BINDING_KEY", tmp_path / "binding.so.key")):
        monkeypatch.setattr(build, name, str(value))

    def run(cmd, what):
        ran.append(what)
        if what in fail:
            raise RuntimeError(what)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    def compile_cu(src, verbose):
        ran.append(os.path.basename(src))
        return src

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "_compile", compile_cu)
    monkeypatch.setattr(build, "nvcc", lambda: "/cuda/bin/nvcc")

    def go(**kw):
        ran.clear()
        build.build(**kw)
        return sorted(ran)

    go.fail, go.ran, go.csrc = fail, ran, csrc
    return go


LIBRARY = ["a.cu", "b.cu", "link"]
BINDING = ["compiling py_binding.cpp", "linking the binding"]


def later(path):
    t = os.path.getmtime(build.__file__) + 1e6
    os.utime(path, (t, t))


def test_each_part_by_itself(steps):
    assert steps() == sorted(LIBRARY + BINDING) and steps() == [] and build.up_to_date()
    later(steps.csrc / "py_binding.cpp")
    assert not build.up_to_date() and steps() == BINDING
    later(build.BINDING)
    assert steps() == []
    later(steps.csrc / "c.cuh")
    assert steps() == LIBRARY
    later(build.LIB)
    assert steps() == [] and steps(force=True) == sorted(LIBRARY + BINDING)


def test_library_without_the_binding(steps, monkeypatch):
    assert steps(library_only=True) == LIBRARY and not os.path.exists(build.BINDING)
    assert steps() == BINDING


def test_without_torch(steps, monkeypatch):
    monkeypatch.setattr(build, "have_torch", lambda: False)
    assert steps() == LIBRARY and build.up_to_date() and steps() == []


@pytest.mark.parametrize("step", BINDING)
def test_a_failing_binding_does_not_build_the_library_again(steps, step):
    steps.fail.add(step)
    with pytest.raises(RuntimeError, match=step):
        steps()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    with pytest.raises(RuntimeError, match=step):
        steps()
    assert not set(steps.ran) & set(LIBRARY)
    steps.fail.clear()
    assert steps() == BINDING and build.up_to_date()


@pytest.mark.parametrize("other", ["2.9.0 1 .cpython-312-x86_64-linux-gnu.so", ""])
def test_a_binding_of_another_torch_is_built_again(steps, monkeypatch, other):
    assert steps() == sorted(LIBRARY + BINDING) and build.binding_matches()
    with open(build.BINDING_KEY, "w") as f:
        f.write(other)
    assert not build.binding_matches() and not build.up_to_date() and steps() == BINDING
    mine = build.binding_key()
    monkeypatch.setattr(build, "binding_key", lambda: mine + "+new")
    assert not build.up_to_date() and steps() == BINDING and build.up_to_date()
    os.remove(build.BINDING_KEY)
    assert steps() == BINDING
    # a link that fails leaves no key beside the old binding
    monkeypatch.setattr(build, "binding_key", lambda: mine)
    steps.fail.add(BINDING[1])
    with pytest.raises(RuntimeError):
        steps()
    assert not build.binding_matches()


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    from io_aware_attention_attn_gb300 import attn
    build.build()
    monkeypatch.setattr(attn, "_native_module", None)
    key = tmp_path / "key"
    key.write_text("2.9.0 1 .cpython-312-x86_64-linux-gnu.so")
    monkeypatch.setattr(build, "BINDING_KEY", str(key))
    with pytest.raises(RuntimeError, match="another torch"):
        attn._native()
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "none"))
    with pytest.raises(RuntimeError, match="is missing"):
        attn._native()
    monkeypatch.undo()
    assert attn._native() is not None


def test_the_library_is_called_without_torch():
    build.build()
    code = ("import sys; sys.modules['torch'] = None\n"
            "from io_aware_attention_attn_gb300 import attn\n"
            "assert attn.paged_workspace_bytes(2, 8, 2, 128) == attn.lib().attn_fwd_paged_workspace_bytes(2, 8, 2, 128) > 0\n"
            "assert attn.version() > 0 and attn.bwd_workspace_bytes(1, 2, 64, 64) > 0\n"
            "assert attn.decode_status(0) is not None")
    r = subprocess.run([sys.executable, "-c", code], cwd=build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
