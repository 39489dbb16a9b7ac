"""What build() does when something is missing or has changed (the compilers are replaced
by a function that writes empty files: nothing is compiled here)."""
import os

import pytest

from compressed_kv_attention_gated_gb300 import build as b


@pytest.fixture
def made(monkeypatch, tmp_path):
    """build() into an empty folder; the commands that it runs."""
    for name in ("LIB", "BINDING", "BINDING_OF"):
        monkeypatch.setattr(b, name, str(tmp_path / "lib" / os.path.basename(getattr(b, name))))
    monkeypatch.setattr(b, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "_nvcc", lambda: "nvcc")
    runs = []

    def compile_(cmd):
        runs.append(cmd)
        if any(r in " ".join(cmd) for r in made.refuse):
            raise RuntimeError("no such header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    def made():
        runs.clear()
        assert b.build() == b.LIB
        return [os.path.basename(c[-3] if "-c" in c else c[c.index("-o") + 1]).split(".tmp")[0] for c in runs]

    made.refuse = ()
    monkeypatch.setattr(b, "_compile", compile_)
    return made


LIBRARY = [*b.CUDA_SOURCES, *b.CXX_SOURCES, "libckv.so"]


def test_everything_is_built_once(made):
    assert sorted(made()) == sorted([*LIBRARY, "binding.cpp", "ckv_binding.so"])
    assert b.up_to_date() and made() == []


@pytest.mark.parametrize("refuse", ["binding.cpp", "-lc10_cuda"])
def test_the_library_does_without_the_binding(made, refuse):
    """No Python or torch headers, or a torch without CUDA: libckv.so is there, the binding is not, and
    one of an earlier build is gone; the next build tries it again."""
    made()
    os.utime(b.BINDING, (0, 0))
    made.refuse = (refuse,)
    with pytest.warns(UserWarning, match="was not built: no such header"):
        made()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING) and not b.up_to_date()
    os.remove(b.LIB)
    with pytest.warns(UserWarning, match="was not built"):
        assert "libckv.so" in made()
    assert os.path.exists(b.LIB)
    made.refuse = ()
    assert made() == ["binding.cpp", "ckv_binding.so"] and b.up_to_date()


def test_the_library_does_without_torch(made, monkeypatch):
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    with pytest.warns(UserWarning, match="torch is not installed"):
        assert sorted(made()) == sorted(LIBRARY)
    assert os.path.exists(b.LIB)


def test_another_torch_gets_a_binding_of_its_own(made, monkeypatch):
    made()
    monkeypatch.setattr(b, "_torch_build", lambda: "another one")
    assert not b.up_to_date()
    assert made() == ["binding.cpp", "ckv_binding.so"]
    assert b.up_to_date()


def test_errors_of_the_library_are_raised(made):
    made.refuse = ("kpool.cu",)
    with pytest.raises(RuntimeError):
        made()
