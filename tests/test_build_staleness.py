"""What build.py compiles again: the extension belongs to one torch and one Python, whose headers it
was compiled against, so another one makes it stale, as changed sources do. No compiler runs here:
the steps are recorded and their outputs created empty."""
import importlib.util
import os
import sysconfig
import types

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_161_gb300")


@pytest.fixture
def steps(tmp_path, monkeypatch):
    """A function that builds into an empty folder and returns the outputs of the steps it took."""
    spec = importlib.util.spec_from_file_location("_pa_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    taken = []

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        taken.append(os.path.basename(out))

    monkeypatch.setattr(mod, "_run", run)
    monkeypatch.setattr(mod, "_cuda_home", lambda: "/cuda")
    monkeypatch.setattr(mod, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(mod, "LIB_DIR", str(tmp_path / "_lib"))
    for name in ("LIB_PATH", "EXT_PATH"):
        monkeypatch.setattr(mod, name, str(tmp_path / "_lib" / os.path.basename(getattr(mod, name))))

    def build():
        taken.clear()
        mod.build()
        return set(taken)

    build.tmp, build.mod = tmp_path, mod
    return build


def _use_torch(monkeypatch, folder, version):
    os.makedirs(folder, exist_ok=True)
    for name, text in (("__init__.py", ""), ("version.py", f"__version__ = {version!r}\n")):
        with open(os.path.join(folder, name), "w") as f:
            f.write(text)
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name: types.SimpleNamespace(origin=os.path.join(folder, "__init__.py")))


EXT = {"torch_binding.cpp.o", "_pa_torch.so.tmp"}


def test_another_torch_or_python_compiles_the_extension_again(steps, monkeypatch):
    a, b = str(steps.tmp / "a" / "torch"), str(steps.tmp / "b" / "torch")
    _use_torch(monkeypatch, a, "2.9.1")
    assert EXT < steps()
    assert steps() == set()
    _use_torch(monkeypatch, a, "2.11.0")  # upgraded in place
    assert EXT <= steps()
    assert steps() == set()
    _use_torch(monkeypatch, b, "2.11.0")  # another environment
    assert EXT <= steps()
    assert steps() == set()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert EXT <= steps()
    assert steps() == set()


def test_a_build_that_stopped_is_taken_again(steps, monkeypatch):
    folder = str(steps.tmp / "torch")
    _use_torch(monkeypatch, folder, "2.9.1")
    steps()
    _use_torch(monkeypatch, folder, "2.11.0")

    def stop(name):
        def run(cmd, verbose, go=steps.mod._run):
            if os.path.basename(cmd[cmd.index("-o") + 1]) == name:
                raise RuntimeError("stopped")
            go(cmd, verbose)

        with monkeypatch.context() as m:
            m.setattr(steps.mod, "_run", run)
            with pytest.raises(RuntimeError):
                steps()

    stop("torch_binding.cpp.o")
    stop("_pa_torch.so.tmp")  # compiled, not linked
    assert EXT <= steps()
    assert steps() == set()
