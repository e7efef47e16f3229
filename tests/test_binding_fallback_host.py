"""The package without _binding.so, as built where Python's headers are missing:
it imports, and its calls convert, refuse and answer as with it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def test_the_host_tests_of_the_calls_pass_without_it(built, tmp_path):
    """The refusals of every many-token and 8-bit call, in a process that cannot import it."""
    (tmp_path / "sitecustomize.py").write_text(
        "import sys\nsys.modules['moe_expert_ffn_smoe_gb300._binding'] = None\n")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT, os.environ.get("PYTHONPATH", "")]))
    code = ("import moe_expert_ffn_smoe_gb300 as m, types, pytest, sys\n"
            "assert isinstance(m._binding, types.SimpleNamespace)\n"
            "sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', 'tests/test_tokens_host.py']))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_build_without_the_headers_is_whole(built, monkeypatch, tmp_path):
    from moe_expert_ffn_smoe_gb300 import _build
    assert _build.up_to_date()
    real = dict(_build.sysconfig.get_paths())
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: dict(real, include=str(tmp_path)))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_binding.so"))
    assert _build.up_to_date()  # nothing is missing
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libsmoe.so"))
    assert not _build.up_to_date()


def test_every_call_of_the_binding_has_its_other_route(built):
    import moe_expert_ffn_smoe_gb300 as m
    names = [n for n in dir(m._binding) if n.startswith("smoe_")]
    assert len(names) == 9 and all(callable(m._by_ctypes(n)) for n in names)
