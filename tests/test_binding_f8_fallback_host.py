"""The package without _binding_f8.so, as built where Python's headers are missing:
its calls convert and refuse as with it."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_host_tests_of_the_calls_pass_without_it(tmp_path):
    import __graft_entry__
    __graft_entry__.build_library()
    (tmp_path / "sitecustomize.py").write_text(
        "import sys\nsys.modules['moe_expert_ffn_smoe_gb300._binding_f8'] = None\n")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT, os.environ.get("PYTHONPATH", "")]))
    code = ("import moe_expert_ffn_smoe_gb300 as m, types, pytest, sys\n"
            "assert isinstance(m._binding_f8, types.SimpleNamespace)\n"
            "sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', 'tests/test_scores_host.py', 'tests/test_f8_host.py']))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
