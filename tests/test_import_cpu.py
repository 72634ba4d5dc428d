"""The package, its build and the library without torch: a host that only builds
the C library has none."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=600)


def test_the_build_needs_no_torch():
    r = _python("import sys; sys.modules['torch'] = None; import deepseek_v4_flash_gb300.build as b; print(len(b.sources()))")
    assert r.returncode == 0, r.stderr
    assert int(r.stdout) > 0


def test_the_binding_loads_without_torch():
    r = _python("import sys; sys.modules['torch'] = None; import deepseek_v4_flash_gb300 as d; "
                "print(d.lib().ds4moe_abi_version() == d.ABI_VERSION, d.AttentionDesc(8, 2, 64).c().head_dim)\n"
                "try: d.Rope(None)\n"
                "except ImportError: print('a call that needs it says so')")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:2] == ["True 64", "a call that needs it says so"]


def test_importing_does_not_import_torch():
    r = _python("import sys, deepseek_v4_flash_gb300; print('torch' in sys.modules)")
    assert r.returncode == 0 and r.stdout.strip() == "False", r.stderr
