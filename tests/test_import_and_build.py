"""The package without torch, or with an extension module that does not load:
the Q4_0 functions still work with raw addresses, and the functions that need
the extension module say why they cannot run."""
import importlib.metadata
import importlib.util
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HIDE = """
import sys

class Hide:
    def find_spec(self, name, path=None, target=None):
        if name == {hidden!r} or name.startswith({hidden!r} + "."):
            raise ModuleNotFoundError("No module named " + repr(name), name=name)

sys.meta_path.insert(0, Hide())
"""

USE = """
import bit_weight_only_matmul_b200 as q4
assert q4.q4_0_bytes(4, 64) == 4 * 2 * 18 and q4.mxfp4_bytes(128, 256) == 17408
A = 1 << 20                            # never dereferenced: the checks come first
for args in ((A, A, A, 2, 64, 100), (A + 8, A, A, 2, 64, 96)):
    try:
        q4.q4_0_gemm(*args, stream=0)
    except q4.Q4Error as e:
        print("refused", e.status)
q4.q4_0_gemm(A, A, A, 0, 64, 96, stream=0)
for call in (lambda: q4.mxfp4_quantize(A, A, 2, 64), lambda: q4.mxfp4_gemm(A, A, A, 2, 64, 64),
             lambda: q4.q4_0_block_norm(A, 2, 64, x=A)):
    try:
        call()
    except ImportError as e:
        print("ImportError", e)
"""


def _run(hidden):
    r = subprocess.run([sys.executable, "-c", HIDE.format(hidden=hidden) + USE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.splitlines()


def test_import_without_torch():
    out = _run("torch")
    assert out[:2] == ["refused 1", "refused 2"]
    assert len(out) == 5 and all(line.startswith("ImportError") and "torch" in line for line in out[2:]), out


def test_import_without_the_extension_module():
    out = _run("bit_weight_only_matmul_b200._binding")
    assert out[:2] == ["refused 1", "refused 2"]
    assert len(out) == 5 and all(line.startswith("ImportError") and "build.py" in line for line in out[2:]), out


def _builder(tmp_path, monkeypatch):
    """build.py with its outputs in tmp_path and a compiler that only notes that it ran."""
    spec = importlib.util.spec_from_file_location("q4_0_b200_build_copy", os.path.join(ROOT, "bit_weight_only_matmul_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b.subprocess, "run", run)
    return b, ran


def test_binding_is_rebuilt_for_another_torch_or_interpreter(tmp_path, monkeypatch):
    b, ran = _builder(tmp_path, monkeypatch)
    b.build_binding()
    b.build_binding()
    assert len(ran) == 1
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0" if name == "torch" else version(name))
    b.build_binding()
    b.build_binding()
    assert len(ran) == 2
    monkeypatch.setattr(sys, "version", "another interpreter")
    b.build_binding()
    b.build_binding()
    assert len(ran) == 3


def test_library_alone_is_built_without_torch(tmp_path, monkeypatch, capsys):
    b, ran = _builder(tmp_path, monkeypatch)
    monkeypatch.setattr(b, "build", lambda *a: "the library")
    find_spec = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find_spec(name, *a))
    assert b.main([]) == 0
    out = capsys.readouterr().out
    assert "the library" in out and "torch" in out and not ran


def test_looking_at_the_package_needs_no_torch():
    code = HIDE.format(hidden="torch") + "import inspect, bit_weight_only_matmul_b200 as q4\n" + \
        "for v in vars(q4).values(): inspect.unwrap(v) if callable(v) else hasattr(v, '__wrapped__')\nprint('seen')"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "seen\n", r.stderr
