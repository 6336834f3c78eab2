"""The package without torch, or with an extension module that does not load:
the Q4_0 functions still work with raw addresses, and the functions that need
the extension module say why they cannot run."""
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
