"""Loading the library: a host-only caller does not pay torch's import, and a process that imports torch later has
one HIP runtime, torch's."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
import numpy as np
import w4a4_integer_gemm_amd as fq
fq.fq_rope_freqs(64)
fq.fq_fp8_pack_weights(np.ones((8, 128), np.float32))
fq.fq_pack_weights(np.ones((8, 128), np.float32), None, 0, 64, 8)
print("torch imported:", "torch" in sys.modules)
import torch
paths = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
print("runtimes:", sorted(paths))
print("of torch:", all(p.startswith(torch.__path__[0]) for p in paths) if len(paths) else None)
"""


def test_host_calls_do_not_import_torch_and_leave_one_runtime():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = dict(line.split(": ", 1) for line in r.stdout.splitlines() if ": " in line)
    assert out["torch imported"] == "False"
    import torch
    if os.path.exists(os.path.join(torch.__path__[0], "lib", "libamdhip64.so")):
        assert out["runtimes"].count("libamdhip64") == 1 and out["of torch"] == "True", out


def test_a_torch_that_cannot_be_loaded_leaves_the_host_calls(tmp_path):
    lib = tmp_path / "torch" / "lib"
    lib.mkdir(parents=True)
    (tmp_path / "torch" / "__init__.py").write_text("raise ImportError('broken')")
    (lib / "libamdhip64.so").write_text("no library")
    code = "import sys; sys.path.insert(0, %r)\nimport w4a4_integer_gemm_amd as fq\nprint(len(fq.fq_rope_freqs(64)[0]))" % str(tmp_path)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["32"], r.stderr[-2000:]
