"""The range-checking build (libramnet_debug.so) on the state space layer: every kernel checks the rows, channels, segments,
chunks and workspace places it computes, and records a failed check in the status word, which the tests' ramnet_sync_status
reports.  Runs cases of every form in a child process with RAMNET_DEBUG=1.
"""
import os
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_slot_recurrent_b200", "csrc", "ssm")

CASES = ("scan_matches or ragged or cut or step_matches or conv or norm or past_32_bits or layer_prompt or captured or "
         "run_out or no_number or resets")


def test_every_kernel_checks_its_indices():
    """Each kernel's body (from its name to the next top-level brace) makes a range check."""
    found = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        src = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r"__global__[^;{]*?\b(k_\w+)\(", src):
            body = src[m.end():src.index("\n}\n", m.end())]
            assert "dcheck(" in body, f"{m.group(1)} in {name}"
            found += 1
    assert found >= 10


@pytest.mark.gpu
def test_debug_build_state_space_layer():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from sparse_slot_recurrent_b200 import build as build_mod
    build_mod.build(debug=True)
    env = dict(os.environ, RAMNET_DEBUG="1", PYTHONPATH=ROOT)
    which = subprocess.run([sys.executable, "-c", "from sparse_slot_recurrent_b200 import ramnet; ramnet.load(); "
                            "print(ramnet.LIB_PATH)"], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert which.returncode == 0, which.stderr
    assert which.stdout.strip().endswith("libramnet_debug.so")
    files = [os.path.join("tests", f) for f in ("test_ssm.py", "test_ssm_edges.py", "test_ssm_forms.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-q", "-x", "-m", "gpu", "-k", CASES, "-p", "no:cacheprovider"],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
