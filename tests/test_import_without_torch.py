"""The package's host calls need no torch: it is imported by the calls that take tensors."""
import os
import subprocess
import sys

from tests.conftest import ROOT


def test_host_calls_without_torch():
    code = ("import sys; sys.modules['torch'] = None\n"  # any import of it raises ImportError
            "import compressed_output_head_amd as ah\n"
            "assert ah.archead_pack_layout(1000, 256, 8, 8, 64)['total_bytes'] > 0\n"
            "assert ah.archead_loss_workspace_bytes(480, 151936, 4) > 0\n"
            "assert ah.archead_logits_backward_workspace_bytes(1000, 256, 8, 8, 64, 4) > 0\n"
            "print(ah.archead_status_string(0))\n")
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=100,
                         env=dict(os.environ, PYTHONPATH=ROOT))
    assert run.returncode == 0, run.stderr
