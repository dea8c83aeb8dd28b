"""The quantizers' debug check of weights without a GPU: no exception leaves a C entry point, whatever the sizes."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
CALL = """
import gemm_w4a16_amd as w
print(w.lib.w4a16_quantize_pack(w.W4A16_FMT_W8_ROW_FP32, 0x10000, {N}, {K}, 0x10000, 0x10000, None, None))
"""


@pytest.mark.parametrize("N,K", [(4, 64), (1 << 26, 1 << 22), (1 << 25, 1 << 20)])
def test_weights_larger_than_the_hosts_memory(N, K):
    """(with no device to copy them from: the call says so, and does not end the process)"""
    env = {**os.environ, "W4A16_DEBUG_CHECKS": "1", "HIP_VISIBLE_DEVICES": "-1"}
    out = subprocess.run([sys.executable, "-c", CALL.format(N=N, K=K)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=110)
    assert out.returncode == 0, out.stderr[-500:]
    assert out.stdout.split()[-1] == "3"  # ERR_DEVICE
