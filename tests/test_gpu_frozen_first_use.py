"""What a process pays for at its first calls, seen from fresh processes."""
import json
import os
import subprocess
import sys

import pytest

import weight_only_int4_wise_b200 as w

pytestmark = pytest.mark.gpu

PROGRAM = """
import json, time
import torch
import weight_only_int4_wise_b200 as w
M, K, N, G = 32, 512, 512, 64
half = dict(device="cuda", dtype=torch.float16)
A, S, C = torch.zeros((M, K), **half), torch.ones((K // G, N), **half), torch.empty((M, N), **half)
wt = torch.zeros(w.w4a16_tiled_bytes(K, N), dtype=torch.uint8, device="cuda")
calls = {
    "plain": lambda: w.w4a16_gemm(A, wt, S, C, M, N, K, G),
    "gated": lambda: w.w4a16_gated_gemm(A, wt, S, wt, S, C, None, None, M, N, K, G, w.ACT_SILU),
}
out = {}
for name, call in calls.items():
    times = []
    for _ in range(20):
        torch.cuda.synchronize()
        start = time.perf_counter()
        assert call() == w.OK
        times.append(time.perf_counter() - start)
    torch.cuda.synchronize()
    out[name] = [times[0], min(times[1:])]
print(json.dumps(out))
"""


def test_the_plain_product_does_not_prepare_the_other_forms():
    # the set-up of a form (attributes, loading its kernels: milliseconds) falls to the first call of that form, not to
    # the first plain product
    root = os.path.dirname(os.path.dirname(os.path.abspath(w.__file__)))
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    times = json.loads(run.stdout.splitlines()[-1])
    for name in ("plain", "gated"):
        first, later = times[name]
        assert first > 20 * later, (name, times)
