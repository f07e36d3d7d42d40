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
    # ... and neither does loading the code of those forms: it takes about 16 ms, and the preparation alone less than 1
    # (not measured against the first plain product, which on a cold machine also waits for the file)
    assert times["gated"][0] > 3e-3, times


CAPTURED = """
import sys
import torch
import weight_only_int4_wise_b200 as w
form, M, K, N, G = sys.argv[1], int(sys.argv[2]), 512, 512, 64
half = dict(device="cuda", dtype=torch.float16)
A, S, C = torch.randn((M, K), **half), torch.rand((K // G, N), **half) * 0.02, torch.zeros((M, N), **half)
wt = torch.randint(0, 255, (w.w4a16_tiled_bytes(K, N),), dtype=torch.uint8, device="cuda")
LA, LB = torch.randn((2, 16, K), **half) * 0.05, torch.randn((2, N, 16), **half) * 0.05
ids = (torch.arange(M, device="cuda") % 3 - 1).int()
call = {
    "gated": lambda: w.gated_gemm(A, wt, S, wt, S, N, G, out=C),
    "adapters": lambda: w.lora_gemm(A, wt, S, N, G, LA, LB, ids, out=C),
    "transposed": lambda: w.gemm_dgrad(A, wt, S, K, G, out=C),
}[form]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
first = C.clone()
C.zero_()
call()
torch.cuda.synchronize()
assert torch.equal(first, C) and bool(C.any())
"""


@pytest.mark.parametrize("form,M", [("gated", 40), ("gated", 300), ("adapters", 8), ("adapters", 300), ("transposed", 40)])
def test_the_first_call_of_a_form_may_be_a_captured_one(form, M):
    root = os.path.dirname(os.path.dirname(os.path.abspath(w.__file__)))
    run = subprocess.run([sys.executable, "-c", CAPTURED, form, str(M)], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr
