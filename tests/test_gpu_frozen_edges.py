"""The operators on frozen 4-bit weights where the ordinary cases cannot see a mistake: NaN gates, and waits that run
out."""
import numpy as np
import pytest
import torch

import frozen_util as f
import workloads
import weight_only_int4_wise_b200 as w
from gpu_util import dev, device_weights, guarded_output, guards_intact

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    w.device_status(clear=True)
    yield
    assert w.device_status(clear=True) == w.OK


class Layer:
    def __init__(self, K, N, G, seed, scale=1.0):
        c = workloads.dense(1, K, N, G, seed)
        self.K, self.N, self.G = K, N, G
        self.S64 = (c.S.astype(np.float64) * scale).astype(np.float16)
        self.S, self.W = dev(self.S64), f.matrix(c.q, self.S64, G)
        self.wt = device_weights(c.q)[1]


def normal(shape, seed, scale=1.0):
    return (np.random.Generator(np.random.PCG64(seed)).standard_normal(shape) * scale).astype(np.float16)


def gated(A, gate, up, act=w.ACT_SILU, **kw):
    return w.gated_gemm(A, gate.wt, gate.S, up.wt, up.S, gate.N, gate.G, act, **kw)


# ---------------------------------------------------------------- NaN gates


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("M,K,N", [(3, 128, 136), (16, 128, 136), (40, 512, 136), (300, 256, 136), (300, 136, 8968)])
def test_a_nan_gate_is_not_lost_forward(M, K, N, act):
    # one column of the gate has a NaN scale, the up projection is finite: the column of H is NaN whatever the activation
    gate, up = Layer(K, N, 64, 1), Layer(K, N, 64, 2)
    A = dev(normal((M, K), 3))
    clean = gated(A, gate, up, act)
    gate.S[0, 5] = float("nan")
    H, g, _ = gated(A, gate, up, act, save=True)
    rest = [n for n in range(N) if n != 5]
    assert torch.isnan(H[:, 5]).all() and torch.isnan(g[:, 5]).all()
    assert torch.equal(H[:, rest], clean[:, rest]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("act", range(5))
def test_a_nan_gate_is_not_lost_backward(act):
    M, K, N, G = 6, 64, 72, 64
    gate, up = Layer(K, N, G, 1), Layer(K, N, G, 2)
    g, u, dH = dev(normal((M, N), 1)), dev(normal((M, N), 2)), dev(normal((M, N), 3, 0.05))
    call = lambda: w.gated_gemm_backward(dH, g, u, gate.wt, gate.S, up.wt, up.S, K, G, act)
    clean = call()
    g[2, 9] = float("nan")
    dA, dG, dU = call()
    assert torch.isnan(dU[2, 9]) and torch.isnan(dA[2]).all()
    assert torch.isnan(dG[2, 9]) or act == w.ACT_IDENTITY  # (the identity's slope is 1 everywhere)
    rows, cols = [m for m in range(M) if m != 2], [n for n in range(N) if n != 9]
    assert torch.equal(dA[rows], clean[0][rows])
    for got, ref in ((dG, clean[1]), (dU, clean[2])):
        assert torch.equal(got[rows], ref[rows]) and torch.equal(got[:, cols], ref[:, cols])


# ---------------------------------------------------------------- waits that run out


def test_transposed_stall_stage_counts_from_each_ranks_range():
    # 16 stages over a cluster of two: no rank has a stage 8 of its own, both have a stage 7
    layer = Layer(256, 1024, 64, 0)
    dC = normal((20, 1024), 1, 0.05)
    ref, err = f.product(dC, layer.W.T)
    for stage, status in ((8, w.OK), (7, w.ERR_TIMEOUT)):
        out = torch.full((20, 256), 7.0, dtype=torch.float16, device="cuda")
        try:
            w.w4a16_set_fault_injection(stage, 2_000_000)
            w.gemm_dgrad(dev(dC), layer.wt, layer.S, 256, 64, out=out)
            torch.cuda.synchronize()
        finally:
            w.w4a16_set_fault_injection(-1, 0)
        assert w.device_status(clear=True) == status
        if status == w.OK:
            assert f.worst(out.cpu().numpy(), ref, f.half_step(ref) + 1.001 * err) <= 1
        else:
            assert (out == 7.0).all()


class Adapters:
    def __init__(self, layer, M, L, R, seed, la_scale=None):
        self.layer = layer
        self.LA = normal((L, R, layer.K), seed, la_scale or 1 / np.sqrt(layer.K))
        self.LB = normal((L, layer.N, R), seed + 1, 0.1)
        self.ids = (np.arange(M) % L).astype(np.int32)
        self.scaling = np.linspace(0.5, 1.5, L).astype(np.float32)

    def run(self, A, **kw):
        x = self.layer
        return w.lora_gemm(A, x.wt, x.S, x.N, x.G, dev(self.LA), dev(self.LB), dev(self.ids), dev(self.scaling), **kw)

    def reference(self, A):
        return f.lora(A, self.layer.W, self.LA, self.LB, self.ids, self.scaling)


@pytest.mark.parametrize("M,K,N", [(40, 1024, 512), (130, 320, 264), (300, 1024, 520)])
def test_adapter_product_with_a_stalled_stage_writes_nothing(M, K, N):
    a = Adapters(Layer(K, N, 64, M), M, 5, 16, M)
    A = normal((M, K), 9)
    out = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
    try:
        w.w4a16_set_fault_injection(0, 2_000_000)
        a.run(dev(A), out=out)
        torch.cuda.synchronize()
    finally:
        w.w4a16_set_fault_injection(-1, 0)
    assert w.device_status(clear=True) == w.ERR_TIMEOUT
    assert (out == 7.0).all()
    ref, bound = a.reference(A)
    assert f.worst(a.run(dev(A)).cpu().numpy(), ref, bound) <= 1


@pytest.mark.parametrize("M", [1, 16])
def test_decode_forms_with_a_short_wait_limit(M):
    # the wait for the activations may or may not run out: each block of columns is right or untouched, and reported
    K, N, G = 4096, 2056, 128
    gate, up = Layer(K, N, G, 1), Layer(K, N, G, 2)
    a = Adapters(gate, M, 3, 16, 5)
    A = normal((M, K), 9)
    (H, _, _), (eH, _, _) = f.gated(A, gate.W, up.W, w.ACT_SILU)
    C, eC = a.reference(A)
    for call, ref, bound in ((lambda **kw: gated(dev(A), gate, up, **kw), H, eH), (lambda **kw: a.run(dev(A), **kw), C, eC)):
        out = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
        try:
            w.w4a16_set_fault_injection(-1, 1)
            call(out=out)
            torch.cuda.synchronize()
        finally:
            w.w4a16_set_fault_injection(-1, 0)
        status = w.device_status(clear=True)
        got = out.cpu().numpy()
        missing = np.isnan(got)
        assert status == (w.ERR_TIMEOUT if missing.any() else status) and status in (w.OK, w.ERR_TIMEOUT)
        blocks = missing.reshape(M, N // 8, 8)
        assert (blocks == blocks[:1, :, :1]).all()  # whole columns in blocks of eight
        assert np.all(np.abs(got.astype(np.float64) - ref)[~missing] <= bound[~missing])
        assert f.worst(call().cpu().numpy(), ref, bound) <= 1
