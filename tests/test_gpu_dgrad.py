"""The products with the transposed 4-bit weights on the GPU: w4a16_gemm_dgrad and w4a16_gated_gemm_backward against
their 64-bit forms, against differences of the forward pass, and against the forward product (adjointness)."""
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


def gradient(M, N, seed, scale=0.05):
    g = np.random.Generator(np.random.PCG64(seed))
    return (g.standard_normal((M, N)) * scale).astype(np.float16)


class Layer:
    def __init__(self, K, N, G, seed):
        c = workloads.dense(1, K, N, G, seed)
        self.K, self.N, self.G, self.S = K, N, G, dev(c.S)
        self.W = f.matrix(c.q, c.S, G)
        self.wt = device_weights(c.q)[1]


@pytest.mark.parametrize("M", [1, 5, 16, 32, 33, 64, 65, 128, 129, 200, 256, 257, 300])
@pytest.mark.parametrize("K,N,G", [(64, 64, 64), (8, 72, 16), (136, 200, 48), (520, 512, 128), (264, 1112, 80),
                                   (192, 2048, 128), (72, 4096, 32), (1112, 136, 16)])
def test_every_form(M, K, N, G):
    layer = Layer(K, N, G, seed=K + N)
    dC = gradient(M, N, M)
    flat, dA, pad = guarded_output(M, K)
    w.gemm_dgrad(dev(dC), layer.wt, layer.S, K, G, out=dA)
    ref, err = f.product(dC, layer.W.T)
    assert f.worst(dA.cpu().numpy(), ref, f.half_step(ref) + 1.001 * err) <= 1
    assert guards_intact(flat, pad, M * K)


def test_full_sizes():
    for M, K, N in [(300, 14336, 4096), (2048, 4096, 512)]:
        layer = Layer(K, N, 128, seed=M)
        dC = gradient(M, N, M)
        dA = w.gemm_dgrad(dev(dC), layer.wt, layer.S, K, 128).cpu().numpy()
        rows = np.random.Generator(np.random.PCG64(M)).choice(M, size=32, replace=False)
        ref, err = f.product(dC[rows], layer.W.T)
        assert f.worst(dA[rows], ref, f.half_step(ref) + 1.001 * err) <= 1


def test_adjoint_of_the_forward_product():
    # <A W, dC> = <A, dC W^T>: both sides from the GPU, summed in 64 bits
    M, K, N, G = 40, 512, 384, 64
    layer = Layer(K, N, G, seed=3)
    A, dC = workloads.dense(M, K, N, G, 5).A, gradient(M, N, 6)
    C = w.gemm(dev(A), layer.wt, layer.S, N, G).cpu().numpy()
    dA = w.gemm_dgrad(dev(dC), layer.wt, layer.S, K, G).cpu().numpy()
    C64, eC = f.product(A, layer.W)
    dA64, eA = f.product(dC, layer.W.T)
    left, right = np.sum(C.astype(np.float64) * dC), np.sum(A.astype(np.float64) * dA)
    bound = np.sum((f.half_step(C64) + eC) * np.abs(dC)) + np.sum((f.half_step(dA64) + eA) * np.abs(A))
    assert abs(left - right) <= bound


@pytest.mark.parametrize("M,K,N,G", [(1, 64, 64, 64), (7, 136, 200, 48), (77, 520, 264, 128), (130, 72, 1112, 16),
                                     (300, 256, 320, 64), (16, 1112, 72, 80), (64, 512, 2048, 128)])
@pytest.mark.parametrize("act", range(5))
def test_gated_backward(M, K, N, G, act):
    gate, up = Layer(K, N, G, seed=K), Layer(K, N, G, seed=N + 7)
    g, u, dH = gradient(M, N, 1, 2.0), gradient(M, N, 2, 2.0), gradient(M, N, 3)
    g[:, ::9] = 0  # relu'(0) = 0
    outs = [guarded_output(M, K), guarded_output(M, N), guarded_output(M, N)]
    w.gated_gemm_backward(dev(dH), dev(g), dev(u), gate.wt, gate.S, up.wt, up.S, K, G, act, out=outs[0][1],
                          out_gate=outs[1][1], out_up=outs[2][1])
    refs, bounds = f.gated_backward(dH, g, u, gate.W, up.W, act)
    for (flat, view, pad), ref, bound in zip(outs, refs, bounds):
        assert f.worst(view.cpu().numpy(), ref, bound) <= 1
        assert guards_intact(flat, pad, view.numel())


@pytest.mark.parametrize("act", range(5))
def test_far_gates_have_finite_slopes(act):
    M, K, N, G = 4, 64, 64, 64
    gate, up = Layer(K, N, G, seed=1), Layer(K, N, G, seed=2)
    g = np.linspace(-6e4, 6e4, M * N).astype(np.float16).reshape(M, N)
    dH, u = gradient(M, N, 3, 0.01), np.ones((M, N), dtype=np.float16)
    dA, dG, dU = w.gated_gemm_backward(dev(dH), dev(g), dev(u), gate.wt, gate.S, up.wt, up.S, K, G, act)
    (rG, rU), (eG, eU) = f.slopes(dH, g, u, act)
    assert f.worst(dG.cpu().numpy(), rG, eG) <= 1 and f.worst(dU.cpu().numpy(), rU, eU) <= 1


@pytest.mark.parametrize("act", [w.ACT_SILU, w.ACT_GELU_ERF, w.ACT_GELU_TANH, w.ACT_IDENTITY])
@pytest.mark.parametrize("M", [6, 40])
def test_forward_and_backward_against_differences(M, act):
    # directional derivative of sum(dH * H(A)) in 64 bits, by central differences, against <dA, direction>
    # from the two GPU calls run together
    K, N, G = 136, 200, 48
    gate, up = Layer(K, N, G, seed=10), Layer(K, N, G, seed=20)
    A, dH = workloads.dense(M, K, N, G, 30).A, gradient(M, N, 40)
    H, g, u = w.gated_gemm(dev(A), gate.wt, gate.S, up.wt, up.S, N, G, act, save=True)
    dA = w.gated_gemm_backward(dev(dH), g, u, gate.wt, gate.S, up.wt, up.S, K, G, act)[0].cpu().numpy()
    d = gradient(M, K, 50, 1.0).astype(np.float64)
    eps = 1e-4
    value = lambda a: np.sum(dH.astype(np.float64) * f.act(a @ gate.W, act) * (a @ up.W))
    slope = (value(A.astype(np.float64) + eps * d) - value(A.astype(np.float64) - eps * d)) / (2 * eps)
    # the kept projections are rounded to fp16: half a step each, carried by |act''| <= 1.2 and |act'| <= 1.13
    G64, U64 = A.astype(np.float64) @ gate.W, A.astype(np.float64) @ up.W
    hg, hu, h = f.half_step(G64) * 1.01, f.half_step(U64) * 1.01, np.abs(dH.astype(np.float64))
    eG = h * (1.2 * hg * np.abs(U64) + 1.13 * hu)
    eU = h * 1.13 * hg
    (_, _, _), (eA, _, _) = f.gated_backward(dH, G64, U64, gate.W, up.W, act)
    bound = np.sum((eA + 1.01 * (eG @ np.abs(gate.W).T + eU @ np.abs(up.W).T)) * np.abs(d))
    # central differences: eps^2 / 6 times a third derivative, and 1e-16 * |value| / eps: far below
    assert abs(np.sum(dA.astype(np.float64) * d) - slope) <= bound + 1e-6 * abs(slope) + 1e-9


def test_infinite_scales_stay_in_their_columns():
    # a column of W with an infinite scale makes dA infinite or NaN only for rows whose gradient reaches it; a
    # column past N never does
    K, N, G = 64, 72, 64
    layer = Layer(K, N, G, seed=4)
    layer.S[0, N - 1] = float("inf")
    dC = gradient(3, N, 5)
    dA = w.gemm_dgrad(dev(dC[:, :N - 8]), Layer(K, N - 8, G, seed=4).wt, Layer(K, N - 8, G, seed=4).S, K, G)
    assert torch.isfinite(dA).all()
    assert not torch.isfinite(w.gemm_dgrad(dev(dC), layer.wt, layer.S, K, G)).all()


def test_rows_do_not_touch_each_other():
    for M in (5, 40, 300):
        layer = Layer(264, 328, 64, seed=M)
        dC = dev(gradient(M, 328, M))
        clean = w.gemm_dgrad(dC, layer.wt, layer.S, 264, 64)
        dC[2] = float("nan")
        got = w.gemm_dgrad(dC, layer.wt, layer.S, 264, 64)
        keep = [m for m in range(M) if m != 2]
        assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[2]).all()


def test_repeats_streams_and_capture():
    M, K, N, G = 70, 512, 1024, 128
    gate, up = Layer(K, N, G, seed=1), Layer(K, N, G, seed=2)
    g, u, dH = dev(gradient(M, N, 1, 2.0)), dev(gradient(M, N, 2, 2.0)), dev(gradient(M, N, 3))
    call = lambda **kw: w.gated_gemm_backward(dH, g, u, gate.wt, gate.S, up.wt, up.S, K, G, **kw)
    ref = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (call(), call(flags=w.FLAG_STATIC_WEIGHTS, stream=side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    dH.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_no_rows():
    layer = Layer(64, 64, 64, seed=0)
    empty = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    assert w.gemm_dgrad(empty, layer.wt, layer.S, 64, 64).shape == (0, 64)
    outs = w.gated_gemm_backward(empty, empty, empty, layer.wt, layer.S, layer.wt, layer.S, 64, 64)
    assert all(x.shape == (0, 64) for x in outs)


def test_helpers_refuse_wrong_operands():
    layer = Layer(128, 64, 64, seed=0)
    dC = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        w.gemm_dgrad(dC, layer.wt, layer.S, 256, 64)  # weights of another K
    with pytest.raises(TypeError):
        w.gemm_dgrad(dC.bfloat16(), layer.wt, layer.S, 128, 64)
    with pytest.raises(ValueError):
        w.gated_gemm_backward(dC, dC[:3], dC, layer.wt, layer.S, layer.wt, layer.S, 128, 64)


def test_a_stalled_stage_ends_with_the_timeout_status():
    # the bounded waits: one stage's ready signal is withheld, the kernel latches the status and writes nothing
    layer = Layer(256, 1024, 64, seed=0)
    for M in (20, 300):
        dC = dev(gradient(M, 1024, 1))
        out = torch.full((M, 256), 7.0, dtype=torch.float16, device="cuda")
        try:
            w.w4a16_set_fault_injection(3, 2_000_000)
            w.gemm_dgrad(dC, layer.wt, layer.S, 256, 64, out=out)
            torch.cuda.synchronize()
        finally:
            w.w4a16_set_fault_injection(-1, 0)
        assert w.device_status(clear=True) == w.ERR_TIMEOUT
        assert (out == 7.0).all()
        again = w.gemm_dgrad(dC, layer.wt, layer.S, 256, 64, out=out)
        ref, err = f.product(dC.cpu().numpy(), layer.W.T)
        assert f.worst(again.cpu().numpy(), ref, f.half_step(ref) + 1.001 * err) <= 1


@pytest.mark.parametrize("M,K,N,G", [(300, 19288, 72, 48), (2000, 2680, 136, 64), (1030, 5000, 264, 128), (260, 19400, 8, 16)])
def test_two_blocks_per_cta(M, K, N, G):
    # enough output blocks that a CTA takes two; the last one alone, ending inside the block
    layer = Layer(K, N, G, seed=K)
    dC = gradient(M, N, M)
    flat, dA, pad = guarded_output(M, K)
    w.gemm_dgrad(dev(dC), layer.wt, layer.S, K, G, out=dA)
    ref, err = f.product(dC, layer.W.T)
    assert f.worst(dA.cpu().numpy(), ref, f.half_step(ref) + 1.001 * err) <= 1
    assert guards_intact(flat, pad, M * K)


def test_calls_on_two_streams_at_once():
    # forms that fill tensor memory, forms that share it and cluster splits, side by side on two streams
    shapes = [(300, 1112, 2856, 64), (40, 512, 1024, 64), (20, 264, 2048, 128), (600, 2048, 4104, 128), (5, 1024, 2048, 64)]
    calls = []
    for i, (M, K, N, G) in enumerate(shapes):
        gate, up = Layer(K, N, G, seed=i), Layer(K, N, G, seed=i + 50)
        A, dC = dev(workloads.dense(M, K, N, G, i).A), dev(gradient(M, N, i))
        calls.append(lambda a=A, g=gate, u=up, s=None: w.gated_gemm(a, g.wt, g.S, u.wt, u.S, g.N, g.G, stream=s))
        calls.append(lambda d=dC, g=gate, s=None: w.gemm_dgrad(d, g.wt, g.S, g.K, g.G, stream=s))
    refs = [c() for c in calls]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for r in range(3):
        for i in range(len(calls)):
            for x in (0, 1):  # the other stream runs the list from its other end
                j = i if x == 0 else len(calls) - 1 - i
                got[x].append((j, calls[j](s=sides[x])))
    torch.cuda.synchronize()
    for lists in got:
        for j, out in lists:
            assert torch.equal(out, refs[j]), j
