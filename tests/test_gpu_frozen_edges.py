"""The operators on frozen 4-bit weights where the ordinary cases cannot see a mistake: NaN gates, waits that run out,
infinite scales beside a clamped load, contractions of which only a few neighbouring k count, outputs that are only
2-byte aligned, the tensor-core forms at decode sizes, full-size transposed products of few rows, offsets past 32
bits."""
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


# ---------------------------------------------------------------- infinite scales beside clamped loads


def infinite_tail(S):
    """The scales as the head of a larger buffer that goes on with infinities."""
    flat = torch.full((S.numel() + 4096,), float("inf"), dtype=torch.float16, device="cuda")
    flat[:S.numel()] = S.reshape(-1)
    return flat[:S.numel()].view_as(S)


@pytest.mark.parametrize("M", [3, 40, 100, 300])
@pytest.mark.parametrize("K,G", [(192, 64), (144, 48), (200, 80), (19400, 6480)])
@pytest.mark.parametrize("column", [0, 71])
def test_transposed_infinite_scale_stays_in_its_group(M, K, G, column):
    # N = 72 ends inside a 64-deep stage: what is decoded past N must be exact zeros, whatever scale a clamped or
    # overrunning load would meet. An infinite scale in one group reaches the k of that group and no other.
    N = 72
    layer, other = Layer(K, N, G, 4), Layer(K, N, G, 5)
    dC, g, u = dev(normal((M, N), 5)), dev(normal((M, N), 6)), dev(normal((M, N), 7))
    calls = (lambda S: w.gemm_dgrad(dC, layer.wt, S, K, G),
             lambda S: w.gated_gemm_backward(dC, g, u, layer.wt, S, other.wt, infinite_tail(other.S), K, G)[0],
             lambda S: w.gated_gemm_backward(dC, g, u, other.wt, infinite_tail(other.S), layer.wt, S, K, G)[0])
    for call in calls:
        clean = call(layer.S)
        assert torch.isfinite(clean).all()
        groups = layer.S.shape[0]
        for group in (1, groups - 1):
            S = infinite_tail(layer.S)
            assert torch.equal(call(S), clean)
            S[group, column] = float("inf")
            got = call(S)
            lo, hi = group * G, min(K, (group + 1) * G)
            assert not torch.isfinite(got[:, lo:hi]).any()
            assert torch.equal(got[:, :lo], clean[:, :lo]) and torch.equal(got[:, hi:], clean[:, hi:])


@pytest.mark.parametrize("M", [2, 16, 40, 300])
@pytest.mark.parametrize("K,G", [(200, 80), (320, 64)])
@pytest.mark.parametrize("N", [72, 8968])
def test_forward_infinite_scale_stays_in_its_column(M, K, G, N):
    gate, up = Layer(K, N, G, 4), Layer(K, N, G, 5)
    a = Adapters(gate, M, 3, 8, 6)
    A = dev(normal((M, K), 7))
    calls = (lambda S: w.gated_gemm(A, gate.wt, S, up.wt, infinite_tail(up.S), N, G, w.ACT_GELU_ERF),
             lambda S: w.gated_gemm(A, up.wt, infinite_tail(up.S), gate.wt, S, N, G, w.ACT_IDENTITY),
             lambda S: w.lora_gemm(A, gate.wt, S, N, G, dev(a.LA), dev(a.LB), dev(a.ids)))
    for call in calls:
        clean = call(infinite_tail(gate.S))
        assert torch.isfinite(clean).all()
        for group in (0, gate.S.shape[0] - 1):
            for column in (0, N - 1):
                S = infinite_tail(gate.S)
                S[group, column] = float("nan")
                got = call(S)
                rest = [n for n in range(N) if n != column]
                assert torch.isnan(got[:, column]).all() and torch.equal(got[:, rest], clean[:, rest])


# ---------------------------------------------------------------- contractions of which a few k count


def windows(K, step=128):
    """Runs of 16 k around every multiple of `step`, and the last eight k."""
    return [(max(0, k - 8), min(K, k + 8)) for k in range(0, K, step)] + [(K - 8, K)]


def windowed(M, K, seed):
    """Batches (A, (lo, hi) per row): every row of A is zero outside its window, so that a result and its error bound
    come from a few terms and none of them can be lost unseen."""
    todo = windows(K)
    rng = np.random.Generator(np.random.PCG64(seed))
    for i in range(0, len(todo), M):
        part = [todo[min(i + m, len(todo) - 1)] for m in range(M)]
        A = np.zeros((M, K), dtype=np.float16)
        for m, (lo, hi) in enumerate(part):
            A[m, lo:hi] = rng.uniform(1.0, 2.0, hi - lo)
        yield A, part


def products(A, part, W, terms):
    """A @ W row by row over the rows' windows, and the bounds of the 32-bit sums (zeros add no error: the sum has as
    many steps that change it as the window has, but the tolerance counts all `terms`)."""
    ref = np.stack([A[m, lo:hi].astype(np.float64) @ W[lo:hi] for m, (lo, hi) in enumerate(part)])
    T = np.stack([np.abs(A[m, lo:hi].astype(np.float64)) @ np.abs(W[lo:hi]) for m, (lo, hi) in enumerate(part)])
    return ref, f.sum_error(terms, T)


@pytest.mark.parametrize("M,K,N,G", [(16, 14336, 64, 128), (9, 14344, 72, 48), (13, 8200, 136, 80), (1, 120008, 8, 64),
                                     (16, 20000, 8, 32), (1, 4104, 4104, 64), (40, 4104, 72, 64), (200, 2056, 8, 48),
                                     (300, 2056, 8968, 64)])
def test_no_part_of_a_long_contraction_is_lost(M, K, N, G):
    gate, up = Layer(K, N, G, K), Layer(K, N, G, K + 1)
    for A, part in windowed(M, K, 3):
        H, g, u = (x.cpu().numpy() for x in gated(dev(A), gate, up, w.ACT_RELU, save=True))
        for got, layer in ((g, gate), (u, up)):
            ref, err = products(A, part, layer.W, K)
            assert f.worst(got, ref, f.half_step(ref) + 1.001 * err) <= 1


@pytest.mark.parametrize("M,K,N,G", [(16, 14336, 64, 128), (11, 14344, 72, 48), (1, 120008, 8, 64), (1, 4104, 4104, 64),
                                     (40, 4104, 72, 64), (300, 2056, 72, 48), (1100, 2056, 136, 64)])
def test_no_part_of_the_adapters_contraction_is_lost(M, K, N, G):
    # the shared projection's scales are small beside the adapters: what counts is V
    layer = Layer(K, N, G, K, scale=2.0 ** -6)
    L, R = min(M, 3), 16
    a = Adapters(layer, M, L, R, K, la_scale=0.25)
    A64, B64 = a.LA.astype(np.float64), a.LB.astype(np.float64)
    for A, part in windowed(M, K, 5):
        got = a.run(dev(A)).cpu().numpy()
        ref, err = products(A, part, layer.W, K)
        for m, (lo, hi) in enumerate(part):
            i, s = a.ids[m], float(a.scaling[a.ids[m]])
            x = A[m, lo:hi].astype(np.float64)
            v = s * (A64[i][:, lo:hi] @ x)
            ev = f.sum_error(K, s * (np.abs(A64[i][:, lo:hi]) @ np.abs(x))) + np.abs(v) * 2.0 ** -24
            ev = ev + f.half_step(np.abs(v) + ev)
            ref[m] += B64[i] @ v
            err[m] += np.abs(B64[i]) @ ev + f.sum_error(R, np.abs(B64[i]) @ np.abs(v))
        assert f.worst(got, ref, f.half_step(ref) + 1.001 * err) <= 1


@pytest.mark.parametrize("M,K,N,G", [(8, 72, 14344, 16), (40, 136, 4104, 64), (100, 264, 2056, 48), (300, 64, 4104, 64),
                                     (300, 19400, 1032, 64)])
def test_no_part_of_the_transposed_contraction_is_lost(M, K, N, G):
    layer = Layer(K, N, G, N)
    for dC, part in windowed(M, N, 4):
        got = w.gemm_dgrad(dev(dC), layer.wt, layer.S, K, G).cpu().numpy()
        ref, err = products(dC, part, layer.W.T, N)
        assert f.worst(got, ref, f.half_step(ref) + 1.001 * err) <= 1


# ---------------------------------------------------------------- forms and alignments that few calls reach


# Group sizes whose index needs more than a multiply-shift at this K: a few rows run on the tensor cores.
@pytest.mark.parametrize("G", [65280, 65552])
@pytest.mark.parametrize("M", [1, 5, 16])
def test_tensor_core_forms_at_decode_sizes(M, G):
    K, N = 66320, 72
    gate, up = Layer(K, N, G, 1), Layer(K, N, G, 2)
    A = normal((M, K), 3, 0.25)
    outs = [guarded_output(M, N) for _ in range(3)]
    gated(dev(A), gate, up, w.ACT_SILU, save=True, out=outs[0][1], out_gate=outs[1][1], out_up=outs[2][1])
    refs, bounds = f.gated(A, gate.W, up.W, w.ACT_SILU)
    for (flat, view, pad), ref, bound in zip(outs, refs, bounds):
        assert f.worst(view.cpu().numpy(), ref, bound) <= 1
        assert guards_intact(flat, pad, M * N)
    a = Adapters(gate, M, 5, 24, 4)
    a.ids[-1] = -1
    flat, out, pad = guarded_output(M, N)
    a.run(dev(A), out=out)
    ref, bound = a.reference(A)
    assert f.worst(out.cpu().numpy(), ref, bound) <= 1
    assert guards_intact(flat, pad, M * N)
    for A, part in list(windowed(M, K, 5))[-3:]:  # the last groups' border and the tail
        g = gated(dev(A), gate, up, w.ACT_RELU, save=True)[1].cpu().numpy()
        ref, err = products(A, part, gate.W, K)
        assert f.worst(g, ref, f.half_step(ref) + 1.001 * err) <= 1


ODD = 65  # elements in front of an output: it starts on a 2-byte boundary


@pytest.mark.parametrize("M,K,N,G", [(4, 200, 136, 48), (16, 512, 264, 64), (40, 1024, 136, 64), (130, 264, 136, 64),
                                     (300, 136, 8968, 48), (200, 264, 14336, 64)])
def test_outputs_on_two_byte_boundaries_forward(M, K, N, G):
    gate, up = Layer(K, N, G, 1), Layer(K, N, G, 2)
    A = normal((M, K), 3)
    refs, bounds = f.gated(A, gate.W, up.W, w.ACT_SILU)
    for pads in ((ODD, 64, 64), (64, ODD, 64), (ODD, ODD, ODD)):
        outs = [guarded_output(M, N, p) for p in pads]
        gated(dev(A), gate, up, w.ACT_SILU, save=True, out=outs[0][1], out_gate=outs[1][1], out_up=outs[2][1])
        for (flat, view, pad), ref, bound in zip(outs, refs, bounds):
            assert f.worst(view.cpu().numpy(), ref, bound) <= 1
            assert guards_intact(flat, pad, M * N)
    a = Adapters(gate, M, 3, 8, 4)
    flat, out, pad = guarded_output(M, N, ODD)
    a.run(dev(A), out=out)
    ref, bound = a.reference(A)
    assert f.worst(out.cpu().numpy(), ref, bound) <= 1
    assert guards_intact(flat, pad, M * N)


@pytest.mark.parametrize("M,K,N,G", [(5, 136, 200, 48), (20, 256, 1024, 64), (100, 136, 2048, 64), (300, 264, 328, 64),
                                     (300, 19288, 72, 48)])
def test_outputs_on_two_byte_boundaries_transposed(M, K, N, G):
    gate, up = Layer(K, N, G, 1), Layer(K, N, G, 2)
    dC, g, u = normal((M, N), 3, 0.05), normal((M, N), 4), normal((M, N), 5)
    flat, dA, pad = guarded_output(M, K, ODD)
    w.gemm_dgrad(dev(dC), gate.wt, gate.S, K, G, out=dA)
    ref, err = f.product(dC, gate.W.T)
    assert f.worst(dA.cpu().numpy(), ref, f.half_step(ref) + 1.001 * err) <= 1
    assert guards_intact(flat, pad, M * K)
    flat, dA, pad = guarded_output(M, K, ODD)
    w.gated_gemm_backward(dev(dC), dev(g), dev(u), gate.wt, gate.S, up.wt, up.S, K, G, out=dA)
    refs, bounds = f.gated_backward(dC, g, u, gate.W, up.W, w.ACT_SILU)
    assert f.worst(dA.cpu().numpy(), refs[0], bounds[0]) <= 1
    assert guards_intact(flat, pad, M * K)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (16, 14336, 4096), (17, 4096, 14336), (64, 14336, 4096),
                                   (128, 4096, 14336), (130, 14336, 4096)])
def test_full_size_transposed_products_of_few_rows(M, K, N):
    layer = Layer(K, N, 128, M)
    dC = normal((M, N), M, 0.05)
    dA = w.gemm_dgrad(dev(dC), layer.wt, layer.S, K, 128).cpu().numpy()
    rows = np.random.Generator(np.random.PCG64(M)).choice(M, size=min(M, 16), replace=False)
    ref, err = f.product(dC[rows], layer.W.T)
    assert f.worst(dA[rows], ref, f.half_step(ref) + 1.001 * err) <= 1


# ---------------------------------------------------------------- offsets past 32 bits


def tail_rows(x, n):
    return x[-n:].cpu().numpy()


def test_many_rows_past_32_bit_offsets():
    # 150000 rows of 14336: rows and outputs past 2^31 elements; the last rows against 64 bits
    M, K, N, G, last = 150_000, 64, 14336, 64, 24
    gate, up = Layer(K, N, G, 1), Layer(K, N, G, 2)
    A = torch.randn((M, K), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").half()
    H, g, u = gated(A, gate, up, w.ACT_SILU, save=True)
    refs, bounds = f.gated(tail_rows(A, last), gate.W, up.W, w.ACT_SILU)
    for got, ref, bound in zip((H, g, u), refs, bounds):
        assert f.worst(tail_rows(got, last), ref, bound) <= 1
    H.mul_(2.0 ** -6)
    dA, dG, dU = w.gated_gemm_backward(H, g, u, gate.wt, gate.S, up.wt, up.S, K, G, w.ACT_SILU)
    refs, bounds = f.gated_backward(*(tail_rows(x, last) for x in (H, g, u)), gate.W, up.W, w.ACT_SILU)
    for got, ref, bound in zip((dA, dG, dU), refs, bounds):
        assert f.worst(tail_rows(got, last), ref, bound) <= 1
    del g, u, dG, dU
    dA = w.gemm_dgrad(H, gate.wt, gate.S, K, G)
    ref, err = f.product(tail_rows(H, last), gate.W.T)
    assert f.worst(tail_rows(dA, last), ref, f.half_step(ref) + 1.001 * err) <= 1
    a = Adapters(gate, last, 3, 8, 4)
    tail_ids = a.ids
    a.ids = np.concatenate([np.full(M - last, 1, dtype=np.int32), tail_ids])
    C = a.run(A)
    a.ids = tail_ids
    ref, bound = a.reference(tail_rows(A, last))
    assert f.worst(tail_rows(C, last), ref, bound) <= 1


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("K,N", [(64, 14336), (14336, 64)])
def test_many_adapters_past_32_bit_offsets(M, K, N):
    # 1200 adapters of rank 128: the stacked matrices of 14336 pass 2^31 elements; the first and last adapter are used
    L, R, G = 1200, 128, 64
    layer = Layer(K, N, G, 1)
    a = Adapters(layer, M, 2, R, 2)
    LA = torch.zeros((L, R, K), dtype=torch.float16, device="cuda")
    LB = torch.zeros((L, N, R), dtype=torch.float16, device="cuda")
    LA[0], LA[-1], LB[0], LB[-1] = dev(a.LA[0]), dev(a.LA[1]), dev(a.LB[0]), dev(a.LB[1])
    A = normal((M, K), 3)
    got = w.lora_gemm(dev(A), layer.wt, layer.S, N, G, LA, LB, dev(a.ids * (L - 1)))
    a.scaling[:] = 1
    ref, bound = a.reference(A)
    assert f.worst(got.cpu().numpy(), ref, bound) <= 1
