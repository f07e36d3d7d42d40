"""The gated projections on the GPU (w4a16_gated_gemm) against their 64-bit form: every launch form (one to sixteen
rows on the skinny kernel, token tiles of 16 to 256 rows, K split over a cluster or not), odd sizes, every activation,
with and without the projections kept."""
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


class Case:
    def __init__(self, M, K, N, G, seed, a_scale=1.0):
        gate = workloads.dense(M, K, N, G, seed, a_scale=a_scale)
        up = workloads.dense(1, K, N, G, seed + 1000)
        self.M, self.K, self.N, self.G = M, K, N, G
        self.A, self.Sg, self.Su = gate.A, gate.S, up.S
        self.Wg, self.Wu = f.matrix(gate.q, gate.S, G), f.matrix(up.q, up.S, G)
        self.wg, self.wu = device_weights(gate.q)[1], device_weights(up.q)[1]

    def run(self, act, save=False, A=None, **kw):
        A = dev(self.A) if A is None else A
        out = w.gated_gemm(A, self.wg, dev(self.Sg), self.wu, dev(self.Su), self.N, self.G, act, save=save, **kw)
        torch.cuda.synchronize()
        return out


def check(c, act, save):
    flats = [guarded_output(c.M, c.N) for _ in range(3 if save else 1)]
    names = ["out", "out_gate", "out_up"]
    c.run(act, save, **{n: v for n, (_, v, _) in zip(names, flats)})
    refs, bounds = f.gated(c.A, c.Wg, c.Wu, act)
    for (flat, view, pad), ref, bound, name in zip(flats, refs, bounds, names):
        assert f.worst(view.cpu().numpy(), ref, bound) <= 1, (name, c.M, c.K, c.N, c.G, act)
        assert guards_intact(flat, pad, c.M * c.N), name


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 129, 200, 256, 300])
@pytest.mark.parametrize("K,N,G", [(64, 64, 64), (72, 8, 16), (200, 136, 48), (512, 520, 128), (1112, 264, 80),
                                   (2048, 192, 128), (4096, 72, 64)])
def test_every_form(M, K, N, G):
    c = Case(M, K, N, G, seed=M + K)
    check(c, act=(M + K // 8) % 5, save=(M + N // 8) % 2 == 0)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("M", [3, 16, 40, 270])
def test_every_activation_with_projections(M, act):
    check(Case(M, 384, 200, 128, seed=act * 10 + M), act, save=True)


@pytest.mark.parametrize("M", [4, 16, 100, 300])
@pytest.mark.parametrize("act", [w.ACT_SILU, w.ACT_GELU_TANH, w.ACT_GELU_ERF])
def test_large_projections_saturate_without_nan(M, act):
    # gates of several thousand of either sign: the activation is x or 0 there, never NaN
    c = Case(M, 256, 128, 128, seed=act, a_scale=300.0)
    H, g, u = c.run(act, save=True)
    refs, _ = f.gated(c.A, c.Wg, c.Wu, act)
    got, ref = H.cpu().numpy().astype(np.float64), refs[0]
    assert not np.isnan(got).any() and np.abs(refs[1]).max() > 500
    small = np.abs(ref) < 60000
    assert np.allclose(got[small], ref[small], rtol=2e-3, atol=np.abs(refs[2]).max() * 1e-3)
    assert np.all(np.abs(got[~small]) > 59000)


def test_full_size_decode_and_prompt():
    for M in (1, 16, 200):
        c = Case(M, 4096, 14336, 128, seed=M)
        H = c.run(w.ACT_SILU).cpu().numpy()
        cols = np.random.Generator(np.random.PCG64(M)).choice(c.N, size=512, replace=False)
        refs, bounds = f.gated(c.A, c.Wg[:, cols], c.Wu[:, cols], w.ACT_SILU)
        assert f.worst(H[:, cols], refs[0], bounds[0]) <= 1


def test_rows_do_not_touch_each_other():
    # a row of NaN or infinities makes its own outputs NaN and no other's
    for M in (5, 16, 40, 300):
        c = Case(M, 256, 136, 64, seed=M)
        clean = c.run(w.ACT_SILU).clone()
        A = dev(c.A)
        A[1] = float("nan")
        A[3, 17] = float("inf")
        got = c.run(w.ACT_SILU, A=A)
        keep = [m for m in range(M) if m not in (1, 3)]
        assert torch.equal(got[keep], clean[keep])
        assert torch.isnan(got[1]).all()


def test_no_rows():
    c = Case(1, 64, 64, 64, seed=0)
    H, g, u = c.run(w.ACT_SILU, save=True, A=torch.empty((0, 64), dtype=torch.float16, device="cuda"))
    assert H.shape == g.shape == u.shape == (0, 64)


def test_strided_activations_and_streams():
    for M in (6, 50):
        c = Case(M, 320, 128, 64, seed=M)
        ref = c.run(w.ACT_SILU).clone()
        wide = torch.zeros((M, 640), dtype=torch.float16, device="cuda")
        wide[:, ::2] = dev(c.A)
        assert torch.equal(c.run(w.ACT_SILU, A=wide[:, ::2]), ref)
        S = [dev(c.Sg), dev(c.Su)]
        A = dev(c.A)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out = w.gated_gemm(A, c.wg, S[0], c.wu, S[1], c.N, c.G)
        other = w.gated_gemm(A, c.wg, S[0], c.wu, S[1], c.N, c.G, flags=w.FLAG_STATIC_WEIGHTS, stream=side)
        side.synchronize()
        assert torch.equal(out, ref) and torch.equal(other, ref)


@pytest.mark.parametrize("M", [1, 16, 100])
def test_captured_calls_replay(M):
    c = Case(M, 512, 256, 128, seed=M)
    A, Sg, Su = dev(c.A), dev(c.Sg), dev(c.Su)
    H = torch.empty((M, c.N), dtype=torch.float16, device="cuda")
    w.gated_gemm(A, c.wg, Sg, c.wu, Su, c.N, c.G, out=H)  # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.gated_gemm(A, c.wg, Sg, c.wu, Su, c.N, c.G, out=H)
    A.copy_(A.flip(0) * 0.5)
    H.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ref, bound = f.gated(A.cpu().numpy(), c.Wg, c.Wu, w.ACT_SILU)
    assert f.worst(H.cpu().numpy(), ref[0], bound[0]) <= 1


def test_repeats_are_bitwise_equal():
    for M in (1, 12, 64, 300):
        c = Case(M, 2048, 256, 128, seed=M)
        ref = c.run(w.ACT_SILU).clone()
        for _ in range(3):
            assert torch.equal(c.run(w.ACT_SILU), ref)


def test_helper_refuses_wrong_operands():
    c = Case(4, 128, 64, 64, seed=1)
    A, Sg, Su = dev(c.A), dev(c.Sg), dev(c.Su)
    with pytest.raises(TypeError):
        w.gated_gemm(A.float(), c.wg, Sg, c.wu, Su, c.N, c.G)
    with pytest.raises(ValueError):
        w.gated_gemm(A, c.wg[:-4096], Sg, c.wu, Su, c.N, c.G)  # a tile short
    with pytest.raises(ValueError):
        w.gated_gemm(A, c.wg, Sg[:1], c.wu, Su, c.N, c.G)      # a group short
    with pytest.raises(ValueError):
        w.gated_gemm(A, c.wg, Sg, c.wu, Su, c.N, c.G, out=torch.empty((4, 32), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        w.gated_gemm(A.cpu(), c.wg, Sg, c.wu, Su, c.N, c.G)
    with pytest.raises(w.W4A16Error):
        w.gated_gemm(A, c.wg, Sg, c.wu, Su, c.N, c.G, act=9)


@pytest.mark.parametrize("M,K,N,G,save", [(200, 264, 14336, 64, True), (300, 136, 8968, 48, False),
                                          (513, 1112, 9480, 128, True), (2000, 200, 4104, 16, True)])
def test_many_columns(M, K, N, G, save):
    # the form with 128 output columns per CTA: odd rows, columns that end inside a block, one and several row tiles
    check(Case(M, K, N, G, seed=M), act=M % 5, save=save)


def test_a_stalled_stage_ends_with_the_timeout_status():
    # the bounded waits of both tensor-core forms: the kernel latches the status and writes nothing
    for M, N in ((40, 512), (300, 8192)):
        c = Case(M, 1024, N, 64, seed=M)
        out = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
        try:
            w.w4a16_set_fault_injection(0, 2_000_000)  # (stages count from each CTA's start: all have a first one)
            c.run(w.ACT_SILU, out=out)
        finally:
            w.w4a16_set_fault_injection(-1, 0)
        assert w.device_status(clear=True) == w.ERR_TIMEOUT
        assert (out == 7.0).all()
        refs, bounds = f.gated(c.A, c.Wg, c.Wu, w.ACT_SILU)
        assert f.worst(c.run(w.ACT_SILU).cpu().numpy(), refs[0], bounds[0]) <= 1


@pytest.mark.parametrize("M,K,N,G", [(16, 14336, 64, 128), (9, 14344, 72, 48), (13, 8200, 136, 80), (1, 30008, 64, 64),
                                     (16, 20000, 8, 32)])
def test_long_contraction_at_decode_sizes(M, K, N, G):
    # K too long for the activations to be staged at once: several pieces, the last one partial
    check(Case(M, K, N, G, seed=M), act=M % 5, save=True)


@pytest.mark.parametrize("M,K,N,G", [(1, 64, 40000, 64), (16, 136, 36008, 16), (7, 8, 4104, 16), (200, 8, 14336, 16)])
def test_many_columns_short_contraction(M, K, N, G):
    check(Case(M, K, N, G, seed=M), act=w.ACT_SILU, save=False)
