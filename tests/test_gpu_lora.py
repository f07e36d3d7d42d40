"""The shared 4-bit projection with one low-rank adapter per row (w4a16_lora_gemm) on the GPU against its 64-bit form:
every launch form, odd sizes, ranks up to 128, rows without an adapter, mixed and contiguous adapters, broken
adapters that other rows must not see, bad indices, streams, workspaces and captures."""
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
    def __init__(self, M, K, N, G, L, R, seed, ids=None):
        c = workloads.dense(M, K, N, G, seed)
        g = np.random.Generator(np.random.PCG64(seed + 77))
        self.M, self.K, self.N, self.G, self.L, self.R = M, K, N, G, L, R
        self.A, self.S, self.W = c.A, c.S, f.matrix(c.q, c.S, G)
        self.wt = device_weights(c.q)[1]
        self.LA = (g.standard_normal((L, R, K)) / np.sqrt(K)).astype(np.float16)
        self.LB = (g.standard_normal((L, N, R)) * 0.1).astype(np.float16)
        self.scaling = (0.5 + g.random(L)).astype(np.float32)
        self.ids = (g.integers(-1, L, size=M) if ids is None else np.asarray(ids)).astype(np.int32)

    def operands(self):
        return (dev(self.A), self.wt, dev(self.S), self.N, self.G, dev(self.LA), dev(self.LB), dev(self.ids),
                dev(self.scaling))

    def run(self, **kw):
        out = w.lora_gemm(*self.operands(), **kw)
        torch.cuda.synchronize()
        return out

    def reference(self):
        return f.lora(self.A, self.W, self.LA, self.LB, self.ids, self.scaling)

    def check(self):
        flat, out, pad = guarded_output(self.M, self.N)
        self.run(out=out)
        ref, bound = self.reference()
        assert f.worst(out.cpu().numpy(), ref, bound) <= 1
        assert guards_intact(flat, pad, self.M * self.N)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 129, 200, 256, 257, 300])
@pytest.mark.parametrize("K,N,G,L,R", [(64, 64, 64, 1, 8), (72, 8, 16, 3, 16), (200, 136, 48, 40, 24),
                                       (512, 520, 128, 5, 64), (1112, 264, 80, 2, 128), (2048, 192, 128, 300, 8),
                                       (192, 4096, 32, 9, 40)])
def test_every_form(M, K, N, G, L, R):
    Case(M, K, N, G, L, R, seed=M + K).check()


@pytest.mark.parametrize("M,ids", [
    (300, [2] * 300),                                   # one request
    (300, [-1] * 300),                                  # no adapter at all
    (300, [0] * 100 + [-1] * 3 + [3] * 197),            # prompts side by side
    (300, [i % 4 for i in range(300)]),                 # interleaved
    (16, [3] * 16), (16, [-1] * 16), (16, [0, 3] * 8), (1, [-1]), (1, [3]),
])
def test_row_orders(M, ids):
    Case(M, 320, 200, 64, 4, 16, seed=M, ids=ids).check()


def test_every_row_its_own_adapter():
    for M in (16, 40, 256, 270):
        Case(M, 256, 136, 64, M, 8, seed=M, ids=np.random.Generator(np.random.PCG64(M)).permutation(M)).check()


def test_full_sizes():
    Case(1, 4096, 4096, 128, 8, 16, seed=1, ids=[5]).check()
    Case(16, 4096, 4096, 128, 16, 64, seed=2, ids=list(range(16))).check()
    Case(512, 4096, 1024, 128, 8, 16, seed=3, ids=[1] * 70 + [4] * 300 + [-1] * 42 + [0] * 100).check()


def test_no_scaling_means_one():
    for M in (4, 40):
        c = Case(M, 128, 64, 64, 3, 8, seed=M)
        a = w.lora_gemm(*c.operands()[:-1])
        c.scaling[:] = 1
        assert torch.equal(a, c.run())


def test_rows_without_adapter_equal_the_plain_product():
    c = Case(300, 512, 264, 128, 3, 16, seed=300)  # (the same kernel without a K split: one order of the sums)
    plain = w.gemm(dev(c.A), c.wt, dev(c.S), c.N, c.G)
    none = c.ids < 0
    assert torch.equal(c.run()[none], plain[none])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("M", [6, 16, 40, 130, 300])
def test_broken_adapter_stays_with_its_rows(M, value):
    c = Case(M, 256, 136, 64, 4, 16, seed=M, ids=[i % 5 - 1 for i in range(M)])
    clean = c.run().clone()
    c.LB[2, 50, 3] = value   # one value of adapter 2's up-projection
    c.LB[1, 60] = value      # a whole column of adapter 1
    c.LA[3, 5, 7] = value    # adapter 3's down-projection
    got = c.run()
    keep = (c.ids < 1)
    assert torch.equal(got[keep], clean[keep])
    two = torch.from_numpy(c.ids == 2).cuda()
    rest = [n for n in range(c.N) if n != 50]
    assert torch.equal(got[two][:, rest], clean[two][:, rest]) and not torch.isfinite(got[two][:, 50]).any()
    one = torch.from_numpy(c.ids == 1).cuda()
    assert not torch.isfinite(got[one][:, 60]).any() and torch.isfinite(got[one][:, 61]).all()
    if (c.ids == 3).any():
        assert not torch.isfinite(got[torch.from_numpy(c.ids == 3).cuda()]).any()


def test_rows_do_not_touch_each_other():
    for M in (5, 16, 40, 300):
        c = Case(M, 256, 136, 64, 3, 16, seed=M)
        clean = c.run().clone()
        c.A[1] = np.nan
        got = c.run()
        keep = [m for m in range(M) if m != 1]
        assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[1]).all()


@pytest.mark.parametrize("M", [4, 50])
def test_bad_index_latches_and_computes_without_adapter(M):
    c = Case(M, 128, 64, 64, 3, 8, seed=M)
    c.ids[2] = 3
    got = c.run()
    assert w.device_status(clear=True) == w.ERR_BAD_ADAPTER
    c.ids[2] = -1
    assert torch.equal(got, c.run())


def test_streams_workspaces_and_repeats():
    for M in (3, 16, 60, 300):
        c = Case(M, 512, 264, 64, 6, 16, seed=M)
        ref = c.run().clone()
        ops = c.operands()
        torch.cuda.synchronize()
        sides = [torch.cuda.Stream() for _ in range(2)]
        outs = []
        for i in range(6):  # calls that overlap on two streams, each with a workspace of its own
            outs.append(w.lora_gemm(*ops, stream=sides[i % 2]))
        ws = torch.empty(w.w4a16_lora_workspace_size(M, 16), dtype=torch.uint8, device="cuda")
        outs += [w.lora_gemm(*ops, workspace=ws) for _ in range(3)]  # one after another in the same workspace
        wide = torch.zeros((M, 1024), dtype=torch.float16, device="cuda")
        wide[:, ::2] = ops[0]
        torch.cuda.synchronize()
        outs.append(w.lora_gemm(wide[:, ::2], *ops[1:], stream=sides[0].cuda_stream))
        torch.cuda.synchronize()
        assert all(torch.equal(x, ref) for x in outs)


@pytest.mark.parametrize("M", [1, 16, 100])
def test_captured_calls_replay_with_new_rows_and_adapters(M):
    c = Case(M, 512, 256, 128, 4, 16, seed=M)
    ops = c.operands()
    w.lora_gemm(*ops)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two captured calls that share nothing
        graph, out = torch.cuda.CUDAGraph(), torch.empty((M, c.N), dtype=torch.float16, device="cuda")
        ws = torch.empty(w.w4a16_lora_workspace_size(M, 16), dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(graph):
            w.lora_gemm(*ops, workspace=ws, out=out)
        graphs.append((graph, out))
    c.ids = (c.ids + 2) % 5 - 1
    c.A = c.A[::-1].copy()
    ops[7].copy_(dev(c.ids.astype(np.int32)))
    ops[0].copy_(dev(c.A))
    for graph, out in graphs:
        graph.replay()
    torch.cuda.synchronize()
    ref, bound = c.reference()
    for _, out in graphs:
        assert f.worst(out.cpu().numpy(), ref, bound) <= 1


def test_a_chain_of_calls_reads_what_the_call_before_wrote():
    # the product starts before the kernel in front of it ends: every operand is the output of the launch just before
    for M in (8, 48):
        c = Case(M, 256, 256, 64, 3, 16, seed=M)
        ops = list(c.operands())
        x, ref = ops[0], ops[0]
        for _ in range(6):
            x = w.lora_gemm(x.clone() * 0.25, *ops[1:])
        torch.cuda.synchronize()
        for _ in range(6):
            y = ref.clone() * 0.25
            torch.cuda.synchronize()
            ref = w.lora_gemm(y, *ops[1:])
            torch.cuda.synchronize()
        assert torch.equal(x, ref)
        # adapters and indices written right before the call
        for _ in range(4):
            ops[6].mul_(1.5)
            ops[7].add_(1).remainder_(3)
            got = w.lora_gemm(*ops)
            torch.cuda.synchronize()
            assert torch.equal(got, w.lora_gemm(*ops))


def test_gated_block_with_adapters_and_its_backward():
    # the operators together: adapters on the input of a gated block, down projection, and the way back
    M, H, I, G = 48, 256, 392, 64
    att = Case(M, H, H, G, 3, 8, seed=1)
    gate, up, down = (workloads.dense(1, *kn, G, s) for kn, s in (((H, I), 2), ((H, I), 3), ((I, H), 4)))
    wt = [device_weights(c.q)[1] for c in (gate, up, down)]
    S = [dev(c.S) for c in (gate, up, down)]
    W = [f.matrix(c.q, c.S, G) for c in (gate, up, down)]
    x = w.lora_gemm(*att.operands())
    h, g, u = w.gated_gemm(x, wt[0], S[0], wt[1], S[1], I, G, save=True)
    y = w.gemm(h, wt[2], S[2], H, G)
    dy = (y * 2.0 ** -8).contiguous()
    dh = w.gemm_dgrad(dy, wt[2], S[2], I, G)
    dx, dg, du = w.gated_gemm_backward(dh, g, u, wt[0], S[0], wt[1], S[1], H, G)
    n = lambda t: t.cpu().numpy()
    ref, bound = att.reference()
    assert f.worst(n(x), ref, bound) <= 1
    refs, bounds = f.gated(n(x), W[0], W[1], w.ACT_SILU)
    assert all(f.worst(n(a), r, b) <= 1 for a, r, b in zip((h, g, u), refs, bounds))
    ref, err = f.product(n(dy), W[2].T)
    assert f.worst(n(dh), ref, f.half_step(ref) + 1.001 * err) <= 1
    refs, bounds = f.gated_backward(n(dh), n(g), n(u), W[0], W[1], w.ACT_SILU)
    assert all(f.worst(n(a), r, b) <= 1 for a, r, b in zip((dx, dg, du), refs, bounds))


def test_no_rows_and_wrong_operands():
    c = Case(4, 128, 64, 64, 3, 8, seed=1)
    A, wt, S, N, G, LA, LB, ids, sc = c.operands()
    assert w.lora_gemm(A[:0], wt, S, N, G, LA, LB, ids[:0], sc).shape == (0, 64)
    with pytest.raises(TypeError):
        w.lora_gemm(A, wt, S, N, G, LA, LB, ids.long(), sc)
    with pytest.raises(TypeError):
        w.lora_gemm(A, wt, S, N, G, LA.float(), LB, ids, sc)
    with pytest.raises(ValueError):
        w.lora_gemm(A, wt, S, N, G, LA, LB.transpose(1, 2), ids, sc)
    with pytest.raises(ValueError):
        w.lora_gemm(A, wt, S, N, G, LA, LB, ids[:3], sc)
    with pytest.raises(w.W4A16Error):
        w.lora_gemm(A, wt, S, N, G, LA, LB, ids, sc, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(w.W4A16Error):
        w.lora_gemm(A, wt, S, N, G, LA[:, :4].contiguous(), LB[:, :, :4].contiguous(), ids, sc)  # rank 4


@pytest.mark.parametrize("M,K,N,G,L,R", [(16, 14336, 64, 128, 5, 16), (11, 14344, 72, 48, 3, 24), (16, 136, 70008, 16, 4, 8),
                                         (1, 64, 80000, 64, 2, 8), (9, 8, 4104, 16, 2, 128), (40, 14336, 72, 64, 3, 8),
                                         (1100, 264, 136, 64, 3, 40), (1030, 4096, 264, 128, 70, 16)])
def test_long_and_wide(M, K, N, G, L, R):
    Case(M, K, N, G, L, R, seed=M + K).check()
