"""Host-side refusals of the operators on frozen 4-bit weights: nothing is enqueued for a bad argument."""
import pytest

import weight_only_int4_wise_b200 as w
from weight_only_int4_wise_b200 import build

FAKE = 0x10000  # a non-null, 16-byte aligned address that is never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_gated_gemm_rejects_bad_arguments_on_host():
    def g(A=FAKE, wg=FAKE, sg=FAKE, wu=FAKE, su=FAKE, H=FAKE, Pg=None, Pu=None, M=4, N=128, K=128, G=64,
          act=w.ACT_SILU, flags=0):
        return w.w4a16_gated_gemm(A, wg, sg, wu, su, H, Pg, Pu, M, N, K, G, act, flags, stream=0)
    for name in ("A", "wg", "sg", "wu", "su", "H"):
        assert g(**{name: None}) == w.ERR_INVALID_ARG, name
    assert g(Pg=FAKE) == w.ERR_INVALID_ARG and g(Pu=FAKE) == w.ERR_INVALID_ARG  # both or neither
    assert g(M=-1) == w.ERR_INVALID_ARG and g(N=0) == w.ERR_INVALID_ARG
    assert g(act=5) == w.ERR_INVALID_ARG and g(act=-1) == w.ERR_INVALID_ARG
    assert g(flags=2) == w.ERR_INVALID_ARG
    assert g(N=100) == w.ERR_UNSUPPORTED and g(K=100) == w.ERR_UNSUPPORTED and g(G=24) == w.ERR_UNSUPPORTED
    assert g(M=1 << 31) == w.ERR_UNSUPPORTED
    for name in ("A", "wg", "sg", "wu", "su"):
        assert g(**{name: FAKE + 8}) == w.ERR_MISALIGNED, name
    assert g(H=FAKE + 1) == w.ERR_MISALIGNED
    assert g(Pg=FAKE + 1, Pu=FAKE) == w.ERR_MISALIGNED
    assert g(M=0) == w.OK and g(M=0, Pg=FAKE, Pu=FAKE) == w.OK


def test_dgrad_rejects_bad_arguments_on_host():
    def g(dC=FAKE, wt=FAKE, s=FAKE, dA=FAKE, M=4, N=128, K=128, G=64, flags=0):
        return w.w4a16_gemm_dgrad(dC, wt, s, dA, M, N, K, G, flags, stream=0)
    for name in ("dC", "wt", "s", "dA"):
        assert g(**{name: None}) == w.ERR_INVALID_ARG, name
    assert g(M=-1) == w.ERR_INVALID_ARG and g(K=0) == w.ERR_INVALID_ARG and g(flags=4) == w.ERR_INVALID_ARG
    assert g(N=100) == w.ERR_UNSUPPORTED and g(K=100) == w.ERR_UNSUPPORTED and g(G=24) == w.ERR_UNSUPPORTED
    for name in ("dC", "wt", "s"):
        assert g(**{name: FAKE + 8}) == w.ERR_MISALIGNED, name
    assert g(dA=FAKE + 1) == w.ERR_MISALIGNED
    assert g(M=0) == w.OK


def test_gated_backward_rejects_bad_arguments_on_host():
    names = ("dH", "Pg", "Pu", "wg", "sg", "wu", "su", "dPg", "dPu", "dA")

    def g(M=4, N=128, K=128, G=64, act=w.ACT_SILU, flags=0, **kw):
        return w.w4a16_gated_gemm_backward(*[kw.get(n, FAKE) for n in names], M, N, K, G, act, flags, stream=0)
    for name in names:
        assert g(**{name: None}) == w.ERR_INVALID_ARG, name
    for name in names[:-1]:
        assert g(**{name: FAKE + 8}) == w.ERR_MISALIGNED, name
    assert g(dA=FAKE + 1) == w.ERR_MISALIGNED
    assert g(act=5) == w.ERR_INVALID_ARG and g(flags=2) == w.ERR_INVALID_ARG and g(M=-1) == w.ERR_INVALID_ARG
    assert g(N=100) == w.ERR_UNSUPPORTED and g(K=100) == w.ERR_UNSUPPORTED and g(G=24) == w.ERR_UNSUPPORTED
    assert g(M=0) == w.OK


def test_lora_rejects_bad_arguments_on_host():
    names = ("A", "wt", "s", "LA", "LB", "ids", "scaling", "C")
    need = w.w4a16_lora_workspace_size(4, 16)

    def g(M=4, N=128, K=128, G=64, L=3, R=16, ws=FAKE, ws_bytes=need, **kw):
        return w.w4a16_lora_gemm(*[kw.get(n, FAKE) for n in names], M, N, K, G, L, R, ws, ws_bytes, stream=0)
    for name in names:
        if name != "scaling":
            assert g(**{name: None}) == w.ERR_INVALID_ARG, name
    assert g(ws=None) == w.ERR_INVALID_ARG and g(ws_bytes=need - 1) == w.ERR_INVALID_ARG
    assert g(M=-1) == w.ERR_INVALID_ARG and g(L=0) == w.ERR_INVALID_ARG and g(R=0) == w.ERR_INVALID_ARG
    assert g(R=12) == w.ERR_UNSUPPORTED and g(R=136) == w.ERR_UNSUPPORTED
    assert g(N=100) == w.ERR_UNSUPPORTED and g(K=100) == w.ERR_UNSUPPORTED and g(G=24) == w.ERR_UNSUPPORTED
    for name in ("A", "wt", "s", "LA", "LB"):
        assert g(**{name: FAKE + 8}) == w.ERR_MISALIGNED, name
    assert g(ws=FAKE + 8) == w.ERR_MISALIGNED
    assert g(ids=FAKE + 2) == w.ERR_MISALIGNED and g(scaling=FAKE + 2) == w.ERR_MISALIGNED
    assert g(C=FAKE + 1) == w.ERR_MISALIGNED
    assert g(M=0) == w.OK and g(M=0, scaling=None) == w.OK


def test_lora_workspace_size():
    r = lambda b: (b + 255) // 256 * 256
    for M, R in [(0, 8), (1, 16), (16, 64), (2048, 128)]:
        assert w.w4a16_lora_workspace_size(M, R) == r(M * R * 2) + r((M + 256) * 4) + r((M // 16 + 1) * 4)
    assert w.w4a16_lora_workspace_size(4, 12) == -1 and w.w4a16_lora_workspace_size(4, w.MAX_RANK + 8) == -1
    assert w.w4a16_lora_workspace_size(-1, 16) == -1
    assert w.status_string(w.ERR_BAD_ADAPTER) != "unknown status"
