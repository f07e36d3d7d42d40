"""The gated feed-forward projections, their backward pass, the transposed product and the product with low-rank
adapters on 4-bit group-wise weights: what each computes in elementary torch operations, in 64 bits, and the calls of
this package that compute it.

The weights of every case are signed 4-bit codes q [K, N] with fp16 scales S [ceil(K / G), N]; the matrix they stand
for is W[k, n] = fp16(q[k, n] * S[k // G, n]). Sizes and distributions are those of workloads/ and the tests: a model's
hidden size 4096 and inner size 14336, groups of 128 and 64, activations of unit variance, scales in [0.002, 0.02].
"""
import math

import torch

own = False

ACTS = ("identity", "relu", "gelu_erf", "gelu_tanh", "silu")  # in the order of the package's ACT_* codes
NIBBLES = (0, 2, 4, 6, 1, 3, 5, 7)  # k of nibble i inside a 32-bit word of the tiled layout


def listed():
    return [
        # one sequence generating: the gate and up projections of one token stream both weight matrices
        dict(name="gated one token", op="gated", M=1, K=4096, N=14336, G=128, act="silu", save=False),
        # a decode batch of 16 sequences, finer groups, the tanh GELU
        dict(name="gated decode batch", op="gated", M=16, K=4096, N=14336, G=64, act="gelu_tanh", save=False),
        # a short prompt through a small model of odd sizes (no multiple of a tile in any direction)
        dict(name="gated odd sizes", op="gated", M=333, K=1112, N=2856, G=48, act="gelu_erf", save=False),
        # a training batch: the forward pass keeps both projections for its backward pass
        dict(name="gated training forward", op="gated", M=2048, K=4096, N=14336, G=128, act="silu", save=True),
        # the same batch backward, to the block's input
        dict(name="gated backward", op="gated_backward", M=2048, K=4096, N=14336, G=128, act="silu"),
        dict(name="gated backward odd sizes", op="gated_backward", M=77, K=1112, N=2856, G=48, act="gelu_erf"),
        # backward through an attention projection, and through the down projection of a short batch
        dict(name="dgrad projection", op="dgrad", M=2048, K=4096, N=4096, G=128),
        dict(name="dgrad down projection", op="dgrad", M=300, K=14336, N=4096, G=64),
        # one sequence with its adapter; 16 sequences with 16 adapters; five prompts side by side; many adapters, odd sizes
        dict(name="lora one token", op="lora", M=1, K=4096, N=4096, G=128, L=8, R=16, segs=0),
        dict(name="lora decode batch", op="lora", M=16, K=4096, N=14336, G=128, L=16, R=64, segs=0),
        dict(name="lora prompts", op="lora", M=2048, K=4096, N=4096, G=128, L=8, R=16, segs=5),
        dict(name="lora odd sizes", op="lora", M=200, K=1112, N=2856, G=48, L=40, R=24, segs=0),
    ]


def draw(rng):
    def eights(lo, hi):  # a multiple of 8, spread over the logarithm
        return 8 * int(round(math.exp(rng.uniform(math.log(lo / 8), math.log(hi / 8)))))

    def rows(hi):
        return min(hi, int(math.exp(rng.uniform(0.0, math.log(hi + 1)))))

    op = rng.choice(("gated", "gated", "gated_backward", "dgrad", "lora", "lora"))
    c = dict(op=op, K=eights(64, 4096), N=eights(64, 14336), G=rng.choice((16, 32, 48, 64, 80, 128, 256)))
    if op == "gated":
        c.update(M=rows(2048), act=rng.choice(ACTS), save=rng.random() < 0.5)
    elif op == "gated_backward":
        c.update(M=rows(2048), act=rng.choice(ACTS))
    elif op == "dgrad":
        c.update(M=rows(2048))
    else:
        c.update(M=rows(2048), L=1 + int(math.exp(rng.uniform(0.0, math.log(63)))), R=eights(8, 128))
        c["segs"] = rng.choice((0, 0, 1, 3, 6)) if c["M"] >= 6 else 0
    return c


def adapter_of_row(c):
    """Which of the batch's adapters (0, 1, ... in order of appearance; -1: none) each row uses."""
    M, L, segs = c["M"], c["L"], c["segs"]
    if segs == 0:  # every row a request of its own; every seventh without an adapter
        return [-1 if M > 1 and i % 7 == 3 else i % L for i in range(M)]
    ends = [M * (j + 1) ** 2 // segs ** 2 for j in range(segs)]  # prompts of uneven lengths, the last of several without one
    out = []
    for j, e in enumerate(ends):
        out += [-1 if segs > 2 and j == segs - 1 else j % L] * (e - len(out))
    return out


def work(c):
    M, K, N, G = c["M"], c["K"], c["N"], c["G"]
    weights = K * N // 2 + -(-K // G) * N * 2
    if c["op"] == "gated":
        return {"bytes": 2 * weights + 2 * M * (K + N * (3 if c["save"] else 1)), "flops": 4 * M * N * K}
    if c["op"] == "gated_backward":  # reads dH, both projections; writes the gradients of both and of the input
        return {"bytes": 2 * weights + 2 * M * (5 * N + K), "flops": 4 * M * N * K}
    if c["op"] == "dgrad":
        return {"bytes": weights + 2 * M * (N + K), "flops": 2 * M * N * K}
    who = adapter_of_row(c)
    used, rows = len(set(who) - {-1}), sum(x >= 0 for x in who)
    return {"bytes": weights + 2 * M * (K + N) + used * 2 * c["R"] * (K + N) + 4 * M,
            "flops": 2 * M * N * K + 2 * rows * c["R"] * (K + N)}


def tiled(q):
    """The layout that the products read (include/w4a16.h): 128-column x 64-row tiles of nibbles, flat bytes."""
    K, N = q.shape
    kt, nt = -(-K // 64), -(-N // 128)
    full = torch.zeros((kt * 64, nt * 128), dtype=torch.uint8, device=q.device)
    full[:K, :N] = q.view(torch.uint8) & 15
    x = full.view(kt, 2, 4, 8, nt, 128)[:, :, :, list(NIBBLES)]  # tile, half, word, nibble, column tile, column
    x = x.permute(4, 0, 1, 5, 2, 3).contiguous()                 # column tile, tile, half, column, word, nibble
    return (x[..., 0::2] | (x[..., 1::2] << 4)).contiguous().view(-1)


def weights(gen, c):
    K, N = c["K"], c["N"]
    q = torch.randint(-8, 8, (K, N), generator=gen, device="cuda", dtype=torch.int8)
    S = torch.rand((-(-K // c["G"]), N), generator=gen, device="cuda").mul_(0.018).add_(0.002).half()
    return {"q": q, "S": S, "wt": tiled(q)}


def normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).half()


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(seed)
    M, K, N = c["M"], c["K"], c["N"]
    s = {"c": c}
    if c["op"] in ("gated", "gated_backward"):
        s["gate"], s["up"] = weights(gen, c), weights(gen, c)
    else:
        s["w"] = weights(gen, c)
    if c["op"] in ("gated", "lora"):
        s["A"] = normal(gen, (M, K))
    if c["op"] == "gated_backward":  # projections as wide as such weights make them; a scaled loss's gradient
        wide = 0.05 * math.sqrt(K)
        s["g"], s["u"], s["dH"] = normal(gen, (M, N), wide), normal(gen, (M, N), wide), normal(gen, (M, N), 0.02)
    if c["op"] == "dgrad":
        s["dC"] = normal(gen, (M, N), 0.02)
    if c["op"] == "lora":
        L, R = c["L"], c["R"]
        s["lora_A"], s["lora_B"] = normal(gen, (L, R, K), 1 / math.sqrt(K)), normal(gen, (L, N, R), 0.05)
        s["scaling"] = torch.rand(L, generator=gen, device="cuda").add_(0.5)
        who = torch.tensor(adapter_of_row(c), device="cuda")
        order = torch.randperm(L, generator=gen, device="cuda")
        s["ids"] = torch.where(who >= 0, order[who.clamp(min=0)], who).int()
    return s


def matrix(w, G):
    """The fp16 matrix that codes and scales stand for, in 32 bits."""
    scale = w["S"].float().repeat_interleave(G, 0)[:w["q"].shape[0]]
    return (w["q"].float() * scale).half().float()


def act_of(x, act):
    if act == "identity":
        return x
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "gelu_erf":
        return 0.5 * x * torch.special.erfc(x * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x))
    return x * torch.sigmoid(x)


def slope_of(x, act):
    if act == "identity":
        return torch.ones_like(x)
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu_erf":
        return 0.5 * torch.special.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        a = 2 * math.sqrt(2 / math.pi)
        t = torch.sigmoid(a * (x + 0.044715 * x * x * x))
        return t + x * t * (1 - t) * a * (1 + 3 * 0.044715 * x * x)
    t = torch.sigmoid(x)
    return t + x * t * (1 - t)


def run(s):
    c = s["c"]
    G = c["G"]
    if own:
        return run_own(s, c)
    if c["op"] == "gated":
        A = s["A"].float()
        g, u = A @ matrix(s["gate"], G), A @ matrix(s["up"], G)
        h = (act_of(g, c["act"]) * u).half()
        return {"h": h, "g": g.half(), "u": u.half()} if c["save"] else {"h": h}
    if c["op"] == "gated_backward":
        g, u, dH = s["g"].float(), s["u"].float(), s["dH"].float()
        dg, du = dH * u * slope_of(g, c["act"]), dH * act_of(g, c["act"])
        dx = dg @ matrix(s["gate"], G).T + du @ matrix(s["up"], G).T
        return {"dx": dx.half(), "dg": dg.half(), "du": du.half()}
    if c["op"] == "dgrad":
        return {"dx": (s["dC"].float() @ matrix(s["w"], G).T).half()}
    A, ids, L, R = s["A"].float(), s["ids"].long(), c["L"], c["R"]
    down = s["lora_A"].float().view(L * R, -1)
    up = s["lora_B"].float().transpose(1, 2).reshape(L * R, -1)
    V = (A @ down.T).view(-1, L, R) * s["scaling"].view(1, L, 1)
    mine = ids.view(-1, 1, 1) == torch.arange(L, device="cuda").view(1, L, 1)
    V = torch.where(mine, V, torch.zeros_like(V)).view(-1, L * R)
    return {"out": (A @ matrix(s["w"], G) + V @ up).half()}


def run_own(s, c):
    import weight_only_int4_wise_b200 as w
    N, K, G = c["N"], c["K"], c["G"]
    if c["op"] == "gated":
        a, b = s["gate"], s["up"]
        act = ACTS.index(c["act"])
        if c["save"]:
            h, g, u = w.gated_gemm(s["A"], a["wt"], a["S"], b["wt"], b["S"], N, G, act, save=True)
            return {"h": h, "g": g, "u": u}
        return {"h": w.gated_gemm(s["A"], a["wt"], a["S"], b["wt"], b["S"], N, G, act)}
    if c["op"] == "gated_backward":
        a, b = s["gate"], s["up"]
        dx, dg, du = w.gated_gemm_backward(s["dH"], s["g"], s["u"], a["wt"], a["S"], b["wt"], b["S"], K, G,
                                           ACTS.index(c["act"]))
        return {"dx": dx, "dg": dg, "du": du}
    if c["op"] == "dgrad":
        return {"dx": w.gemm_dgrad(s["dC"], s["w"]["wt"], s["w"]["S"], K, G)}
    return {"out": w.lora_gemm(s["A"], s["w"]["wt"], s["w"]["S"], N, G, s["lora_A"], s["lora_B"], s["ids"],
                               s["scaling"])}


def exact(case, seed):
    """The same from the definitions, in 64 bits: one column block of the weights at a time, one adapter at a time."""
    s, c = prepare(case, seed), case
    M, K, N, G = c["M"], c["K"], c["N"], c["G"]

    def block(w, lo, hi):  # columns lo..hi of W in 64 bits: the exact product rounded to fp16
        rows = torch.arange(K, device="cuda") // G
        return (w["q"][:, lo:hi].double() * w["S"][rows, lo:hi].double()).half().double()

    def sigma(x):
        return 1 / (1 + torch.exp(-x))

    def value_and_slope(x):
        if c["act"] == "identity":
            return x, torch.ones_like(x)
        if c["act"] == "relu":
            on = (x > 0).double()
            return x * on, on
        if c["act"] == "gelu_erf":
            phi = (1 + torch.erf(x / math.sqrt(2.0))) / 2
            return x * phi, phi + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        if c["act"] == "gelu_tanh":
            r = math.sqrt(2 / math.pi)
            t = torch.tanh(r * (x + 0.044715 * x ** 3))
            return x * (1 + t) / 2, (1 + t) / 2 + x * (1 - t * t) / 2 * r * (1 + 3 * 0.044715 * x ** 2)
        return x * sigma(x), sigma(x) * (1 + x * (1 - sigma(x)))

    out, step = {}, 2048
    if c["op"] == "gated":
        A = s["A"].double()
        g = torch.cat([A @ block(s["gate"], lo, min(N, lo + step)) for lo in range(0, N, step)], 1)
        u = torch.cat([A @ block(s["up"], lo, min(N, lo + step)) for lo in range(0, N, step)], 1)
        out = {"h": value_and_slope(g)[0] * u}
        return dict(out, g=g, u=u) if c["save"] else out
    if c["op"] == "gated_backward":
        a, da = value_and_slope(s["g"].double())
        dH = s["dH"].double()
        dg, du = dH * s["u"].double() * da, dH * a
        dx = torch.zeros((M, K), dtype=torch.float64, device="cuda")
        for lo in range(0, N, step):
            hi = min(N, lo + step)
            dx += torch.einsum("mn,kn->mk", dg[:, lo:hi], block(s["gate"], lo, hi))
            dx += torch.einsum("mn,kn->mk", du[:, lo:hi], block(s["up"], lo, hi))
        return {"dx": dx, "dg": dg, "du": du}
    if c["op"] == "dgrad":
        dx = torch.zeros((M, K), dtype=torch.float64, device="cuda")
        for lo in range(0, N, step):
            hi = min(N, lo + step)
            dx += torch.einsum("mn,kn->mk", s["dC"][:, lo:hi].double(), block(s["w"], lo, hi))
        return {"dx": dx}
    A = s["A"].double()
    y = torch.cat([A @ block(s["w"], lo, min(N, lo + step)) for lo in range(0, N, step)], 1)
    for i in range(c["L"]):
        rows = (s["ids"] == i).nonzero().view(-1)
        v = torch.einsum("mk,rk->mr", A[rows], s["lora_A"][i].double()) * s["scaling"][i].double()
        y[rows] += torch.einsum("mr,nr->mn", v, s["lora_B"][i].double())
    return {"out": y}
