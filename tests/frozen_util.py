"""64-bit forms of the operators on frozen 4-bit weights (gated projections, transposed product, their
backward pass, low-rank adapters), and the error bounds their tests use.

W[k, n] = fp16(q[k, n] * S[k // G, n]) is exact data here: an fp16 product of a 4-bit and an 11-bit number, formed in
64 bits and rounded once, as the operators define it.

Bounds. A product sum of `terms` terms, accumulated in 32 bits in steps of 16 terms, whose partial sums never exceed
T = sum |a| |w| in magnitude: a step rounds (or truncates, aligning its 17 addends to the largest) by at most
2^-21 T, and at most 16 partial sums are added afterwards, so the error is below (terms / 16 + 16) * 2^-21 * T.
An fp16 result adds half a step: 2^-11 of its magnitude, or 2^-25 in the subnormal range.
Activations and their derivatives are evaluated with a few 32-bit operations and one library function of a few ulp:
2^-18 relative to the larger of their terms covers them; |act'| <= 1.13 and |act''| <= 1.2 for every activation
carry a projection's error over."""
from __future__ import annotations

import numpy as np
from scipy.special import erf

ACTS = ("identity", "relu", "gelu_erf", "gelu_tanh", "silu")


def matrix(q: np.ndarray, S: np.ndarray, G: int) -> np.ndarray:
    K = q.shape[0]
    s = np.repeat(S.astype(np.float64), G, axis=0)[:K]
    return (q.astype(np.float64) * s).astype(np.float16).astype(np.float64)


def sigma(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def act(x: np.ndarray, a: int) -> np.ndarray:
    name = ACTS[a]
    if name == "identity":
        return x
    if name == "relu":
        return np.maximum(x, 0)
    if name == "gelu_erf":
        return x * 0.5 * (1 + erf(x / np.sqrt(2)))
    if name == "gelu_tanh":
        return x * sigma(2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))
    return x * sigma(x)


def slope(x: np.ndarray, a: int) -> np.ndarray:
    name = ACTS[a]
    if name == "identity":
        return np.ones_like(x)
    if name == "relu":
        return (x > 0).astype(np.float64)
    if name == "gelu_erf":
        return 0.5 * (1 + erf(x / np.sqrt(2))) + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        c = 2 * np.sqrt(2 / np.pi)
        t = sigma(c * (x + 0.044715 * x ** 3))
        return t + x * t * (1 - t) * c * (1 + 3 * 0.044715 * x * x)
    t = sigma(x)
    return t + x * t * (1 - t)


def sum_error(terms: int, T: np.ndarray) -> np.ndarray:
    return (terms / 16 + 16) * 2.0 ** -21 * T


def half_step(ref: np.ndarray) -> np.ndarray:
    return np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25)


def product(A: np.ndarray, W: np.ndarray):
    """A @ W and the bound of its 32-bit sum's error."""
    A = A.astype(np.float64)
    return A @ W, sum_error(W.shape[0], np.abs(A) @ np.abs(W))


def gated(A, Wg, Wu, a):
    """(H, g, u) and the bounds of their fp16 results' errors."""
    g, eg = product(A, Wg)
    u, eu = product(A, Wu)
    v = act(g, a)
    H = v * u
    # error of act: 1.13 eg from its argument and, from its evaluation, 2^-18 of itself or of a small term of |g| <= 1
    ev = 1.13 * eg + 2.0 ** -18 * np.maximum(np.abs(v), np.minimum(np.abs(g), 1.0) * 2.0 ** -4)
    eh = ev * np.abs(u) + (np.abs(v) + ev) * eu
    return (H, g, u), (half_step(H) + 1.001 * eh, half_step(g) + 1.001 * eg, half_step(u) + 1.001 * eu)


def worst(got: np.ndarray, ref: np.ndarray, bound: np.ndarray) -> float:
    """The largest error in units of its bound (below 1 everywhere if the result is right)."""
    err = np.abs(got.astype(np.float64) - ref)
    return float(np.max(err / bound, initial=0.0)) if np.all(np.isfinite(got)) else float("inf")


def slopes(dH, g, u, a):
    """(dG, dU) of the gated product from fp16 projections, and the bounds of their fp16 results' errors."""
    dH, g, u = (x.astype(np.float64) for x in (dH, g, u))
    d, v = slope(g, a), act(g, a)
    # evaluation: 2^-18 of the derivative's terms (none above 1.2, or of act's); three fp32 products
    ed = 2.0 ** -18 * np.maximum(np.abs(d), 2.0 ** -4)
    ev = 2.0 ** -18 * np.maximum(np.abs(v), np.minimum(np.abs(g), 1.0) * 2.0 ** -4)
    dG, dU = dH * u * d, dH * v
    return (dG, dU), (half_step(dG) + np.abs(dH * u) * ed, half_step(dU) + np.abs(dH) * ev)


def gated_backward(dH, g, u, Wg, Wu, a):
    """(dA, dG, dU) and their bounds; dA's counts the rounding of dG and dU to fp16 before their products."""
    (dG, dU), (eG, eU) = slopes(dH, g, u, a)
    dA = dG @ Wg.T + dU @ Wu.T
    T = np.abs(dG) @ np.abs(Wg).T + np.abs(dU) @ np.abs(Wu).T
    eA = sum_error(2 * Wg.shape[1], T) + eG @ np.abs(Wg).T + eU @ np.abs(Wu).T
    return (dA, dG, dU), (half_step(dA) + 1.001 * eA, eG, eU)


def lora(A, W, LA, LB, ids, scaling):
    """The product with one adapter per row, and the bound of its fp16 result's error: V = scaling * A LA^T is
    rounded to fp16 before its product."""
    A64 = A.astype(np.float64)
    C, e = product(A, W)
    for m, i in enumerate(ids):
        if not 0 <= i < LA.shape[0]:
            continue
        a, b, s = LA[i].astype(np.float64), LB[i].astype(np.float64), float(scaling[i])
        v = s * (a @ A64[m])
        ev = sum_error(A.shape[1], abs(s) * (np.abs(a) @ np.abs(A64[m]))) + np.abs(v) * 2.0 ** -24
        ev = ev + half_step(np.abs(v) + ev)
        C[m] += b @ v
        e[m] += np.abs(b) @ ev + sum_error(LA.shape[1], np.abs(b) @ np.abs(v))
    return C, half_step(C) + 1.001 * e
