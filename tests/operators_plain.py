"""Plain float64 numpy forms of the fused-epilogue, grouped, row-grouping and row-joining operators, written
from their definitions, and the error bounds their tests hold the kernels to."""

import math

import numpy as np

U32, UBF = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative to the value

_erf = np.vectorize(math.erf, otypes=[np.float64])


def signs(packed):
    """uint32 [..., K/32] -> +-1 float64 [..., K], least significant bit first."""
    b = np.unpackbits(np.ascontiguousarray(packed).view(np.uint8), axis=-1, bitorder="little")
    return 2.0 * b - 1.0


def activate(z, act):
    with np.errstate(all="ignore"):
        if act == "relu":
            return np.where(z < 0, 0.0, z)
        if act == "gelu":
            return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
        if act == "gelu_tanh":
            return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        if act == "silu":
            return z / (1 + np.exp(-z))
    return z


def activate_exact(z, act):
    """(act(z), tol) of float64 values z that are exact in fp32, in forms that do not cancel where act is small, and what
    evaluating act in fp32 may be off by:

    gelu, z/2 erfc(x), x = -z/sqrt 2: the constant and its product are off by U32 each, which erfc turns into at most
    2 U32 |x| (2/sqrt pi) e^(-x^2) / erfc(x) <= 2 U32 (1 + z^2) for z < 0, to U32 for
    z >= 0; erfc itself is within 4 steps (8 U32), the last product U32.
    gelu_tanh, z / (1 + e^(-2y)): y's two terms have one sign, so its seven roundings are off by 7 U32 |y|, 14 U32 |y| in
    the exponential's argument; exp is within 2 steps (4 U32), and of both the share e/(1 + e) enters the sum (U32); the
    quotient is within 2 steps (4 U32). silu: exp, sum and quotient, 9 U32. One more U32 each for products of these. none
    and relu are exact.
    A factor or denominator at the end of the normal range may be taken as 0: |z| 2^-126, and half the smallest step."""
    with np.errstate(all="ignore"):
        if act == "gelu":
            o = 0.5 * z * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2))
            steps = np.where(z < 0, 2 * (1 + z * z), 1) + 10
        elif act == "gelu_tanh":
            y = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            share = 1 / (1 + np.exp(2 * y))
            o, steps = z / (1 + np.exp(-2 * y)), (14 * np.abs(y) + 4) * share + 6
        elif act == "silu":
            o, steps = z / (1 + np.exp(-z)), 10.0
        else:
            return activate(z, act), np.zeros_like(z)
        return o, np.abs(o) * steps * U32 + np.abs(z) * 2.0 ** -126 + 2.0 ** -150


def layer(packed, s, u, bias=None, act=None, glu=False, residual=None):
    """(o, tol): o in float64, and the largest error an fp32 computation may make before its result is rounded.

    z is a sum of K exact products: the kernels add them in at most K/16 + 16 dependent fp32 steps (a tensor
    instruction adds 16 products; 16 more for partial sums and the epilogue), each off by at most 2^-23 of the
    partial sum it makes (truncation: twice the half step), and the partial sums of +-u in random sign order
    stay below 4 sqrt(sum u^2). Inputs that are not of random sign are compared at their own tolerance.
    act has a slope of at most 1.13, a gate multiplies the errors of its factors, and evaluating act takes under
    16 roundings more (the library's exp and erfc are within 3 of them each)."""
    u = np.asarray(u, np.float64)
    z = s * (u @ signs(packed).T)
    K = u.shape[1]
    dz = (K / 16 + 16) * 2.0 ** -23 * 4 * np.abs(s) * np.sqrt((u * u).sum(1))[:, None]
    if bias is not None:
        z = z + bias
    dz = dz + 2 * U32 * np.abs(z)
    if glu:
        a, b, da, db = z[:, 0::2], z[:, 1::2], dz[:, 0::2], dz[:, 1::2]
        fa = activate(a, act)
        dfa = 1.13 * da + 16 * U32 * np.abs(fa)
        o, tol = fa * b, dfa * np.abs(b) + np.abs(fa) * db + dfa * db
    else:
        o = activate(z, act)
        tol = 1.13 * dz + 16 * U32 * np.abs(o)
    tol = tol + 4 * U32 * np.abs(o)
    if residual is not None:
        o = o + np.asarray(residual, np.float64)
        tol = tol + 2 * U32 * (np.abs(o) + np.abs(np.asarray(residual, np.float64)))
    return o, tol


def grouped(packed, s, u, offsets, n, rows=None, bias=None, act=None, glu=False):
    """(o, tol, written): slots of no expert hold zeros and are not marked as written."""
    width = packed.shape[1] // 2 if glu else packed.shape[1]
    o, tol, written = np.zeros((n, width)), np.zeros((n, width)), np.zeros(n, bool)
    for e in range(packed.shape[0]):
        lo, hi = min(max(int(offsets[e]), 0), n), min(max(int(offsets[e + 1]), 0), n)
        if hi <= lo:
            continue
        at = np.arange(lo, hi) if rows is None else np.asarray(rows[lo:hi])
        there = (at >= 0) & (at < u.shape[0])
        x = np.where(there[:, None], np.asarray(u, np.float64)[np.where(there, at, 0)], 0.0)
        o[lo:hi], tol[lo:hi] = layer(packed[e], s[e], x, None if bias is None else bias[e], act, glu)
        written[lo:hi] = True
    return o, tol, written


def group(ids, experts):
    T, k = ids.shape
    flat = ids.reshape(-1)
    kept = np.flatnonzero((flat >= 0) & (flat < experts))
    order = kept[np.argsort(flat[kept], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])])
    rows, slots = np.full(T * k, -1), np.full(T * k, -1)
    rows[: order.size] = order // k
    slots[order] = np.arange(order.size)
    return offsets, rows, slots.reshape(T, k)


def combine(y, slots, weights, residual=None):
    """(o, tol): topk products and sums in fp32, one rounding each."""
    y = np.asarray(y, np.float64)
    T, k = slots.shape
    o, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < y.shape[0]:
                term = float(weights[t, j]) * y[slots[t, j]]
                o[t] += term
                mag[t] += np.abs(term)
    if residual is not None:
        o, mag = o + residual, mag + np.abs(residual)
    return o, (k + 2) * 2 * U32 * mag


def assert_close(got, want, tol, bf16):
    """got within tol plus one rounding to its type, element by element."""
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape
    limit = tol + (UBF if bf16 else U32) * (np.abs(want) + tol)
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax((np.abs(got - want) / limit)[bad])), np.argwhere(bad)[:5].tolist())
