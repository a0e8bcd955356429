"""Plain 64-bit forms of the microscaled 4-bit and expert operators, their
tolerances and their inputs (shared by the CPU and the GPU tests)."""
import math

import numpy as np
import torch

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx_quantize_ref(x: np.ndarray):
    """x [rows, K] (float64 of BF16 or fp32 values) -> codes [rows, K] (0..15), scale bytes [rows, K/32], by search:
    the nearest level, on a tie the one with an even index."""
    rows, K = x.shape
    v = x.reshape(rows, K // 32, 32)
    fine = np.isfinite(v).all(-1)
    a = np.where(fine, np.abs(np.where(np.isfinite(v), v, 0)).max(-1), 0)
    _, e = np.frexp(a)                                   # a = m 2^e, 1/2 <= m < 1
    s = np.where(a > 0, np.clip(e - 3, -127, 127), -127)
    m = np.abs(np.where(fine[..., None], v, 0)) / np.ldexp(1.0, s)[..., None]
    d = np.abs(m[..., None] - LEVELS)
    best = d.min(-1, keepdims=True)
    tie = d == best
    even = tie & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), tie.argmax(-1))
    code = code + 8 * np.signbit(v)
    code = np.where(fine[..., None], code, 0)
    return code.reshape(rows, K).astype(np.uint8), np.where(fine, s + 127, 255).astype(np.uint8)


def mx_values_ref(code: np.ndarray, sbyte: np.ndarray) -> np.ndarray:
    v = np.where(code >= 8, -LEVELS[code & 7], LEVELS[code & 7]).reshape(code.shape[0], -1, 32)
    s = np.ldexp(1.0, sbyte.astype(np.int64) - 127)[..., None]
    return np.where(sbyte[..., None] == 255, np.nan, v * s).reshape(code.shape)


def scale_at(rows: int, K: int):
    """Index of every (row, block) scale byte in one matrix's tiles, by the header's formula, and the tiles' bytes."""
    kt = -(-K // 256)
    at = np.empty((rows, K // 32), np.int64)
    for r in range(rows):
        for b in range(K // 32):
            at[r, b] = ((r // 128) * kt + b // 8) * 1024 + (b // 4 % 2) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    return at, -(-rows // 128) * kt * 1024


def pack_ref(code: np.ndarray, sbyte: np.ndarray):
    """Packed codes and scale tiles of one matrix."""
    at, size = scale_at(*code.shape)
    tiles = np.zeros(size, np.uint8)
    tiles[at] = sbyte
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), tiles


def route_ref(logits: np.ndarray, k: int, score: str, renorm: bool, scale: float):
    """The router token by token in float64: ids, weights, offsets, rows, pos."""
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        x = np.array([-math.inf if math.isnan(v) else min(float(v), float(np.finfo(np.float32).max)) for v in logits[t]])
        order = sorted((e for e in range(E) if x[e] > -math.inf), key=lambda e: (-x[e], e))[:k]
        if not order:
            continue
        if score == "softmax":
            p = np.exp(x - x.max())
            q = p[order] / (p[order].sum() if renorm else p.sum())
        else:
            q = np.array([1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in x[order]])
            if renorm:
                q = q / q.sum() if q.sum() > 0 else q * 0
        ids[t, :len(order)] = order
        w[t, :len(order)] = q * scale
    slots = sorted((int(ids[t, j]), t, j) for t in range(T) for j in range(k) if ids[t, j] >= 0)
    rows, pos = np.full(T * k, -1, np.int32), np.full((T, k), -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    for s, (e, t, j) in enumerate(slots):
        rows[s], pos[t, j] = t, s
        offsets[e + 1:] += 1
    return ids, w, offsets, rows, pos


# Tolerances.  Products of BF16 (or 4-bit) values are exact in fp32; a sum of
# K of them whose additions are off by at most 2^-23 relative each (truncation)
# is off by at most K 2^-23 sum|x||w|.  Rounding to BF16 adds 2^-8 |ref|.
def product_tolerance(absolute: torch.Tensor, K: int) -> torch.Tensor:
    return K * 2.0 ** -23 * absolute


def split_tolerance(X: torch.Tensor, W: torch.Tensor) -> torch.Tensor:
    """BF16 rows against 4-bit weights: a value may enter the product off by 2^-21 (1 + 2^-8) of the largest of its
    block of 32.  The largest is scaled into [2^7, 2^8) and lo has steps of 2^-13 there, so rounding is off by 2^-14 at
    most; below 2^-14 a value with significand 1 + m/128 is taken as m/128 2^-14, which for m = 127, whose tie goes up to
    2^-13, is (2 - 255/256) 2^-14."""
    top = X.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
    return 2.0 ** -21 * (1 + 2.0 ** -8) * (top @ W.abs().T)


def swiglu_ref(g: torch.Tensor, u: torch.Tensor) -> torch.Tensor:
    return g * torch.sigmoid(g) * u


def swiglu_tolerance(g, u, dg, du):
    """First order through h = silu(g) u (|silu'| <= 1.1) plus the product term; the fast exponential is off by at most
    (2 + 1.2 |g|) 2^-23, the division and the products by 6 more."""
    silu = g * torch.sigmoid(g)
    return 1.1 * u.abs() * dg + silu.abs() * du + 1.1 * dg * du + (8 + 1.2 * g.abs()) * 2.0 ** -23 * (silu * u).abs() + 1e-37


def check(y: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor):
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside; first at {bad.nonzero()[0].tolist()}, worst {float((err / tol).nan_to_num(1e9).max()):.3g}x"


def grouped_ref(X, W, offsets, rows, up, mx):
    """(reference, tolerance) over the slots inside the offsets; X, W, up in float64."""
    ys, ts = [], []
    K = X.shape[1]
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        x = X[lo:hi] if rows is None else X[rows[lo:hi].long()]
        part = lambda w: (x @ w.T, product_tolerance(x.abs() @ w.abs().T, K) + (split_tolerance(x, w) if mx else 0))  # noqa: E731
        g, dg = part(W[e])
        if up is not None:
            u, du = part(up[e])
            ys.append(swiglu_ref(g, u))
            ts.append(swiglu_tolerance(g, u, dg, du))
        else:
            ys.append(g)
            ts.append(dg)
    return torch.cat(ys), torch.cat(ts)
