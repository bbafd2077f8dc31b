"""Plain definitions of the 4-bit formats, the products, the router and the combination, in 64 bits
(numpy / torch on the CPU), written from include/qgemm.h and sharing nothing with the library."""
from __future__ import annotations

import numpy as np

BLOCK = {3: 32, 4: 16}                       # by format number: MXFP4, NVFP4
MAG = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e2m1(x):
    """Codes of the e2m1 values nearest to x (ties to the even code, at most 6); the sign is x's."""
    a = np.abs(x)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    v = np.minimum(np.rint(a / step) * step, 6.0)
    return (np.searchsorted(MAG, v) + 8 * np.signbit(x)).astype(np.uint8)


def e4m3_table():
    b = np.arange(128)
    v = np.where(b < 8, b / 512.0, (1 + (b % 8) / 8.0) * 2.0 ** (b // 8 - 7.0))
    v[127] = np.nan
    return v


def e4m3(r):
    """Bytes of the e4m3 values nearest to r >= 0 (ties to even, at most 448)."""
    r = np.minimum(r, 448.0)
    e = np.maximum(np.floor(np.log2(np.where(r > 0, r, 1))), -6)
    q = 2.0 ** (e - 3)
    v = np.rint(r / q) * q
    return np.searchsorted(e4m3_table()[:127], v).astype(np.uint8)


def quantize(x, fmt):
    """Rows x (float64, exactly the stored values) -> codes [M][K], scale bytes [M][K/B], row scales."""
    M, K = x.shape
    B = BLOCK[fmt]
    row = np.ones(M)
    with np.errstate(all="ignore"):
        if fmt == 4:
            top = np.abs(x).max(1)
            bad = ~np.isfinite(x).all(1)
            e = np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 1
            row = np.where(top == 0, 1.0, 2.0 ** np.clip(e - 10, -116, 117))
            y = np.where(bad[:, None], 0.0, x / row[:, None]).reshape(M, K // B, B)
            row[bad] = np.nan
            top = np.abs(y).max(2)
            byte = e4m3((top / 6).astype(np.float32).astype(np.float64))
            s = e4m3_table()[byte][..., None]
            q = np.where(s > 0, y / np.where(s > 0, s, 1), np.copysign(0.0, y))
            return e2m1(q).reshape(M, K), byte, row
        y = x.reshape(M, K // B, B)
        top = np.abs(y).max(2)
        bad = ~np.isfinite(y).all(2)
        e = np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 1
        se = np.where(top == 0, -127, np.maximum(e - 2, -127))
        byte = np.where(bad, 255, se + 127).astype(np.uint8)
        q = np.where(bad[..., None], 0.0, y / 2.0 ** np.where(bad, 0, se)[..., None])
    return e2m1(q).reshape(M, K), byte, None


def values(codes, byte, row, fmt):
    """float64 values of codes [M][K], scale bytes [M][K/B] and row scales (None: 1)."""
    v = MAG[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127)) if fmt == 3 else e4m3_table()[byte & 127]
    v = v * np.repeat(s, BLOCK[fmt], -1)
    return v if row is None else v * np.asarray(row, np.float64)[:, None]


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def rows_layout(byte, K, fmt):
    n = K // BLOCK[fmt]
    out = np.zeros((byte.shape[0], (n + 15) // 16 * 16), np.uint8)
    out[:, :n] = byte
    return out


def tiled_layout(byte, K, fmt):
    n, rows = K // BLOCK[fmt], byte.shape[0]
    kt, rt = (n + 3) // 4, (rows + 127) // 128
    out = np.zeros((rt, kt, 512), np.uint8)
    for r in range(rows):
        for j in range(n):
            out[r // 128, j // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4] = byte[r, j]
    return out


def activate(v, act):
    with np.errstate(over="ignore"):
        if act == 1:
            return np.maximum(v, 0)
        if act == 2:
            return v / (1 + np.exp(-v))
        if act == 3:
            return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
        if act == 4:
            return v[:, 0::2] / (1 + np.exp(-v[:, 0::2])) * v[:, 1::2]
    return v


def product(A, B, a_scale, b_scale, bias, act, residual):
    """(result, bound): the product in float64 and how far float32 accumulation may be from it.

    The products of two operand values are exact in float32. A sum over K of which every 32 products
    or more are added into a float32 accumulator by rounding or truncation at 2^-22 of its size is
    within K / 32 * 2^-22 * sum |a b| of the exact one; scaling and bias add three float32 roundings.
    SiLU, GELU and SwiGLU have slopes of at most 1.13 and are evaluated to 2^-18 of their value."""
    with np.errstate(all="ignore"):
        s = (1 if a_scale is None else np.asarray(a_scale, np.float64)[:, None]) * (1 if b_scale is None else np.asarray(b_scale, np.float64))
        v = A @ B.T * s
        err = (A.shape[1] / 32 + 1) * 2.0 ** -22 * (np.abs(A) @ np.abs(B).T) * np.abs(s)
        if bias is not None:
            v = v + bias
        err = err + 3 * 2.0 ** -24 * (np.abs(v) + (0 if bias is None else np.abs(bias)))
        out = activate(v, act)
        if act == 4:
            g, u, eg, eu = v[:, 0::2], v[:, 1::2], err[:, 0::2], err[:, 1::2]
            err = 1.13 * eg * (np.abs(u) + eu) + np.abs(activate(g, 2)) * eu + 2.0 ** -18 * np.abs(out)
        elif act:
            err = 1.13 * err + 2.0 ** -18 * np.abs(out)
        if residual is not None:
            out = out + residual
            err = err + 2.0 ** -24 * np.abs(out)
    return out, err


def route(x, k, renorm):
    """expert, weight (float64), slot, row, offsets of logits x [T][E] (float64)."""
    T, E = x.shape
    expert, weight, slot = np.full((T, k), -1), np.zeros((T, k)), np.full((T, k), -1)
    for t in range(T):
        ok = [e for e in range(E) if x[t, e] > -np.inf]
        pick = sorted(ok, key=lambda e: (-x[t, e], e))[:k]
        if not pick:
            continue
        top = x[t, pick[0]]
        f = lambda e: 1.0 if x[t, e] == top else np.exp(x[t, e] - top)
        over = sum(f(e) for e in (pick if renorm else ok))
        expert[t, : len(pick)] = pick
        weight[t, : len(pick)] = [f(e) / over for e in pick]
    row, offsets = [], [0]
    where = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if expert[t, j] >= 0:
                where[expert[t, j]].append((t, j))
    for e in range(E):
        for t, j in where[e]:
            slot[t, j] = len(row)
            row.append(t)
        offsets.append(len(row))
    row += [-1] * (T * k - len(row))
    return expert, weight, slot, np.array(row, dtype=np.int64), np.array(offsets)
