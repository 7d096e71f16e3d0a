"""CPU reference of the MXFP4 form and of the expert routing.  Test and
benchmark infrastructure only; the product never imports it.

Plain numpy in 64 bits, from the definitions: E2M1 codes are found by
nearest-value search over the value table (ties to the even code), scales by
frexp, and products are formed on the decoded values.
"""
from __future__ import annotations

import numpy as np

from .nvfp4_oracle import bf16_to_f32

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_round(v: np.ndarray) -> np.ndarray:
    """Codes 0..7 of non-negative values: nearest, ties to the even code, saturating."""
    v = np.asarray(v, dtype=np.float64)
    d = np.abs(v[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    near = d == best                              # one code, or two neighbours on a tie
    first = near.argmax(-1)
    last = 7 - near[..., ::-1].argmax(-1)
    return np.where(first % 2 == 0, first, last).astype(np.uint8)


def quantize(bits: np.ndarray):
    """bf16 bit patterns [rows, cols] -> (packed codes [rows, cols/2], scale bytes [rows, cols/32])."""
    x = bf16_to_f32(bits).astype(np.float64)
    R, Cc = x.shape
    b = x.reshape(R, Cc // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.abs(np.where(bad[..., None], 0.0, b)).max(-1)
    _, e = np.frexp(amax)                         # amax = m 2^e, 0.5 <= m < 1
    byte = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    scale = np.ldexp(1.0, byte - 127)
    with np.errstate(invalid="ignore"):
        code = e2m1_round(np.abs(b) / scale[..., None]) | (np.signbit(b).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).reshape(R, Cc).astype(np.uint8)
    byte = np.where(bad, 255, byte).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte


def dequantize(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """The fp64 values of packed codes and linear scale bytes."""
    v = np.empty((codes.shape[0], 2 * codes.shape[1]))
    for h, c in enumerate((codes & 15, codes >> 4)):
        v[:, h::2] = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return (v.reshape(*byte.shape, 32) * scale[..., None]).reshape(v.shape)


def sf_swizzle(byte: np.ndarray) -> np.ndarray:
    """Linear scale bytes [rows, cols/32] in 128x4 atoms, by the address formula."""
    R, S = byte.shape
    s4 = (S + 3) // 4
    out = np.zeros((R + 127) // 128 * 512 * s4, dtype=np.uint8)
    r, c = np.meshgrid(np.arange(R), np.arange(S), indexing="ij")
    out[512 * ((r // 128) * s4 + c // 4) + 16 * (r % 32) + 4 * ((r % 128) // 32) + c % 4] = byte
    return out


# ----------------------------------------------------------------- routing --

def scores(x: np.ndarray, score: str) -> np.ndarray:
    """fp64 scores of the logits [T, E]; masked logits (-inf, NaN) have score 0."""
    x = np.asarray(x, dtype=np.float64)
    ok = x > -np.inf
    x = np.where(ok, np.minimum(x, float(np.finfo(np.float32).max)), -np.inf)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(ok, 1.0 / (1.0 + np.exp(-x)), 0.0)
    m = np.where(ok.any(1), x.max(1, initial=-np.inf), 0.0)[:, None]
    e = np.where(ok, np.exp(x - m), 0.0)
    total = e.sum(1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route_keys(x, bias, score):
    """(ordering keys, s + bias), -inf where an expert cannot be chosen."""
    x = np.asarray(x, dtype=np.float64)
    s = scores(x, score)
    with np.errstate(invalid="ignore"):
        sb = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    key = np.minimum(x, float(np.finfo(np.float32).max)) if bias is None else sb
    ok = (x > -np.inf) & (key > -np.inf)
    return np.where(ok, key, -np.inf), np.where(ok, sb, -np.inf)


def route_topk(x, k, bias=None, score="sigmoid", num_groups=1, topk_groups=1, group_top=2,
               renormalize=True, scale=1.0):
    """(ids [T, k], weights [T, k], margins [T]).  The margin is the smallest
    difference of a token's choice between neighbours of its order (chosen keys,
    the first rejected one, group scores) among those that fp32 rounds: below
    their rounding error the choice is not determined by the definition in 64
    bits.  Keys without a bias are the logits themselves, exact, and so are
    group scores that are their largest."""
    key, sb = route_keys(x, bias, score)
    T, E = key.shape
    s = scores(x, score)
    ids = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    margins = np.full(T, np.inf)
    per = E // num_groups
    for t in range(T):
        row = key[t].copy()
        if num_groups > 1 and topk_groups < num_groups:
            g = np.sort((sb[t] if group_top == 2 else key[t]).reshape(num_groups, per), axis=1)[:, ::-1]
            gs = g[:, 0].copy()
            if group_top == 2 and per > 1:
                two = g[:, 1] > -np.inf
                gs[two] += g[two, 1]
            order = np.argsort(-gs, kind="stable")
            ranked = gs[order]
            if ranked[topk_groups] > -np.inf and (bias is not None or group_top == 2):
                margins[t] = min(margins[t], ranked[topk_groups - 1] - ranked[topk_groups])
            dropped = order[topk_groups:]
            for gi in dropped:
                row[gi * per:(gi + 1) * per] = -np.inf
        order = np.argsort(-row, kind="stable")
        order = order[row[order] > -np.inf]
        take = order[:k]
        near = row[order[:k + 1]]
        if len(near) > 1 and bias is not None:
            margins[t] = min(margins[t], np.min(near[:-1] - near[1:]))
        ids[t, :len(take)] = take
        w = s[t, take]
        if renormalize:
            total = w.sum()
            w = w / total if total > 0 else np.zeros_like(w)
        weights[t, :len(take)] = w * scale
    return ids, weights, margins


def route_topk_backward(x, ids, grad, score="sigmoid", renormalize=True, scale=1.0):
    """fp64 gradient of sum(grad * weights) with respect to the logits, the
    choice held fixed: the Jacobian of the definition, written out."""
    s = scores(x, score)
    T, E = s.shape
    out = np.zeros((T, E))
    for t in range(T):
        j = np.flatnonzero((ids[t] >= 0) & (ids[t] < E))
        e, d = ids[t, j], np.asarray(grad[t, j], dtype=np.float64) * scale
        ds = np.zeros(E)
        if renormalize:
            # over the chosen alone: unaffected by a softmax sum that underflows
            if score == "softmax":
                xe = np.minimum(np.asarray(x, dtype=np.float64)[t, e], float(np.finfo(np.float32).max))
                if len(xe) and xe.max() > -np.inf:
                    w = np.exp(xe - xe.max())
                    w = w / w.sum()
                    out[t, e] = w * (d - (d * w).sum())
                continue
            total = s[t, e].sum()
            ds[e] = (d - (d * s[t, e]).sum() / total) / total if total > 0 else 0.0
        else:
            ds[e] = d
        if score == "sigmoid":
            out[t] = ds * s[t] * (1.0 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out
