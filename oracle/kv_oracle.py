"""CPU reference of the NVFP4 key-value cache and of attention over it, numpy in
64 bits.  Rows are packed by nvfp4_oracle.quantize under a static scale; the
products and the softmax follow the definitions directly.  Tests only."""
import numpy as np

from . import nvfp4_oracle as o


def pack_rows(x_bits: np.ndarray, g: np.ndarray):
    """bf16 bits [tokens, heads, hd], g [heads] -> codes [tokens, heads, hd/2], sf [tokens, heads, hd/16]."""
    T, H, hd = x_bits.shape
    codes = np.zeros((T, H, hd // 2), np.uint8)
    sf = np.zeros((T, H, hd // 16), np.uint8)
    for h in range(H):
        codes[:, h], sf[:, h] = o.quantize(np.ascontiguousarray(x_bits[:, h]), np.float32(g[h]))[:2]
    return codes, sf


def values(codes: np.ndarray, sf: np.ndarray, g: np.ndarray) -> np.ndarray:
    """What packed rows stand for: [.., heads, hd] in 64 bits, unrounded."""
    mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    table = np.concatenate([mag, -mag])
    v = np.empty((*codes.shape[:-1], codes.shape[-1] * 2))
    v[..., 0::2], v[..., 1::2] = table[codes & 15], table[codes >> 4]
    b = sf.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    s = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0)) * np.where(b >= 128, -1, 1)
    s = np.where((b & 127) == 127, np.nan, s)
    return v * np.repeat(s * g.astype(np.float64)[:, None], 16, -1)


def gather(codes, sf, g, table, n: int, page: int):
    """[n, heads, hd] values of a sequence and a mask that leaves out keys of pages outside the cache."""
    j = np.arange(n)
    ids = table[j // page].astype(np.int64) if n else np.zeros(0, np.int64)
    ok = (ids >= 0) & (ids < codes.shape[0])
    at = np.where(ok, ids, 0)
    return values(codes[at, :, j % page], sf[at, :, j % page], g), ok


def attention(q, k, v, ok, pos, scale: float, causal: bool, window: int):
    """q [rows, Hq, hd], k and v [n, Hkv, hd], pos [rows]: the queries' positions.
    Returns out [rows, Hq, hd], lse [rows, Hq] and the sums the tolerances need:
    sum_j w_j |v_j|, sum_j |v_j| / sum_j exp(s_j - max), the largest sum_d |q_d k_jd|."""
    rows, Hq, hd = q.shape
    n, Hkv = k.shape[:2]
    G = Hq // Hkv
    out, lse = np.zeros((rows, Hq, hd)), np.full((rows, Hq), -np.inf)
    s_abs, v_sum, qk = np.zeros((rows, Hq, hd)), np.zeros((rows, Hq, hd)), np.zeros((rows, Hq))
    for r in range(rows):
        see = ok.copy()
        if causal:
            j = np.arange(n)
            see &= j <= pos[r]
            if window:
                see &= j > pos[r] - window
        if not see.any():
            continue
        for h in range(Hq):
            kk, vv = k[see, h // G], v[see, h // G]
            s = scale * (kk @ q[r, h])
            if np.isnan(s).any():
                out[r, h], lse[r, h] = np.nan, np.nan
                continue
            m = s.max()
            e = np.exp(s - m)
            w = e / e.sum()
            seen_nan = np.isnan(vv).any(0)
            out[r, h] = np.where(seen_nan, np.nan, w @ np.nan_to_num(vv))
            lse[r, h] = m + np.log(e.sum())
            s_abs[r, h], v_sum[r, h] = w @ np.abs(vv), np.abs(vv).sum(0) / e.sum()
            qk[r, h] = (np.abs(kk) @ np.abs(q[r, h])).max()
    return out, lse, s_abs, v_sum, qk
