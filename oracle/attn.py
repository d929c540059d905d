"""Plain numpy oracle of the attention-side operators, in 64 bits: norm and rotation of
queries and keys, the 4-bit cache's coding, causal attention over the coded values.
Written from include/sherry.h's definitions; shares no code with the kernels.
"""
import numpy as np

PAGE = 64


def to_bf16(x):
    """float32 rounded to the nearest bf16 (ties to even), as float32; NaN stays NaN."""
    x = np.ascontiguousarray(x, np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def rope(x, w, pos, inv_freq, eps, interleaved):
    """x [T, H, D] -> [T, H, D] float64."""
    y = np.asarray(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    half = len(inv_freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    out = y.copy()
    ia = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    ib = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


def kv4_encode(x):
    """Rows [..., D] float32 -> (codes uint8, step, low end: float32 holding bf16 values)."""
    with np.errstate(all="ignore"):
        x = np.asarray(x, np.float32)
        lo, hi = x.min(-1), x.max(-1)   # a NaN stays
        s = to_bf16((hi - lo) * np.float32(1.0 / 15.0))
        m = to_bf16(lo)
        bad = ~(np.isfinite(s) & np.isfinite(m))
        flat = ~bad & (s < np.float32(2.0) ** -120)
        inv = np.where(bad | flat, np.float32(0), np.float32(1) / s)
        q = np.clip(np.rint((x - m[..., None]) * inv[..., None]), 0, 15)
        codes = np.where((bad | flat)[..., None], 0, q).astype(np.uint8)
        s = np.where(flat, np.float32(0), np.where(bad, np.float32(np.nan), s)).astype(np.float32)
        m = np.where(bad, np.float32(np.nan), m).astype(np.float32)
    return codes, s, m


def kv4_values(codes, s, m):
    """float64 values of coded rows."""
    return m[..., None].astype(np.float64) + s[..., None].astype(np.float64) * codes


def kv4_pack(cache, page, slot, head, kv, codes, s, m):
    """One coded row into a cache array uint8 [pages, H, 2, 64 * (D / 2 + 4)]."""
    d = codes.shape[-1]
    blk = cache[page, head, kv]
    blk[slot * d // 2:(slot + 1) * d // 2] = codes[0::2] | (codes[1::2] << 4)
    pair = np.array([s, m], np.float32).view(np.uint32) >> 16
    at = PAGE * d // 2 + 4 * slot
    blk[at:at + 4] = pair.astype(np.uint16).view(np.uint8)


def kv4_unpack(cache, page, slot, head, kv):
    """(codes, step, low end) of one row of a cache array."""
    blk = cache[page, head, kv]
    d = (blk.size // PAGE - 4) * 2
    b = blk[slot * d // 2:(slot + 1) * d // 2]
    codes = np.stack([b & 15, b >> 4], -1).reshape(-1)
    at = PAGE * d // 2 + 4 * slot
    pair = (blk[at:at + 4].copy().view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    return codes, pair[0], pair[1]


def attend(q, k, v, last, scale):
    """One head: q [n, D], k and v [L, D] float64, row i sees keys 0 .. last[i] -> [n, D]; rows
    that see nothing give zeros."""
    out = np.zeros(q.shape, np.float64)
    for i in range(q.shape[0]):
        e = min(int(last[i]) + 1, k.shape[0])
        if e <= 0:
            continue
        x = k[:e] @ q[i] * scale
        p = np.exp(x - x.max())
        out[i] = (p @ v[:e]) / p.sum()
    return out
