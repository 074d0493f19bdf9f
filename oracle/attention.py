"""FP64 restatement of the attention-layer operators (numpy, plain loops over sequences).

Conventions as in the C ABI: a batch is packed rows with ``q_lens`` new tokens per sequence,
the last of ``kv_lens``; a cache is E4M3 bytes [num_blocks, kv_heads, block, D] with FP32 scales
[num_blocks, kv_heads]; ``table`` is [n_seqs, max_blocks].
"""
from __future__ import annotations

import numpy as np

from .nvfp4_oracle import e2m1_decode, e4m3_decode, e4m3_encode_signed

MIN_SCALE = 2.0 ** -100


def rope_table(max_pos: int, rot: int, base: float = 10000.0) -> np.ndarray:
    angle = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1)


def head_norm_rope(x, w, offset, eps, positions, table, interleaved) -> np.ndarray:
    """x: [tokens, heads, D]; w: [D]; table: [max_pos, R] or None."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + eps) * (offset + np.asarray(w, dtype=np.float64))
    if table is None:
        return y
    half = table.shape[1] // 2
    c, s = (np.asarray(table, dtype=np.float64)[positions][:, None, i * half:(i + 1) * half] for i in range(2))
    out = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        out[:, :, a] = y[:, :, a] * c[..., i] - y[:, :, b] * s[..., i]
        out[:, :, b] = y[:, :, b] * c[..., i] + y[:, :, a] * s[..., i]
    return out


def block_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-100 with 448 s >= amax."""
    s = MIN_SCALE
    while 448.0 * s < amax:
        s *= 2.0
    return s


def _encode(x) -> np.ndarray:
    """E4M3 bytes of x, saturating; NaN gives 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    return np.where(nan, 0x7F, e4m3_encode_signed(np.clip(np.where(nan, 0.0, x), -448.0, 448.0))).astype(np.uint8)


def append(rows, q_lens, kv_lens, table, codes, scales, block: int):
    """Appends rows [tokens, kv_heads, D] to (codes, scales), in place."""
    rows = np.asarray(rows, dtype=np.float64)
    start = 0
    for s, (n, total) in enumerate(zip(q_lens, kv_lens)):
        past = total - n
        for b in range(past // block, -(-total // block)) if n else ():
            at, lo = int(table[s][b]), b * block
            first, last = max(past, lo), min(total, lo + block)
            new = rows[start + first - past:start + last - past]
            for h in range(rows.shape[1]):
                x = new[:, h]
                mags = np.abs(x)[np.isfinite(x)]
                scale = block_scale(mags.max() if mags.size else 0.0)
                if first > lo:
                    old = float(scales[at, h])
                    if old >= scale:
                        scale = old
                    else:
                        codes[at, h, :first - lo] = _encode(e4m3_decode(codes[at, h, :first - lo]) * (old / scale))
                scales[at, h] = scale
                codes[at, h, first - lo:last - lo] = _encode(x / scale)
        start += n


def attention(q, q_lens, kv_lens, table, k, v, k_scales, v_scales, scale, causal):
    """q: [tokens, heads, D].  Returns (out, mags) with mags = sum_j p_j |v_j| / sum_j p_j, the
    size that rounding errors of the weights are relative to.  Blocks outside the cache hold
    no tokens."""
    q = np.asarray(q, dtype=np.float64)
    nb, hk, block, d = k.shape
    heads = q.shape[1]
    out, mags = np.zeros_like(q), np.zeros_like(q)
    start = 0
    for s, (n, total) in enumerate(zip(q_lens, kv_lens)):
        ids = [int(table[s][b]) for b in range(-(-total // block))]
        have = np.repeat([0 <= i < nb for i in ids], block)[:total].astype(bool)
        ids = [i if 0 <= i < nb else 0 for i in ids]
        for h in range(heads):
            a = h // (heads // hk)
            dec = lambda c, sc: (e4m3_decode(c[ids, a]) * np.asarray(sc, dtype=np.float64)[ids, a][:, None, None]).reshape(-1, d)[:total]
            if total == 0:
                continue
            kk, vv = dec(k, k_scales), dec(v, v_scales)
            for i in range(n):
                seen = have.copy()
                if causal:
                    seen[max(0, total - n + i + 1):] = False
                if not seen.any():
                    continue
                x = kk[seen] @ q[start + i, h] * scale
                p = np.exp(x - np.max(x))
                p /= p.sum()
                out[start + i, h] = p @ vv[seen]
                mags[start + i, h] = p @ np.abs(vv[seen])
        start += n
    return out, mags


def matvec(x, codes, sf, segments):
    """x: [M, K]; codes [N, K], sf [N, K/16] logical bytes.  Returns (y, mags)."""
    w = e2m1_decode(codes) * np.repeat(e4m3_decode(sf), 16, axis=1)
    gs = np.concatenate([np.full(n1 - n0, float(g)) for n0, n1, g in segments])
    x = np.asarray(x, dtype=np.float64)
    return x @ w.T / gs, np.abs(x) @ np.abs(w).T / gs
