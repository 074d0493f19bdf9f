"""Random paged caches and batches for the attention-layer tests, on host and device alike."""
from __future__ import annotations

import numpy as np

from oracle import attention as ref

BF16_HALF = 2.0 ** -8    # half a BF16 step relative to the value
F16_HALF = 2.0 ** -11


def bf16(x):
    """FP32 array rounded to BF16 (as FP32) and the device tensor of it."""
    import torch
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.float().numpy().astype(np.float64), t.cuda()


def batch(q_lens, kv_lens, block, rng, spare=2, max_blocks=None):
    """(cu, lens, table) device tensors and the table as numpy, blocks shuffled; -1 where a
    sequence needs none."""
    import torch
    need = [-(-n // block) for n in kv_lens]
    cols = max(max(need), 1) if max_blocks is None else max_blocks
    count = sum(need) + spare
    ids = rng.permutation(count)
    table = np.full((len(kv_lens), cols), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return dev(cu), dev(np.asarray(kv_lens, np.int32)), dev(table), table, count


def filled_cache(count, hk, block, d, rng, log_spread=1.0):
    """Random codes (no NaN) and power-of-two scales: numpy (k, v, ks, vs)."""
    def codes():
        x = rng.standard_normal((count, hk, block, d)) * 100.0
        return ref._encode(x)
    scales = lambda: (2.0 ** np.round(-6 + log_spread * rng.standard_normal((count, hk)))).astype(np.float32)
    return codes(), codes(), scales(), scales()


def to_cache(nv, k, v, ks, vs):
    import torch
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return nv.BlockKVCache(dev(k), dev(v), dev(ks), dev(vs))


def attention_bound(out, mags, biggest_v, half_step, kv_max):
    """Allowed |error| of an attention output.  A weight is rounded to FP16 (half a step
    2^-11 of it); its exponent x = s c + e carries a few FP32 roundings of magnitudes up to
    2^7 (4 * 2^7 * 2^-24 * ln 2 < 2^-15), ex2 is good to 2^-22, and a sum of up to 2^10 terms in one chain to
    2^-14: together below 2^-11 + 2^-13 of sum p |v|.  Weights below 2^-30 of the largest may vanish.
    Then the result is rounded once."""
    return half_step * np.abs(out) + (F16_HALF + 2.0 ** -13) * mags + kv_max * 2.0 ** -30 * biggest_v


def counted(cu, tokens):
    """The sequences of a batch that count: bounds in order and within the rows, and no earlier
    usable bound behind the start."""
    out, high = [], 0
    for s in range(len(cu) - 1):
        b, e = int(cu[s]), int(cu[s + 1])
        if 0 <= b <= e <= tokens and b >= high:
            out.append(s)
        if b <= tokens:
            high = max(high, b)
    return out


def broken_bounds(n, longest, rng, share=0.1, first=0):
    """Bounds of n sequences of up to `longest` new tokens, a share of them (from index `first` on) replaced by
    anything from -5 to 50 behind the last row."""
    cu = np.concatenate([[0], np.cumsum(rng.integers(0, longest + 1, n))])
    tokens = int(cu[-1])
    wrong = np.flatnonzero(rng.random(n + 1) < share)
    wrong = wrong[wrong >= first]
    cu[wrong] = rng.integers(-5, tokens + 50, len(wrong))
    return cu.astype(np.int32), tokens
