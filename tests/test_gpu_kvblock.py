"""GPU parity of the append to the block-scaled 8-bit cache: codes and scales are exact."""
import numpy as np
import pytest

from attention_testutil import batch, bf16, filled_cache, to_cache
from oracle import attention as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import torch
    from nvfp4_w4a4_quantized_02_b200 import build
    build.build()
    import nvfp4_w4a4_quantized_02_b200 as nv
    assert torch.cuda.is_available()
    return nv


def _rows(tokens, hk, d, rng):
    """K or V rows of sizes that vary by token, with the odd outlier."""
    x = rng.standard_normal((tokens, hk, d)) * np.exp2(rng.integers(-6, 7, (tokens, 1, 1)))
    x[rng.random(x.shape) < 0.002] *= 300.0
    return bf16(x)


def _check(nv, cache, host, where=""):
    import torch
    torch.cuda.synchronize()
    for got, want, name in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), host, ("k", "v", "k_scales", "v_scales")):
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=want.dtype == np.float32), name + where


CASES = [
    ([1], [1], 1, 64, 16), ([1], [17], 2, 128, 16), ([16], [16], 1, 128, 16), ([5, 1, 0, 40], [20, 1, 30, 40], 2, 64, 32),
    ([1] * 30, list(range(1, 300, 10)), 2, 128, 64), ([300], [333], 3, 256, 128), ([129, 63], [129, 127], 1, 256, 64),
    ([200, 7], [231, 128], 8, 64, 128), ([33], [64], 2, 128, 32), ([2, 2, 2], [17, 16, 15], 1, 64, 16),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_append_is_exact(nv, case):
    q_lens, kv_lens, hk, d, block = case
    rng = np.random.default_rng(sum(kv_lens))
    cu, lens, table_d, table, count = batch(q_lens, kv_lens, block, rng)
    host = filled_cache(count, hk, block, d, rng, 3.0)
    cache = to_cache(nv, *host)
    (k, k_d), (v, v_d) = (_rows(sum(q_lens), hk, d, rng) for _ in range(2))
    nv.kv_append(k_d.reshape(len(k), -1), v_d.reshape(len(v), -1), cu, lens, table_d, cache)
    ref.append(k, q_lens, kv_lens, table, host[0], host[2], block)
    ref.append(v, q_lens, kv_lens, table, host[1], host[3], block)
    _check(nv, cache, host)
    assert nv.device_status() == 0


@pytest.mark.parametrize("d,block", [(64, 16), (128, 64), (256, 128)])
def test_token_by_token(nv, d, block):
    """A cache that starts as arbitrary memory, grown one token at a time, with growing scales."""
    import torch
    rng = np.random.default_rng(7)
    n = block + 9
    table = np.array([[2, 0]], np.int32)
    host = (np.full((3, 2, block, d), 0x7F, np.uint8), np.full((3, 2, block, d), 0xFF, np.uint8),
            np.full((3, 2), np.nan, np.float32), np.full((3, 2), -1.0, np.float32))
    cache = to_cache(nv, *host)
    x, x_d = bf16(rng.standard_normal((n, 2, d)) * np.exp2(np.arange(n) / 4.0)[:, None, None])
    table_d = torch.from_numpy(table).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for t in range(n):
        lens = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        row = x_d[t:t + 1].reshape(1, -1)
        nv.kv_append(row, row, cu, lens, table_d, cache)
        ref.append(x[t:t + 1], [1], [t + 1], table, host[0], host[2], block)
        ref.append(x[t:t + 1], [1], [t + 1], table, host[1], host[3], block)
        _check(nv, cache, host, f" after token {t}")


def test_scale_borders_ties_and_non_finite(nv):
    import torch
    d, block = 64, 16
    values = [448.0, 450.0, 447.0, 0.0, 1e-38, 3e38, 2.0 ** -100, 1.75 * 2.0 ** 20, 1.7578125 * 2.0 ** 20]
    rows = np.zeros((len(values), 1, d))
    for t, x in enumerate(values):
        rows[t, 0] = x * np.linspace(-1, 1, d)
        rows[t, 0, 0] = x
    rows[3, 0, 1] = -0.0
    rows[1, 0, 5:9] = [np.inf, -np.inf, np.nan, 449.0]
    x, x_d = bf16(rows)
    n = len(values)
    host = filled_cache(n, 1, block, d, np.random.default_rng(1))
    cache = to_cache(nv, *host)
    table = np.arange(n, dtype=np.int32)[::-1].reshape(n, 1).copy()
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    r = x_d.reshape(n, d)
    nv.kv_append(r, r, cu, one, torch.from_numpy(table).cuda(), cache)
    for i in (0, 1):
        ref.append(x, [1] * n, [1] * n, table, host[i], host[2 + i], block)
    _check(nv, cache, host)
    only_bad = torch.full((1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    nv.kv_append(only_bad, only_bad, cu[:2].contiguous(), one[:1], torch.from_numpy(table[:1].copy()).cuda(), cache)
    assert float(cache.k_scales[n - 1, 0]) == 2.0 ** -100 and (cache.k[n - 1, 0, 0] == 0x7F).all()


def test_strided_rows_and_rows_behind_the_last_sequence(nv):
    import torch
    rng = np.random.default_rng(2)
    q_lens, kv_lens, hk, d, block = [3, 40], [50, 47], 2, 128, 32
    cu, lens, table_d, table, count = batch(q_lens, kv_lens, block, rng)
    host = filled_cache(count, hk, block, d, rng)
    cache = to_cache(nv, *host)
    wide, wide_d = bf16(rng.standard_normal((50, 5 * 256)))
    cut = lambda i: wide[:43, i * 256:(i + 1) * 256].reshape(43, hk, d)
    nv.kv_append(wide_d[:, 256:512], wide_d[:, 768:1024], cu, lens, table_d, cache)
    ref.append(cut(1), q_lens, kv_lens, table, host[0], host[2], block)
    ref.append(cut(3), q_lens, kv_lens, table, host[1], host[3], block)
    _check(nv, cache, host)


def test_bad_sequences_and_blocks_are_skipped_and_reported(nv):
    import torch
    rng = np.random.default_rng(3)
    q_lens, kv_lens, hk, d, block = [20, 5, 30], [40, 25, 30], 1, 64, 16
    cu, lens, table_d, table, count = batch(q_lens, kv_lens, block, rng)
    (x, x_d) = _rows(55, hk, d, rng)
    r = x_d.reshape(55, d)
    start = np.concatenate([[0], np.cumsum(q_lens)])
    for what in ("short", "long", "block", "bounds"):
        host = filled_cache(count, hk, block, d, rng)
        cache = to_cache(nv, *host)
        l, t, c, tb = list(kv_lens), table.copy(), cu.clone(), table_d.clone()
        skip = {1}
        if what == "short":
            l[1] = 4
        elif what == "long":
            l[1] = table.shape[1] * block + 1
        elif what == "block":
            skip = set()
            tb[2, 1] = count + 3
        else:
            c[1] = 400
            skip = {0, 1}
        nv.kv_append(r, r, c, torch.tensor(l, dtype=torch.int32, device="cuda"), tb, cache)
        for s in range(3):
            if s in skip:
                continue
            part = x[start[s]:start[s + 1]]
            for i in (0, 1):
                if what == "block" and s == 2:  # its second block is nowhere: only the first is written
                    ref.append(part[:16], [16], [16], t[2:3], host[i], host[2 + i], block)
                else:
                    ref.append(part, [q_lens[s]], [kv_lens[s]], t[s:s + 1], host[i], host[2 + i], block)
        _check(nv, cache, host, " " + what)
        assert nv.device_status() == 7


def test_graph_and_side_stream(nv):
    import torch
    rng = np.random.default_rng(4)
    q_lens, kv_lens, hk, d, block = [1] * 5, [17, 33, 1, 64, 100], 2, 128, 64
    cu, lens, table_d, table, count = batch(q_lens, kv_lens, block, rng)
    host = filled_cache(count, hk, block, d, rng)
    (x, x_d) = _rows(5, hk, d, rng)
    r = x_d.reshape(5, -1)
    cache, again = to_cache(nv, *host), to_cache(nv, *host)
    g = torch.cuda.CUDAGraph()
    nv.kv_append(r, r, cu, lens, table_d, again)  # first use outside the capture
    with torch.cuda.graph(g):
        nv.kv_append(r, r, cu, lens, table_d, cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.replay()
        g.replay()  # the same tokens again: the scales have grown already, nothing changes
    torch.cuda.current_stream().wait_stream(side)
    for i in (0, 1):
        ref.append(x, q_lens, kv_lens, table, host[i], host[2 + i], block)
    _check(nv, cache, host)
    _check(nv, again, host)


def test_many_sequences(nv):
    import torch
    rng = np.random.default_rng(5)
    q_lens = [int(x) for x in rng.integers(0, 3, 700)]
    q_lens[13] = 200
    kv_lens = [q + int(x) for q, x in zip(q_lens, rng.integers(0, 40, 700))]
    cu, lens, table_d, table, count = batch(q_lens, kv_lens, 16, rng)
    host = filled_cache(count, 1, 16, 64, rng, 3.0)
    cache = to_cache(nv, *host)
    (k, k_d), (v, v_d) = (_rows(sum(q_lens), 1, 64, rng) for _ in range(2))
    # the first sequence starts behind the first row
    pad = lambda t: torch.cat([torch.full((4, 64), 7.0, dtype=t.dtype, device="cuda"), t.reshape(len(t), -1)])
    nv.kv_append(pad(k_d), pad(v_d), cu + 4, lens, table_d, cache)
    ref.append(k, q_lens, kv_lens, table, host[0], host[2], 16)
    ref.append(v, q_lens, kv_lens, table, host[1], host[3], 16)
    _check(nv, cache, host)
    assert nv.device_status() == 0
