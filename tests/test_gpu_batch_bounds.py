"""Bounds that step back: sequences that count are served as ever, the others' rows and blocks stay,
nothing is written outside the workspace."""
import numpy as np
import pytest

from attention_testutil import broken_bounds, counted, filled_cache, to_cache
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


def _i32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _attend(nv, q, cu, lens, table, cache, heads):
    """The call with a workspace of the stated size between guard bytes."""
    import torch
    d, hk = cache.k.shape[3], cache.k.shape[1]
    need = nv.attention_workspace_bytes(len(q), len(lens), heads, hk, d)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((len(q), heads * d), 7.0, dtype=torch.float32, device="cuda")
    nv.attention(q, _i32(cu), _i32(lens), _i32(table), cache, out=out, out_dtype="f32", workspace=ws[:need])
    assert bool((ws[need:] == 0xA5).all())
    return out


def _case(nv, cu, tokens, heads, hk, d, kv, seed):
    """Random queries and cache; every sequence has kv tokens (or its own many) in blocks of 16."""
    import torch
    rng = np.random.default_rng(seed)
    n = len(cu) - 1
    cols = 40  # 640 tokens: units are cut over CTAs at every head size
    cache = to_cache(nv, *filled_cache(64, hk, 16, d, rng))
    table = rng.integers(0, 64, (n, cols))  # sequences may share blocks that they only read
    q = torch.from_numpy(rng.standard_normal((tokens, heads * d)).astype(np.float32)).to(torch.bfloat16).cuda()
    lens = rng.integers(0, kv + 1, n)
    return q, lens, table, cache


def _check(nv, cu, tokens, heads, hk, d, kv, seed):
    import torch
    q, lens, table, cache = _case(nv, cu, tokens, heads, hk, d, kv, seed)
    nv.device_status()
    got = _attend(nv, q, cu, lens, table, cache, heads)
    good, n = counted(cu, tokens), len(cu) - 1
    assert nv.device_status() == (0 if len(good) == n else 7)
    # The same work in the same order, in bounds that do not step back: gaps are sequences that a
    # length below zero takes out.
    bounds, ls, tb, at = [0], [], [], 0
    for s in good:
        b, e = int(cu[s]), int(cu[s + 1])
        if b > at:
            bounds.append(b), ls.append(-1), tb.append(table[s])
        bounds.append(e), ls.append(lens[s]), tb.append(table[s])
        at = e
    while len(ls) < n:  # as many sequences, so that the work is cut alike
        bounds.append(at), ls.append(0), tb.append(table[0])
    if not good:
        assert bool((got == 7.0).all())
        return
    want = _attend(nv, q, bounds, ls, np.array(tb), cache, heads)
    nv.device_status()
    assert torch.equal(got, want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_claimed_again_and_again(nv, d):
    # 128 sequences over the same five rows: by their own bounds every other one would pass, and make
    # 2048 units where the workspace has room for 1056
    cu = np.array([0, 5] * 64 + [0], np.int32)
    _check(nv, cu, 5, 48, 8, d, 600, 1)


@pytest.mark.parametrize("n,longest,first", [(6, 5, 0), (40, 5, 0), (40, 60, 0), (200, 4, 0), (300, 4, 150), (700, 30, 0), (1500, 20, 700)])
@pytest.mark.parametrize("d", [64, 256])
def test_random_bounds(nv, n, longest, first, d):
    rng = np.random.default_rng(n + longest + d)
    for share in (0.02, 0.3):
        cu, tokens = broken_bounds(n, longest, rng, share, first)
        if tokens:
            _check(nv, cu, tokens, 6, 1, d, 600, n)


def test_prompts_behind_a_step_back(nv):
    cu = np.array([0, 200, 120, 260, 200, 330, 331, 300, 500], np.int32)
    for d in (64, 128, 256):
        _check(nv, cu, 500, 2, 1, d, 600, 3)


@pytest.mark.parametrize("n,longest,first", [(6, 30, 0), (40, 5, 0), (300, 4, 200), (700, 3, 0), (700, 3, 600)])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 32), (256, 128)])
def test_append(nv, n, longest, first, d, block):
    import torch
    rng = np.random.default_rng(n + longest + d)
    for share in (0.02, 0.3):
        cu, tokens = broken_bounds(n, longest, rng, share, first)
        if tokens == 0:
            continue
        good = counted(cu, tokens)
        new = [int(cu[s + 1] - cu[s]) if s in set(good) else 0 for s in range(n)]
        lens = [x + int(p) for x, p in zip(new, rng.integers(0, 40, n))]
        need = [-(-x // block) for x in lens]
        table, ids, at = np.full((n, max(max(need), 1)), -1), rng.permutation(sum(need) + 1), 0
        for s, m in enumerate(need):
            table[s, :m], at = ids[at:at + m], at + m
        host = filled_cache(sum(need) + 1, 1, block, d, rng, 3.0)
        cache = to_cache(nv, *host)
        x = torch.from_numpy(rng.standard_normal((tokens, d)).astype(np.float32)).to(torch.bfloat16)
        nv.device_status()
        nv.kv_append(x.cuda(), x.cuda(), _i32(cu), _i32(lens), _i32(table), cache)
        assert nv.device_status() == (0 if len(good) == n else 7)
        rows = x.double().numpy().reshape(tokens, 1, d)
        for s in good:
            part = rows[cu[s]:cu[s + 1]]
            for i in (0, 1):
                ref.append(part, [new[s]], [lens[s]], table[s:s + 1], host[i], host[2 + i], block)
        for got, want in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), host):
            assert np.array_equal(got.cpu().numpy(), want)
