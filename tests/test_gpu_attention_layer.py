"""The attention-layer operators one after another, as a serving step runs them: projection,
head norms with rotation, append, attention, output projection; a prompt, then single tokens."""
import numpy as np
import pytest

from attention_testutil import BF16_HALF, bf16
from nvfp4_testutil import logical
from oracle import attention as ref

pytestmark = pytest.mark.gpu

D, BLOCK = 64, 16


@pytest.fixture(scope="module")
def nv():
    import torch
    from nvfp4_w4a4_quantized_02_b200 import build
    build.build()
    import nvfp4_w4a4_quantized_02_b200 as nv
    assert torch.cuda.is_available()
    return nv


def test_prompt_then_tokens(nv):
    """Prompt of two sequences, then 20 steps of single tokens, each checked against FP64 run
    on the operators' own inputs."""
    import torch
    rng = np.random.default_rng(0)
    hid = 512
    w_qkv = nv.quantize_fused([bf16(rng.standard_normal((n * D, hid)) * 0.05)[1] for n in (8, 2, 2)])
    w_o = nv.quantize(bf16(rng.standard_normal((hid, 8 * D)) * 0.05)[1])
    w_q, w_k = (bf16(1 + 0.1 * rng.standard_normal(D))[1] for _ in range(2))
    heads, hk = 8, 2
    rope = nv.rope_table(256, 32)
    prompt = [40, 75]
    table = np.array([[5, 1, 9, 3, 0, 11, 12], [2, 8, 4, 7, 6, 10, 13]], np.int32)
    table_d = torch.from_numpy(table).cuda()
    cache = nv.block_kv_cache(14, hk, BLOCK, D)
    for t in (cache.k, cache.v):
        t.fill_(0x7F)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    lens = list(prompt)
    for step in range(21):
        new = prompt if step == 0 else [1, 1]
        if step:
            lens = [n + 1 for n in lens]
        rows = sum(new)
        x = bf16(rng.standard_normal((rows, hid)))[1]
        pos = torch.cat([torch.arange(n - c, n) for n, c in zip(lens, new)]).cuda()
        cu, kv = i32([0, new[0], rows]), i32(lens)
        qkv = (nv.linear(nv.quantize(x), w_qkv[0], segments=w_qkv[1]) if step == 0 else
               nv.matvec(x, w_qkv[0], segments=w_qkv[1]))
        q_in, k_in, v_in = qkv[:, :heads * D], qkv[:, heads * D:(heads + hk) * D], qkv[:, (heads + hk) * D:]
        q, k = nv.qk_norm_rope(q_in, k_in, w_q, w_k, pos, rope)
        before = [t.cpu().numpy().copy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
        nv.kv_append(k, v_in, cu, kv, table_d, cache)
        o = nv.attention(q, cu, kv, table_d, cache)
        y = nv.linear(nv.quantize(o), w_o) if step == 0 else nv.matvec(o, w_o)
        torch.cuda.synchronize()
        f = lambda t: t.float().cpu().numpy().astype(np.float64)
        want_q = ref.head_norm_rope(f(q_in).reshape(rows, heads, D), f(w_q), 0.0, 1e-6, pos.cpu().numpy(), rope.cpu().numpy(), False)
        top = np.abs(want_q).max()
        assert np.max(np.abs(f(q).reshape(want_q.shape) - want_q)) <= (BF16_HALF + 2.0 ** -18) * 1.5 * top
        ref.append(f(k).reshape(rows, hk, D), new, lens, table, before[0], before[2], BLOCK)
        ref.append(f(v_in).reshape(rows, hk, D), new, lens, table, before[1], before[3], BLOCK)
        for got, want in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), before):
            held = np.unique(np.concatenate([table[s, :-(-n // BLOCK)] for s, n in enumerate(lens)]))
            assert np.array_equal(got.cpu().numpy()[held], want[held])
        want, mags = ref.attention(f(q).reshape(rows, heads, D), new, lens, table, *before, float(np.float32(D ** -0.5)), True)
        assert not np.any(np.abs(f(o).reshape(want.shape) - want) > BF16_HALF * np.abs(want) + 2.0 ** -10 * mags)
        if step:
            codes, sf = logical(w_o)
            want, mags = ref.matvec(f(o), codes, sf, [(0, hid, float(w_o.gs))])
            assert not np.any(np.abs(f(y) - want) > BF16_HALF * np.abs(want) + 2.0 ** -13 * mags)
    assert nv.device_status() == 0


def test_token_step_in_a_graph(nv):
    """A token step captured once and replayed with new inputs, lengths and positions in place."""
    import torch
    rng = np.random.default_rng(1)
    hid, heads, hk = 512, 8, 2
    w_qkv = nv.quantize_fused([bf16(rng.standard_normal((n * D, hid)) * 0.05)[1] for n in (8, 2, 2)])
    w_q = bf16(np.ones(D))[1]
    rope = nv.rope_table(64, D)
    table = torch.tensor([[1, 3], [2, 0]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    x, pos = torch.zeros((2, hid), dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    kv = torch.ones(2, dtype=torch.int32, device="cuda")

    def step(cache, out):
        qkv = nv.matvec(x, w_qkv[0], segments=w_qkv[1])
        q, k = nv.qk_norm_rope(qkv[:, :512], qkv[:, 512:640], w_q, w_q, pos, rope)
        nv.kv_append(k, qkv[:, 640:], cu, kv, table, cache)
        return nv.attention(q, cu, kv, table, cache, out=out)

    def fresh():
        c = nv.block_kv_cache(4, hk, BLOCK, D)
        for t in (c.k, c.v, c.k_scales, c.v_scales):
            t.zero_()
        return c
    a, b = fresh(), fresh()
    out_a, out_b = (torch.zeros((2, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    step(fresh(), out_a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, out_a)
    for t in range(30):
        x.copy_(bf16(rng.standard_normal((2, hid)))[1])
        pos.fill_(t)
        kv.fill_(t + 1)
        g.replay()
        step(b, out_b)
        torch.cuda.synchronize()
        assert torch.equal(out_a, out_b), t
    assert torch.equal(a.k, b.k) and torch.equal(a.v_scales, b.v_scales)
