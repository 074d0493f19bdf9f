"""CPU checks of the attention-layer entry points: refusals before any device work, the
oracle's own invariants."""
import ctypes

import numpy as np
import pytest

import nvfp4_w4a4_quantized_02_b200 as nv
from nvfp4_w4a4_quantized_02_b200 import build as nvbuild
from oracle import attention as ref
from oracle import e4m3_decode

vp = ctypes.c_void_p
P = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    nvbuild.build()
    return nv.lib()


def _cache(k=P, v=P, ks=P, vs=P, blocks=8, block=64, heads=2, d=128):
    return nv.BlockCache(k, v, ks, vs, blocks, block, heads, d)


def _batch(cu=P, lens=P, table=P, n=2, tokens=4, cols=3, ld=3):
    return nv.Batch(cu, lens, table, n, tokens, cols, ld)


BATCH_REFUSALS = [
    (dict(), dict(cu=None), 1), (dict(), dict(lens=None), 1), (dict(), dict(table=None), 1),
    (dict(k=None), dict(), 1), (dict(vs=None), dict(), 1),
    (dict(), dict(n=0), 1), (dict(), dict(tokens=-1), 1), (dict(), dict(cols=0), 1), (dict(), dict(ld=2), 1),
    (dict(blocks=0), dict(), 1), (dict(heads=0), dict(), 1),
    (dict(block=48), dict(), 2), (dict(block=8), dict(), 2), (dict(block=256), dict(), 2),
    (dict(d=96), dict(), 2), (dict(d=512), dict(), 2),
    (dict(), dict(n=70000), 2), (dict(), dict(tokens=1 << 31), 2), (dict(), dict(cols=1 << 30, ld=1 << 30), 2),
    (dict(), dict(cols=(1 << 25) - 8, ld=1 << 25), 2),  # 2^31 - 512 cached tokens of 64 a block
    (dict(k=P + 8), dict(), 3), (dict(ks=P + 2), dict(), 3), (dict(), dict(cu=P + 2), 3),
]


@pytest.mark.parametrize("c,b,want", BATCH_REFUSALS)
def test_append_and_attention_refuse_bad_batches(L, c, b, want):
    cache, batch = _cache(**c), _batch(**b)
    assert L.nvfp4_kv_append(P, 256, P, 256, batch, cache, None) == want
    assert L.nvfp4_attention(P, 512, 4, batch, cache, 0.1, 1, P, 0, 512, P, 1 << 40, None) == want


def test_append_refusals(L):
    call = lambda k=P, ld_k=256, v=P, ld_v=256: L.nvfp4_kv_append(k, ld_k, v, ld_v, _batch(), _cache(), None)
    assert call(k=None) == 1 and call(v=None) == 1
    assert call(ld_k=248) == 1 and call(ld_v=128) == 1
    assert call(k=P + 8) == 3 and call(ld_v=260) == 3


def test_attention_refusals(L):
    def call(q=P, ld_q=512, heads=4, scale=0.1, out=P, kind=0, ld=512, ws=P, ws_bytes=1 << 40):
        return L.nvfp4_attention(q, ld_q, heads, _batch(), _cache(), scale, 1, out, kind, ld, ws, ws_bytes, None)
    assert call(q=None) == 1 and call(out=None) == 1 and call(ws=None) == 1
    assert call(heads=3) == 1 and call(heads=0) == 1          # not a multiple of the kv heads
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(kind=2) == 1 and call(kind=-1) == 1
    assert call(ld_q=504) == 1 and call(ld=504) == 1
    assert call(ld_q=516) == 3 and call(ld=516) == 3 and call(q=P + 8) == 3 and call(out=P + 4) == 3
    assert call(kind=1, ld=514) == 3 and call(ws=P + 8) == 3
    need = nv.attention_workspace_bytes(4, 2, 4, 2, 128)
    assert need > 0 and call(ws_bytes=need - 1) == 1
    assert nv.attention_workspace_bytes(4, 0, 4, 2, 128) == 0 and nv.attention_workspace_bytes(4, 2, 3, 2, 128) == 0
    # more tokens, sequences or kv heads never need less
    assert nv.attention_workspace_bytes(400, 2, 4, 2, 128) >= need <= nv.attention_workspace_bytes(4, 3, 4, 2, 128)


def test_norm_rope_refusals(L):
    def call(q=P, ld_q=512, k=P, ld_k=256, tokens=3, h=4, hk=2, d=128, wq=P, eps=1e-6, off=0.0, pos=P, table=P,
             most=16, rot=64, qo=P, ld_qo=512, ko=P, ld_ko=256):
        return L.nvfp4_qk_norm_rope(q, ld_q, k, ld_k, tokens, h, hk, d, wq, P, off, eps, pos, table, most, rot, 0, qo,
                                    ld_qo, ko, ld_ko, None)
    assert call(q=None) == 1 and call(wq=None) == 1 and call(ko=None) == 1
    assert call(tokens=-1) == 1 and call(h=0) == 1 and call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(off=float("inf")) == 1
    assert call(pos=None) == 1 and call(table=None) == 1 and call(most=0) == 1
    assert call(d=96) == 2 and call(rot=24) == 2 and call(rot=144) == 2
    assert call(ld_q=504) == 1 and call(ld_ko=128) == 1
    assert call(q=P + 2) == 3 and call(ld_k=260) == 3 and call(pos=P + 4) == 3 and call(table=P + 8) == 3
    assert L.nvfp4_rope_table(None, 4, 64, 1e4, None) == 1 and L.nvfp4_rope_table(P, 0, 64, 1e4, None) == 1
    assert L.nvfp4_rope_table(P, 4, 24, 1e4, None) == 2 and L.nvfp4_rope_table(P, 4, 64, -1.0, None) == 1
    assert L.nvfp4_rope_table(P + 8, 4, 64, 1e4, None) == 3


def test_matvec_refusals(L):
    def call(x=P, ld_x=512, M=1, codes=P, scales=P, rows=64, K=512, segs=((0, 64, P),), out=P, kind=0, ldo=64):
        s = (nv.Segment * max(len(segs), 1))(*[nv.Segment(*t) for t in segs])
        return L.nvfp4_matvec(x, ld_x, M, nv.Operand(codes, scales, rows, K), s, len(segs), out, kind, ldo, None)
    assert call(x=None) == 1 and call(codes=None) == 1 and call(out=None) == 1
    assert call(M=0) == 1 and call(rows=0) == 1 and call(segs=()) == 1 and call(kind=2) == 1
    assert call(M=17) == 2 and call(K=480, ld_x=480) == 2
    assert call(ld_x=504) == 1 and call(ldo=63) == 1
    assert call(segs=((0, 32, P),)) == 1 and call(segs=((0, 32, P), (40, 64, P))) == 1 and call(segs=((0, 64, None),)) == 1
    assert call(x=P + 8) == 3 and call(codes=P + 8) == 3 and call(ld_x=516) == 3 and call(out=P + 1) == 3


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    cache = nv.block_kv_cache(2, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        nv.attention(x, i32, i32[:2], i32.reshape(1, 3), cache)
    with pytest.raises(ValueError):
        nv.kv_append(x, x, i32, i32[:2], i32.reshape(1, 3), cache)
    with pytest.raises(ValueError):
        nv.qk_norm_rope(x, x, x[0, :64], x[0, :64])
    with pytest.raises(ValueError):
        nv.matvec(x, nv.NVFP4Tensor(None, None, None, 16, 256))


def test_oracle_scale_and_append_invariants():
    for a, want in ((448.0, 1.0), (449.0, 2.0), (447.0, 1.0), (224.0, 0.5), (0.0, 2.0 ** -100), (1e-40, 2.0 ** -100)):
        assert ref.block_scale(a) == want
    rng = np.random.default_rng(0)
    # appended token by token or at once: the same scale, and values within one rounding more
    rows = rng.standard_normal((20, 1, 16)) * np.exp2(rng.integers(-3, 4, (20, 1, 1)))
    once = (np.zeros((2, 1, 16, 16), np.uint8), np.ones((2, 1), np.float32))
    steps = (once[0].copy(), once[1].copy())
    ref.append(rows, [20], [20], [[1, 0]], *once, 16)
    for t in range(20):
        ref.append(rows[t:t + 1], [1], [t + 1], [[1, 0]], *steps, 16)
    assert np.array_equal(once[1], steps[1])
    a, b = (e4m3_decode(c) * s[..., None, None] for c, s in (once, steps))
    assert np.max(np.abs(a - b)) <= 2.0 ** -10 * 16  # subnormal codes only: half a step 2^-10 of s <= 16


def test_oracle_attention_is_causal_and_normalised():
    rng = np.random.default_rng(1)
    k, v = (ref._encode(rng.standard_normal((3, 1, 16, 64)) * 50) for _ in range(2))
    one = np.ones((3, 1), np.float32)
    q = rng.standard_normal((5, 2, 64))
    out, _ = ref.attention(q, [5], [37], [[2, 0, 1]], k, v, one, one, 0.01, True)
    later = v.copy()
    later[1, 0, 4] = 0x7F  # position 36, the last one
    again, _ = ref.attention(q, [5], [37], [[2, 0, 1]], k, later, one, one, 0.01, True)
    assert np.array_equal(out[:4], again[:4]) and np.isnan(again[4]).all()
    same, _ = ref.attention(q, [5], [37], [[2, 0, 1]], k, np.full_like(v, 0x38), one, one, 0.01, False)
    assert np.allclose(same, 1.0)
