"""GPU parity of the head norms with the position rotation, against FP64."""
import numpy as np
import pytest

from attention_testutil import BF16_HALF, bf16
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


def _rows(tokens, heads, hk, d, rng, mul=1.0):
    """q and k as column ranges of one wider matrix: FP64 values and device views."""
    x, x_d = bf16(rng.standard_normal((tokens, (heads + 2 * hk) * d)) * mul)
    w, w_d = bf16(1.0 + 0.3 * rng.standard_normal((2, d)))
    cols = ((0, heads), (heads, heads + hk))
    return [x[:, a * d:b * d].reshape(tokens, b - a, d) for a, b in cols], [x_d[:, a * d:b * d] for a, b in cols], w, w_d


def _check(got, want, d):
    """One rounding to BF16; FP32 before it: the sum of d squares (d / 2 * 2^-24, halved by the
    root), the root, the quotient and three products, each 2^-24 of the terms, which are at most
    sqrt(2) times the pair's length."""
    got = got.float().cpu().numpy().astype(np.float64).reshape(want.shape)
    size = np.sqrt(2.0) * np.abs(want).max(axis=2, keepdims=True)
    bound = BF16_HALF * np.abs(want) + (d / 4 + 8) * 2.0 ** -24 * size
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert not np.any(np.abs(got - want) > bound)


@pytest.mark.parametrize("tokens", [1, 3, 33, 700])
@pytest.mark.parametrize("heads,hk,d,rot", [(48, 8, 128, 128), (6, 1, 256, 64), (3, 3, 64, 16), (5, 2, 128, 96), (1, 1, 64, 64),
                                            (7, 1, 256, 256), (4, 2, 128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_matches_oracle(nv, tokens, heads, hk, d, rot, interleaved):
    import torch
    rng = np.random.default_rng(tokens + rot)
    x, x_d, w, w_d = _rows(tokens, heads, hk, d, rng, 3.0)
    pos = rng.integers(0, 5000, tokens)
    table = nv.rope_table(5000, rot, 1e6) if rot else None
    out = nv.qk_norm_rope(x_d[0], x_d[1], w_d[0], w_d[1], torch.from_numpy(pos).cuda() if rot else None, table,
                          interleaved=interleaved)
    t = table.cpu().numpy() if rot else None
    for i in range(2):
        _check(out[i], ref.head_norm_rope(x[i], w[i], 0.0, np.float32(1e-6), pos, t, interleaved), d)
    assert nv.device_status() == 0


def test_table(nv):
    t = nv.rope_table(300_000, 64, 10000.0).cpu().numpy()
    want = ref.rope_table(300_000, 64, 10000.0)
    # FP64 angles of up to 3e5 (half a step 2^-35), rounded once to FP32
    assert np.max(np.abs(t - want)) <= 2.0 ** -25 + 2.0 ** -33


def test_weight_offset_eps_and_in_place(nv):
    import torch
    rng = np.random.default_rng(1)
    x, x_d, w, w_d = _rows(9, 4, 2, 128, rng)
    pos = rng.integers(0, 64, 9)
    table = nv.rope_table(64, 128)
    wide = torch.zeros((9, 8 * 128), dtype=torch.bfloat16, device="cuda")
    q, k = wide[:, :512], wide[:, 512:768]
    q.copy_(x_d[0])
    k.copy_(x_d[1])
    got = nv.qk_norm_rope(q, k, w_d[0], w_d[1], torch.from_numpy(pos).cuda(), table, eps=0.5, weight_offset=1.0, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and not wide[:, 768:].any()
    for i in range(2):
        _check(got[i], ref.head_norm_rope(x[i], w[i], 1.0, 0.5, pos, table.cpu().numpy(), False), 128)


@pytest.mark.parametrize("mul,eps", [(2.0 ** 100, 1e-6), (2.0 ** 120, 0.0), (2.0 ** -100, 0.0), (2.0 ** -120, 0.0), (2.0 ** -70, 1e-30),
                                     (2.0 ** -100, 1e-6)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_squares_outside_fp32(nv, mul, eps, d):
    rng = np.random.default_rng(2)
    x, x_d, w, w_d = _rows(5, 3, 1, d, rng, 1.0)
    big = [a.double().mul(mul).to(a.dtype) for a in x_d]
    big[0][2, :d] = x_d[0][2, :d]  # one head of ordinary size among them
    x = [b.double().cpu().numpy().reshape(a.shape) for a, b in zip(x, big)]  # what the operator gets
    out = nv.qk_norm_rope(big[0], big[1], w_d[0], w_d[1], eps=eps)
    for i in range(2):
        _check(out[i], ref.head_norm_rope(x[i], w[i], 0.0, float(np.float32(eps)), None, None, False), d)


def test_zero_and_non_finite_heads(nv):
    import torch
    rng = np.random.default_rng(3)
    x, x_d, w, w_d = _rows(4, 3, 1, 128, rng)
    q = x_d[0].clone()
    q[0, :128] = 0
    q[1, 130] = float("nan")
    q[2, 5] = float("inf")
    out, _ = nv.qk_norm_rope(q, x_d[1], w_d[0], w_d[1])
    out = out.float().reshape(4, 3, 128)
    assert not out[0, 0].any() and out[1, 1].isnan().all() and not out[1, 0].isnan().any() and not out[1, 2].isnan().any()
    assert out[2, 0, 5].isnan() and not out[2, 0, :5].any() and not out[2, 0, 6:].any()


def test_positions_outside_the_table(nv):
    import torch
    rng = np.random.default_rng(4)
    x, x_d, w, w_d = _rows(6, 4, 2, 64, rng)
    pos = torch.tensor([0, -1, 3, 16, 15, 2 ** 40], device="cuda")
    table = nv.rope_table(16, 64)
    q, k = torch.full_like(x_d[0], 5.0), torch.full_like(x_d[1], 5.0)
    q, k = q.contiguous(), k.contiguous()
    nv.qk_norm_rope(x_d[0], x_d[1], w_d[0], w_d[1], pos, table, q_out=q, k_out=k)
    for t in range(6):
        assert bool((q[t] == 5.0).all() and (k[t] == 5.0).all()) == (t in (1, 3, 5))
    assert nv.device_status() == 7


def test_no_tokens(nv):
    import torch
    q = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    a, b = nv.qk_norm_rope(q, q[:, :128], w, w)
    assert a.shape == (0, 256) and b.shape == (0, 128)


@pytest.mark.parametrize("tokens", [3, 6000])  # a warp per head group, a warp per token
@pytest.mark.parametrize("w", [0.0, 2.0 ** -60, 2.0 ** 70])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_in_place_among_heads_outside_fp32(nv, tokens, w, d):
    """Finished heads whose results are themselves outside FP32's range of squares stay finished."""
    import torch
    rng = np.random.default_rng(5)
    x, x_d, _, _ = _rows(tokens, 9, 5, d, rng)
    q, k = (t.contiguous().clone() for t in x_d)
    for t in (q, k):
        t.reshape(tokens, -1, d)[:, 1::3] *= 2.0 ** 100
        t.reshape(tokens, -1, d)[:, 2::3] *= 2.0 ** -100
    weight = torch.full((d,), w, dtype=torch.bfloat16, device="cuda")
    pos = torch.from_numpy(rng.integers(0, 64, tokens)).cuda()
    table = nv.rope_table(64, 32)
    for interleaved in (False, True):
        want = nv.qk_norm_rope(q, k, weight, weight, pos, table, eps=0.0, interleaved=interleaved)
        a, b = q.clone(), k.clone()
        nv.qk_norm_rope(a, b, weight, weight, pos, table, eps=0.0, interleaved=interleaved, q_out=a, k_out=b)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        assert bool(want[0].isfinite().all()) and (w > 0 or not want[0].any())
        some = slice(0, 50)
        host = q[some].double().cpu().numpy().reshape(-1, 9, d)
        _check(a[some], ref.head_norm_rope(host, np.full(d, w), 0.0, 0.0, pos[some].cpu().numpy(), table.cpu().numpy(), interleaved), d)


@pytest.mark.parametrize("rot", [0, 32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_infinities_behind_the_rotation_stay_alone(nv, rot, d):
    """y = x / rms: next to an infinity finite values are 0, and only rotated pairs share it."""
    import torch
    rng = np.random.default_rng(6)
    x, x_d, w, w_d = _rows(4, 3, 1, d, rng)
    q = x_d[0].clone()
    q[1, d + 41] = float("inf")       # behind the rotated range, odd
    q[2, 2 * d + 50] = -float("inf")  # and even
    q[3, 7] = float("inf")            # within it, if there is one
    pos = torch.tensor([3, 5, 7, 9], device="cuda") if rot else None
    table = nv.rope_table(16, rot) if rot else None
    out = nv.qk_norm_rope(q, x_d[1], w_d[0], w_d[1], pos, table, interleaved=True)[0].float().reshape(4, 3, d).cpu().numpy()
    want = np.zeros((4, 3, d), bool)
    want[1, 1, 41] = want[2, 2, 50] = want[3, 0, 7] = True
    if rot:
        want[3, 0, 6] = True
    assert np.array_equal(np.isnan(out), want)
    for t, h in ((1, 1), (2, 2), (3, 0)):
        assert not np.any(out[t, h][~want[t, h]])
