"""GPU parity of the products of a few BF16 tokens with an NVFP4 weight, against FP64."""
import numpy as np
import pytest

from attention_testutil import BF16_HALF, bf16
from nvfp4_testutil import make_operand, to_dev_f32
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


def _weight(n, k, rng):
    codes = rng.integers(0, 16, (n, k)).astype(np.uint8)
    sf = rng.integers(0x08, 0x7F, (n, k // 16)).astype(np.uint8)
    return codes, sf


def _check(got, want, mags, k, half_step):
    """Operands are exact, so the error is that of K additions in FP32 (2^-23 of the partial
    sum each, were they truncated) and one rounding of the result."""
    got = got.double().cpu().numpy()
    bound = half_step * np.abs(want) + (k + 8) * 2.0 ** -23 * mags
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert not np.any(np.abs(got - want) > bound)


@pytest.mark.parametrize("m", [1, 2, 5, 8, 9, 16])
@pytest.mark.parametrize("n,k", [(16, 64), (128, 256), (1000, 1024), (130, 1088), (5120, 6144), (37, 4160), (2304, 320)])
def test_matches_oracle(nv, m, n, k):
    rng = np.random.default_rng(m * n + k)
    codes, sf = _weight(n, k, rng)
    x, x_d = bf16(rng.standard_normal((m, k)))
    want, mags = ref.matvec(x, codes, sf, [(0, n, 3.0)])
    w = make_operand(codes, sf, 3.0)
    _check(nv.matvec(x_d, w, out_dtype="f32"), want, mags, k, 2.0 ** -23)
    _check(nv.matvec(x_d, w), want, mags, k, BF16_HALF)


def test_segments_of_odd_sizes_and_strides(nv):
    import torch
    rng = np.random.default_rng(1)
    n, k = 300, 512
    codes, sf = _weight(n, k, rng)
    w = make_operand(codes, sf, 1.0)
    cuts = [(0, 7, 2.0), (7, 133, 0.25), (133, 300, 11.0)]
    segs = [(a, b, to_dev_f32([g])) for a, b, g in cuts]
    x, x_d = bf16(rng.standard_normal((3, 3 * k)))
    out = torch.full((4, 2 * n + 1), 9.0, dtype=torch.bfloat16, device="cuda")
    nv.matvec(x_d[:, k:2 * k], w, segments=segs, out=out[:3, :n])
    want, mags = ref.matvec(x[:, k:2 * k], codes, sf, cuts)
    _check(out[:3, :n], want, mags, k, BF16_HALF)
    assert (out[3] == 9.0).all() and (out[:, n:] == 9.0).all()


def test_sizes_of_x_far_apart(nv):
    rng = np.random.default_rng(2)
    n, k = 64, 4096
    codes, sf = _weight(n, k, rng)
    x = rng.standard_normal((4, k))
    x[0] *= 2.0 ** 90
    x[1] *= 2.0 ** -90
    x[2, 1024:2048] *= 2.0 ** 40  # one chunk of the row
    x[3] = 0.0
    x, x_d = bf16(x)
    want, mags = ref.matvec(x, codes, sf, [(0, n, 1.0)])
    _check(nv.matvec(x_d, make_operand(codes, sf, 1.0), out_dtype="f32"), want, mags, k, 2.0 ** -23)


def test_non_finite_inputs_stay_in_their_row(nv):
    rng = np.random.default_rng(3)
    n, k = 200, 2048
    codes, sf = _weight(n, k, rng)
    codes[codes % 8 == 0] = 1  # no zero code: 0 * inf is NaN
    x, x_d = bf16(rng.standard_normal((3, k)))
    x_d[1, 5] = float("nan")
    x_d[2, 1500] = float("inf")
    sf[17, 3] = 0x7F  # a NaN scale
    got = nv.matvec(x_d, make_operand(codes, sf, 1.0), out_dtype="f32").cpu().numpy()
    assert np.isnan(got[1]).all() and np.isnan(got[:, 17]).all()
    rest = np.delete(got, 17, axis=1)
    assert np.isfinite(rest[0]).all() and np.isinf(rest[2]).all()


def test_agrees_with_the_library_quantiser(nv):
    """A weight quantised by the library: the product is that of its dequantised values."""
    import torch
    rng = np.random.default_rng(4)
    w, w_d = bf16(rng.standard_normal((256, 1024)) * 0.02)
    x, x_d = bf16(rng.standard_normal((2, 1024)))
    q = nv.quantize(w_d)
    y = nv.matvec(x_d, q, out_dtype="f32").double().cpu().numpy()
    assert np.linalg.norm(y - x @ w.T) <= 0.15 * np.linalg.norm(x @ w.T)  # the 4-bit weight itself
    assert torch.equal(nv.matvec(x_d, q), nv.matvec(x_d, q))


def test_graph_replay(nv):
    import torch
    rng = np.random.default_rng(5)
    codes, sf = _weight(512, 2048, rng)
    w = make_operand(codes, sf, 1.0)
    x, x_d = bf16(rng.standard_normal((1, 2048)))
    want = nv.matvec(x_d, w)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.matvec(x_d, w, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_refusals_of_the_binding(nv):
    import torch
    w = nv.quantize(torch.ones(64, 64, dtype=torch.bfloat16, device="cuda"))
    x = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="out must not be x"):
        nv.matvec(x, w, out=x)
    with pytest.raises(ValueError, match="global scale"):
        nv.matvec(x, w, segments=[(0, 32, w.gs), (32, 64, w.gs.cpu())])
