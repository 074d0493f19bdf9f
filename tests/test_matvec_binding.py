"""CPU checks of what the binding of the product refuses, with host tensors that claim to be on a device."""
import pytest
import torch

import nvfp4_w4a4_quantized_02_b200 as nv


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


def _t(t):
    return t.as_subclass(OnDevice)


@pytest.fixture
def call(monkeypatch):
    """The binding with a launch that only notes what it gets."""
    launched = []
    monkeypatch.setattr(nv, "_launch", lambda *a: launched.append(a))

    def run(rows=200, cols=128, tokens=3, **change):
        w = dict(codes=_t(torch.zeros((rows, cols // 2), dtype=torch.uint8)),
                 scales=_t(torch.zeros(nv.scale_bytes(rows, cols), dtype=torch.uint8)),
                 gs=_t(torch.ones(1)), rows=rows, cols=cols)
        segments = change.pop("segments", None)
        w["rows"] = change.pop("claimed_rows", rows)
        w.update(change)
        launched.clear()
        out = nv.matvec(_t(torch.zeros((tokens, cols), dtype=torch.bfloat16)), nv.NVFP4Tensor(**w), segments=segments)
        return out, launched
    return run


def test_whole_weights_pass(call):
    for rows, cols in ((200, 128), (1, 64), (128, 192), (129, 4160)):
        out, launched = call(rows, cols)
        assert out.shape == (3, rows) and len(launched) == 1


@pytest.mark.parametrize("change", [
    dict(codes=_t(torch.zeros((200, 64), dtype=torch.int8))),
    dict(codes=_t(torch.zeros((200, 128), dtype=torch.uint8)[:, ::2])),
    dict(codes=_t(torch.zeros((64, 200), dtype=torch.uint8).t())),
    dict(codes=_t(torch.zeros((199, 64), dtype=torch.uint8))),
    dict(scales=_t(torch.zeros(256 * 8, dtype=torch.float32))),
    dict(scales=_t(torch.zeros((256, 16), dtype=torch.uint8)[:, :8])),
    dict(scales=_t(torch.zeros(200 * 8, dtype=torch.uint8))),  # rows padded to 128 have scales too
    dict(claimed_rows=300),
], ids=lambda c: next(iter(c)))
def test_weights_that_are_not_what_the_kernel_reads_are_refused(call, change):
    with pytest.raises(ValueError, match="the weight must be"):
        call(**change)


def test_global_scales_of_other_types_are_refused(call):
    for gs in (torch.ones(1, dtype=torch.float64), torch.ones(1, dtype=torch.bfloat16), torch.ones(0)):
        with pytest.raises(ValueError, match="a global scale must be"):
            call(gs=_t(gs))
        with pytest.raises(ValueError, match="a global scale must be"):
            call(segments=[(0, 8, _t(torch.ones(1))), (8, 200, _t(gs))])
    with pytest.raises(ValueError, match="another device"):
        call(gs=torch.ones(1))


def test_no_tokens_launch_nothing(call):
    out, launched = call(tokens=0)
    assert out.shape == (0, 200) and not launched
    with pytest.raises(ValueError, match="the weight must be"):
        call(tokens=0, claimed_rows=300)
