"""Calls on another stream than the current one, without any order between the two: results and
workspaces must not lie in memory that kernels queued on the current stream still use."""
import numpy as np
import pytest

from attention_testutil import batch, filled_cache, to_cache
from nvfp4_testutil import make_operand

pytestmark = pytest.mark.gpu
WAIT = 40_000_000  # cycles: some 20 ms


@pytest.fixture(scope="module")
def nv():
    import torch
    from nvfp4_w4a4_quantized_02_b200 import build
    build.build()
    import nvfp4_w4a4_quantized_02_b200 as nv
    assert torch.cuda.is_available()
    return nv


def _calls(nv):
    """Calls that allocate their results: name -> call with a stream, which returns a tuple of tensors."""
    import torch
    rng = np.random.default_rng(0)
    bf = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()
    x, y, w = bf(200, 512), bf(200, 256), bf(128)
    cu, lens, table, _, count = batch([1, 3, 196], [700, 30, 300], 16, rng)
    cache = to_cache(nv, *filled_cache(count, 2, 16, 128, rng))
    weight = make_operand(rng.integers(0, 16, (40000, 512)).astype(np.uint8), rng.integers(8, 0x7F, (40000, 32)).astype(np.uint8), 2.0)
    return {
        "norm": lambda s: nv.qk_norm_rope(x, y, w, w, stream=s),
        "attention": lambda s: (nv.attention(x, cu, lens, table, cache, stream=s),),
        "attention, FP32": lambda s: (nv.attention(x, cu, lens, table, cache, out_dtype="f32", stream=s),),
        "matvec": lambda s: (nv.matvec(x[:16], weight, stream=s),),
        "table": lambda s: (nv.rope_table(3000, 64, stream=s),),
    }


def test_memory_with_a_reader_on_the_current_stream_is_left_alone(nv):
    import torch
    side = torch.cuda.Stream()
    for name, call in _calls(nv).items():
        want = call(None)
        need = [t.clone() for t in want]
        del want
        torch.cuda.synchronize()
        # tensors of the results' sizes, read late on the current stream, and free for the allocator at once
        held = [torch.full_like(t, 3.0) for t in need]
        seen = [torch.empty_like(t) for t in need]
        torch.cuda.synchronize()
        torch.cuda._sleep(WAIT)
        for a, b in zip(seen, held):
            a.copy_(b)
        del held, a, b
        got = call(side)
        side.synchronize()
        mine = [t.clone() for t in got]  # on the current stream, behind the readers
        torch.cuda.synchronize()
        assert all(bool((t == 3.0).all()) for t in seen), name
        assert all(torch.equal(a, b) for a, b in zip(mine, need)), name


def test_results_with_a_reader_on_the_current_stream_are_left_alone(nv):
    import torch
    side = torch.cuda.Stream()
    for name, call in _calls(nv).items():
        got = call(side)
        side.synchronize()
        want = [t.clone() for t in got]
        seen = [torch.empty_like(t) for t in got]
        torch.cuda.synchronize()
        torch.cuda._sleep(WAIT)
        for a, b in zip(seen, got):
            a.copy_(b)
        del got, a, b
        other = []
        with torch.cuda.stream(side):
            for t in want:
                other.append(torch.full_like(t, 3.0))  # would take the freed results' place
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(seen, want)), name


def test_capture_with_a_forked_stream(nv):
    import torch
    side = torch.cuda.Stream()
    for name, call in _calls(nv).items():
        want = call(None)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            got = call(side)
            main.wait_stream(side)
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
