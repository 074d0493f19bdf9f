"""GPU parity of attention over the block-scaled 8-bit cache, against FP64."""
import numpy as np
import pytest

from attention_testutil import BF16_HALF, attention_bound, batch, bf16, filled_cache, to_cache
from oracle import attention as ref
from oracle import e4m3_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import torch
    from nvfp4_w4a4_quantized_02_b200 import build
    build.build()
    import nvfp4_w4a4_quantized_02_b200 as nv
    assert torch.cuda.is_available()
    return nv


def run_case(nv, q_lens, kv_lens, heads, hk, d, block, causal, seed=0, scale=None, out_dtype="f32", q_mul=1.0,
             edit=None, spread=1.0, q_edit=None):
    """Runs one batch and checks it against the oracle; returns (got, want)."""
    import torch
    rng = np.random.default_rng(seed)
    cu, lens, table_d, table, count = batch(q_lens, kv_lens, block, rng)
    k, v, ks, vs = filled_cache(count, hk, block, d, rng, spread)
    if edit is not None:
        edit(k, v, ks, vs, table)
        import torch
        table_d = torch.from_numpy(table).cuda()
    x = rng.standard_normal((sum(q_lens), heads, d)) * q_mul
    if q_edit is not None:
        q_edit(x)
    q, q_d = bf16(x)
    scale = d ** -0.5 if scale is None else scale
    got = nv.attention(q_d.reshape(-1, heads * d), cu, lens, table_d, to_cache(nv, k, v, ks, vs), softmax_scale=scale,
                       causal=causal, out_dtype=out_dtype)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy().reshape(q.shape)
    want, mags = ref.attention(q, q_lens, kv_lens, table, k, v, ks, vs, float(np.float32(scale)), causal)
    biggest = np.nanmax(np.abs(e4m3_decode(v)) * vs[..., None, None]) if v.size else 0.0
    half = BF16_HALF if out_dtype == "bf16" else 2.0 ** -24
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bound = attention_bound(want, mags, biggest, half, max(kv_lens))
    over = np.abs(got - want) - bound
    assert not np.any(over > 0), f"{np.nanmax(over)} over the bound at {np.unravel_index(np.nanargmax(over), over.shape)}"
    return got, want


# one row group, odd lengths, tile and block borders, empty sequences
DECODE = [
    ([1], [1], 1, 1, 128, 16), ([1], [15], 6, 1, 128, 16), ([1], [16], 8, 2, 64, 16), ([1], [17], 6, 1, 256, 16),
    ([1], [700], 48, 8, 128, 64), ([1, 1, 1], [129, 1, 1000], 12, 2, 128, 32), ([1, 0, 1], [40, 33, 128], 6, 1, 64, 128),
    ([2, 3, 5], [2, 70, 513], 6, 2, 128, 16), ([5], [300], 4, 4, 256, 64), ([4, 1], [64, 65], 8, 1, 64, 64),
    ([1] * 40, list(range(1, 400, 10)), 2, 1, 128, 16), ([1], [4097], 3, 1, 128, 128), ([1, 1], [2000, 0], 6, 1, 256, 32),
]
# query rows around the tiles of 128 and 256, ragged batches, short prompts on long caches
PROMPT = [
    ([33], [33], 1, 1, 128, 16), ([128], [128], 1, 1, 128, 64), ([129], [129], 1, 1, 64, 64), ([100], [1000], 6, 2, 128, 32),
    ([257, 40], [257, 300], 1, 1, 256, 16), ([64, 1, 90], [500, 77, 90], 6, 1, 64, 16), ([50], [61], 8, 1, 256, 128),
    ([11, 200, 0, 43], [11, 201, 5, 1111], 4, 1, 128, 16), ([130], [130], 2, 2, 256, 64), ([300], [700], 1, 1, 128, 128),
]


@pytest.mark.parametrize("case", DECODE + PROMPT, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_matches_oracle(nv, case, causal):
    run_case(nv, *case, causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 60])
def test_bf16_output(nv, d, q_len):
    run_case(nv, [q_len, 1], [q_len + 100, 9], 6, 2, d, 16, True, out_dtype="bf16", seed=3)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [3, 70])
def test_rows_that_see_nothing_are_zero(nv, d, q_len):
    # more new tokens than the cache holds: the first rows' positions are negative
    got, _ = run_case(nv, [q_len, 2], [2, 0], 4, 1, d, 16, True)
    assert not got[:q_len - 2].any() and not got[q_len:].any() and got[q_len - 2:q_len].any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 4, 75])
def test_nan_behind_the_end_and_in_later_tokens(nv, d, q_len):
    kv, block = 75 + 64, 16

    def edit(k, v, ks, vs, table):
        last = table[0, (kv - 1) // block]
        for c in (k, v):
            c[last, :, (kv - 1) % block + 1:] = 0x7F           # behind the end of the sequence
        spare = np.setdiff1d(np.arange(k.shape[0]), table)
        k[spare], v[spare], ks[spare], vs[spare] = 0xFF, 0x7F, np.nan, np.nan
        v[last, 0, (kv - 1) % block, 5] = 0xFF                  # the last token: only the last row sees it
        if q_len > 2:
            k[table[0, (kv - 2) // block], 1, (kv - 2) % block, 3] = 0x7F
    got, _ = run_case(nv, [q_len], [kv], 4, 2, d, block, True, edit=edit)
    assert np.isnan(got).any() and not np.isnan(got[0]).all()


@pytest.mark.parametrize("q_len", [1, 50])
def test_nan_everyone_sees(nv, q_len):
    def edit(k, v, ks, vs, table):
        v[table[0, 0], 0, 3, 17] = 0x7F
        k[table[0, 1], 1, 2, 1] = 0xFF
    got, _ = run_case(nv, [q_len], [300], 4, 2, 128, 16, True, edit=edit)
    assert np.isnan(got[:, :2, 17]).all() and np.isnan(got[:, 2:]).all() and not np.isnan(got[:, :2, 18]).any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 90])
def test_value_scales_far_apart(nv, d, q_len):
    run_case(nv, [q_len], [500], 2, 1, d, 16, True, spread=8.0, seed=5, q_mul=0.02)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 90])
def test_scores_that_keep_growing(nv, d, q_len):
    # every block's keys outweigh the ones before: the running maximum moves at every tile
    def edit(k, v, ks, vs, table):
        for b, at in enumerate(table[0]):
            ks[at] = 2.0 ** -8 * 1.03125 ** b
            k[at] = 0x48  # 4.0

    def q_edit(x):
        x[:] = np.abs(x) + 0.5
    run_case(nv, [q_len], [1500], 2, 1, d, 16, True, edit=edit, q_edit=q_edit, scale=0.6)


@pytest.mark.parametrize("q_len", [1, 90])
@pytest.mark.parametrize("q_mul,scale", [(2.0 ** 100, 2.0 ** -104), (2.0 ** -100, 2.0 ** 97), (1.0, -0.1), (1.0, 0.0)])
def test_query_sizes_and_scales(nv, q_len, q_mul, scale):
    run_case(nv, [q_len], [200], 4, 2, 128, 32, True, q_mul=q_mul, scale=scale)


@pytest.mark.parametrize("q_len", [2, 90])
def test_non_finite_queries_stay_in_their_row(nv, q_len):
    def q_edit(x):
        x[0, 1, 3] = np.nan
        x[1, 0, 7] = np.nan
        x[1, 2] = 0.0
    got, _ = run_case(nv, [q_len], [200], 3, 1, 128, 32, True, q_edit=q_edit)
    assert np.isnan(got[0, 1]).all() and not np.isnan(got[0, 0]).any() and not np.isnan(got[1, 2]).any()


@pytest.mark.parametrize("q_len", [1, 90])
def test_other_scales_than_powers_of_two(nv, q_len):
    def edit(k, v, ks, vs, table):
        ks *= 1.37
        vs *= 0.777
    run_case(nv, [q_len], [333], 6, 1, 128, 64, True, edit=edit, out_dtype="bf16")


@pytest.mark.parametrize("q_len", [1, 90])
def test_bad_blocks_are_reported_and_hold_nothing(nv, q_len):
    def edit(k, v, ks, vs, table):
        table[0, 3] = 10 ** 6
        table[0, 5] = -7
    run_case(nv, [q_len], [333], 6, 1, 128, 16, True, edit=edit)
    assert nv.device_status() == 7 and nv.device_status() == 0


def _inputs(nv, q_lens, kv_lens, heads, hk, d, block, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    cu, lens, table_d, table, count = batch(q_lens, kv_lens, block, rng)
    cache = to_cache(nv, *filled_cache(count, hk, block, d, rng))
    q = torch.from_numpy(rng.standard_normal((sum(q_lens), heads * d)).astype(np.float32)).to(torch.bfloat16).cuda()
    return q, cu, lens, table_d, cache


def test_bad_sequences_are_skipped_and_reported(nv):
    import torch
    q, cu, lens, table, cache = _inputs(nv, [1, 70, 1], [30, 90, 40], 4, 2, 64, 16)
    good = nv.attention(q, cu, lens, table, cache)
    for at, value in ((0, -1), (1, 10 ** 6), (2, table.shape[1] * 16 + 1)):
        bad = lens.clone()
        bad[at] = value
        out = torch.full_like(good, 7.0)
        nv.attention(q, cu, bad, table, cache, out=out)
        rows = torch.arange(cu[at], cu[at + 1], device="cuda")
        keep = torch.ones(len(q), dtype=torch.bool, device="cuda")
        keep[rows] = False
        assert (out[rows] == 7.0).all() and torch.equal(out[keep], good[keep])
        assert nv.device_status() == 7
    wrong = cu.clone()
    wrong[1] = 5000
    out = torch.full_like(good, 7.0)
    nv.attention(q, wrong, lens, table, cache, out=out)
    assert torch.equal(out[71:], good[71:]) and (out[:71] == 7.0).all() and nv.device_status() == 7


def test_strides_and_rows_behind_the_last_sequence(nv):
    import torch
    for q_lens in ([1, 3], [80, 1]):
        q, cu, lens, table, cache = _inputs(nv, q_lens, [100, 40], 6, 2, 64, 16)
        want = nv.attention(q, cu, lens, table, cache)
        n = len(q)
        wide = torch.full((n + 5, 3 * 384 + 8), 3.0, dtype=torch.bfloat16, device="cuda")
        wide[:n, 384:768] = q
        out = torch.full((n + 5, 400), 9.0, dtype=torch.bfloat16, device="cuda")
        tables = torch.full((2, table.shape[1] + 3), -5, dtype=torch.int32, device="cuda")
        tables[:, :table.shape[1]] = table
        nv.attention(wide[:, 384:768], cu, lens, tables[:, :table.shape[1]], cache, out=out[:, :384])
        assert torch.equal(out[:n, :384], want) and (out[n:] == 9.0).all() and (out[:, 384:] == 9.0).all()
        assert nv.device_status() == 0


def test_empty_calls(nv):
    import torch
    q, cu, lens, table, cache = _inputs(nv, [1], [20], 2, 1, 64, 16)
    assert nv.attention(q[:0], torch.zeros_like(cu), lens, table, cache).shape == (0, 128)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert nv.attention(q, none, none[:0], table[:0], cache).shape == q.shape


def test_repeats_are_identical_on_other_streams_and_in_graphs(nv):
    import torch
    for q_lens, kv_lens, d in (([1] * 9, [5000, 3, 700, 90, 1, 64, 1200, 33, 2500], 128), ([400, 1, 200], [900, 800, 200], 128),
                               ([300, 2], [2000, 500], 256)):
        q, cu, lens, table, cache = _inputs(nv, q_lens, kv_lens, 6, 1, d, 16)
        want = nv.attention(q, cu, lens, table, cache)
        for _ in range(20):
            assert torch.equal(nv.attention(q, cu, lens, table, cache), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        on_side = nv.attention(q, cu, lens, table, cache, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(on_side, want)
        # two graphs that share a workspace, replayed one after the other
        ws = torch.empty(nv.attention_workspace_bytes(len(q), len(lens), 6, 1, d), dtype=torch.uint8, device="cuda")
        outs, graphs = [], []
        half = (q * 0.5).contiguous()
        for x in (q, half):
            out = torch.zeros_like(want)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                nv.attention(x, cu, lens, table, cache, out=out, workspace=ws)
            outs.append(out)
            graphs.append(g)
        ws.fill_(0xFF)
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], nv.attention(half, cu, lens, table, cache))
    assert nv.device_status() == 0


def test_offsets_beyond_32_bits(nv):
    import torch
    # 4.3 GB per tensor; the sequences live in the last blocks
    d, block, count = 128, 64, (1 << 32) // (64 * 128) + 1000
    for q_len in (1, 80):
        q, cu, lens, table, small = _inputs(nv, [q_len], [200], 2, 1, d, block)
        want = nv.attention(q, cu, lens, table, small)
        big = nv.block_kv_cache(count, 1, block, d)
        far = table + (count - small.k.shape[0])
        at = far[0].long()
        big.k[at], big.v[at] = small.k[table[0].long()], small.v[table[0].long()]
        big.k_scales[at], big.v_scales[at] = small.k_scales[table[0].long()], small.v_scales[table[0].long()]
        assert torch.equal(nv.attention(q, cu, lens, far, big), want)
        del big


def test_mixed_batch_equals_separate_calls(nv):
    import torch
    q_lens, kv_lens = [1, 500, 3, 1, 60], [3000, 800, 50, 1, 4000]
    q, cu, lens, table, cache = _inputs(nv, q_lens, kv_lens, 6, 2, 128, 32)
    whole = nv.attention(q, cu, lens, table, cache, out_dtype="f32")
    for s, n in enumerate(q_lens):
        lo = int(cu[s])
        one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        part = nv.attention(q[lo:lo + n], one, lens[s:s + 1], table[s:s + 1], cache, out_dtype="f32")
        # a unit cut elsewhere sums in another order, and takes its weights from other references:
        # each side is within its FP16 rounding of them
        assert torch.allclose(part, whole[lo:lo + n], rtol=0, atol=2.0 ** -10 * float(whole.abs().max()))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 90])
def test_whole_leading_tiles_of_bad_blocks(nv, q_len, d):
    def edit(k, v, ks, vs, table):
        table[0, :17] = 10 ** 6  # the first 272 tokens: more than two tiles
    got, _ = run_case(nv, [q_len], [700], 3, 1, d, 16, True, edit=edit)
    assert got.any()
    assert nv.device_status() == 7


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [2, 70])
def test_nothing_but_bad_blocks(nv, q_len, d):
    def edit(k, v, ks, vs, table):
        table[:] = -1
    got, _ = run_case(nv, [q_len], [400], 3, 1, d, 16, True, edit=edit)
    assert not got.any() and nv.device_status() == 7


def test_many_sequences(nv):
    """More sequences than threads of a CTA, short and long in turn."""
    rng = np.random.default_rng(11)
    q_lens = [int(x) for x in rng.integers(0, 4, 900)]
    q_lens[::97] = [45] * len(q_lens[::97])
    kv_lens = [q + int(x) for q, x in zip(q_lens, rng.integers(0, 60, 900))]
    kv_lens[500] = 3000
    run_case(nv, q_lens, kv_lens, 1, 1, 64, 16, True)
    assert nv.device_status() == 0


def test_first_sequence_starts_behind_the_first_row(nv):
    import torch
    for q_lens in ([2, 1], [50, 40]):
        q, cu, lens, table, cache = _inputs(nv, q_lens, [60, 41], 4, 2, 128, 16)
        want = nv.attention(q, cu, lens, table, cache)
        more = torch.cat([torch.full_like(q[:3], 5.0), q])
        out = torch.full_like(more, 9.0)
        nv.attention(more, cu + 3, lens, table, cache, out=out)
        assert torch.equal(out[3:], want) and (out[:3] == 9.0).all()


def test_two_streams_at_once(nv):
    import torch
    runs = []
    for i, (q_lens, kv_lens) in enumerate((([1] * 6, [4000, 10, 700, 90, 2000, 64]), ([300, 200], [900, 700]))):
        args = _inputs(nv, q_lens, kv_lens, 6, 2, 128, 64, seed=i)
        runs.append((args, nv.attention(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for args, want, stream in runs:
            with torch.cuda.stream(stream):
                got.append((nv.attention(*args), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)


def test_changed_lengths_between_replays(nv):
    """A captured call follows the lengths, tables and queries that are in its buffers when it runs."""
    import torch
    q, cu, lens, table, cache = _inputs(nv, [1, 1, 1], [900, 900, 900], 4, 2, 128, 16)
    out = torch.zeros_like(q)
    nv.attention(q, cu, lens, table, cache, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.attention(q, cu, lens, table, cache, out=out)
    for n in ([1, 2, 3], [900, 1, 450], [16, 17, 0]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        assert torch.equal(out, nv.attention(q, cu, lens, table, cache)), n


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([40], [4500]), ([60, 1, 45], [3333, 2100, 45]), ([130], [2200])], ids=str)
def test_few_prompt_rows_on_a_long_cache(nv, d, q_lens, kv_lens):
    """The cache is cut over several CTAs, whose results are joined."""
    run_case(nv, q_lens, kv_lens, 2, 1, d, 32, True, seed=8)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_joined_parts_keep_masks_and_nan(nv, d):
    def edit(k, v, ks, vs, table):
        v[table[0, 100], 0, 3, 9] = 0x7F       # position 1603: everyone sees it, value 9
        v[table[0, -1], 0, 5, 17] = 0xFF       # among the new tokens
        k[table[0, -1], 0, 6, 1] = 0x7F
        table[0, 20:60] = -3
    got, _ = run_case(nv, [50], [4090], 2, 1, d, 16, True, edit=edit)
    assert np.isnan(got[:, :, 9]).all() and not np.isnan(got[0, 0, 8]) and nv.device_status() == 7


def test_output_over_the_input_is_refused(nv):
    q, cu, lens, table, cache = _inputs(nv, [1, 3], [40, 50], 2, 1, 64, 16)
    with pytest.raises(ValueError, match="out must not be q"):
        nv.attention(q, cu, lens, table, cache, out=q)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_tiles", [1, 2, 3, 4, 7, 9])
def test_prompts_around_tile_ends(nv, d, n_tiles):
    """One token less, as many and one more than whole tiles of 128 cached tokens, causal or not."""
    for extra in (-1, 0, 1):
        kv = 128 * n_tiles + extra
        for causal in (True, False):
            run_case(nv, [65, 70], [kv, max(kv - 57, 70)], 2, 1, d, 16, causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("growth", [0.0, 2.5, 9.0])
def test_denominators_of_long_rows_with_the_smallest_value_scale(nv, d, q_len, growth):
    """700000 tokens of one value at the smallest scale: the output is that value.  The scores of
    the first tile are lower, so that the others' weights exceed the reference by 2^growth."""
    import torch
    block, kv = 128, 700_000
    k = torch.zeros((2, 1, block, d), dtype=torch.uint8, device="cuda")
    k[1, :, :, 0] = 0x38  # 1.0
    v = torch.full_like(k, 0x3C)  # 1.5
    one = torch.ones((2, 1), device="cuda")
    cache = nv.BlockKVCache(k, v, one, one * 2.0 ** -100)
    table = torch.ones((1, -(-kv // block)), dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    q = torch.zeros((q_len, d), dtype=torch.bfloat16, device="cuda")
    q[:, 0] = growth
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = nv.attention(q, i32(0, q_len), i32(kv), table, cache, softmax_scale=float(np.log(2.0)), causal=False, out_dtype="f32")
    # FP16's rounding of one weight for all, 2^-11; sums of 700000 / 16 terms in one chain at worst, each
    # addition within 2^-23, above and below
    bound = 2.0 ** -11 + 2 * 700_000 / 16 * 2.0 ** -23
    want = 1.5 * 2.0 ** -100
    assert float((got.double() / want - 1.0).abs().max()) <= bound


def wide_queries(rng, rows, heads, d, outlier):
    """Queries with one value per row `outlier` times the others."""
    x = rng.standard_normal((rows, heads, d))
    x[:, :, 5] = outlier * rng.choice([-1.0, 1.0], (rows, heads))
    return x


def narrow_keys(rng, count, block, d):
    """Keys of two values, and next to nothing where the queries have their outlier."""
    k = np.zeros((count, 1, block, d))
    k[..., [8, 9]] = rng.standard_normal((count, 1, block, 2)) * 100.0
    k = ref._encode(k)
    k[..., 5] = rng.choice([0x00, 0x01, 0x81], (count, 1, block))
    return k


def wide_query_bound(q, k, ks, scale, parts):
    """Largest error of a score.  Of prompts (`parts`) a value is exact down to 2^-10 of the row's largest, and
    below it within half a step 2^-9 of the row scaled to (224, 448]; of few tokens down to 2^-29 of it,
    and below within half a step 2^-24 of [2^14, 2^15)."""
    top = np.abs(q).max(axis=2)
    dq = top[..., None] * (2.0 ** -10 / 224 if parts else 2.0 ** -25 / 2.0 ** 14)
    if parts:
        dq = np.where(np.abs(q) >= 2.0 ** -10 * top[..., None], 0.0, dq)
    reach = np.abs(e4m3_decode(k) * ks[..., None, None]).max(axis=(0, 1, 2))
    return scale * (np.broadcast_to(dq, q.shape) * reach).sum(axis=2)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [3, 50])
@pytest.mark.parametrize("log_outlier", [0, 4, 8, 11, 14])
def test_queries_far_apart_within_a_row(nv, d, q_len, log_outlier):
    import torch
    rng = np.random.default_rng(log_outlier)
    heads, kv, block = 2, 300, 32
    cu, lens, table_d, table, count = batch([q_len], [kv], block, rng)
    _, v, ks, vs = filled_cache(count, 1, block, d, rng)
    k, scale = narrow_keys(rng, count, block, d), 0.25
    q, q_d = bf16(wide_queries(rng, q_len, heads, d, 2.0 ** log_outlier))
    got = nv.attention(q_d.reshape(q_len, -1), cu, lens, table_d, to_cache(nv, k, v, ks, vs), softmax_scale=scale, out_dtype="f32")
    got = got.double().cpu().numpy().reshape(q.shape)
    want, mags = ref.attention(q, [q_len], [kv], table, k, v, ks, vs, scale, True)
    dx = wide_query_bound(q, k, ks, scale, q_len * heads > 32)[..., None]
    biggest = np.abs(e4m3_decode(v) * vs[..., None, None]).max()
    # scores off by dx either way move a weight's share by e^(2 dx)
    bound = attention_bound(want, mags, biggest, 2.0 ** -24, kv) + np.expm1(2 * dx) * mags
    assert not np.any(np.abs(got - want) > bound)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 50])
@pytest.mark.parametrize("log_scale", [0, 6])
@pytest.mark.parametrize("gap", [6, 14, 20, 26, 30])
def test_weights_far_below_the_largest(nv, d, q_len, log_scale, gap):
    """A block whose tokens outweigh all others by 2^gap and whose values are zero, at a larger
    scale or not: the output is what the small weights make of the others' values."""
    import torch
    rng = np.random.default_rng(gap)
    block, kv = 16, 200
    cu, lens, table_d, table, count = batch([q_len], [kv], block, rng)
    _, v, ks, _ = filled_cache(count, 1, block, d, rng)
    k, ks, vs = np.zeros_like(v), np.ones_like(ks), np.ones_like(ks)
    first = table[0, 0]
    k[first, ..., 0], v[first], vs[first] = 0x38, 0, 2.0 ** log_scale
    x = np.zeros((q_len, 1, d))
    x[..., 0] = gap
    q, q_d = bf16(x)
    scale = float(np.float32(np.log(2.0)))
    got = nv.attention(q_d.reshape(q_len, -1), cu, lens, table_d, to_cache(nv, k, v, ks, vs), softmax_scale=scale, causal=False,
                       out_dtype="f32").double().cpu().numpy().reshape(q.shape)
    want, mags = ref.attention(q, [q_len], [kv], table, k, v, ks, vs, scale, False)
    # a weight times its value scale is within half a step 2^-24 of FP16 of 2^12 (few tokens) or 2^6 (prompts) for
    # the largest one; the first block's 16 tokens make up the denominator at least
    least = 2.0 ** (log_scale - (37 if q_len == 1 else 31)) * np.abs(e4m3_decode(v)).sum(axis=(0, 1, 2)) / 16
    bound = 2.0 ** -24 * np.abs(want) + (2.0 ** -11 + 2.0 ** -13) * mags + least
    assert not np.any(np.abs(got - want) > bound)
