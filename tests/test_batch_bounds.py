"""CPU checks of the rule by which sequences of a batch count: what the sizes of workspaces, grids
and slot ranges rest on."""
import numpy as np
import pytest

from attention_testutil import broken_bounds, counted


@pytest.mark.parametrize("n,longest", [(1, 5), (6, 5), (50, 40), (300, 3), (200, 300)])
def test_sequences_that_count_share_no_rows_and_no_slots(n, longest):
    rng = np.random.default_rng(n + longest)
    for _ in range(50):
        cu, tokens = broken_bounds(n, longest, rng, share=rng.choice([0.0, 0.05, 0.5, 1.0]))
        good = counted(cu, tokens)
        rows = np.zeros(tokens, int)
        for s in good:
            rows[cu[s]:cu[s + 1]] += 1
        assert rows.max(initial=0) <= 1
        for group in (1, 6, 8):  # row blocks of 8 and of 256 query rows
            new = [int(cu[s + 1] - cu[s]) * group for s in good]
            assert sum(-(-x // 8) for x in new if x <= 32) <= min((tokens * group + 7) // 8 + n, 4 * n)
            prompts = min(tokens * group // 33, n)
            for tile in (128, 256):
                assert sum(-(-x // tile) for x in new if x > 32) <= tokens * group // tile + prompts
        for log_block in (4, 7):
            slots = [(int(cu[s]) >> log_block) + 2 * s for s in good], [(int(cu[s + 1]) >> log_block) + 2 * (s + 1) for s in good]
            assert all(e <= b for e, b in zip(slots[1], slots[0][1:]))
            assert not good or slots[1][-1] <= (tokens >> log_block) + 2 * n


def test_examples():
    assert counted([0, 5, 0, 5, 0, 5], 5) == [0]
    assert counted([0, 100, 50, 100, 120], 200) == [0, 3]    # the third starts inside the first
    assert counted([0, 5000, 71, 72], 72) == [2]             # a bound that is no row binds nobody
    assert counted([3, 3, 7, -1, 7, 9], 9) == [0, 1, 4]
    assert counted([0, 2, 4], 4) == [0, 1]
