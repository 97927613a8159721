"""QK-Clip: head counts at the ends of their type. Nothing is launched: the calls have no weights (cols = 0)."""
import pytest

import adamw_hybrid_optimizer_muon_b200 as ma

TOP = 0x6000_0000_0000  # made up, never followed
MOST = (1 << 31) - 1


@pytest.mark.parametrize("heads,kv", [(MOST, 1), (MOST, MOST), (1 << 30, 1 << 30), (MOST - 1, 2), (2048, 1), (1025, 1025)])
def test_head_counts_whose_sum_passes_the_limit_are_refused(heads, kv):
    # the sum of the first four is beyond 32 bits
    assert heads % kv == 0
    assert ma.lib().ma_qk_clip(heads, kv, 1, 1, 0, None, None, TOP, 100.0, 0.5, None) == ma.MA_ERR_UNSUPPORTED
