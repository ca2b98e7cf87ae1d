"""Rules of ScoreMod that the fp32 fields of pa_score_mod cannot hold: no GPU is touched."""
import pytest

import paged_kv_cache_107_gb300 as pk


@pytest.mark.parametrize("cap", [1e-46, 1e-60, 5e-324])
def test_a_cap_that_fp32_rounds_to_zero_is_refused(cap):
    """0 would mean no cap at all, the opposite of a cap that takes every score to 0."""
    with pytest.raises(pk.PagedAttentionError, match="softcap"):
        pk.ScoreMod(softcap=cap)._check(16, 2)


@pytest.mark.parametrize("cap", [0.0, 0, 1e-6, 50, 1e30])
def test_other_caps_pass(cap):
    assert pk.ScoreMod(softcap=cap)._check(16, 2).softcap == pytest.approx(float(cap), rel=2e-7)
