"""Rules of ScoreMod that the fp32 fields of pa_score_mod cannot hold, and what the header says of
arrays that are read early: no GPU is touched."""
import os
import re

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


HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "pa.h")


@pytest.mark.parametrize("call,arrays", [("pa_decode_mod", ["prefix_lens"]),
                                         ("pa_decode_shared", ["group_starts", "prefix_lens"])])
def test_the_header_names_the_arrays_that_are_read_early(call, arrays):
    """The launch rule of a dependent launch binds every array read before the wait for the
    previous kernel, those of the rules and groups included."""
    text = re.sub(r"\s*\n \* ?", " ", open(HEADER).read())
    about = text[text.index(f"{call} — "):]
    about = re.split(r" (?:Both: a softcap|pa_prefill_mod — )|\*/", about)[0]
    rules = [s for s in re.split(r"(?<=\.) ", about) if "context_lens and block_tables" in s]
    assert rules and all(any(a in s for s in rules) for a in arrays), about
