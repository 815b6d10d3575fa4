"""The parity tests of the attention-layer operators once more, with comparisons that no NaN
passes (tests/layer_checks.py)."""
import pytest

import test_gpu_attn
import test_gpu_rope
from layer_checks import numbers
from test_gpu_attn import (jb, test_256_queries_to_a_key_head, test_cache_past_32_bit_offsets,  # noqa: F401
                           test_chunk_at_the_end_of_a_long_context, test_decode, test_last_round_in_pieces,
                           test_many_sequences, test_non_finite_values_that_no_query_sees, test_packed,
                           test_pages_out_of_range_read_as_zeros, test_plan_hints_change_no_result,
                           test_rows_behind_the_last_sequence_stay, test_scale_and_large_scores)
from test_gpu_rope import (test_backward, test_forward, test_in_place_strides_and_far_positions,  # noqa: F401
                           test_layer_in_serving)

pytestmark = pytest.mark.gpu


def strict(check, near):
    def check_numbers(d, r, new, kv, *args, **kw):
        numbers(r["o"], sum(new))
        numbers(r["lse"].unsqueeze(-1), sum(new))
        check(d, r, new, kv, *args, **kw)

    def near_numbers(got, want, t):
        numbers(got)
        near(got, want, t)
    return check_numbers, near_numbers


@pytest.fixture(autouse=True)
def comparisons_that_no_nan_passes(monkeypatch):
    check, near = strict(test_gpu_attn.check, test_gpu_rope.near)
    monkeypatch.setattr(test_gpu_attn, "check", check)
    monkeypatch.setattr(test_gpu_rope, "check", check)
    monkeypatch.setattr(test_gpu_rope, "near", near)
