"""Host-side refusals at the borders of what a decoding step's operators document."""
from test_step_operators_abi import ALIAS, INVALID, lib, logits, pytestmark  # noqa: F401


def test_histories_that_a_count_cannot_hold(lib):  # noqa: F811
    # a token may be there as often as the history is wide, and its count has 30 bits
    assert logits(lib, history_width=1 << 30, history=1 << 40, rows=1) == INVALID
    assert logits(lib, history_width=(1 << 30) - 1, history=1 << 40, rows=1) not in (INVALID, ALIAS)
