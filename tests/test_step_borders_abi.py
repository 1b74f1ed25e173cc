"""Host-side refusals at the borders of what a decoding step's operators document, and what their tests' checks refuse."""
import numpy as np
import pytest
import torch

from test_logits_gpu import make, reference
from test_step_borders_gpu import wrong_logits
from test_step_operators_abi import ALIAS, INVALID, lib, logits, pytestmark  # noqa: F401


def test_histories_that_a_count_cannot_hold(lib):  # noqa: F811
    # a token may be there as often as the history is wide, and its count has 30 bits
    assert logits(lib, history_width=1 << 30, history=1 << 40, rows=1) == INVALID
    assert logits(lib, history_width=(1 << 30) - 1, history=1 << 40, rows=1) not in (INVALID, ALIAS)


def test_the_check_of_penalised_logits_refuses_nan():
    # the 64-bit values themselves pass; a NaN among the touched, the masked or the others does not
    rng = np.random.default_rng(1)
    x = torch.as_tensor(rng.standard_normal((3, 500)).astype(np.float32))
    rules = make(rng, 3, 500, width=50, biases=4, mask=0.9)
    want, size, touched = reference(x.double().numpy(), rules)
    right = torch.where(torch.as_tensor(touched | np.isneginf(want)), torch.as_tensor(want).float(), x)
    wrong_logits(right, x, want, size, touched, "fp32", 4)
    masked = np.isneginf(want)
    for places in (touched & ~masked, masked, ~touched & ~masked):
        bad = right.clone()
        r, t = np.argwhere(places)[0]
        bad[r, t] = float("nan")
        with pytest.raises(AssertionError):
            wrong_logits(bad, x, want, size, touched, "fp32", 4)
