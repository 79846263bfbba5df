"""Attention over packed prompts on the GPU where the cut of a batch and values reach their
limits, against its reference (oracle/serving.py)."""
import numpy as np
import pytest
import torch

from test_kv4_gpu import hq  # noqa: F401  (the fixture)
from test_prompt_gpu import call, check, offsets, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", range(4))
def test_equal_sequences_cut_into_pieces(hq, case):
    """Batches that are cut, with several sequences of one length, or more keys than the sort by length tells
    apart: the same bits in every call."""
    new, old, nh, G, cap, dtype = (
        ([128] * 2, [20000] * 2, 8, 2, 0.0, "bf16"), ([1] * 5, [19000] * 5, 2, 4, 0.0, "f16"),
        ([1] * 9, [5000] * 9, 1, 3, 20.0, "bf16"), ([1, 3, 2], [131300, 140000, 135000], 1, 1, 0.0, "bf16"))[case]
    rng = np.random.default_rng(71 + case)
    starts, k_starts = offsets(new), offsets([a + b for a, b in zip(new, old)])
    q, k, v = tensors(rng, starts[-1], k_starts[-1], nh, G, dtype, "plain")
    first = call(hq, q, k, v, starts, k_starts, 128 ** -0.5, cap)
    for _ in range(30):
        again = call(hq, q, k, v, starts, k_starts, 128 ** -0.5, cap)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    if case > 0:
        check(q, k, v, starts, k_starts, 128 ** -0.5, cap, first)
