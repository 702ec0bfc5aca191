"""Beam search's selection at sizes and arguments beyond those of test_beams.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_weight_direct_gb300 as swd  # noqa: E402
from test_sequence import F16, Draw  # noqa: E402


@pytest.mark.gpu
def test_sums_of_parts_that_round_alike():
    """2^28 tokens, every eighth likely and the others alike: so are the sums of the
    16,384 parts of the row, and added to one number one after the other they would
    all be rounded to the same side.  A thread's eight loads of five additions count 23
    roundings of 2^-24 of their sum (earlier ones are of less of it), the trees over
    lanes, warps and lanes 18; an exponential is good to 2^-22, its argument, below 2,
    to 2^-23: 47 times 2^-24."""
    V = 1 << 28
    if torch.cuda.get_device_properties(0).total_memory < 8 << 30:
        pytest.skip("needs 2 GB of device memory")
    logits = torch.zeros(1, 1, V, dtype=F16, device="cuda")
    for low in (-0.17, -0.52, -0.77, -0.87, -0.92, -0.97):
        logits[0, 0] = low
        logits[0, 0, ::8] = 0
        exact = math.log(V / 8 * (1 + 7 * math.exp(float(logits[0, 0, 1]))))
        start = torch.tensor([[exact]], device="cuda")  # (so that the score, near zero, keeps the sum's error)
        score, token, _, _ = swd.beam_select(logits, start)
        assert int(token) == 0
        assert abs(float(score) - (float(start) - exact)) <= 47 * 2.0 ** -24, low


@pytest.mark.gpu
def test_beams_and_eos_of_any_kind_of_whole_number():
    d = Draw(23)
    logits, scores = d(2, 3, 40), d(2, 3)
    want = swd.beam_select(logits, scores, beams=4, eos=7)
    for beams, eos in ((np.int64(4), np.int32(7)), (torch.tensor(4), torch.tensor(7))):
        assert all(torch.equal(a, b) for a, b in zip(swd.beam_select(logits, scores, beams=beams, eos=eos), want))
    for bad in ("2", 2.0, [2], None.__class__, torch.tensor([1, 2])):
        with pytest.raises(swd.SpconvError):
            swd.beam_select(logits, scores, eos=bad)
        with pytest.raises(swd.SpconvError):
            swd.beam_select(logits, scores, beams=bad)
