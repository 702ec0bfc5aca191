"""The block norms at sizes and values beyond those of test_residual_norm.py."""
import pytest

torch = pytest.importorskip("torch")

import sparse_weight_direct_gb300 as swd  # noqa: E402
from test_residual_norm import PARTS, check_all, inputs  # noqa: E402
from test_sequence import F32  # noqa: E402

# more channels than a thread of the single tokens' kernel or a cluster keeps
MANY = [(2, 20000, 1), (1, 1 << 18, 1), (1, (1 << 17) + 1, 1), (1, 20000, 7), (1, 1 << 16, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", MANY, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("value", [1.1, 0.7])
def test_squares_that_round_alike(case, value):
    """All channels alike: squares added to one number one after the other are all
    rounded to the same side, 900 E of the sum by 32,768 of them.  The bounds are
    those of any other input: sums in runs and a tree."""
    s, dsum, dout, _ = inputs(case, F32, PARTS[0], seed=20)
    for k in ("x", "y"):
        s[k] = torch.full_like(s[k], value)
    s["z"] = torch.full_like(s["z"], 0.5)
    for k in ("post", "scale", "pre"):
        s[k] = torch.full_like(s[k], 0.9)
    check_all(s, dsum, dout, None)
    if case[2] == 1:
        check_all({k: v[:, :, 0].contiguous() if v.dim() == 3 else v for k, v in s.items()}, None, None, None, back=False)
