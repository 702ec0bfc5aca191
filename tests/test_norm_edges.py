"""The block norms at sizes and values beyond those of test_residual_norm.py."""
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

from test_residual_norm import PARTS, check_all, inputs  # noqa: E402
from test_sequence import F32, TYPE_IDS, TYPES  # noqa: E402

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


def test_every_plan_fits(tmp_path):
    """All plans over types, inputs, whole and odd rows, lengths and channels, on the host: within a
    block's shared memory, with clusters to run them, and over all channels and positions."""
    from sparse_weight_direct_gb300 import build as b
    exe = str(tmp_path / "norm_plan_test")
    cmd = [b._nvcc(), "-std=c++17", "-O1", *b.ARCH, "-I", os.path.join(b.ROOT, "include"), "-I", b.CSRC,
           os.path.join(b.ROOT, "tests", "c_abi", "norm_plan_test.cu"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("parts", ["x pre", "y"])
@pytest.mark.parametrize("case", [(1, 22528, 16), (1, 23552, 8), (1, 45000, 24), (1, 47104, 64)], ids=lambda c: "x".join(map(str, c)))
def test_weights_beside_a_tile(case, parts, dtype):
    """One input's tiles leave little room for the weights of the channels that they hold."""
    check_all(*inputs(case, dtype, parts, seed=22), back=False)
