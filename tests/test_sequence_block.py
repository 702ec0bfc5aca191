"""The pruned selective-scan block of examples/pruned_sequence_block.py: prompts
of different lengths, tokens, adapters and pruned projections together, each
against plain products in 64 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import sequence_reference as ref  # noqa: E402


def plain(block, x, length, i):
    """One request's outputs in 64 bits: (width, length)"""
    x = ref.f64(x)[:, :length]
    W = [torch.from_numpy(w.dense).double() for w in (block.w_in, block.w_x, block.w_dt, block.w_out)]
    xz = W[0] @ x
    if i >= 0:
        xz = xz + float(block.scale[i]) * (ref.f64(block.b[i]) @ (ref.f64(block.a[i]) @ x))
    u, z = xz[:block.inner], xz[block.inner:]
    (u, _), _, _ = ref.conv(u[None], block.conv_w, block.conv_b, True, None, None)
    p = W[1] @ u[0]
    R, S = block.R, block.S
    (y, _), _ = ref.scan(u, (W[2] @ p[:R])[None], block.A, p[None, R:R + S], p[None, R + S:], block.D,
                         z[None], block.dt_bias, True, None, None)
    return W[3] @ y[0]


@pytest.mark.gpu
def test_block_against_plain_products():
    """Every stage is good to about 2^-20 of its terms and none of the six
    amplifies more than a few times: 1e-4 of the largest output."""
    import pruned_sequence_block as example
    block = example.PrunedSequenceBlock(seed=3)
    lengths = (13, 1, 33)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, block.w_in.C, 33, generator=g).cuda()
    index = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 0, 7], dtype=torch.int32, device="cuda")
    out = block.prompts(x, torch.tensor(lengths, dtype=torch.int32, device="cuda"), index, slots)
    for n, k in enumerate(lengths):
        want = plain(block, x[n], k, int(index[n]))
        far = (ref.f64(out[n, :, :k]) - want).abs().max()
        assert float(far) <= 1e-4 * float(want.abs().max()), n


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,more", [((19, 1, 32, 7), 5), ((1,), 3), ((64, 63, 2), 2)])
def test_tokens_continue_prompts(lengths, more):
    import pruned_sequence_block as example
    assert example.run(lengths, more, seed=len(lengths)) < 1e-5


@pytest.mark.gpu
def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "pruned_sequence_block.py")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "agree with one pass" in r.stdout


def test_pruned_linear_is_its_csr():
    import pruned_sequence_block as example
    w = example.PrunedLinear(12, 20, 0.2, np.random.default_rng(0))
    dense = np.zeros((12, 20), np.float32)
    for m in range(12):
        for k in range(w.rowptr[m], w.rowptr[m + 1]):
            dense[m, w.colidx[k]] = w.value[k]
    assert np.array_equal(dense, w.dense) and (np.diff(w.rowptr) > 0).all()
