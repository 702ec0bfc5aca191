"""A selective-scan block whose projections are pruned 1x1 layers, serving
requests of different lengths with an adapter each: prompts first, then token
by token.

    python examples/pruned_sequence_block.py

Everything is channels-first: a projection is spconv's 1x1 layer over N x C x 1
x L positions (1 x 1 for a token), its output is the next operator's input as
it lies.

    xz       = W_in x                  pruned, shared by all requests
    xz      += s_i B_i A_i x           each request's own adapter
    u, z     = halves of xz
    u        = silu(short convolution of u)
    dt, B, C = W_x u                   pruned
    delta    = W_dt dt                 pruned
    y        = selective scan of u, delta, A, B, C, D, gated by z
    out      = W_out y                 pruned

The block's states (K-1 inputs of the convolution, S numbers of the scan for each
channel) live in pools; a request's token names its slot.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sparse_weight_direct_gb300 as swd  # noqa: E402


class PrunedLinear:
    """M x C pruned weights as 1x1 layers: packed once for each number of
    positions that they meet (1 for tokens, the prompts' padded length)."""

    def __init__(self, M, C, density, rng):
        keep = rng.random((M, C)) < density
        keep[np.arange(M), rng.integers(0, C, M)] = True  # no empty row
        self.dense = np.where(keep, rng.normal(0, (density * C) ** -0.5, (M, C)), 0).astype(np.float32)
        self.M, self.C = M, C
        self.rowptr = np.concatenate([[0], np.cumsum(keep.sum(1))]).astype(np.int32)
        self.colidx = np.nonzero(keep)[1].astype(np.int32)
        self.value = self.dense[keep]
        self.packed = {}

    def __call__(self, x):
        """(N, C, L) -> (N, M, L)"""
        N, C, L = x.shape
        if L not in self.packed:
            self.packed[L] = swd.pack(self.rowptr, self.colidx, self.value, C=C, H=1, W=L, M=self.M,
                                      R=1, S=1, batch_hint=N)
        return swd.forward(x.view(N, C, 1, L), self.packed[L]).view(N, self.M, L)


class PrunedSequenceBlock:
    def __init__(self, width=64, inner=128, states=16, taps=4, dt_rank=8, adapters=3, rank=8,
                 density=0.1, slots=8, seed=0):
        rng = np.random.default_rng(seed)
        self.inner, self.S, self.R = inner, states, dt_rank
        self.w_in = PrunedLinear(2 * inner, width, density, rng)
        self.w_x = PrunedLinear(dt_rank + 2 * states, inner, density, rng)
        self.w_dt = PrunedLinear(inner, dt_rank, 0.5, rng)
        self.w_out = PrunedLinear(width, inner, density, rng)

        def normal(*shape, scale=1.0):
            return torch.from_numpy(rng.normal(0, scale, shape).astype(np.float32)).cuda()

        self.conv_w, self.conv_b = normal(inner, taps, scale=taps ** -0.5), normal(inner, scale=0.1)
        self.A = -torch.arange(1, states + 1, device="cuda", dtype=torch.float32).repeat(inner, 1)
        self.D = torch.ones(inner, device="cuda")
        self.dt_bias = normal(inner, scale=0.5) - 3.0
        self.a = normal(adapters, rank, width, scale=width ** -0.5)
        self.b = normal(adapters, 2 * inner, rank, scale=rank ** -0.5)
        self.scale = torch.full((adapters,), 0.5, device="cuda")
        self.conv_pool = torch.zeros(slots, inner, taps - 1, device="cuda")
        self.scan_pool = torch.zeros(slots, inner, states, device="cuda")

    def _project(self, x, index):
        xz = self.w_in(x)
        return swd.adapter_add(xz, x, self.a, self.b, index, scale=self.scale, out=xz)

    def _parts(self, u):
        p = self.w_x(u)
        R, S = self.R, self.S
        return self.w_dt(p[:, :R].contiguous()), p[:, R:R + S], p[:, R + S:]

    def prompts(self, x, lengths, index, slots):
        """x: (N, width, L), each request's first lengths[n] positions; its
        states go to slots[n].  Outputs behind a length mean nothing."""
        xz = self._project(x, index)
        u, z = xz[:, :self.inner], xz[:, self.inner:]
        conv, scan = self.conv_pool[:len(x)].clone(), self.scan_pool[:len(x)].clone()
        u = swd.short_conv(u, self.conv_w, self.conv_b, final_state=conv, lengths=lengths)
        delta, B, C = self._parts(u)
        y = swd.scan(u, delta, self.A, B, C, D=self.D, z=z, delta_bias=self.dt_bias,
                     final_state=scan, lengths=lengths)
        self.conv_pool[slots.long()] = conv
        self.scan_pool[slots.long()] = scan
        return self.w_out(y)

    def token(self, x, index, slots):
        """x: (N, width), the next token of the requests in slots[n]."""
        xz = self._project(x[:, :, None], index)[:, :, 0]
        u, z = xz[:, :self.inner], xz[:, self.inner:]
        u = swd.short_conv_step(u, self.conv_pool, self.conv_w, self.conv_b, slots=slots)
        delta, B, C = self._parts(u[:, :, None])
        y = swd.scan_step(self.scan_pool, u, delta[:, :, 0], self.A, B[:, :, 0], C[:, :, 0],
                          D=self.D, z=z, delta_bias=self.dt_bias, slots=slots)
        return self.w_out(y[:, :, None])[:, :, 0]


def run(lengths=(19, 1, 32, 7), more=5, seed=0):
    """Prompts, then `more` tokens of every request, against one pass over the
    whole sequences: the largest difference relative to the outputs' size."""
    block = PrunedSequenceBlock(seed=seed)
    N, width, total = len(lengths), block.w_in.C, max(lengths) + more
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, width, total, generator=g).cuda()
    index = torch.tensor([n % 4 - 1 for n in range(N)], dtype=torch.int32, device="cuda")
    slots = torch.tensor([(3 * n + 2) % 8 for n in range(N)], dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    whole = block.prompts(x, lens + more, index, slots)
    first = block.prompts(x[:, :, :max(lengths)].contiguous(), lens, index, slots)
    worst = 0.0
    for n, k in enumerate(lengths):
        worst = max(worst, float((first[n, :, :k] - whole[n, :, :k]).abs().max()))
    for t in range(more):
        now = torch.stack([x[n, :, k + t] for n, k in enumerate(lengths)])
        out = block.token(now, index, slots)
        want = torch.stack([whole[n, :, k + t] for n, k in enumerate(lengths)])
        worst = max(worst, float((out - want).abs().max()))
    return worst / float(whole.abs().max())


if __name__ == "__main__":
    off = run()
    print(f"prompts and tokens agree with one pass to {off:.1e} of the largest output")
    sys.exit(0 if off < 1e-5 else 1)
