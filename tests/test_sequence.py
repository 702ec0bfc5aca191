"""The sequence operators (short causal convolution, selective scan, low-rank
adapters) against plain 64-bit forms (sequence_reference.py, which derives the
bounds), at the sizes and masks where they can go wrong: one position, lengths
of zero and one, odd lengths, tiles' ends, strided halves of a projection,
padding that holds NaN, slots outside the pool, another stream, graph capture,
offsets past 32 bits.  Refusals of wrong arguments are checked at the C entry
without a GPU and at the Python one."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import sequence_reference as ref  # noqa: E402
import sparse_weight_direct_gb300 as swd  # noqa: E402
from sparse_weight_direct_gb300 import _lib  # noqa: E402
from sparse_weight_direct_gb300._lib import AdapterArgs, ScanArgs, ShortConvArgs  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
TYPE_IDS = ["f32", "bf16", "f16"]


class Draw:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(dtype).cuda()


def lengths_of(N, L):
    """An empty sequence, one of one position, a full one and others between; a
    negative length and one past L count as 0 and L."""
    some = [L, 0, 1, max(L - 1, 0), -3, L + 7, L // 2, (L * 3) // 4]
    return torch.tensor([some[i % len(some)] for i in range(N)], dtype=torch.int32, device="cuda")


def poison(t, lengths):
    """t with NaN behind each length."""
    t = t.clone()
    for n, k in enumerate(lengths.tolist()):
        t[n, ..., max(k, 0):] = float("nan")
    return t


def wide(t, channels_before=3):
    """The same values as a slice of a larger tensor: another batch stride, an
    offset, and rows that keep their alignment only if L is even enough."""
    big = torch.full((t.shape[0], t.shape[1] + channels_before, *t.shape[2:]), float("nan"),
                     dtype=t.dtype, device=t.device)
    big[:, channels_before:] = t
    return big[:, channels_before:]


# ------------------------------------------------------------------ short convolution

CONV = [  # N, C, L, K
    (1, 1, 1, 1), (1, 1, 1, 4), (3, 5, 1, 3), (2, 3, 2, 4), (8, 7, 9, 4), (8, 33, 64, 4), (5, 12, 65, 2),
    (8, 6, 131, 3), (2, 4, 2051, 4), (1, 600, 24, 4), (70, 1220, 32, 4),
]


def conv_inputs(case, dtype, ragged, seed=0):
    N, C, L, K = case
    d = Draw(seed)
    x, dy = d(N, C, L, dtype=dtype), d(N, C, L, dtype=dtype)
    lens = lengths_of(N, L) if ragged else None
    if ragged:
        x, dy = poison(x, lens), poison(dy, lens)
    return (x, dy, d(C, K, scale=K ** -0.5), d(C, scale=0.3), d(N, C, K - 1, dtype=dtype),
            d(N, C, K - 1, dtype=dtype), lens)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CONV)
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("ragged,full", [(False, True), (True, True), (True, False), (False, False)])
def test_short_conv(case, dtype, ragged, full):
    """Forward and gradients; full: with bias, silu, state and strided inputs."""
    x, dy, w, b, st, df, lens = conv_inputs(case, dtype, ragged)
    if not full:
        b = st = df = None
    else:
        x, dy = wide(x), wide(dy)
    final = torch.full((x.shape[0], x.shape[1], case[3] - 1), float("nan"), dtype=dtype, device="cuda")
    y = swd.short_conv(x, w, b, silu=full, state=st, final_state=final, lengths=lens)
    (wy, by), (wf, bf), _ = ref.conv(x, w, b, full, st, lens)
    ref.check(y, wy, by, "y")
    assert torch.equal(final.cpu().double(), wf)
    got = swd.short_conv_backward(dy, x, w, b, silu=full, state=st, dfinal_state=df, lengths=lens)
    want = ref.conv_backward(dy, x, w, b, full, st, df, lens)
    for name, g, (value, bound) in zip(("dx", "dweight", "dbias", "dstate"), got, want):
        if not full and name in ("dbias", "dstate"):
            assert g is None
        else:
            ref.check(g, value, bound, name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("C,L", [(45000, 16), (700, 520)])
def test_short_conv_batch_equals_its_sequences(dtype, C, L):
    """Threads that take one sequence after the other give the bits of calls with
    one sequence each; the weights' gradients are their sums."""
    d = Draw(21)
    N, K = 8, 4
    x, dy, w, b = d(N, C, L, dtype=dtype), d(N, C, L, dtype=dtype), d(C, K, scale=0.5), d(C)
    st, df = d(N, C, K - 1, dtype=dtype), d(N, C, K - 1, dtype=dtype)
    final = torch.empty_like(st)
    y = swd.short_conv(x, w, b, state=st, final_state=final)
    dx, dw, db, ds = swd.short_conv_backward(dy, x, w, b, state=st, dfinal_state=df)
    sw, sb = torch.zeros_like(dw), torch.zeros_like(db)
    for n in range(N):
        one = slice(n, n + 1)
        f = torch.empty_like(st[one])
        assert torch.equal(swd.short_conv(x[one], w, b, state=st[one], final_state=f), y[one])
        assert torch.equal(f, final[one])
        gx, gw, gb, gs = swd.short_conv_backward(dy[one], x[one], w, b, state=st[one], dfinal_state=df[one])
        assert torch.equal(gx, dx[one]) and torch.equal(gs, ds[one])
        sw += gw
        sb += gb
    # sums of N L terms below 3 or so in another order
    tol = N * L * 2.0 ** -23 * 8
    assert float((dw - sw).abs().max()) <= tol and float((db - sb).abs().max()) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("N,C", [(1, 1), (5, 33), (3, 1000), (64, 128)])
def test_short_conv_step(K, dtype, N, C):
    """Slots in another order, one outside the pool; the rest of the pool stays."""
    d = Draw(1)
    x, w, b = d(N, C, dtype=dtype), d(C, K, scale=K ** -0.5), d(C, scale=0.3)
    pool = d(N + 2, C, K - 1, dtype=dtype)
    slots = torch.arange(N, dtype=torch.int32).flip(0) + 1
    if N > 2:
        slots[1], slots[2] = -1, N + 2
    before = pool.clone()
    y = swd.short_conv_step(x, pool, w, b, slots=slots.cuda())
    left = before.clone()
    for n, s in enumerate(slots.tolist()):
        if not 0 <= s < N + 2:
            assert not y[n].any()
            continue
        (wy, by), (wf, _), _ = ref.conv(x[n][None, :, None], w, b, True, before[s][None], None)
        ref.check(y[n][None, :, None], wy, by, "y")
        left[s] = wf[0].to(dtype)
    assert torch.equal(pool, left)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
def test_short_conv_pieces_and_tokens_equal_one_pass(dtype):
    """A sequence in two calls that hand over the state, and token by token:
    the same sums in the same order, so the same bits."""
    d = Draw(2)
    N, C, L, K = 3, 20, 37, 4
    x, w, b = d(N, C, L, dtype=dtype), d(C, K, scale=0.5), d(C)
    whole = torch.empty(N, C, K - 1, dtype=dtype, device="cuda")
    y = swd.short_conv(x, w, b, final_state=whole)
    mid, end = torch.empty_like(whole), torch.empty_like(whole)
    y1 = swd.short_conv(x[..., :17], w, b, final_state=mid)
    y2 = swd.short_conv(x[..., 17:], w, b, state=mid, final_state=end)
    assert torch.equal(torch.cat([y1, y2], 2), y) and torch.equal(end, whole)
    pool = torch.zeros_like(whole)
    for t in range(L):
        assert torch.equal(swd.short_conv_step(x[..., t].contiguous(), pool, w, b), y[..., t])
    assert torch.equal(pool, whole)


# ------------------------------------------------------------------ selective scan

SCAN = [  # N, channels, L, S, groups
    (1, 1, 1, 1, 1), (3, 2, 1, 16, 1), (2, 5, 3, 4, 1), (8, 6, 31, 16, 2), (8, 33, 32, 16, 1),
    (2, 40, 33, 8, 2), (8, 3, 70, 3, 3), (2, 36, 129, 16, 1), (1, 10, 40, 17, 1), (2, 4, 50, 64, 2),
    (1, 70, 200, 5, 2), (1, 3, 700, 16, 1),
]


def scan_inputs(case, dtype, ragged, seed=0):
    N, ch, L, S, G = case
    d = Draw(seed)
    s = dict(u=d(N, ch, L, dtype=dtype), delta=d(N, ch, L, dtype=dtype, scale=0.7),
             A=-(torch.arange(1, S + 1, device="cuda") * torch.exp(d(ch, S, scale=0.1))),
             B=d(N, G, S, L, dtype=dtype), C=d(N, G, S, L, dtype=dtype), D=d(ch),
             z=d(N, ch, L, dtype=dtype), delta_bias=d(ch, scale=0.5) - 3.0)
    lens = lengths_of(N, L) if ragged else None
    dy = d(N, ch, L, dtype=dtype)
    if ragged:
        for k in ("u", "delta", "B", "C", "z"):
            s[k] = poison(s[k], lens)
        dy = poison(dy, lens)
    return s, dy, d(N, ch, S, scale=0.5), d(N, ch, S, scale=0.5), lens


@pytest.mark.gpu
@pytest.mark.parametrize("case", SCAN)
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("ragged,full", [(False, True), (True, True), (True, False), (False, False)])
def test_scan(case, dtype, ragged, full):
    """Forward and gradients; full: every optional input, softplus, strided
    inputs; otherwise the bare recurrence with positive step sizes."""
    s, dy, state, dfinal, lens = scan_inputs(case, dtype, ragged)
    if full:
        for k in ("u", "delta", "z"):
            s[k] = wide(s[k])
    else:
        s["D"] = s["z"] = s["delta_bias"] = None
        s["delta"] = s["delta"].abs() * 0.1
        state = dfinal = None
        if case[4] == 1:
            s["B"], s["C"] = s["B"][:, 0], s["C"][:, 0]
    final = torch.full((case[0], case[1], case[3]), float("nan"), device="cuda")
    y = swd.scan(**s, softplus=full, state=state, final_state=final, lengths=lens)
    (wy, by), (wf, bf), want = ref.scan(**s, softplus=full, state=state, lengths=lens, grad=(dy, dfinal))
    ref.check(y, wy, by, "y")
    ref.check(final, wf, bf, "final_state")
    got = swd.scan_backward(dy, **s, softplus=full, state=state, dfinal_state=dfinal, lengths=lens)
    for name, g in got.items():
        if not full and name in ("dD", "dz", "ddelta_bias", "dstate"):
            assert g is None
            continue
        value, bound = want[name]
        if name in ("dB", "dC") and g.dim() == 3:
            g = g[:, None]
        ref.check(g, value, bound, name)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["u", "delta", "A", "B", "C", "D", "z", "delta_bias", "state"])
def test_scan_gradients_against_differences(which):
    """<gradient, direction> against a central difference of the 64-bit form
    along a random direction (its own error is below 1e-6 of its terms)."""
    s, dy, state, dfinal, lens = scan_inputs((3, 6, 37, 16, 2), F32, False, seed=5)
    lens = torch.tensor([37, 20, 1], dtype=torch.int32, device="cuda")
    s["state"] = state
    got = swd.scan_backward(dy, **s, dfinal_state=dfinal, lengths=lens)["d" + which]
    direction = Draw(6)(*s[which].shape).double().cpu()

    def value(step):
        moved = {k: v.double().cpu() for k, v in s.items()}
        moved[which] = moved[which] + step * direction
        st = moved.pop("state")
        (y, _), (h, _) = ref.scan(**moved, softplus=True, state=st, lengths=lens)
        return float((y * dy.double().cpu()).sum() + (h * dfinal.double().cpu()).sum())

    eps = 1e-5
    want = (value(eps) - value(-eps)) / (2 * eps)
    terms = got.double().cpu() * direction
    assert abs(float(terms.sum()) - want) <= 2e-5 * float(terms.abs().sum()) + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["x", "weight", "bias", "state"])
def test_short_conv_gradients_against_differences(which):
    x, dy, w, b, st, df, _ = conv_inputs((3, 5, 21, 4), F32, False, seed=7)
    lens = torch.tensor([21, 2, 0], dtype=torch.int32, device="cuda")
    s = dict(x=x, weight=w, bias=b, state=st)
    grads = swd.short_conv_backward(dy, x, w, b, state=st, dfinal_state=df, lengths=lens)
    got = dict(zip(("x", "weight", "bias", "state"), grads))[which]
    direction = Draw(8)(*s[which].shape).double().cpu()

    def value(step):
        m = {k: v.double().cpu() for k, v in s.items()}
        m[which] = m[which] + step * direction
        (y, _), (f, _), _ = ref.conv(m["x"], m["weight"], m["bias"], True, m["state"], lens)
        return float((y * dy.double().cpu()).sum() + (f * df.double().cpu()).sum())

    want = (value(1e-5) - value(-1e-5)) / 2e-5
    terms = got.double().cpu() * direction
    assert abs(float(terms.sum()) - want) <= 2e-5 * float(terms.abs().sum()) + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("N,ch,S,G", [(1, 1, 1, 1), (5, 33, 16, 1), (3, 40, 8, 2), (2, 6, 64, 3), (4, 7, 5, 1),
                                      (33, 256, 16, 1)])
def test_scan_step(dtype, N, ch, S, G):
    """One token per request, slots in another order, one outside the pool."""
    s, _, _, _, _ = scan_inputs((N, ch, 1, S, G), dtype, False, seed=3)
    d = Draw(4)
    pool = d(N + 2, ch, S)
    slots = torch.arange(N, dtype=torch.int32).flip(0) + 1
    if N > 2:
        slots[1], slots[2] = -7, N + 2
    before = pool.clone()
    one = {k: v[..., 0].contiguous() if k in ("u", "delta", "B", "C", "z") else v for k, v in s.items()}
    y = swd.scan_step(pool, **one, slots=slots.cuda())
    touched = set()
    for n, k in enumerate(slots.tolist()):
        if not 0 <= k < N + 2:
            assert not y[n].any()
            continue
        at = {k2: v[n:n + 1] if k2 in ("u", "delta", "B", "C", "z") else v for k2, v in s.items()}
        (wy, by), (wf, bf) = ref.scan(**at, softplus=True, state=before[k:k + 1], lengths=None)
        ref.check(y[n][None, :, None], wy, by, "y")
        ref.check(pool[k:k + 1], wf, bf, "state")
        touched.add(k)
    for k in range(N + 2):
        if k not in touched:
            assert torch.equal(pool[k], before[k])


@pytest.mark.gpu
def test_scan_extreme_step_sizes():
    """Step sizes far outside softplus's bend on both sides: the decay vanishes
    or is one, nothing overflows."""
    N, ch, L, S = 1, 4, 40, 16
    s, dy, _, _, _ = scan_inputs((N, ch, L, S, 1), F32, False, seed=9)
    s["delta_bias"] = torch.tensor([-80.0, -20.0, 30.0, 90.0], device="cuda")
    s["delta"] = s["delta"] * 0
    y = swd.scan(**s)
    (wy, by), _, want = ref.scan(**s, softplus=True, state=None, lengths=None, grad=(dy, None))
    ref.check(y, wy, by, "y")
    for name, g in swd.scan_backward(dy, **s).items():
        if g is not None:
            ref.check(g, *want[name], name)


@pytest.mark.gpu
def test_scan_repeats_bit_for_bit():
    s, dy, state, dfinal, lens = scan_inputs((2, 130, 300, 16, 1), BF16, False, seed=10)
    a = swd.scan_backward(dy, **s, state=state, dfinal_state=dfinal)
    b = swd.scan_backward(dy, **s, state=state, dfinal_state=dfinal)
    assert torch.equal(swd.scan(**s, state=state), swd.scan(**s, state=state))
    for k in a:
        assert torch.equal(a[k], b[k]), k


# ------------------------------------------------------------------ adapters

ADAPTER = [  # N, P, C, M, R, adapters
    (1, 1, 1, 1, 1, 1), (5, 1, 64, 48, 16, 3), (7, 1, 257, 129, 31, 4), (3, 2, 40, 24, 8, 2),
    (4, 7, 70, 33, 4, 3), (3, 33, 96, 65, 16, 2), (2, 64, 128, 128, 32, 2), (3, 130, 100, 72, 64, 2),
    (9, 16, 512, 40, 13, 5), (130, 1, 128, 64, 16, 9), (2, 784, 40, 48, 8, 2), (1, 96, 1000, 200, 33, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ADAPTER)
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("strided", [False, True])
def test_adapter_add(case, dtype, strided):
    N, P, C, M, R, K = case
    d = Draw(11)
    x = d(N, C, P, dtype=dtype)
    y = d(N, M, P, dtype=dtype)
    a, b = d(K, R, C, dtype=dtype, scale=C ** -0.5), d(K, M, R, dtype=dtype, scale=R ** -0.5)
    index = torch.tensor([(3 * n) % (K + 2) - 1 for n in range(N)], dtype=torch.int32)  # -1 and K: none
    scale = d(K).abs() + 0.5 if strided else None
    if strided:
        x = wide(x)
    elif P == 1:
        x, y = x[..., 0].contiguous(), y[..., 0].contiguous()
    before = y.clone()
    out = swd.adapter_add(y, x, a, b, index.cuda(), scale=scale)
    ref.check(out, *ref.adapter(y, x, a, b, index, scale), "out")
    assert torch.equal(y, before)
    assert swd.adapter_add(y, x, a, b, index.cuda(), scale=scale, out=y) is y
    assert torch.equal(y, out)
    for n, i in enumerate(index.tolist()):
        if not 0 <= i < K:
            assert torch.equal(out[n], before[n])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("P", [1, 40])
def test_adapter_add_is_exact_on_whole_numbers(dtype, P):
    """Small whole numbers: every product and sum is exact, whatever the order."""
    g = torch.Generator().manual_seed(12)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(dtype).cuda()  # noqa: E731
    N, C, M, R, K = 4, 24, 20, 4, 3
    x, y, a, b = ints(N, C, P), ints(N, M, P), ints(K, R, C), ints(K, M, R)
    a[:, :, 4:] = 0  # sums stay below 2^8, which bfloat16 holds
    index = torch.tensor([0, 2, -1, 1], dtype=torch.int32)
    out = swd.adapter_add(y, x, a, b, index.cuda())
    want, _ = ref.adapter(y, x, a, b, index, None)
    assert float(want.abs().max()) <= 256
    assert torch.equal(out.cpu().double(), want)


@pytest.mark.gpu
def test_adapter_values_of_others_stay_out():
    """NaN and infinities of one request, or of an adapter that none uses, do
    not reach another request."""
    d = Draw(13)
    for P in (1, 24):
        x, y = d(4, 32, P, dtype=BF16), d(4, 16, P, dtype=BF16)
        a, b = d(3, 8, 32, dtype=BF16), d(3, 16, 8, dtype=BF16)
        x[1], a[2], b[2] = float("nan"), float("inf"), float("nan")
        index = torch.tensor([0, 1, -1, 0], dtype=torch.int32)
        out = swd.adapter_add(y, x, a, b, index.cuda())
        keep = [0, 2, 3]
        want, bound = ref.adapter(y[keep], x[keep], a[:2], b[:2], index[keep], None)
        ref.check(out[keep], want, bound, "out")
        assert torch.isnan(out[1]).all()


# ------------------------------------------------------------------ streams, graphs, offsets


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_on_another_stream(raw):
    """Each call enqueued on a stream of its own, inputs made there, memory
    given back to the allocator while the stream is still busy."""
    d = Draw(14)
    stream = torch.cuda.Stream()
    sx = stream.cuda_stream if raw else stream
    x, w = d(2, 64, 4096), d(64, 4)
    s, dy, state, dfinal, _ = scan_inputs((2, 64, 512, 16, 1), F32, False)
    y0, xa, a, b = d(2, 32, 512), d(2, 64, 512), d(2, 8, 64), d(2, 32, 8)
    index = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    want = (swd.short_conv(x, w), swd.scan(**s), swd.adapter_add(y0, xa, a, b, index))
    grads = swd.scan_backward(dy, **s)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            busy = busy @ busy
            busy = busy / busy.norm()
    got = (swd.short_conv(x, w, stream=sx), swd.scan(**s, stream=sx),
           swd.adapter_add(y0, xa, a, b, index, stream=sx))
    more = swd.scan_backward(dy, **s, stream=sx)
    del busy
    junk = [torch.full((2, 64, 4096), float("nan"), device="cuda") for _ in range(8)]  # reuse what was freed
    torch.cuda.synchronize()
    del junk
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    for k in grads:
        assert grads[k] is None and more[k] is None or torch.equal(grads[k], more[k])


@pytest.mark.gpu
def test_captured_into_a_graph():
    """Tokens of a whole block captured once and replayed on new inputs."""
    d = Draw(15)
    N, C, S, K = 4, 96, 16, 4
    x, w, b = d(N, C), d(C, K), d(C)
    s, _, _, _, _ = scan_inputs((N, C, 1, S, 1), F32, False)
    one = {k: v[..., 0].contiguous() if k in ("u", "delta", "B", "C", "z") else v for k, v in s.items()}
    conv_state, scan_state = d(N, C, K - 1), d(N, C, S)
    a, bb, index = d(2, 8, C), d(2, C, 8), torch.tensor([1, -1, 0, 1], dtype=torch.int32, device="cuda")

    def token(cs, ss):
        one["u"] = swd.short_conv_step(x, cs, w, b)
        y = swd.scan_step(ss, **one)
        return swd.adapter_add(y, x, a, bb, index)

    warm = token(conv_state.clone(), scan_state.clone())
    del warm
    c1, s1, c2, s2 = conv_state.clone(), scan_state.clone(), conv_state.clone(), scan_state.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(c1, s1)
    for step in range(3):
        x.copy_(d(N, C))
        graph.replay()
        want = token(c2, s2)
        assert torch.equal(out, want) and torch.equal(c1, c2) and torch.equal(s1, s2)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows more than 2^32 elements apart, and a state number whose offset does
    not fit 32 bits."""
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 40 GB of device memory")
    apart = (1 << 32) + 64
    d = Draw(16)
    L, C, S = 100, 3, 16
    big = torch.empty(apart + C * 128, dtype=BF16, device="cuda")
    x = big.as_strided((2, C, L), (apart, 128, 1))
    x.copy_(d(2, C, L, dtype=BF16))
    w = d(C, 4)
    assert torch.equal(swd.short_conv(x, w), swd.short_conv(x.contiguous(), w))
    s, dy, _, _, _ = scan_inputs((2, C, L, S, 1), BF16, False)
    s["u"] = x
    near = dict(s, u=x.contiguous())
    assert torch.equal(swd.scan(**s), swd.scan(**near))
    g, h = swd.scan_backward(dy, **s), swd.scan_backward(dy, **near)
    assert all(torch.equal(g[k], h[k]) for k in g if g[k] is not None)
    y, a, b = d(2, 5, L, dtype=BF16), d(1, 8, C, dtype=BF16), d(1, 5, 8, dtype=BF16)
    index = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert torch.equal(swd.adapter_add(y, x, a, b, index), swd.adapter_add(y, x.contiguous(), a, b, index))
    del big, x, s, near
    C = 4096
    slots = (1 << 31) // (C * S) + 8
    pool = torch.zeros(slots, C, S, device="cuda")
    s, _, _, _, _ = scan_inputs((1, C, 1, S, 1), F32, False)
    one = {k: v[..., 0].contiguous() if k in ("u", "delta", "B", "C", "z") else v for k, v in s.items()}
    small = d(1, C, S)
    pool[slots - 1] = small[0]
    y1 = swd.scan_step(pool, **one, slots=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    y2 = swd.scan_step(small, **one)
    assert torch.equal(y1, y2) and torch.equal(pool[slots - 1], small[0])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(0, 5, 7), (2, 0, 7), (2, 5, 0)])
def test_empty_sizes(shape):
    """No sequence, no channel or no position: states pass through, weights'
    gradients are zero."""
    N, C, L = shape
    d = Draw(17)
    x, w, b, st = d(N, C, L), d(C, 4), d(C), d(N, C, 3)
    final = torch.empty_like(st)
    assert swd.short_conv(x, w, b, state=st, final_state=final).shape == shape
    assert torch.equal(final, st)
    dx, dw, db, ds = swd.short_conv_backward(x, x, w, b, state=st, dfinal_state=st)
    assert not dw.any() and not db.any() and torch.equal(ds, st)
    S = 16
    st, B = d(N, C, S), d(N, 1, S, L)
    A = -d(C, S).abs()
    final = torch.empty_like(st)
    assert swd.scan(x, x, A, B, B, b, x, b, state=st, final_state=final).shape == shape
    assert torch.equal(final, st)
    g = swd.scan_backward(x, x, x, A, B, B, b, x, b, state=st, dfinal_state=st)
    assert not g["dA"].any() and not g["dD"].any() and torch.equal(g["dstate"], st)
    y = d(N, 6, L)
    index = torch.zeros(N, dtype=torch.int32, device="cuda")
    out = swd.adapter_add(y, x, d(1, 4, C), d(1, 6, 4), index)
    if C == 0:
        assert torch.equal(out, y)


# ------------------------------------------------------------------ refusals

GOOD = 0x10000  # an aligned address that is never read: every call here is refused


def conv_args(**change):
    a = ShortConvArgs(2, 3, 5, 4, 0, 1)
    a.x_stride_n, a.x_stride_c, a.dy_stride_n, a.dy_stride_c = 15, 5, 15, 5
    for i, n in enumerate("x weight bias state y final_state pool dy dfinal_state dx dstate dweight dbias workspace".split()):
        setattr(a, n, GOOD + 0x10000 * i)
    a.workspace_bytes = 1 << 16
    for k, v in change.items():
        setattr(a, k, v)
    return a


def scan_args(**change):
    a = ScanArgs(2, 4, 5, 16, 2, 0, 1)
    for n in ("u", "delta", "z", "dy"):
        setattr(a, n + "_stride_n", 20)
        setattr(a, n + "_stride_c", 5)
    for n in "bc":
        for k, v in (("n", 160), ("g", 80), ("s", 5)):
            setattr(a, f"{n}_stride_{k}", v)
    names = ("u delta z B C A D delta_bias state y final_state pool dy dfinal_state du ddelta dz dB dC dA dD "
             "ddelta_bias dstate workspace").split()
    for i, n in enumerate(names):
        setattr(a, n, GOOD + 0x10000 * i)
    a.workspace_bytes = 1 << 30
    for k, v in change.items():
        setattr(a, k, v)
    return a


def adapter_args(**change):
    a = AdapterArgs(2, 5, 4, 6, 8, 3, 0)
    a.x_stride_n, a.x_stride_c = 20, 5
    for i, n in enumerate("x a b index scale y out".split()):
        setattr(a, n, GOOD + 0x10000 * i)
    for k, v in change.items():
        setattr(a, k, v)
    return a


BAD, BEYOND = _lib.SPCONV_ERR_INVALID_ARG, _lib.SPCONV_ERR_UNSUPPORTED
REFUSED = [
    ("spconv_short_conv", conv_args, [(dict(N=-1), BAD), (dict(C=-1), BAD), (dict(L=-1), BAD), (dict(K=0), BAD),
     (dict(K=5), BEYOND), (dict(dtype=3), BAD), (dict(dtype=-1), BAD), (dict(silu=2), BAD), (dict(x=None), BAD),
     (dict(weight=None), BAD), (dict(y=None), BAD), (dict(x=GOOD + 2), BAD), (dict(dtype=1, x=GOOD + 1), BAD),
     (dict(y=GOOD), BAD), (dict(final_state=GOOD + 4), BAD), (dict(x_stride_n=-1), BAD), (dict(weight=GOOD + 2), BAD),
     (dict(L=0x7fffffff), BEYOND)]),
    ("spconv_short_conv_backward", conv_args, [(dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dweight=None), BAD),
     (dict(dx=GOOD), BAD), (dict(K=9), BEYOND), (dict(dy_stride_c=-4), BAD), (dict(dstate=GOOD + 8), BAD),
     (dict(N=4096, L=4096, workspace_bytes=0), BAD), (dict(N=4096, L=4096, workspace=None), BAD)]),
    ("spconv_short_conv_step", conv_args, [(dict(num_slots=1), BAD), (dict(num_slots=2, x_stride_c=5), BAD),
     (dict(num_slots=2, x_stride_c=1, pool=None), BAD), (dict(num_slots=2, x_stride_c=1, x=None), BAD),
     (dict(num_slots=-1, x_stride_c=1), BAD), (dict(num_slots=2, x_stride_c=1, K=6), BEYOND),
     (dict(N=70000, num_slots=70000, x_stride_c=1), BEYOND)]),
    ("spconv_scan", scan_args, [(dict(N=-1), BAD), (dict(S=0), BAD), (dict(S=65), BEYOND), (dict(groups=0), BAD),
     (dict(groups=3), BAD), (dict(dtype=7), BAD), (dict(softplus=2), BAD), (dict(u=None), BAD), (dict(A=None), BAD),
     (dict(B=None), BAD), (dict(y=None), BAD), (dict(y=GOOD), BAD), (dict(u=GOOD + 2), BAD), (dict(A=GOOD + 1), BAD),
     (dict(b_stride_s=-5), BAD), (dict(N=70000), BEYOND), (dict(L=0x7fffffff), BEYOND),
     (dict(final_state=GOOD + 16), BAD)]),
    ("spconv_scan_backward", scan_args, [(dict(dy=None), BAD), (dict(dz=None), BAD), (dict(z=None), BAD),
     (dict(dA=None), BAD), (dict(du=GOOD), BAD), (dict(workspace=None), BAD), (dict(workspace_bytes=16), BAD),
     (dict(workspace=GOOD + 4), BAD), (dict(S=65), BEYOND), (dict(N=70000, workspace_bytes=1 << 40), BEYOND)]),
    ("spconv_scan_step", scan_args, [(dict(num_slots=1), BAD), (dict(num_slots=2), BAD),
     (dict(num_slots=2, u_stride_c=1, delta_stride_c=1, z_stride_c=1, b_stride_s=1, c_stride_s=1, pool=None), BAD),
     (dict(num_slots=2, u_stride_c=1, delta_stride_c=1, z_stride_c=1, b_stride_s=1, c_stride_s=1, y=GOOD), BAD),
     (dict(N=70000), BEYOND)]),
    ("spconv_adapter_add", adapter_args, [(dict(N=-1), BAD), (dict(R=0), BAD), (dict(R=65), BEYOND),
     (dict(P=1 << 27), BEYOND), (dict(M=1 << 27), BEYOND), (dict(C=1 << 27), BEYOND),
     (dict(adapters=-1), BAD), (dict(dtype=3), BAD), (dict(x=None), BAD), (dict(a=None), BAD), (dict(b=None), BAD),
     (dict(index=None), BAD), (dict(y=None), BAD), (dict(out=None), BAD), (dict(out=GOOD), BAD),
     (dict(out=GOOD + 0x50000 + 4), BAD), (dict(x=GOOD + 2), BAD), (dict(x_stride_n=-1), BAD),
     (dict(index=GOOD + 2), BAD)]),
]


@pytest.mark.parametrize("name,make,change,status", [(n, m, c, s) for n, m, cs in REFUSED for c, s in cs],
                         ids=[f"{n[7:]}-{'-'.join(c)}" for n, _, cs in REFUSED for c, _ in cs])
def test_refused_at_the_c_entry(name, make, change, status):
    """Refused before anything is enqueued: no GPU is needed to be told so."""
    assert getattr(_lib.lib(), name)(ctypes.byref(make(**change)), None) == status


@pytest.mark.parametrize("name", [n for n, _, _ in REFUSED])
def test_null_arguments_refused(name):
    assert getattr(_lib.lib(), name)(None, None) == BAD


def test_argument_structures_match_the_header():
    """The sizes that the header's structures have for a C compiler."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "s.c"), "w") as f:
            f.write('#include <stdio.h>\n#include <stddef.h>\n#include "spconv.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu",'
                    "sizeof(spconv_short_conv_args),sizeof(spconv_scan_args),sizeof(spconv_adapter_args),"
                    "offsetof(spconv_short_conv_args,dweight),offsetof(spconv_scan_args,dstate),"
                    "offsetof(spconv_adapter_args,out));return 0;}\n")
        exe = os.path.join(d, "s")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), os.path.join(d, "s.c"), "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    want = [ctypes.sizeof(ShortConvArgs), ctypes.sizeof(ScanArgs), ctypes.sizeof(AdapterArgs),
            ShortConvArgs.dweight.offset, ScanArgs.dstate.offset, AdapterArgs.out.offset]
    assert [int(v) for v in out.split()] == want


@pytest.mark.gpu
def test_refused_at_the_python_entry():
    d = Draw(18)
    x, w, b = d(2, 3, 8), d(3, 4), d(3)
    A, B = -d(3, 16).abs(), d(2, 16, 8)
    bad = [
        lambda: swd.short_conv(x.cpu(), w), lambda: swd.short_conv(x.double(), w),
        lambda: swd.short_conv(x, w.half()), lambda: swd.short_conv(x, w[:2]),
        lambda: swd.short_conv(x.transpose(1, 2), w), lambda: swd.short_conv(x, d(3, 5)),
        lambda: swd.short_conv(x, w, b[:2]), lambda: swd.short_conv(x, w, state=d(2, 3, 4)),
        lambda: swd.short_conv(x, w, lengths=torch.ones(2, device="cuda")),
        lambda: swd.short_conv(x, w, out=x), lambda: swd.short_conv(x[0], w),
        lambda: swd.short_conv_backward(x.half(), x, w),
        lambda: swd.short_conv_step(x[..., 0], d(2, 3, 3), w),
        lambda: swd.short_conv_step(d(2, 3), d(4, 3, 3), w),
        lambda: swd.scan(x, x.half(), A, B, B), lambda: swd.scan(x, x, A[:, :8], B, B),
        lambda: swd.scan(x, x, A, B, B[:1]), lambda: swd.scan(x, x, A, d(2, 2, 16, 8), d(2, 2, 16, 8)),
        lambda: swd.scan(x, x, A, B, None), lambda: swd.scan(x, x, A, B, B, final_state=d(2, 3, 8)),
        lambda: swd.scan(x, x, -d(3, 65).abs(), d(2, 65, 8), d(2, 65, 8)),
        lambda: swd.scan_backward(x[:1], x, x, A, B, B),
        lambda: swd.scan_step(d(3, 3, 16), d(2, 3), d(2, 3), A, d(2, 16), d(2, 16)),
        lambda: swd.adapter_add(d(2, 5, 8), x, d(1, 65, 3), d(1, 5, 65), torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: swd.adapter_add(d(2, 5, 8), x, d(1, 4, 3), d(1, 5, 4), torch.zeros(2, device="cuda")),
        lambda: swd.adapter_add(d(2, 5, 7), x, d(1, 4, 3), d(1, 5, 4), torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: swd.adapter_add(None, x, d(1, 4, 3), d(1, 5, 4), torch.zeros(2, dtype=torch.int32, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(swd.SpconvError):
            call()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("L", [40, 300, 1030])
def test_positions_behind_the_end_leave_no_trace(dtype, L):
    """A padded sequence gives the bits of the sequence alone, in outputs, states
    and gradients, wherever its end lies in a tile or a chunk."""
    s, dy, state, dfinal, _ = scan_inputs((1, 40, L, 16, 1), dtype, False, seed=20)
    for k in (1, 7, 32, 33, L // 2 + 3, L - 1):
        lens = torch.tensor([k], dtype=torch.int32, device="cuda")
        cut = {n: v[..., :k].contiguous() if n in ("u", "delta", "B", "C", "z") else v for n, v in s.items()}
        a, b = torch.empty_like(state), torch.empty_like(state)
        y = swd.scan(**s, state=state, final_state=a, lengths=lens)
        assert not y[..., k:].any()
        # (cut into other chunks the states are joined at other places)
        swd.scan(**cut, state=state, final_state=b)
        tight = 2.0 ** -19 if L >= 256 else 0.0
        assert float((a - b).abs().max()) <= tight * float(b.abs().max())
        g = swd.scan_backward(dy, **s, state=state, dfinal_state=dfinal, lengths=lens)
        for n in ("du", "ddelta", "dB", "dC", "dz"):
            assert not g[n][..., k:].any(), n
