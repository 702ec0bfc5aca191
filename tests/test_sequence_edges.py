"""The sequence operators where values, sizes or streams are out of the ordinary:
sums of very different size, infinities, memory of another stream, sizes near
2^31, outputs that overlap what a call reads."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import sequence_reference as ref  # noqa: E402
import sparse_weight_direct_gb300 as swd  # noqa: E402
import test_sequence as base  # noqa: E402
from sparse_weight_direct_gb300 import _lib  # noqa: E402
from test_sequence import BF16, F32, GOOD, TYPE_IDS, TYPES, Draw, adapter_args, conv_args, scan_args  # noqa: E402

# ------------------------------------------------------------------ adapters: sums of very different size


def adapter_bound(y, x, a, b, index):
    """ref.adapter with the inner sums held in 32 bits for every type: sums of C
    and R terms within n 2^-24 of their absolute terms, products within E."""
    want, _ = ref.adapter(y, x, a, b, index, None)
    bound = 2.0 ** -23 * ref.f64(y).abs()
    K, R, C = a.shape
    for n, i in enumerate(index.tolist()):
        terms = ref.f64(b[i]).abs() @ (ref.f64(a[i]).abs() @ ref.f64(x[n]).abs())
        bound[n] += ((C + R) * 2.0 ** -24 + ref.E) * terms
    return want, bound


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 2, 40, 64])
@pytest.mark.parametrize("R", [8, 32, 63])
@pytest.mark.parametrize("apart", [10, 15, 20])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
def test_adapter_small_sums_beside_large_ones(dtype, apart, R, P):
    """Adapters joined along the rank: half of a's rows are 2^apart larger, and
    half of the outputs read the other half only.  Those outputs are as good as
    without the large rows."""
    d = Draw(31)
    N, C, M = 2, 48, 40
    x = d(N, C, P, dtype=dtype)
    a, b = d(1, R, C, scale=C ** -0.5), d(1, M, R)
    a[:, : R // 2] *= 2.0 ** (apart / 2)
    a[:, R // 2:] *= 2.0 ** (-apart / 2)
    b[:, M // 2:, : R // 2] = 0
    b[:, : M // 2, R // 2:] = 0
    a, b, y = a.to(dtype), b.to(dtype), torch.zeros(N, M, P, dtype=dtype, device="cuda")
    index = torch.zeros(N, dtype=torch.int32)
    out = swd.adapter_add(y, x, a, b, index.cuda())
    ref.check(out, *adapter_bound(y, x, a, b, index), "out")


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 2, 40, 64])
@pytest.mark.parametrize("R", [16, 30, 64])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
def test_adapter_differences_of_large_whole_sums(dtype, R, P):
    """b takes the difference of two rows of v, whole numbers of up to 20 bits
    that are nearly alike: every product and sum is exact in 32 bits, so v has
    to keep all of its bits between the products."""
    g = torch.Generator().manual_seed(32)
    ints = lambda most, *s: torch.randint(-most, most + 1, s, generator=g).to(dtype).cuda()  # noqa: E731
    N, C, M = 2, 32, 24
    x, a = ints(200, N, C, P), ints(200, 1, R, C)
    x[:, 0], a[:, :, 0] = ints(9, N, P), ints(9, 1, R)
    a[:, R // 2:] = a[:, : R // 2]
    a[:, R // 2:, 0] += ints(9, 1, R // 2)
    b = torch.zeros(1, M, R, dtype=dtype, device="cuda")
    for m in range(M):
        b[0, m, m % (R // 2)], b[0, m, R // 2 + m % (R // 2)] = 1, -1
    y = ints(20, N, M, P)
    index = torch.zeros(N, dtype=torch.int32)
    want, _ = ref.adapter(y, x, a, b, index, None)
    v = ref.f64(a[0]) @ ref.f64(x[0])
    assert float(v.abs().max()) >= 1 << 16 and float(want.abs().max()) <= 256
    out = swd.adapter_add(y, x, a, b, index.cuda())
    assert torch.equal(out.cpu().double(), want)


# ------------------------------------------------------------------ adapters: infinities


def same_values(got, want, bound, open_, what):
    """NaN where `want` is, infinities alike, the rest within the bound; nothing
    is asked where it is open."""
    got, want, bound = (torch.where(open_.to(t.device), torch.zeros_like(t), t) for t in (got, want, bound))
    g, fine = ref.f64(got), torch.isfinite(want)
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what
    assert torch.equal(g[torch.isinf(want)], want[torch.isinf(want)]), what
    zero = torch.zeros_like(want)
    ref.check(torch.where(fine.to(got.device), got, torch.zeros_like(got)), torch.where(fine, want, zero),
              torch.where(fine, bound, zero), what)


INF = float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 2, 40, 64])
@pytest.mark.parametrize("R", [1, 8, 33])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("where", ["x", "a", "b", "x and a", "x largest", "v overflows", "scale"])
def test_adapter_infinities(dtype, R, P, where):
    """One infinite input reaches the outputs that its products reach with the
    sign that the definition gives it, whatever the other factor's bits, and no
    other position, row or request.  Rows of one term: no other term hides it."""
    d = Draw(33)
    N, C, M, K = 3, 20, 24, 2
    most = torch.finfo(dtype).max
    x, y, scale = d(N, C, P, dtype=dtype), d(N, M, P, dtype=dtype), torch.ones(K, device="cuda")
    a, b = d(K, R, C, dtype=dtype), d(K, M, R, dtype=dtype)
    # factors that meet the infinity: whole in few bits, and not
    some = torch.tensor([0.5, 0.3, -0.3, 0.001, -2.0, 1.0, 3.0, -0.7], device="cuda")
    a[:, :, 3], b[:, :, 0] = some[torch.arange(R) % 8].to(dtype), some[torch.arange(M) % 8].to(dtype)
    x[:, 3, :] = some[(torch.arange(P) + 2) % 8].to(dtype)
    if "x" in where.split():
        x[0, 3, P // 2] = most if "largest" in where else -INF
    if "a" in where.split():
        a[0, 0, 3] = INF
    if where == "b":
        b[0, 5, 0] = -INF
        b[0, 7, R - 1] = INF
    if where == "v overflows":  # (of 32-bit sums: not from half precision)
        x[0, 3, P // 2], a[0, 0, 3] = most, most
    if where == "scale":
        scale[0] = INF
    index = torch.tensor([0, 1, -1], dtype=torch.int32)
    out = swd.adapter_add(y, x, a, b, index.cuda(), scale=scale)
    # the definition in 32 bits (an overflow is one), then in 64 for the finite values
    # (by plain sums: a library's product may split its terms)
    v = (a.float()[[0, 1, 0], :, :, None] * x.float()[:, None]).sum(2)
    far, size = torch.zeros(N, M, P, device="cuda"), torch.zeros(N, M, P, device="cuda")
    for r in range(R):
        br, vr = b.float()[[0, 1, 0], :, r, None], v[:, None, r]
        far, size = far + br * vr, size + torch.where(torch.isfinite(br) & torch.isfinite(vr), (br * vr).abs(), 0.0)
    far = y.float() + scale[[0, 1, 0], None, None] * far
    want, bound = ref.adapter(y, x, a, b, index, scale)
    far = ref.f64(far)
    far[2] = ref.f64(y)[2]
    want = torch.where(torch.isfinite(far), want, far)
    # a finite result half a unit beyond the type's largest rounds to an infinity
    edge = most * (1 + torch.finfo(dtype).eps / 4 / (1 - torch.finfo(dtype).eps / 2))
    bound = torch.where(torch.isfinite(bound), bound, torch.zeros_like(bound))
    # open: what finite terms add up to where their sum may overflow in one order
    # and not in another, and the side of that edge that a sum ends on
    open_ = (want.abs() - edge).abs() <= bound
    if R > 1:
        open_ |= torch.isinf(ref.f64(size))
    open_[2] = False
    want = torch.where(want.abs() >= edge, torch.sign(want) * INF, want)
    same_values(out, want, bound, open_, where)
    assert R > 1 or where not in ("x", "b") or torch.isinf(want).any()


# ------------------------------------------------------------------ another stream


def calls_on_streams():
    """name -> call(stream), its inputs made ready."""
    d = Draw(41)
    N, C, L, S = 2, 48, 512, 16
    x, dy, w, b = d(N, C, L), d(N, C, L), d(C, 4), d(C)
    A, B, Cm = -d(C, S).abs(), d(N, S, L), d(N, S, L)
    y, a, bb, index = d(N, 40, L), d(2, 8, C), d(2, 40, 8), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    one = x[..., 0].contiguous()
    pool, states = d(N, C, 3), d(N, C, S)
    step = (one, one * 0.1, A, B[..., 0].contiguous(), Cm[..., 0].contiguous())
    return {
        "short_conv": lambda s: swd.short_conv(x, w, b, stream=s),
        "short_conv_backward": lambda s: swd.short_conv_backward(dy, x, w, b, stream=s),
        "short_conv_step": lambda s: swd.short_conv_step(one, pool.clone() if s is None else pool, w, b, stream=s),
        "scan": lambda s: swd.scan(x, x * 0.1 if s is None else x, A, B, Cm, stream=s),
        "scan_backward": lambda s: swd.scan_backward(dy, x, x, A, B, Cm, stream=s),
        "scan_step": lambda s: swd.scan_step(states.clone() if s is None else states, *step, stream=s),
        "adapter_add": lambda s: swd.adapter_add(y, x, a, bb, index, stream=s),
    }


def tensors_of(result):
    if isinstance(result, dict):
        result = tuple(result.values())
    return [t for t in (result if isinstance(result, tuple) else (result,)) if t is not None]


def busy(steps=20):
    """Some tens of milliseconds of work on the current stream."""
    m = torch.full((4096, 4096), 1.0 / 4096, device="cuda")
    out = torch.empty_like(m)

    def go():
        for _ in range(steps):
            torch.mm(m, m, out=out)
    go()
    torch.cuda.synchronize()
    return go


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", ["short_conv", "short_conv_backward", "short_conv_step", "scan", "scan_backward",
                                  "scan_step", "adapter_add"])
def test_memory_that_the_current_stream_still_reads(name, raw, monkeypatch):
    """Tensors of the sizes that a call allocates are copied out at the end of a
    long queue on the current stream and given back; a call on an independent
    stream, which waits for nothing, leaves them alone."""
    from sparse_weight_direct_gb300 import sequence
    call = calls_on_streams()[name]
    call(None)  # (torch is loaded by the first call)
    sizes = []
    with monkeypatch.context() as m:
        for f in ("_empty", "_empty_like"):
            plain = getattr(sequence, f)

            def spy(*args, _plain=plain, **more):
                t = _plain(*args, **more)
                sizes.append(t.numel() * t.element_size())
                return t
            m.setattr(sequence, f, spy)
        first = call(None)
    assert sizes
    work = busy()
    side = torch.cuda.Stream()
    del first
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    victims = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    kept = [torch.zeros_like(v) for v in victims]
    torch.cuda.synchronize()
    work()
    for k, v in zip(kept, victims):
        k.copy_(v)
    end = torch.cuda.Event()
    end.record()
    del victims, v
    got = tensors_of(call(side.cuda_stream if raw else side))
    early = not end.query()
    torch.cuda.synchronize()
    assert early, "the queue was too short to show anything"
    for k in kept:
        assert bool((k == 7).all())
    assert got


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["short_conv", "short_conv_backward", "scan", "scan_backward", "adapter_add"])
def test_outputs_of_another_stream_given_back_while_read(name):
    """Outputs that the current stream still reads when they are given back are not
    overwritten by the next call on the stream that made them."""
    call = calls_on_streams()[name]
    work, side = busy(), torch.cuda.Stream()
    first = tensors_of(call(side))
    torch.cuda.synchronize()
    want = [t.clone() for t in first]
    kept = [torch.empty_like(t) for t in first]
    torch.cuda.synchronize()
    work()
    for k, t in zip(kept, first):
        k.copy_(t)
    del first, t
    with torch.cuda.stream(side):
        junk = [torch.full_like(k, float("nan")) for k in kept]
    again = tensors_of(call(side))
    torch.cuda.synchronize()
    del junk, again
    for k, w in zip(kept, want):
        assert torch.equal(k, w)


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_forward_leaves_memory_that_the_current_stream_still_reads(raw):
    """The convolution's output, where the call allocates it."""
    import workloads
    L = workloads.LAYERS["tiny"]
    w = swd.pack(*workloads.make_weights(L), C=L.C, H=L.H, W=L.W, M=L.M, R=L.R, S=L.S, stride=L.stride, pad=L.pad)
    x = torch.from_numpy(workloads.make_input(L)).cuda()
    want = swd.forward(x, w)
    work, side = busy(), torch.cuda.Stream()
    torch.cuda.synchronize()
    victims = [torch.full_like(want, 7) for _ in range(2)]
    kept = [torch.zeros_like(want) for _ in victims]
    torch.cuda.synchronize()
    work()
    for k, v in zip(kept, victims):
        k.copy_(v)
    end = torch.cuda.Event()
    end.record()
    del victims, v
    got = swd.forward(x, w, stream=side.cuda_stream if raw else side)
    early = not end.query()
    torch.cuda.synchronize()
    assert early, "the queue was too short to show anything"
    for k in kept:
        assert bool((k == 7).all())
    assert torch.equal(got, want)
    w.close()


# ------------------------------------------------------------------ refusals at the C entry


def refused(name, args):
    return getattr(_lib.lib(), name)(ctypes.byref(args), None)


def test_conv_without_positions_needs_its_weight():
    """The kernel that writes the final state reads the weight: a call without one
    is refused, with or without positions."""
    assert refused("spconv_short_conv", conv_args(L=0, weight=None)) == _lib.SPCONV_ERR_INVALID_ARG
    assert refused("spconv_short_conv", conv_args(L=0, weight=None, final_state=None)) == _lib.SPCONV_ERR_INVALID_ARG


@pytest.mark.parametrize("name,make,change", [
    ("spconv_short_conv", conv_args, dict(N=0x7fffffff, C=1, L=1)),
    ("spconv_short_conv", conv_args, dict(N=0x7fff0001, C=1, L=1)),
    ("spconv_short_conv", conv_args, dict(N=1, C=0x7fffffff, L=1)),
    ("spconv_short_conv_backward", conv_args, dict(N=0x7fffffff, C=1, L=1)),
    ("spconv_short_conv_backward", conv_args, dict(N=1, C=0x7fffffff, L=1)),
    ("spconv_short_conv_step", conv_args, dict(N=1, C=0x7fffffff, num_slots=1, x_stride_c=1)),
    ("spconv_scan", scan_args, dict(N=1, channels=0x7fffffff, groups=1, L=1)),
    ("spconv_scan_backward", scan_args, dict(N=1, channels=0x7fffffff, groups=1, L=1)),
    ("spconv_scan_step", scan_args, dict(N=1, channels=0x7fffffff, groups=1, num_slots=1, u_stride_c=1,
                                         delta_stride_c=1, z_stride_c=1, b_stride_s=1, c_stride_s=1)),
])
def test_sizes_near_2_to_the_31_are_refused(name, make, change):
    """Counts of sequences and channels that a block's reach would take past 32 bits."""
    assert refused(name, make(**change)) == _lib.SPCONV_ERR_UNSUPPORTED


# ------------------------------------------------------------------ no channels


def test_gradients_of_no_channels_need_their_outputs():
    """dB and dC have elements without any channel: sums over none."""
    for change in (dict(dB=None), dict(dC=None), dict(dB=GOOD + 2)):
        assert refused("spconv_scan_backward", scan_args(channels=0, **change)) == _lib.SPCONV_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [None, 1, 3])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
def test_gradients_of_no_channels_are_zero(dtype, groups):
    N, L, S = 2, 7, 16
    x, A = torch.zeros(N, 0, L, dtype=dtype, device="cuda"), torch.zeros(0, S, device="cuda")
    B = torch.ones(*((N, S, L) if groups is None else (N, groups, S, L)), dtype=dtype, device="cuda")
    junk = [torch.full_like(B, float("nan")) for _ in range(4)]  # what the outputs' memory holds
    torch.cuda.synchronize()
    del junk
    g = swd.scan_backward(x, x, x, A, B, B)
    assert g["dB"].shape == B.shape and not g["dB"].any() and not g["dC"].any()


# ------------------------------------------------------------------ outputs over what a call reads

STEP = dict(num_slots=2, u_stride_c=1, delta_stride_c=1, z_stride_c=1, b_stride_s=1, c_stride_s=1)
READ_AND_WRITTEN = [
    ("spconv_short_conv", conv_args, {}, "y final_state", "x weight bias state lengths"),
    ("spconv_short_conv_backward", conv_args, {}, "dx dstate dweight dbias",
     "x weight bias state lengths dy dfinal_state"),
    ("spconv_short_conv_backward", conv_args, dict(N=4096, L=4096, workspace_bytes=1 << 30),
     "dx dstate dweight dbias workspace", "x weight bias state dy dfinal_state"),
    ("spconv_short_conv_step", conv_args, dict(num_slots=2, x_stride_c=1), "y pool", "x weight bias slots"),
    ("spconv_scan", scan_args, {}, "y final_state", "u delta z B C A D delta_bias state lengths"),
    ("spconv_scan", scan_args, dict(N=1, L=4096, workspace_bytes=1 << 30), "y final_state workspace",
     "u delta z B C A D delta_bias state"),
    ("spconv_scan_backward", scan_args, {},
     "du ddelta dz dB dC dA dD ddelta_bias dstate workspace",
     "u delta z B C A D delta_bias state lengths dy dfinal_state"),
    ("spconv_scan_step", scan_args, STEP, "y pool", "u delta z B C A D delta_bias slots"),
    ("spconv_adapter_add", adapter_args, {}, "out", "x a b index scale"),
]


@pytest.mark.parametrize("name,make,change,out,read", READ_AND_WRITTEN,
                         ids=[f"{n[7:]}-{i}" for i, (n, *_) in enumerate(READ_AND_WRITTEN)])
def test_outputs_over_inputs_are_refused(name, make, change, out, read):
    """Every output that lies over an input or over another output: all pointers
    a gigabyte apart but for the two."""
    fields = [f for f, t in make()._fields_ if t is ctypes.c_void_p]
    far = {f: (1 << 40) + (i << 34) for i, f in enumerate(fields)}
    given = {f: far[f] if f in (out + " " + read).split() else None for f in fields}
    if name == "spconv_adapter_add":
        given["y"] = far["y"]  # (out may be y itself)
    for o in out.split():
        for other in (out + " " + read).split():
            if o != other:
                args = make(**{**change, **given, o: far[other]})
                assert refused(name, args) == _lib.SPCONV_ERR_INVALID_ARG, (o, other)


# ------------------------------------------------------------------ refusals at the Python entry


@pytest.mark.gpu
def test_sizes_past_32_bits_are_refused():
    """Views of one element with 2^31 of them along a dimension, a pool of 2^31
    states, and flags that are none: SpconvError, and nothing is allocated."""
    many = 1 << 31
    one = torch.zeros(1, device="cuda")
    wide = lambda *shape: one.as_strided(shape, (0,) * len(shape))  # noqa: E731
    w, A = torch.zeros(1, 2, device="cuda"), torch.zeros(1, 1, device="cuda")
    bf, x = torch.zeros(1, 1, 1, dtype=BF16, device="cuda"), torch.zeros(1, 1, 1, device="cuda")
    pool = torch.empty(many, 1, 1, dtype=BF16, device="cuda")  # 4 GB
    index = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = [
        lambda: swd.short_conv(wide(many, 1, 1), w), lambda: swd.short_conv(wide(1, many, 1), w),
        lambda: swd.short_conv_backward(wide(many, 1, 1), wide(many, 1, 1), w),
        lambda: swd.short_conv_step(wide(many, 1), x, w),
        lambda: swd.short_conv_step(bf[..., 0], pool, w, slots=index),
        lambda: swd.scan(wide(many, 1, 1), wide(many, 1, 1), A, wide(many, 1, 1), wide(many, 1, 1)),
        lambda: swd.scan_backward(*[wide(many, 1, 1)] * 3, A, *[wide(many, 1, 1)] * 2),
        lambda: swd.scan_step(x, wide(many, 1), wide(many, 1), A, wide(many, 1), wide(many, 1)),
        lambda: swd.adapter_add(x, wide(1, many, 1), x, x, index),
        lambda: swd.short_conv(x, w, silu=1 << 40), lambda: swd.scan(x, x, A, x, x, softplus="no"),
    ]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    for i, call in enumerate(calls):
        with pytest.raises(swd.SpconvError):
            call()
            pytest.fail(f"call {i} was not refused")
    assert torch.cuda.max_memory_allocated() - before < 1 << 20


def test_calls_pack_the_structures_of_the_header():
    """What the Python calls pack is the structure that is compared with the
    header, up to its workspace."""
    from sparse_weight_direct_gb300 import sequence
    for pack, structure in ((sequence._pack_conv, _lib.ShortConvArgs), (sequence._pack_scan, _lib.ScanArgs),
                            (sequence._pack_adapter, _lib.AdapterArgs)):
        names = [n for n, _ in structure._fields_ if "workspace" not in n]
        packed = pack(*range(1, len(names) + 1))
        if hasattr(structure, "workspace"):
            packed += sequence._pack_workspace(1 << 40, 1 << 41)
        assert len(packed) == ctypes.sizeof(structure)
        read = structure.from_buffer_copy(packed)
        assert [getattr(read, n) for n in names] == list(range(1, len(names) + 1))
        if hasattr(structure, "workspace"):
            assert (read.workspace, read.workspace_bytes) == (1 << 40, 1 << 41)


# ------------------------------------------------------------------ sizes as served


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("case", [
    # N, P, C, M, R, adapters: clusters of eight and four blocks, aligned and not
    (2, 64, 512, 520, 16, 2), (2, 70, 256, 300, 32, 2), (2, 1, 1100, 600, 16, 2), (5, 1, 256, 300, 33, 2),
    # more tiles of y for a warp than it has on their way, in one block and in eight
    (1, 64, 40, 1040, 8, 1), (1, 128, 512, 8200, 48, 1),
    # more rows of b than a block takes at a time
    (3, 1, 512, 4200, 16, 2), (2, 1, 64, 1100, 64, 2),
], ids=lambda c: "x".join(map(str, c)))
def test_adapter_clusters_and_rounds(case, dtype):
    base.test_adapter_add(case, dtype, False)
    base.test_adapter_add(case, dtype, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", [(1, 40, 640, 64, 1), (1, 33, 300, 20, 1), (2, 20, 520, 33, 2), (8, 4, 600, 48, 2)],
                         ids=lambda c: "x".join(map(str, c)))
def test_scan_of_many_states_in_chunks(case, ragged, dtype):
    """More than 16 states in sequences that are cut."""
    N, ch, L, S, G = case
    assert _lib.lib().spconv_scan_workspace(ctypes.byref(scan_args(N=N, channels=ch, L=L, S=S, groups=G))) > 0
    base.test_scan(case, dtype, ragged, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("L", [40, 300, 1030])
def test_a_padded_sequence_is_the_sequence_alone(dtype, L):
    """Outputs, states and gradients of a sequence with NaN behind its end against
    those of the sequence alone, wherever the end lies in a tile or a chunk.  The
    gradients go by tiles and segments of fixed places here: bit for bit.  So does
    the forward pass up to 127 positions; longer ones are cut into other chunks, so
    that states are joined at other places."""
    s, dy, state, dfinal, _ = base.scan_inputs((1, 40, L, 16, 1), dtype, False, seed=20)
    rows = ("u", "delta", "B", "C", "z")
    for k in (1, 7, 32, 33, L // 2 + 3, L - 1):
        lens = torch.tensor([k], dtype=torch.int32, device="cuda")
        far = {n: base.poison(v, lens) if n in rows else v for n, v in s.items()}
        cut = {n: v[..., :k].contiguous() if n in rows else v for n, v in s.items()}
        ends = torch.empty_like(state), torch.empty_like(state)
        y = swd.scan(**far, state=state, final_state=ends[0], lengths=lens)
        alone = swd.scan(**cut, state=state, final_state=ends[1])
        assert not y[..., k:].any()
        tight = 2.0 ** -19 if L >= 128 else 0.0
        for a, b in ((y[..., :k], alone), ends):
            a, b = a.double(), b.double()
            unit = 2 * ref.HALF[dtype] * b.abs() if tight else 0.0
            assert ((a - b).abs() <= tight * b.abs().max() + unit).all(), k
        g = swd.scan_backward(base.poison(dy, lens), **far, state=state, dfinal_state=dfinal, lengths=lens)
        h = swd.scan_backward(dy[..., :k].contiguous(), **cut, state=state, dfinal_state=dfinal)
        for n, v in g.items():
            if n in ("du", "ddelta", "dB", "dC", "dz"):
                assert not v[..., k:].any(), n
                v = v[..., :k]
            assert torch.equal(v, h[n]), (n, k)
    w, b = base.Draw(22)(40, 4), base.Draw(23)(40)
    st = base.Draw(24)(1, 40, 3, dtype=dtype)
    for k in (1, 7, 32, 33, L // 2 + 3, L - 1):
        lens = torch.tensor([k], dtype=torch.int32, device="cuda")
        far, fdy = base.poison(s["u"], lens), base.poison(dy, lens)
        near, ndy = s["u"][..., :k].contiguous(), dy[..., :k].contiguous()
        ends = torch.empty_like(st), torch.empty_like(st)
        y = swd.short_conv(far, w, b, state=st, final_state=ends[0], lengths=lens)
        assert torch.equal(y[..., :k], swd.short_conv(near, w, b, state=st, final_state=ends[1]))
        assert not y[..., k:].any() and torch.equal(*ends)
        g = swd.short_conv_backward(fdy, far, w, b, state=st, dfinal_state=st, lengths=lens)
        h = swd.short_conv_backward(ndy, near, w, b, state=st, dfinal_state=st)
        assert not g[0][..., k:].any() and torch.equal(g[0][..., :k], h[0]) and torch.equal(g[3], h[3])
        for i in (1, 2):  # sums of at most L terms, each below 2^5, in another order
            assert float((g[i] - h[i]).abs().max()) <= L * 2.0 ** -23 * 8
