"""Cases of the sequence operators that stand beside the sparse-weight convolution: the short causal
convolution, the selective state space scan and the low-rank adapters of many requests, each in the
forms a model calls them (prompts, gradients, single tokens).

Activations are channels-first, N x C x L with the positions contiguous: the N x C x H x W layout of
the convolution with H * W = L.  Weights and recurrent states of the scan are float32.
"""
import torch

own = False  # False: run() computes the plain forms; True: it calls the package's operators

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a batch of prompts through the convolution in front of a scan, a model of width 2048 expanded twice
        dict(name="conv_prompt", op="conv", type="bf16", N=8, C=4096, L=2048, K=4, ragged=False, state=False),
        # requests of different lengths (an empty one and a single token among them) that continue a cached state
        dict(name="conv_ragged", op="conv", type="f32", N=6, C=515, L=785, K=3, ragged=True, state=True),
        # the convolution's gradients in a training step
        dict(name="conv_backward", op="conv_backward", type="bf16", N=4, C=2048, L=2048, K=4, ragged=False, state=False),
        # a few requests' next tokens: latency
        dict(name="conv_step", op="conv_step", type="bf16", N=4, C=1024, K=4),
        # the same batch of prompts through the scan
        dict(name="scan_prompt", op="scan", type="bf16", N=4, C=4096, L=2048, S=16, G=1, ragged=False, state=False),
        # one long prompt of odd length on a narrow model, continuing a state: little to do side by side
        dict(name="scan_long", op="scan", type="f32", N=1, C=1000, L=8191, S=16, G=1, ragged=False, state=True),
        # the scan's gradients in a training step
        dict(name="scan_backward", op="scan_backward", type="bf16", N=2, C=2048, L=2048, S=16, G=1, ragged=False, state=False),
        # gradients over sequences of different lengths, two groups, eight states, in full precision
        dict(name="scan_backward_ragged", op="scan_backward", type="f32", N=5, C=264, L=333, S=8, G=2, ragged=True, state=True),
        # a full serving batch's next tokens
        dict(name="scan_step", op="scan_step", type="bf16", N=128, C=4096, S=16, G=1),
        # next tokens of 48 requests over 32 adapters (one request in 33 without), a square projection
        dict(name="adapter_tokens", op="adapter", type="bf16", N=48, P=1, C=4096, M=4096, R=16, K=32),
        # prompts beside an expanding projection, adapters of rank 32
        dict(name="adapter_prompt", op="adapter", type="bf16", N=8, P=1024, C=2048, M=4096, R=32, K=6),
        # images beside the 512-channel layer of the sparsity sweep (28 x 28 positions), float32 as that layer is
        dict(name="adapter_layer", op="adapter", type="f32", N=8, P=784, C=512, M=512, R=8, K=3),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["conv", "conv_backward", "conv_step", "scan", "scan", "scan_backward", "scan_step", "adapter", "adapter"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "conv_step":
        return dict(op=op, type=kind, N=_log(rng, 1, 256), C=_log(rng, 64, 8192), K=rng.choice([2, 3, 4]))
    if op == "scan_step":
        N = _log(rng, 1, 128)
        G = rng.choice([1, 1, 2])
        return dict(op=op, type=kind, N=N, C=G * _log(rng, 32, 4096 // G), S=rng.choice([4, 8, 16, 16]), G=G)
    if op == "adapter":
        P = rng.choice([1, 1, _log(rng, 2, 1024), _log(rng, 16, 1024)])
        N = _log(rng, 1, 128) if P == 1 else _log(rng, 1, 8)
        return dict(op=op, type=kind, N=N, P=P, C=_log(rng, 64, 2048), M=_log(rng, 64, 2048), R=rng.choice([4, 8, 16, 16, 31, 32, 64]), K=_log(rng, 1, 16))
    C = _log(rng, 32, 4096)
    L = _log(rng, 1, 4096)
    N = _log(rng, 1, 8)
    most = {"conv": 32, "conv_backward": 16, "scan": 16 if kind == "f32" else 32, "scan_backward": 8}[op] << 20  # elements of one activation
    while N * C * L > most:
        N, L = max(1, N // 2), L if N > 1 else L // 2
    c = dict(op=op, type=kind, N=N, C=C, L=L, ragged=rng.random() < 0.5, state=rng.random() < 0.5)
    if op.startswith("conv"):
        c["K"] = rng.choice([2, 3, 4])
    else:
        c["G"] = rng.choice([1, 1, 2])
        c["C"] += c["C"] % c["G"]
        c["S"] = rng.choice([4, 8, 16, 16])
    return c


def _lengths(c):
    """Lengths of a case's sequences: an empty one, a single token and shorter and full ones where it is ragged."""
    N, L = c["N"], c["L"]
    if not c["ragged"]:
        return [L] * N
    return [L if i % 4 == 0 else 0 if i == 1 else 1 if i == 2 else max(1, (L * (i + 3)) // (N + 4)) for i in range(N)]


def _index(c):
    """Each request's adapter, -1 for none."""
    return [(5 * i) % (c["K"] + 1) - 1 if c["N"] > 1 else 0 for i in range(c["N"])]


def prepare(case, seed):
    c, op = case, case["op"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES[c["type"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    f32 = torch.float32
    s = dict(case=c)
    if op == "adapter":
        N, P, C, M, R, K = (c[k] for k in ("N", "P", "C", "M", "R", "K"))
        s["x"], s["y"] = normal(N, C, P), normal(N, M, P)
        s["a"], s["b"] = normal(K, R, C, scale=C ** -0.5), normal(K, M, R, scale=R ** -0.5)
        s["index"] = torch.tensor(_index(c), dtype=torch.int32, device=dev)
        s["scale"] = torch.rand(K, generator=g, device=dev) + 0.5
        return s
    N, C = c["N"], c["C"]
    step = op.endswith("step")
    shape = (N, C) if step else (N, C, c["L"])
    if not step:
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev) if c["ragged"] else None
    if op.startswith("conv"):
        K = c["K"]
        s["x"] = normal(*shape)
        s["weight"] = normal(C, K, scale=K ** -0.5, dtype=f32)
        s["bias"] = normal(C, scale=0.2, dtype=f32)
        s["state"] = normal(N, C, K - 1) if step or c["state"] else None
        if op == "conv_backward":
            s["dy"] = normal(*shape)
            s["dfinal"] = normal(N, C, K - 1) if c["state"] else None
        return s
    S, G = c["S"], c["G"]
    bc = (N, G, S) if step else (N, G, S, c["L"])
    # the activations behind the short convolution: silu of a normal value
    s["u"] = torch.nn.functional.silu(torch.randn(*shape, generator=g, device=dev) * 1.5).to(dt)
    s["delta"] = normal(*shape, scale=0.7)
    # step sizes of 0.001 to 0.1, spread over their logarithm, as the inverse of softplus
    size = torch.exp(torch.rand(C, generator=g, device=dev) * 4.6 - 6.9)
    s["delta_bias"] = size + torch.log(-torch.expm1(-size))
    s["A"] = -torch.arange(1, S + 1, device=dev, dtype=f32) * torch.exp(normal(C, S, scale=0.1, dtype=f32))
    s["B"], s["C"] = normal(*bc), normal(*bc)
    s["D"] = 1 + normal(C, scale=0.1, dtype=f32)
    s["z"] = normal(*shape)
    s["state"] = normal(N, C, S, scale=0.3, dtype=f32) if step or c["state"] else None
    if op == "scan_backward":
        s["dy"] = normal(*shape)
        s["dfinal"] = normal(N, C, S, scale=0.3, dtype=f32) if c["state"] else None
    return s


# ------------------------------------------------------------------ the package's operators


def _run_own(s):
    import sparse_weight_direct_gb300 as swd
    c = s["case"]
    op = c["op"]
    if op == "adapter":
        return swd.adapter_add(s["y"], s["x"], s["a"], s["b"], s["index"], scale=s["scale"])
    if op == "conv":
        final = torch.empty((c["N"], c["C"], c["K"] - 1), dtype=s["x"].dtype, device=s["x"].device)
        y = swd.short_conv(s["x"], s["weight"], s["bias"], silu=True, state=s["state"], final_state=final, lengths=s["lengths"])
        return y, final
    if op == "conv_backward":
        return swd.short_conv_backward(s["dy"], s["x"], s["weight"], s["bias"], silu=True, state=s["state"], dfinal_state=s["dfinal"], lengths=s["lengths"])
    if op == "conv_step":
        return swd.short_conv_step(s["x"], s["state"], s["weight"], s["bias"], silu=True), s["state"]
    args = (s["u"], s["delta"], s["A"], s["B"], s["C"])
    more = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=True)
    if op == "scan":
        final = torch.empty((c["N"], c["C"], c["S"]), dtype=torch.float32, device=s["u"].device)
        return swd.scan(*args, **more, state=s["state"], final_state=final, lengths=s["lengths"]), final
    if op == "scan_backward":
        return swd.scan_backward(s["dy"], *args, **more, state=s["state"], dfinal_state=s["dfinal"], lengths=s["lengths"])
    return swd.scan_step(s["state"], *args, **more), s["state"]


# ------------------------------------------------------------------ the plain forms


def _valid(s, L):
    """N x 1 x L: the positions inside each sequence, or None where all are."""
    if s["lengths"] is None:
        return None
    return torch.arange(L, device=s["lengths"].device)[None, None, :] < s["lengths"][:, None, None]


def _silu_grad(v):
    g = torch.sigmoid(v)
    return g * (1 + v * (1 - g))


def _padded(s, x, K):
    """The inputs behind their state (zeros without one): N x C x (K - 1 + L)."""
    left = s["state"].float() if s["state"] is not None else x.new_zeros(x.shape[0], x.shape[1], K - 1)
    return torch.cat([left, x], dim=2)


def _last(s, x, K):
    """Places in the padded inputs of each sequence's last K - 1: N x 1 x (K - 1)."""
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((x.shape[0],), x.shape[2], device=x.device)
    return n[:, None, None] + torch.arange(K - 1, device=x.device)[None, None, :]


def _plain_conv(s):
    x, w, K, L = s["x"].float(), s["weight"], s["case"]["K"], s["x"].shape[2]
    p = _padded(s, x, K)
    v = s["bias"][None, :, None] + sum(w[None, :, k, None] * p[:, :, k:k + L] for k in range(K))
    y = v * torch.sigmoid(v)
    ok = _valid(s, L)
    y = y if ok is None else torch.where(ok, y, 0.0)
    final = torch.gather(p, 2, _last(s, x, K).expand(-1, x.shape[1], -1))
    return y.to(s["x"].dtype), final.to(s["x"].dtype)


def _plain_conv_backward(s):
    x, w, K, L = s["x"].float(), s["weight"], s["case"]["K"], s["x"].shape[2]
    p = _padded(s, x, K)
    v = s["bias"][None, :, None] + sum(w[None, :, k, None] * p[:, :, k:k + L] for k in range(K))
    g = s["dy"].float() * _silu_grad(v)
    ok = _valid(s, L)
    g = g if ok is None else torch.where(ok, g, 0.0)
    dw = torch.stack([(g * p[:, :, k:k + L]).sum((0, 2)) for k in range(K)], 1)
    dp = torch.zeros_like(p)
    for k in range(K):
        dp[:, :, k:k + L] += w[None, :, k, None] * g
    if s["dfinal"] is not None:
        dp.scatter_add_(2, _last(s, x, K).expand(-1, x.shape[1], -1).contiguous(), s["dfinal"].float())
    dt = s["x"].dtype
    return dp[:, :, K - 1:].to(dt), dw, g.sum((0, 2)), dp[:, :, :K - 1].to(dt) if s["state"] is not None else None


def _plain_conv_step(s):
    x, w = s["x"].float(), s["weight"]
    p = torch.cat([s["state"].float(), x[:, :, None]], 2)
    v = s["bias"] + (p * w).sum(2)
    s["state"].copy_(p[:, :, 1:])
    return (v * torch.sigmoid(v)).to(s["x"].dtype), s["state"]


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _recurrence(a, b):
    """h_t = a_t h_(t-1) + b_t over the last dimension from h = 0: the steps joined two by two, then four by four."""
    n, L = 1, b.shape[-1]
    while n < L:
        b = torch.cat([b[..., :n], b[..., n:] + a[..., n:] * b[..., :-n]], -1)
        a = torch.cat([a[..., :n], a[..., n:] * a[..., :-n]], -1) if 2 * n < L else a
        n *= 2
    return b


def _scan_parts(s):
    """Step sizes, decays, states and the ungated output, all in float32; N x C x S x L for what has states."""
    c = s["case"]
    L, per = s["u"].shape[2], c["C"] // c["G"]
    ok = _valid(s, L)
    raw = s["delta"].float() + s["delta_bias"][None, :, None]
    dt = _softplus(raw)
    if ok is not None:
        dt = torch.where(ok, dt, 0.0)
    u = s["u"].float()
    B = s["B"].float().repeat_interleave(per, 1)
    C = s["C"].float().repeat_interleave(per, 1)
    a = torch.exp(dt[:, :, None, :] * s["A"][None, :, :, None])
    b = (dt * u)[:, :, None, :] * B
    if s["state"] is not None:
        b[..., 0] += a[..., 0] * s["state"]
    h = _recurrence(a, b)
    y = (h * C).sum(2) + s["D"][None, :, None] * u
    return ok, raw, dt, u, B, C, a, h, y


def _plain_scan(s):
    ok, _, _, _, _, _, _, h, y = _scan_parts(s)
    z = s["z"].float()
    y = y * z * torch.sigmoid(z)
    y = y if ok is None else torch.where(ok, y, 0.0)
    return y.to(s["u"].dtype), h[..., -1].contiguous()


def _plain_scan_backward(s):
    c, kind = s["case"], s["u"].dtype
    N, per = c["N"], c["C"] // c["G"]
    ok, raw, dt, u, B, C, a, h, y = _scan_parts(s)
    z, dy = s["z"].float(), s["dy"].float()
    if ok is not None:
        dy = torch.where(ok, dy, 0.0)
    dz = dy * y * _silu_grad(z)
    do = dy * z * torch.sigmoid(z)
    grouped = lambda v: v.view(N, c["G"], per, c["S"], -1).sum(2)  # noqa: E731
    dC = grouped(do[:, :, None, :] * h)
    # the states' gradients: g_t = C_t do_t + a_(t+1) g_(t+1), from the last position back
    src = C * do[:, :, None, :]
    if s["dfinal"] is not None:
        src[..., -1] += s["dfinal"]
    after = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1)
    g = _recurrence(after.flip(-1), src.flip(-1)).flip(-1)
    first = s["state"][..., None] if s["state"] is not None else torch.zeros_like(h[..., :1])
    before = a * torch.cat([first, h[..., :-1]], -1)
    dB = grouped(g * (dt * u)[:, :, None, :])
    gB = (g * B).sum(2)
    moved = g * before
    ddt = gB * u + (moved * s["A"][None, :, :, None]).sum(2)
    draw_ = ddt * torch.sigmoid(raw)
    draw_ = draw_ if ok is None else torch.where(ok, draw_, 0.0)
    return dict(du=(gB * dt + do * s["D"][None, :, None]).to(kind), ddelta=draw_.to(kind), dA=(moved * dt[:, :, None, :]).sum((0, 3)),
                dB=dB.to(kind), dC=dC.to(kind), dD=(do * u).sum((0, 2)), dz=dz.to(kind), ddelta_bias=draw_.sum((0, 2)),
                dstate=g[..., 0] * a[..., 0] if s["state"] is not None else None)


def _plain_scan_step(s):
    c = s["case"]
    per = c["C"] // c["G"]
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    u, z = s["u"].float(), s["z"].float()
    B = s["B"].float().repeat_interleave(per, 1)
    C = s["C"].float().repeat_interleave(per, 1)
    s["state"].mul_(torch.exp(dt[:, :, None] * s["A"])).add_((dt * u)[:, :, None] * B)
    y = (s["state"] * C).sum(2) + s["D"] * u
    return (y * z * torch.sigmoid(z)).to(s["u"].dtype), s["state"]


def _plain_adapter(s):
    on = s["index"] >= 0
    i = s["index"].clamp(min=0).long()
    v = torch.matmul(s["a"].float()[i], s["x"].float())
    d = torch.matmul(s["b"].float()[i], v) * s["scale"][i][:, None, None]
    return (s["y"].float() + torch.where(on[:, None, None], d, 0.0)).to(s["y"].dtype)


PLAIN = {"conv": _plain_conv, "conv_backward": _plain_conv_backward, "conv_step": _plain_conv_step, "scan": _plain_scan,
         "scan_backward": _plain_scan_backward, "scan_step": _plain_scan_step, "adapter": _plain_adapter}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the work of a pass


def work(case):
    c, op = case, case["op"]
    e = 4 if c["type"] == "f32" else 2
    if op == "adapter":
        index = _index(c)
        with_one, kinds = sum(i >= 0 for i in index), len({i for i in index if i >= 0})
        N, P, C, M, R = (c[k] for k in ("N", "P", "C", "M", "R"))
        return dict(bytes=e * (with_one * C * P + 2 * N * M * P + kinds * R * (C + M)) + 4 * (N + c["K"]), flops=2 * with_one * P * R * (C + M))
    N, C = c["N"], c["C"]
    if op.endswith("step"):
        held, tokens = N, N
    else:
        held, tokens = N * c["L"], sum(_lengths(c))
    if op.startswith("conv"):
        K = c["K"]
        weights, state = 4 * C * (K + 1), e * N * C * (K - 1)
        if op == "conv":
            return dict(bytes=e * C * (tokens + held) + weights + state * (1 + c["state"]), flops=tokens * C * (2 * K + 5))
        if op == "conv_backward":
            return dict(bytes=e * C * (2 * tokens + held) + 2 * weights + 3 * state * c["state"], flops=tokens * C * (6 * K + 12))
        return dict(bytes=2 * e * C * N + weights + 2 * state, flops=N * C * (2 * K + 5))
    S, G = c["S"], c["G"]
    weights, state = 4 * C * (S + 2), 4 * N * C * S
    if op == "scan":
        return dict(bytes=e * (C * (3 * tokens + held) + 2 * G * S * tokens) + weights + state * (1 + c["state"]), flops=tokens * C * (7 * S + 12))
    if op == "scan_backward":
        return dict(bytes=e * (C * (4 * tokens + 3 * held) + 2 * G * S * (tokens + held)) + 2 * weights + 3 * state * c["state"], flops=tokens * C * (22 * S + 30))
    return dict(bytes=e * N * (4 * C + 2 * G * S) + weights + 2 * state, flops=N * C * (7 * S + 12))


# ------------------------------------------------------------------ the definitions in 64 bits, position by position


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op == "adapter":
        out = d["y"].clone()
        for n, i in enumerate(_index(c)):
            if i >= 0:
                out[n] += d["scale"][i] * (d["b"][i] @ (d["a"][i] @ d["x"][n]))
        return out
    N, C = c["N"], c["C"]
    step = op.endswith("step")
    sigmoid = torch.special.expit
    if op.startswith("conv"):
        x = d["x"][:, :, None] if step else d["x"]
        L, K = x.shape[2], c["K"]
        zero = x.new_zeros(N, C, K - 1)
        seen = torch.cat([d["state"] if d["state"] is not None else zero, x], 2)
        v = torch.nn.functional.conv1d(seen, d["weight"][:, None, :], d["bias"], groups=C)
        if step:
            return (v * sigmoid(v))[:, :, 0], seen[:, :, 1:]
        lens = _lengths(c)
        if op == "conv":
            y, final = v * sigmoid(v), zero.clone()
            for n, k in enumerate(lens):
                y[n, :, k:] = 0
                final[n] = seen[n, :, k:k + K - 1]
            return y, final
        g = d["dy"] * (sigmoid(v) + v * sigmoid(v) * sigmoid(-v))
        for n, k in enumerate(lens):
            g[n, :, k:] = 0
        dseen = torch.nn.functional.conv_transpose1d(g, d["weight"][:, None, :], groups=C)
        if d["dfinal"] is not None:
            for n, k in enumerate(lens):
                dseen[n, :, k:k + K - 1] += d["dfinal"][n]
        dw = torch.stack([torch.einsum("ncl,ncl->c", g, seen[:, :, k:k + L]) for k in range(K)], 1)
        return dseen[:, :, K - 1:], dw, g.sum((0, 2)), dseen[:, :, :K - 1] if d["state"] is not None else None
    S, G = c["S"], c["G"]
    wide = lambda v: torch.repeat_interleave(v, C // G, 1)  # noqa: E731
    last = lambda v: v.unsqueeze(-1) if step else v  # noqa: E731
    u, z, B, Cm = last(d["u"]), last(d["z"]), last(d["B"]), last(d["C"])
    raw = last(d["delta"]) + d["delta_bias"][:, None]
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    L = u.shape[2]
    lens = [1] * N if step else _lengths(c)
    live = (torch.arange(L, device=u.device)[None, :] < torch.tensor(lens, device=u.device)[:, None]).double()
    A = d["A"]
    h = d["state"].clone() if d["state"] is not None else u.new_zeros(N, C, S)
    keep = op == "scan_backward"
    y, states = torch.empty_like(u), []
    for t in range(L):
        on = live[:, t, None]
        if keep:
            states.append(h)
        h = torch.exp((on * dt[:, :, t])[:, :, None] * A) * h + (on * dt[:, :, t] * u[:, :, t])[:, :, None] * wide(B[..., t])
        y[:, :, t] = torch.einsum("ncs,ncs->nc", h, wide(Cm[..., t])) + d["D"] * u[:, :, t]
    gate = z * sigmoid(z)
    if not keep:
        out = y * gate * live[:, None, :]
        return out[:, :, 0] if step else out, h
    dy = d["dy"] * live[:, None, :]
    dz = dy * y * (sigmoid(z) + z * sigmoid(z) * sigmoid(-z))
    do = dy * gate
    g = d["dfinal"].clone() if d["dfinal"] is not None else u.new_zeros(N, C, S)
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(Cm)
    du, ddt = torch.zeros_like(u), torch.zeros_like(u)
    fold = lambda v: v.view(N, G, C // G, S).sum(2)  # noqa: E731
    after = h
    for t in reversed(range(L)):
        on = live[:, t, None]
        size = on * dt[:, :, t]
        a = torch.exp(size[:, :, None] * A)
        g = g + do[:, :, t, None] * wide(Cm[..., t])
        dC[..., t] = fold(do[:, :, t, None] * after)
        dB[..., t] = fold(g * (size * u[:, :, t])[:, :, None])
        gb = torch.einsum("ncs,ncs->nc", g, wide(B[..., t]))
        kept = g * a * states[t]
        dA += torch.einsum("ncs,nc->cs", kept, size)
        du[:, :, t] = gb * size + d["D"] * do[:, :, t]
        ddt[:, :, t] = on * (gb * u[:, :, t] + torch.einsum("ncs,cs->nc", kept, A))
        g, after = g * a, states[t]
    draw_ = ddt * sigmoid(raw)
    return dict(du=du, ddelta=draw_, dA=dA, dB=dB, dC=dC, dD=(do * u).sum((0, 2)), dz=dz, ddelta_bias=draw_.sum((0, 2)),
                dstate=g if d["state"] is not None else None)
