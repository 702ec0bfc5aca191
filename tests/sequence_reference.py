"""Plain 64-bit forms of the sequence operators, position by position, for the
tests: each returns its outputs and, beside each, how far a computation in 32
bits may be from it before the output's own rounding.

The bounds follow the formulas with every term in absolute value (`mag`) and
E = 2^-21 for what one step may add relative to its terms: a fast exponential
is good to about 2^-22 and its argument to 2^-24 of |dt A|, a product and two
sums to 2^-24 each.  A recurrence carries its error on: err_t = a err_(t-1) +
E (2 + |dt A|) mag_t.
"""
import torch

E = 2.0 ** -21
# half a unit in the last place, relative: 24, 8 and 11 bits of significand
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-30, torch.bfloat16: 1e-30, torch.float16: 2.0 ** -25}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def check(got, want, bound, what):
    """|got - want| <= bound + the rounding of got's type."""
    got_type = got.dtype
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = bound + HALF[got_type] * (want.abs() + bound) + TINY[got_type]
    far = (got - want).abs()
    bad = ~(far <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float((far / tol).nan_to_num(float('inf')).max()):.3g} of the bound")


def sig(v):
    return torch.special.expit(v)


def lens_of(lengths, N, L):
    return [L] * N if lengths is None else [min(max(int(k), 0), L) for k in lengths]


def conv(x, weight, bias, silu, state, lengths):
    """(y, bound), (final, 0), and what the gradients use: v, p, live, mag"""
    x, w, b, st = f64(x), f64(weight), f64(bias), f64(state)
    N, C, L = x.shape
    K = w.shape[1]
    lens = lens_of(lengths, N, L)
    for n, k in enumerate(lens):
        x[n, :, k:] = 0
    p = torch.cat([st if st is not None else x.new_zeros(N, C, K - 1), x], 2)
    v = x.new_zeros(N, C, L) + (b[None, :, None] if b is not None else 0)
    mag = v.abs()
    for k in range(K):
        v = v + w[None, :, k, None] * p[:, :, k:k + L]
        mag = mag + (w[None, :, k, None] * p[:, :, k:k + L]).abs()
    live = torch.zeros(N, 1, L, dtype=torch.float64)
    final = x.new_zeros(N, C, K - 1)
    for n, k in enumerate(lens):
        live[n, :, :k] = 1
        final[n] = p[n, :, k:k + K - 1]
    y = (v * sig(v) if silu else v) * live
    # silu is 1.1-Lipschitz; its own evaluation: an exponential and a quotient
    bound = 1.1 * E * mag + (E * (2 + v.abs()) * y.abs() if silu else 0)
    return (y, bound), (final, 0 * final), (v, p, live, mag, lens)


def conv_backward(dy, x, weight, bias, silu, state, dfinal, lengths):
    _, _, (v, p, live, mag, lens) = conv(x, weight, bias, silu, state, lengths)
    w = f64(weight)
    K, L = w.shape[1], v.shape[2]
    s = sig(v)
    slope = s * (1 + v * (1 - s)) if silu else torch.ones_like(v)
    d = torch.where(live > 0, f64(dy), 0.0)
    g = d * slope
    # |silu''| <= 1/2
    ge = d.abs() * (0.5 * E * mag + E * (3 + v.abs())) if silu else 0 * g
    dp, dpe = torch.zeros_like(p), torch.zeros_like(p)
    for k in range(K):
        dp[:, :, k:k + L] += w[None, :, k, None] * g
        dpe[:, :, k:k + L] += w[None, :, k, None].abs() * (ge + E * g.abs())
    if dfinal is not None:
        for n, k in enumerate(lens):
            dp[n, :, k:k + K - 1] += f64(dfinal)[n]
            dpe[n, :, k:k + K - 1] += E * f64(dfinal)[n].abs()
    # sums of N L terms in a tree and in short runs: 32 roundings of the running sum at most count
    dw = torch.stack([(g * p[:, :, k:k + L]).sum((0, 2)) for k in range(K)], 1)
    dwe = torch.stack([((ge + 8 * E * g.abs()) * p[:, :, k:k + L].abs()).sum((0, 2)) for k in range(K)], 1)
    return ((dp[:, :, K - 1:] * live, dpe[:, :, K - 1:]), (dw, dwe),
            (g.sum((0, 2)), (ge + 8 * E * g.abs()).sum((0, 2))), (dp[:, :, :K - 1], dpe[:, :, :K - 1]))


def scan(u, delta, A, B, C, D, z, delta_bias, softplus, state, lengths, grad=None):
    """(y, bound), (final, bound); with grad = (dy, dfinal): those and a dict of
    (gradient, bound)."""
    u, delta, A, B, C, D, z, bias, h = (f64(t) for t in (u, delta, A, B, C, D, z, delta_bias, state))
    N, ch, L = u.shape
    S = A.shape[1]
    if B.dim() == 3:
        B, C = B[:, None], C[:, None]
    G = B.shape[1]
    lens = lens_of(lengths, N, L)
    live = torch.zeros(N, 1, L, dtype=torch.float64)
    for n, k in enumerate(lens):
        live[n, :, :k] = 1
    clean = lambda t: torch.where(live.expand(N, t.shape[1], L) > 0, t, 0.0)  # noqa: E731
    u, delta = clean(u), clean(delta)
    z = clean(z) if z is not None else None
    B = torch.where(live[:, :, None] > 0, B, 0.0)
    C = torch.where(live[:, :, None] > 0, C, 0.0)
    wide = lambda t: t.repeat_interleave(ch // G, 1)  # noqa: E731
    raw = delta + (bias[None, :, None] if bias is not None else 0)
    dt = (torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw) * live
    D_ = D if D is not None else torch.zeros(ch, dtype=torch.float64)
    h = h if h is not None else torch.zeros(N, ch, S, dtype=torch.float64)
    m, e = h.abs(), torch.zeros_like(h)
    y, ye = torch.zeros_like(u), torch.zeros_like(u)
    hs, ms, es = [h], [m], [e]
    for t in range(L):
        on = live[:, :, t, None]
        w = dt[:, :, t, None] * A
        a = torch.exp(w)
        src = (dt[:, :, t] * u[:, :, t])[:, :, None] * wide(B[..., t])
        h, m = a * h + src, a * m + src.abs()
        # the step size itself is good to 4 E: it moves a by |dt A| of that
        e = a * e + on * E * (2 + 4 * w.abs()) * m + 4 * E * src.abs()
        c = wide(C[..., t])
        y[:, :, t] = (h * c).sum(2) + D_ * u[:, :, t]
        ye[:, :, t] = (c.abs() * (e + 2 * E * m)).sum(2) + E * (D_ * u[:, :, t]).abs()
        hs.append(h), ms.append(m), es.append(e)
    gate = z * sig(z) if z is not None else torch.ones_like(u)
    zabs = z.abs() if z is not None else torch.zeros_like(u)
    out = y * gate * live
    bound = (ye * gate.abs() + E * (2 + zabs) * out.abs()) * live
    if grad is None:
        return (out, bound), (h, e)
    dy, dfinal = clean(f64(grad[0])), f64(grad[1])
    slope = sig(z) * (1 + z * sig(-z)) if z is not None else torch.zeros_like(u)
    do = dy * gate
    doe = E * (2 + zabs) * do.abs()
    r = {}
    if z is not None:
        r["dz"] = (dy * y * slope, dy.abs() * (ye * slope.abs() + E * (4 + zabs) * (y.abs() + ye)))
    g = dfinal if dfinal is not None else torch.zeros(N, ch, S, dtype=torch.float64)
    gm, ge = g.abs(), torch.zeros_like(g)
    fold = lambda t: t.view(N, G, ch // G, S).sum(2)  # noqa: E731
    zeros = torch.zeros_like
    dA, dAe = zeros(A), zeros(A)
    dB, dBe, dC, dCe = zeros(B), zeros(B), zeros(C), zeros(C)
    du, due, dd, dde = zeros(u), zeros(u), zeros(u), zeros(u)
    for t in reversed(range(L)):
        w = dt[:, :, t, None] * A
        a = torch.exp(w)
        b, c, o = wide(B[..., t]), wide(C[..., t]), do[:, :, t, None]
        g, gm = g + o * c, gm + (o * c).abs()
        ge = ge + doe[:, :, t, None] * c.abs() + E * gm
        dC[..., t] = fold(o * hs[t + 1])
        dCe[..., t] = fold((o.abs() + doe[:, :, t, None]) * (es[t + 1] + 4 * E * ms[t + 1]))
        s = (dt[:, :, t] * u[:, :, t])[:, :, None]
        dB[..., t] = fold(g * s)
        dBe[..., t] = fold((ge + 8 * E * gm) * s.abs())
        gb = (g * b).sum(2)
        gbe = ((ge + 4 * E * gm) * b.abs()).sum(2)
        q = g * a * hs[t]
        qe = a * ((ge + 4 * E * (1 + w.abs()) * gm) * (ms[t] + es[t]) + gm * es[t])
        dA += (q * dt[:, :, t, None]).sum(0)
        dAe += ((qe + 8 * E * q.abs()) * dt[:, :, t, None].abs()).sum(0)
        du[:, :, t] = gb * dt[:, :, t] + D_ * do[:, :, t]
        due[:, :, t] = (gbe + 4 * E * gb.abs()) * dt[:, :, t].abs() + D_.abs() * (doe + E * do.abs())[:, :, t]
        dd[:, :, t] = gb * u[:, :, t] + (q * A).sum(2)
        dde[:, :, t] = (gbe + E * gb.abs()) * u[:, :, t].abs() + ((qe + 4 * E * q.abs()) * A.abs()).sum(2)
        g, gm, ge = g * a, gm * a, a * (ge + E * (2 + 4 * w.abs()) * gm)
    if softplus:
        dde = dde * sig(raw) + E * (2 + raw.abs()) * (dd * sig(raw)).abs()
        dd = dd * sig(raw)
    dd, dde = dd * live, dde * live
    r.update(du=(du, due), ddelta=(dd, dde), dA=(dA, dAe), dB=(dB, dBe), dC=(dC, dCe),
             dD=((do * u).sum((0, 2)), ((doe + 8 * E * do.abs()) * u.abs()).sum((0, 2))),
             ddelta_bias=(dd.sum((0, 2)), (dde + 8 * E * dd.abs()).sum((0, 2))), dstate=(g, ge))
    return (out, bound), (h, e), r


def adapter(y, x, a, b, index, scale):
    """(out, bound): sums over C and R of n terms in any order, each within
    n 2^-24 of its absolute terms, and 16-bit products whose inner sum is kept
    to at least 16 bits."""
    half = x.dtype != torch.float32
    y, x, a, b, scale = f64(y), f64(x), f64(a), f64(b), f64(scale)
    flat = x.dim() == 2
    if flat:
        y, x = y[..., None], x[..., None]
    out, bound = y.clone(), 2.0 ** -23 * y.abs()
    K, R, C = a.shape
    rel = (C + R) * 2.0 ** -24 + (2.0 ** -16 if half else E)
    for n, i in enumerate(index.tolist()):
        if 0 <= i < K:
            s = float(scale[i]) if scale is not None else 1.0
            out[n] += s * (b[i] @ (a[i] @ x[n]))
            bound[n] += rel * abs(s) * (b[i].abs() @ (a[i].abs() @ x[n].abs()))
    return (out[..., 0], bound[..., 0]) if flat else (out, bound)
