"""Plain 64-bit implementations of the dense-state layer's operators, token by token, with the
error bounds that the tests hold the kernels to.

u = 2^-24 is half a step of fp32 relative to the value; half(t) the same for the output type."""

import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "sigmoid":
        return torch.sigmoid(x)
    return x


def conv(x, w, bias, state, act, lens):
    """x [rows, C] in 64 bits, sequences one after another with lengths `lens`; state
    [B, K-1, C].  Returns y, new state and the bound on y's error before it is rounded: K + 1
    roundings of partial sums of size at most mag (with its inputs exact); silu' <= 1.1; the
    activation itself is good to a few steps of its value, at most |x|."""
    K = w.shape[1]
    ys, mags, new, at = [], [], [], 0
    for b, n in enumerate(lens):
        full = torch.cat([state[b], x[at:at + n]])
        y = torch.zeros_like(full[K - 1:])
        mag = torch.zeros_like(y)
        for j in range(K):
            y = y + full[j:j + n] * w[:, j]
            mag = mag + (full[j:j + n] * w[:, j]).abs()
        if bias is not None:
            y, mag = y + bias, mag + bias.abs()
        ys.append(act64(y, act))
        mags.append(mag)
        new.append(full[n:])
        at += n
    y, mag = torch.cat(ys), torch.cat(mags)
    return y, torch.stack(new), U * (1.1 * (K + 1) * mag + 8 * (mag + 1))


def softplus64(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def ssm(k, q, v, dt, A, M, D, dt_bias, softplus, gate, act, lens, weights=0.0):
    """Rows one after another: k, q [R, G, N], v, gate [R, H, P], dt [R, H]; M [B, H, N, P]; all
    in 64 bits.  Returns y, M and bounds on the errors of y (before its rounding) and M.

    The state's bound E follows the recurrence: every token decays it and adds the roundings of
    that token's update, of which there are a few of relative size U and the exponential's,
    whose argument d A carries a relative error of a few U (hence the factor 1 + |d A|; a kernel
    that adds up arguments over a block rounds each partial sum once more).  A read of N terms
    adds the roundings of its sums.  `weights`: half a step of the type to which a kernel rounds
    a token's weight in another token's read, relative to the sum of the magnitudes."""
    H, G = v.shape[1], k.shape[1]
    head = torch.arange(H, device=v.device) // (H // G)
    raw = dt + (dt_bias if dt_bias is not None else 0.0)
    d = softplus64(raw) if softplus else torch.clamp(raw, min=0)
    da = d * A
    # the step size itself: its argument's rounding and that of softplus (slope at most 1)
    erel = (4 * U * (d + raw.abs())) / d.clamp(min=1e-300) if softplus else U * torch.ones_like(d)
    erel = erel.clamp(max=1.0)
    M = M.clone()
    y, yb, Mb = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(M)
    at = 0
    for b, n in enumerate(lens):
        m, mabs, E = M[b], M[b].abs(), torch.zeros_like(M[b])
        for t in range(at, at + n):
            kk, qq = k[t, head][:, :, None], q[t, head][:, :, None]
            al = torch.exp(da[t])[:, None, None]
            add = kk * (d[t][:, None] * v[t])[:, None, :]
            m = al * m + add
            mabs = al * mabs + add.abs()
            c = (16 * U * (1 + da[t].abs()) + erel[t] * (1 + da[t].abs()))[:, None, None]
            E = al * E + c * mabs
            y[t] = (qq * m).sum(1)
            ab = (qq.abs() * mabs).sum(1)
            yb[t] = (qq.abs() * E).sum(1) + (8 * U + weights) * ab
        M[b], Mb[b] = m, E
        at += n
    if D is not None:
        y = y + D[:, None] * v
        yb = yb + 2 * U * (D[:, None] * v).abs()
    if gate is not None:
        f = act64(gate, act)
        yb = yb * f.abs() + 8 * U * (y * f).abs()
        y = y * f
    return y, M, yb + 2 * U * y.abs(), Mb


def block_norm(u, r, post, post_gamma, gate, act, scale, pre_gamma, eps):
    """Returns r', n and the bounds on their errors before they are rounded.  A mean of D squares
    is good to (log2-depth and per-thread sums) 16 U relative, its rsqrt to 10 U; every factor
    adds 2 U, the activation 8 U; n divides by the row's norm, whose relative error is at most
    that of its largest terms: |dr| adds up over the row in the root of the mean of squares."""
    f, fe = u, torch.zeros_like(u)
    if post:
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps)
        if post_gamma is not None:
            f = f * post_gamma
        fe = 16 * U * f.abs()
    if gate is not None:
        g = act64(gate, act)
        fe = fe * g.abs() + 10 * U * (f * g).abs()
        f = f * g
    if scale is not None:
        fe = fe * scale.abs() + 2 * U * (f * scale).abs()
        f = f * scale
    r = r + f
    re = fe + U * r.abs()
    ms = r.square().mean(-1, keepdim=True) + eps
    inv = torch.rsqrt(ms)
    n = r * inv
    ne = re * inv + n.abs() * (16 * U + (re.square().mean(-1, keepdim=True) / ms).sqrt())
    if pre_gamma is not None:
        n, ne = n * pre_gamma, ne * pre_gamma.abs()
    return r, n, re, ne + 2 * U * n.abs()


def check(got, ref, bound, what):
    """|got - ref| <= bound + half a step of got's type, everywhere (and got is finite)."""
    g = got.double()
    lim = bound + half(got.dtype) * (ref.abs() + bound) + torch.finfo(got.dtype).tiny
    bad = ~((g - ref).abs() <= lim)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{g[i].item()} for {ref[i].item()} (bound {lim[i].item():.3g})")
