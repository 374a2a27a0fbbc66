"""The bounds of _dense_reads.py tell apart, without a GPU, reads that hold the state and the weights
in two bf16 parts from reads that hold one of them in one: planted in a plain implementation, not in
a kernel."""

import pytest
import torch

from tests import _dense as ref
from tests import _dense_reads as reads


def bf16(x):
    return x.to(torch.bfloat16).double()


def held(x, parts):
    """x in so many bf16 parts."""
    out, left = torch.zeros_like(x), x.clone()
    for _ in range(parts):
        out, left = out + bf16(left), left - bf16(left)
    return out


def blockwise(k, q, v, dt, A, M, dt_bias, lens, state, weights):
    """y of the scan in 64 bits, a block at a time, with the state before the block and a token's
    weight in so many bf16 parts."""
    H, G = v.shape[1], k.shape[1]
    head = torch.arange(H) // (H // G)
    d = ref.softplus64(dt + dt_bias)
    y, at = torch.zeros_like(v), 0
    for b, n in enumerate(lens):
        m = M[b].clone()
        for t0 in range(0, n, reads.BLOCK):
            r = slice(at + t0, at + min(t0 + reads.BLOCK, n))
            c = torch.cumsum(d[r] * A, 0)                              # [L, H]
            kk, qq = k[r][:, head], q[r][:, head]
            w = torch.einsum("thn,shn->hts", qq, kk) * d[r].T[:, None]
            w = torch.tril(w * torch.exp((c.T[:, :, None] - c.T[:, None]).clamp(max=0)))
            y[r] = torch.einsum("hts,shp->thp", held(w, weights), v[r]) + torch.einsum(
                "thn,hnp->thp", qq * torch.exp(c)[..., None], held(m, state))
            left_over = torch.exp(c[-1] - c) * d[r]
            m = torch.exp(c[-1])[:, None, None] * m + torch.einsum(
                "shn,shp->hnp", kk, v[r] * left_over[..., None])
        at += n
    return y


@pytest.mark.parametrize("case", ["kept", "still", "fresh"])
def test_one_bf16_part_is_told_from_two(case):
    """Of the state in a sequence that continues from one, with steps that decay it or are all 0 (y is
    then the state's read); of the weights in a sequence that starts from nothing."""
    g = torch.Generator().manual_seed(3)
    randn = lambda *s: bf16(torch.randn(*s, generator=g))  # noqa: E731
    lens, H, G, N, P = [300, 140], 2, 1, 32, 16
    R = sum(lens)
    k, q, v, dt = randn(R, G, N) * 0.5, randn(R, G, N) * 0.5, randn(R, H, P), randn(R, H)
    if case == "still":
        dt[:] = float("-inf")
    A = -(0.05 + 0.1 * torch.rand(H, generator=g).double())
    bias = torch.full((H,), -3.0, dtype=torch.float64)
    M = torch.randn(2, H, N, P, generator=g).double()
    if case == "fresh":
        M.zero_()
    ry, _, yb, _ = ref.ssm(k, q, v, dt, A, M, None, bias, True, None, "silu", lens)
    own, before = reads.magnitudes(k, q, v, dt, A, M, bias, True, lens)
    if case == "still":
        yb = reads.still_bound(N, before)
    lim = reads.bound(yb, own, before, None, "silu")
    y = lambda s, w: blockwise(k, q, v, dt, A, M, bias, lens, s, w).to(torch.bfloat16)  # noqa: E731
    ref.check(y(2, 2), ry, lim, "y")
    ref.check(y(6, 6), ry, yb, "y")  # both in fp32
    with pytest.raises(AssertionError):
        ref.check(y(2, 1) if case == "fresh" else y(1, 2), ry, lim, "y")
