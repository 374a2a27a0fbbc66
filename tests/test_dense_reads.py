"""The bounds of _dense_reads.py tell apart, without a GPU, reads that hold the state in two bf16
parts from reads that hold it in one: planted in a plain implementation, not in a kernel."""

import pytest
import torch

from tests import _dense as ref
from tests import _dense_reads as reads


def bf16(x):
    return x.to(torch.bfloat16).double()


def blockwise(k, q, v, dt, A, M, dt_bias, lens, parts, weights=True):
    """y of the scan in 64 bits, a block at a time, with a token's weight rounded to bf16 and the
    state before the block in `parts` bf16 parts."""
    H, G = v.shape[1], k.shape[1]
    head = torch.arange(H) // (H // G)
    d = ref.softplus64(dt + dt_bias)
    y, at = torch.zeros_like(v), 0
    for b, n in enumerate(lens):
        m = M[b].clone()
        for t0 in range(0, n, reads.BLOCK):
            held, left = torch.zeros_like(m), m.clone()
            for _ in range(parts):
                held, left = held + bf16(left), left - bf16(left)
            r = slice(at + t0, at + min(t0 + reads.BLOCK, n))
            c = torch.cumsum(d[r] * A, 0)                              # [L, H]
            kk, qq = k[r][:, head], q[r][:, head]
            w = torch.einsum("thn,shn->hts", qq, kk) * d[r].T[:, None]
            w = torch.tril(w * torch.exp((c.T[:, :, None] - c.T[:, None]).clamp(max=0)))
            w = bf16(w) if weights else w
            y[r] = torch.einsum("hts,shp->thp", w, v[r]) + torch.einsum(
                "thn,hnp->thp", qq * torch.exp(c)[..., None], held)
            left_over = torch.exp(c[-1] - c) * d[r]
            m = torch.exp(c[-1])[:, None, None] * m + torch.einsum(
                "shn,shp->hnp", kk, v[r] * left_over[..., None])
        at += n
    return y


@pytest.mark.parametrize("still", [False, True])
def test_one_bf16_part_of_the_state_is_told_from_two(still):
    """In a sequence that decays, and in one whose steps are all 0 so that y is the state's read."""
    g = torch.Generator().manual_seed(3)
    randn = lambda *s: bf16(torch.randn(*s, generator=g))  # noqa: E731
    lens, H, G, N, P = [300, 140], 2, 1, 32, 16
    R = sum(lens)
    k, q, v, dt = randn(R, G, N) * 0.5, randn(R, G, N) * 0.5, randn(R, H, P), randn(R, H)
    if still:
        dt[:] = float("-inf")
    A = -(0.05 + 0.1 * torch.rand(H, generator=g).double())
    bias = torch.full((H,), -3.0, dtype=torch.float64)
    M = torch.randn(2, H, N, P, generator=g).double()
    ry, _, yb, _ = ref.ssm(k, q, v, dt, A, M, None, bias, True, None, "silu", lens)
    own, before = reads.magnitudes(k, q, v, dt, A, M, bias, True, lens)
    if still:
        yb = reads.still_bound(N, before)
    lim = reads.bound(yb, own, before, None, "silu")
    two = blockwise(k, q, v, dt, A, M, bias, lens, 2)
    ref.check(two.to(torch.bfloat16), ry, lim, "y")
    one = blockwise(k, q, v, dt, A, M, bias, lens, 1)
    with pytest.raises(AssertionError):
        ref.check(one.to(torch.bfloat16), ry, lim, "y")
    # rounded weights where a kernel rounds none are told apart as well
    none = blockwise(k, q, v, dt, A, M, bias, lens, 6, weights=False)
    ref.check(none.to(torch.bfloat16), ry, yb, "y")
    if not still:
        with pytest.raises(AssertionError):
            ref.check(two.to(torch.bfloat16), ry, yb, "y")
