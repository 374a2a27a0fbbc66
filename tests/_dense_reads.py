"""What a read of the dense state adds up, told apart by how a kernel may hold it: the tokens of the
reader's own block of 128 and the state before that block.  The block-wise scan holds the weights of
the first and the values of the second as two bf16 parts.

With |q| |k| |v| d e^{dA} the magnitude of a token's share of a read and |q| |M| that of the state's,
either is off by half a step of half a step of bf16, 2^-16 of its magnitude.  Everything else is
fp32 and covered by the bound of tests/_dense.py with weights = 0."""

import torch

from tests import _dense as ref

BLOCK = 128


def magnitudes(k, q, v, dt, A, M, dt_bias, softplus, lens):
    """[R, H, P] each: sums of the magnitudes of what a token's read takes from its own block's
    tokens and from the state before its block.  Arguments in 64 bits, as for ref.ssm."""
    H, G = v.shape[1], k.shape[1]
    head = torch.arange(H, device=v.device) // (H // G)
    raw = dt + (dt_bias if dt_bias is not None else 0.0)
    d = ref.softplus64(raw) if softplus else torch.clamp(raw, min=0)
    own, before = torch.zeros_like(v), torch.zeros_like(v)
    at = 0
    for b, n in enumerate(lens):
        old, new = M[b].abs(), torch.zeros_like(M[b])
        for t in range(n):
            if t % BLOCK == 0:
                old, new = old + new, torch.zeros_like(new)
            r = at + t
            kk, qq = k[r, head].abs()[:, :, None], q[r, head].abs()[:, :, None]
            al = torch.exp(d[r] * A)[:, None, None]
            old, new = al * old, al * new + kk * (d[r][:, None] * v[r]).abs()[:, None, :]
            own[r], before[r] = (qq * new).sum(1), (qq * old).sum(1)
        at += n
    return own, before


def bound(yb, own, before, gate, act):
    """The bound on a block-wise y before its rounding: yb, from ref.ssm with weights = 0, and the
    roundings of the reads, through the gate."""
    reads = 2.0 ** -16 * (own + before)
    return yb + (reads * ref.act64(gate, act).abs() if gate is not None else reads)


def still_bound(N, before):
    """The fp32 part of that bound for tokens whose steps are all 0, so that y is q^T M of the state as
    it is: 2 N products of one read, added up in any order."""
    return 2 * N * ref.U * before
