"""y of the state-space calls on the GPU held to what each kernel may round (_dense_reads.py): the
step and the token-by-token scan nothing but y itself, the block-wise scan the weights of a
block's tokens and the state before the block to two bf16 parts."""

import pytest
import torch

from tests import _dense as ref
from tests import _dense_reads as reads

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sdm():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sparse_memory_linear_b200 as m
    torch.cuda.set_device(0)
    yield m
    torch.cuda.synchronize()
    assert m.sdm_get_device_status() == 0


def inputs(seed, lead, H, G, N, P, B, gate):
    """Slow decays, so that reads are mostly of tokens and states long past."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*s, dtype=BF, by=1.0):
        return (torch.randn(*s, generator=g, device=DEV) * by).to(dtype)

    i = dict(k=randn(*lead, G, N, by=0.5), q=randn(*lead, G, N, by=0.5), v=randn(*lead, H, P),
             dt=randn(*lead, H), A=-(0.05 + 0.2 * torch.rand(H, generator=g, device=DEV)),
             dt_bias=randn(H, dtype=torch.float32, by=0.5) - 3.0,
             D=randn(H, dtype=torch.float32), gate=randn(*lead, H, P) if gate else None)
    return i, randn(B, H, N, P, dtype=torch.float32)


def d64(i):
    """The tensors in 64 bits, rows one after another."""
    return {n: None if t is None else t.double() if n in ("A", "dt_bias", "D")
            else t.double().reshape((-1,) + t.shape[-1 if n == "dt" else -2:])
            for n, t in i.items()}


def bounds(i, M, lens, block):
    f = d64(i)
    ry, rM, yb, Mb = ref.ssm(f["k"], f["q"], f["v"], f["dt"], f["A"], M.double(), f["D"],
                             f["dt_bias"], True, f["gate"], "silu", lens)
    if block:
        own, before = reads.magnitudes(f["k"], f["q"], f["v"], f["dt"], f["A"], M.double(),
                                       f["dt_bias"], True, lens)
        yb = reads.bound(yb, own, before, f["gate"], "silu")
    return ry, rM, yb, Mb


@pytest.mark.parametrize("B,T,H,G,N,P,gate,block", [
    (2, 23, 4, 2, 64, 64, True, False), (1, 130, 2, 1, 136, 40, True, False),
    (1, 300, 1, 1, 256, 64, False, False), (2, 300, 4, 2, 64, 64, True, True),
    (1, 1100, 1, 1, 128, 64, False, True), (3, 129, 2, 1, 24, 80, True, True),
])
def test_scan_reads(sdm, B, T, H, G, N, P, gate, block):
    i, M = inputs(T + N, (B, T), H, G, N, P, B, gate)
    ry, rM, yb, Mb = bounds(i, M, [T] * B, block)
    y = sdm.sdm_ssm_forward(M=M, init="continue", **i)
    ref.check(y.reshape(B * T, H, P), ry, yb, "y")
    ref.check(M, rM, Mb, "M")


@pytest.mark.parametrize("B,H,G,N,P,gate", [(3, 4, 2, 64, 64, True), (2, 3, 1, 256, 72, False),
                                            (17, 8, 1, 128, 128, True)])
def test_step_reads(sdm, B, H, G, N, P, gate):
    i, M = inputs(N + P, (B,), H, G, N, P, B, gate)
    ry, rM, yb, Mb = bounds(i, M, [1] * B, False)
    y = sdm.sdm_ssm_step(M=M, **i)
    ref.check(y, ry, yb, "y")
    ref.check(M, rM, Mb, "M")


@pytest.mark.parametrize("N,block", [(128, True), (40, True), (256, False)])
def test_reads_that_cancel(sdm, N, block):
    """Steps of size 0 (dt = -infinity) and pairs of state rows that nearly cancel: y is a small
    difference of large terms of the state as it is, which one bf16 part of it would lose."""
    B, T, H, P = 2, 200, 2, 64
    i, M = inputs(7, (B, T), H, 1, N, P, B, False)
    i["dt"][:] = float("-inf")
    i["D"] = None
    i["q"][..., 1::2] = -i["q"][..., ::2]
    M[:, :, 1::2] = M[:, :, ::2] * (1 + 2.0 ** -10)
    M0 = M.clone()
    y = sdm.sdm_ssm_forward(M=M, init="continue", **i)
    assert torch.equal(M, M0)
    f = d64(i)
    own, before = reads.magnitudes(f["k"], f["q"], f["v"], f["dt"], f["A"], M0.double(),
                                   f["dt_bias"], True, [T] * B)
    assert not own.any()
    ry = torch.einsum("btn,bhnp->bthp", f["q"].view(B, T, N), M0.double()).reshape(B * T, H, P)
    yb = reads.still_bound(N, before)
    ref.check(y.reshape(B * T, H, P), ry, reads.bound(yb, own, before, None, "") if block else yb,
              "y")
