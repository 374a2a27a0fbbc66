"""Refusals of the dense-state layer's calls at the C boundary, without a GPU: bad pointers,
sizes, strides, enums and overlaps return an error before anything is launched.  As in
test_abi.py the addresses are made up and never dereferenced, so these run only where no CUDA
device is visible."""

import ctypes

import pytest
import torch

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="made-up device addresses are passed only without a GPU")
GAP = 1 << 36  # further apart than any buffer of these calls is long


def at(i):
    return GAP * (i + 1)


@pytest.fixture(scope="module")
def sdm():
    from sparse_memory_linear_b200.build import build_library
    build_library()
    import sparse_memory_linear_b200 as m
    m.library()
    return m


def refused(sdm, status, call):
    n = sdm.sdm_launch_count()
    assert call() == status
    assert sdm.sdm_launch_count() == n


def conv(sdm, step=False, shape=None, **over):
    s = dict(B=2, T=16, C=64, K=4, in_dtype=1, x_stride=0)
    s.update(shape or {})
    a = dict(x=at(0), w=at(1), bias=at(2), state=at(3), init=1, act=0, cu=None, y=at(4))
    a.update(over)
    S = sdm.SdmConvShape(*s.values())
    lib = sdm.library()
    if step:
        return lambda: lib.sdm_conv_step(a["x"], a["w"], a["bias"], a["state"], a["act"], a["y"],
                                         S, None)
    return lambda: lib.sdm_conv_forward(a["x"], a["w"], a["bias"], a["state"], a["init"],
                                        a["act"], a["cu"], a["y"], S, None)


@host_only
@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w=None), dict(y=None), dict(x=at(0) + 8), dict(w=at(1) + 4),
    dict(bias=at(2) + 4), dict(state=at(3) + 2), dict(y=at(4) + 8), dict(act=3), dict(act=-1),
    dict(y=at(0)), dict(state=at(0) + 64), dict(y=at(3)), dict(state=None),
    dict(shape=dict(B=0)), dict(shape=dict(C=60)), dict(shape=dict(C=0)),
    dict(shape=dict(in_dtype=2)), dict(shape=dict(x_stride=56)), dict(shape=dict(x_stride=68)),
    dict(shape=dict(x_stride=-64)),
])
def test_conv_refuses(sdm, step, bad):
    refused(sdm, 1, conv(sdm, step, **bad))


@host_only
def test_conv_refuses_more(sdm):
    refused(sdm, 1, conv(sdm, init=0))
    refused(sdm, 1, conv(sdm, init=3))
    refused(sdm, 1, conv(sdm, shape=dict(T=-1)))
    refused(sdm, 1, conv(sdm, cu=at(5) + 2))
    refused(sdm, 1, conv(sdm, cu=at(4)))  # offsets inside y
    for K in (0, 1, 5):
        refused(sdm, 2, conv(sdm, shape=dict(K=K)))
        refused(sdm, 2, conv(sdm, True, shape=dict(K=K)))


def ssm(sdm, step=False, shape=None, **over):
    s = dict(B=2, T=16, H=4, G=2, N=64, d_v=64, in_dtype=1, softplus=1, k_stride=0, q_stride=0,
             v_stride=0, dt_stride=0, gate_stride=0)
    s.update(shape or {})
    a = dict(k=at(0), q=at(1), v=at(2), dt=at(3), A=at(4), dt_bias=at(5), D=at(6), M=at(7),
             init=1, gate=at(8), act=0, cu=None, y=at(9), ws=at(10), ws_bytes=1 << 30)
    a.update(over)
    S = sdm.SdmSsmShape(*s.values())
    lib = sdm.library()
    head = [a[n] for n in ("k", "q", "v", "dt", "A", "dt_bias", "D", "M")]
    if step:
        return lambda: lib.sdm_ssm_step(*head, a["gate"], a["act"], a["y"], S, None)
    return lambda: lib.sdm_ssm_forward(*head, a["init"], a["gate"], a["act"], a["cu"], a["y"],
                                       a["ws"], a["ws_bytes"], S, None)


@host_only
@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("bad", [
    dict(k=None), dict(q=None), dict(v=None), dict(dt=None), dict(A=None), dict(M=None),
    dict(y=None), dict(k=at(0) + 8), dict(v=at(2) + 2), dict(dt=at(3) + 1), dict(M=at(7) + 8),
    dict(gate=at(8) + 8), dict(D=at(6) + 4), dict(act=5), dict(y=at(2)), dict(y=at(7)),
    dict(M=at(0)), dict(y=at(8)), dict(M=at(4)),
    dict(shape=dict(B=0)), dict(shape=dict(H=0)), dict(shape=dict(G=3)), dict(shape=dict(G=0)),
    dict(shape=dict(N=0)), dict(shape=dict(N=60)), dict(shape=dict(N=264)),
    dict(shape=dict(d_v=4)), dict(shape=dict(d_v=264)), dict(shape=dict(in_dtype=7)),
    dict(shape=dict(k_stride=64)), dict(shape=dict(v_stride=260)), dict(shape=dict(dt_stride=3)),
    dict(shape=dict(gate_stride=255)), dict(shape=dict(q_stride=-128)),
])
def test_ssm_refuses(sdm, step, bad):
    refused(sdm, 1, ssm(sdm, step, **bad))


@host_only
def test_ssm_refuses_more(sdm):
    refused(sdm, 1, ssm(sdm, init=0))
    refused(sdm, 1, ssm(sdm, shape=dict(T=-1)))
    refused(sdm, 1, ssm(sdm, cu=at(11) + 1))
    # a long prompt of few heads is cut into segments: scratch for the states between them
    long = dict(T=8192)
    need = sdm.sdm_ssm_workspace_size(sdm.SdmSsmShape(2, 8192, 4, 2, 64, 64, 1, 1, 0, 0, 0, 0, 0))
    assert need >= 2 * 2 * 4 * 64 * 64 * 4
    refused(sdm, 1, ssm(sdm, shape=long, ws=None))
    refused(sdm, 1, ssm(sdm, shape=long, ws=at(10) + 16))
    refused(sdm, 1, ssm(sdm, shape=long, ws_bytes=need - 1))
    assert sdm.sdm_ssm_workspace_size(sdm.SdmSsmShape(2, 16, 4, 3, 64, 64, 1, 1, 0, 0, 0, 0,
                                                      0)) == 0


def norm(sdm, **over):
    a = dict(u=at(0), gate=at(1), act=0, post=1, post_gamma=at(2), scale=at(3), r=at(4),
             r_dtype=0, pre_gamma=at(5), eps=1e-6, r_out=at(6), n=at(7), rows=9, D=64, dt=1)
    a.update(over)
    return lambda: sdm.library().sdm_block_norm(*a.values(), None)


@host_only
@pytest.mark.parametrize("bad", [
    dict(u=None), dict(r=None), dict(r_out=None), dict(u=at(0) + 8), dict(gate=at(1) + 2),
    dict(r=at(4) + 4), dict(n=at(7) + 8), dict(post_gamma=at(2) + 4), dict(act=9), dict(eps=-1.0),
    dict(eps=float("nan")), dict(rows=-1), dict(D=60), dict(D=0), dict(D=16392), dict(dt=2),
    dict(r_dtype=-1), dict(r_out=at(0)), dict(r_out=at(4) + 16), dict(n=at(4)), dict(n=at(6)),
    dict(n=at(0) + 16), dict(n=at(1) + 16), dict(r_out=at(5)), dict(n=at(2)),
])
def test_block_norm_refuses(sdm, bad):
    refused(sdm, 1, norm(sdm, **bad))


@host_only
def test_binding_wants_cuda_tensors(sdm):
    x, w = torch.zeros(1, 4, 64), torch.zeros(64, 4)
    with pytest.raises(ValueError):
        sdm.sdm_conv_forward(x, w)
    with pytest.raises(ValueError):
        sdm.sdm_conv_step(x[0], w, torch.zeros(4, 3, 64))
    k = torch.zeros(1, 4, 1, 64)
    with pytest.raises(ValueError):
        sdm.sdm_ssm_forward(k, k, k, k[..., 0, :1], torch.zeros(1), torch.zeros(1, 1, 64, 64))
    with pytest.raises(ValueError):
        sdm.sdm_block_norm(x, x)
