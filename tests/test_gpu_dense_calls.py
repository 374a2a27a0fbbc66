"""How the dense-state layer's calls are made on the GPU: streams by handle, large and small
batches, refusals before any launch."""

import random

import pytest
import torch

from tests import _dense as ref

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


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, by=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * by).to(dtype)


def ssm_inputs(g, lead, H, G, N, P, t, B):
    i = dict(k=randn(g, *lead, G, N, dtype=t, by=0.5), q=randn(g, *lead, G, N, dtype=t, by=0.5),
             v=randn(g, *lead, H, P, dtype=t), dt=randn(g, *lead, H, dtype=t),
             A=-(0.5 + 15 * torch.rand(H, generator=g, device=DEV)),
             dt_bias=randn(g, H, by=0.5) - 3.0, D=randn(g, H))
    return i, randn(g, B, H, N, P)


@pytest.mark.parametrize("side", [False, True])
def test_null_handle_is_the_default_stream(sdm, side):
    """stream=0, the handle of the default stream, orders a call behind that stream's work (whether
    or not it is the current one) and that stream's work behind the call."""
    g = gen(1)
    i, M = ssm_inputs(g, (2, 60), 2, 1, 64, 64, BF, 2)
    x, w = randn(g, 2, 60, 64, dtype=BF), randn(g, 64, 4)
    state, u, r = randn(g, 2, 3, 64, dtype=BF), randn(g, 60, 256, dtype=BF), randn(g, 60, 256)
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0

    def calls(states, **kw):
        Ms, Mt, cs, ct = states
        tok = {n: (t[:, 3] if n in ("k", "q", "v", "dt") else t) for n, t in i.items()}
        return [sdm.sdm_conv_forward(x, w, cs, init="continue", **kw),
                sdm.sdm_conv_step(x[:, 3], w, ct, **kw),
                sdm.sdm_ssm_forward(M=Ms, init="continue", **i, **kw),
                sdm.sdm_ssm_step(M=Mt, **tok, **kw), *sdm.sdm_block_norm(u, r, **kw), *states]

    def states():
        return [M.clone(), M.clone(), state.clone(), state.clone()]

    want = calls(states())
    live = list(i.values()) + [x, u, r]
    kept = [t.clone() for t in live]
    for t in live:
        t.zero_()
    new = states()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream() if side else default):
        with torch.cuda.stream(default):
            torch.cuda._sleep(20_000_000)  # about 10 ms, and only then the inputs
            for t, src in zip(live, kept):
                t.copy_(src)
        got = calls(new, stream=0)
        with torch.cuda.stream(default):
            got = [t.clone() for t in got]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9, 150])
def test_steps_of_size_0_keep_the_state_at_any_decay_rate(sdm, dt, T):
    """A up to the largest finite value: exp(0 A) is 1, for tokens whose dt is -infinity."""
    i, M = ssm_inputs(gen(9), (1, T), 2, 1, 64, 64, BF if dt == "bf16" else torch.float32, 1)
    i["A"] = torch.tensor([-torch.finfo(torch.float32).max, -2.5e38], device=DEV)
    i["dt"][:] = float("-inf")
    keep = M.clone()
    y = sdm.sdm_ssm_forward(M=M, init="continue", **i)
    assert torch.equal(M, keep) and torch.isfinite(y).all()
    one = {n: (t[:, 0] if n in ("k", "q", "v", "dt") else t) for n, t in i.items()}
    ys = sdm.sdm_ssm_step(M=M, **one)
    assert torch.equal(M, keep) and torch.isfinite(ys).all()


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_activations_of_fp32_values(sdm, act):
    """Relative to the result, at large negative arguments too: with e = e^-|x| by expf (2 ulp, 4 U),
    1 + e (U), its reciprocal (1 ulp, 2 U) and two products (2 U) 9 U, and 2 ulp of a denormal e
    times |x| and three roundings of denormals."""
    x = torch.cat([torch.linspace(-95, 95, 40000, device=DEV),
                   randn(gen(3), 960)]).reshape(1, -1, 64).contiguous()
    want = ref.act64(x.double(), act)
    lim = 9 * ref.U * want.abs() + 100 * 2.0 ** -148
    w = torch.zeros(64, 4, device=DEV)
    w[:, 3] = 1.0  # a sum of one term: the activation's argument is exact
    state = torch.zeros(1, 3, 64, device=DEV)
    for y in (sdm.sdm_conv_forward(x, w, act=act),
              sdm.sdm_block_norm(torch.ones_like(x), torch.zeros_like(x), post_norm=False, gate=x,
                                 act=act, want_n=False)[0],
              torch.cat([sdm.sdm_conv_step(x[:, t], w, state, act=act) for t in range(40)], 0)):
        y = y.double().reshape(-1, 64)
        n = y.shape[0]
        err = (y - want.reshape(-1, 64)[:n]).abs()
        assert (err <= lim.reshape(-1, 64)[:n]).all(), (err / lim.reshape(-1, 64)[:n]).max()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_packed_batches_of_many_sequences(sdm, dt):
    """More sequences than the 32 that a warp looks at together and the 256 that a block does, the
    ones that are cut into segments among the first and behind both."""
    g = random.Random(4)
    lens = [g.randint(0, 40) for _ in range(300)]
    lens[5], lens[40], lens[290], lens[299] = 700, 1500, 2600, 0
    B, H, G, N, P, n = len(lens), 2, 1, 32, 24, sum(lens)
    assert n // B >= 24
    t = BF if dt == "bf16" else torch.float32
    i, M = ssm_inputs(gen(5), (n + 7,), H, G, N, P, t, B)
    cu = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    M0, y = M.double(), torch.full_like(i["v"], 7.0)
    sdm.sdm_ssm_forward(M=M, init="continue", cu=cu, y=y, **i)
    f = {k: x.double()[:n] if k in ("k", "q", "v", "dt") else x.double() for k, x in i.items()}
    ry, rM, yb, Mb = ref.ssm(f["k"], f["q"], f["v"], f["dt"], f["A"], M0, f["D"], f["dt_bias"],
                             True, None, "silu", lens,
                             weights=2.0 ** -8 + 2.0 ** -16 if dt == "bf16" else 0.0)
    ref.check(y[:n], ry, yb, "y")
    ref.check(M, rM, Mb, "M")
    assert (y[n:] == 7).all()
    # the convolution of the same rows
    C = H * P
    x, w, state = i["v"].flatten(1)[:n].contiguous(), randn(gen(6), C, 4), \
        randn(gen(7), B, 3, C, dtype=t)
    s0 = state.double()
    yc = sdm.sdm_conv_forward(x, w, state, init="continue", cu=cu)
    rc, rs, bound = ref.conv(x.double(), w.double(), None, s0, "silu", lens)
    ref.check(yc, rc, bound, "y")
    assert torch.equal(state.double(), rs)


@pytest.mark.parametrize("H,G,N,P,lens", [
    (48, 4, 40, 72, [300, 40, 0, 129, 700, 25, 128, 64, 1, 511]), (37, 1, 128, 64, [2048] * 4),
    (3, 1, 128, 200, [5000, 100]),
])
def test_scans_of_many_pieces_repeat_bit_for_bit(sdm, H, G, N, P, lens):
    """Tiles are loaded over the ones before as soon as those are released: a read that came too late
    would give a value of another block now and then."""
    B, n = len(lens), sum(lens)
    i, M = ssm_inputs(gen(11), (n,), H, G, N, P, BF, B)
    cu = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    for gate in (None, randn(gen(12), n, H, P, dtype=BF)):
        first = None
        for _ in range(25):
            Ms = M.clone()
            y = sdm.sdm_ssm_forward(M=Ms, init="continue", cu=cu, gate=gate, **i)
            first = first or (y, Ms)
            assert torch.equal(y, first[0]) and torch.equal(Ms, first[1])
