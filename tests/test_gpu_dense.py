"""The dense-state layer's operators on the GPU (sdm_conv_*, sdm_ssm_*, sdm_block_norm) against
plain 64-bit implementations (tests/_dense.py), within bounds derived there; odd and ragged
sizes, packed batches with empty and single-token sequences, pitched rows, values that a
sequence must not see, and a whole layer run for prompts and single tokens."""

import pytest
import torch

from tests import _dense as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# a token's weight in another token's read may be held in bf16 (half a step 2^-8), and so
# may the kept state that a block reads, as two bf16 parts (2^-16)
WEIGHTS = {"bf16": 2.0 ** -8 + 2.0 ** -16, "f32": 0.0}


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


def pitched(t, lead, extra):
    """The same values in rows that are `extra` elements further apart, NaN in between."""
    flat = t.reshape((-1,) + t.shape[lead:]).flatten(1)
    big = torch.full((flat.shape[0], flat.shape[1] + extra), float("nan"), dtype=t.dtype,
                     device=t.device)
    big[:, :flat.shape[1]] = flat
    return big[:, :flat.shape[1]].unflatten(1, t.shape[lead:]).unflatten(0, t.shape[:lead]) \
        if lead > 1 else big[:, :flat.shape[1]].unflatten(1, t.shape[lead:])


def cu_of(lens, at=0):
    cu = [at]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def d64(t):
    return None if t is None else t.double()


# ------------------------------------------------------------------------------ convolution
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,K,init,act,bias", [
    (1, 1, 8, 4, "zero", "silu", True), (2, 2, 8, 4, "continue", "silu", True),
    (3, 3, 72, 4, "continue", "identity", False), (1, 16, 136, 2, "zero", "sigmoid", True),
    (5, 17, 1280, 3, "continue", "silu", True), (2, 63, 264, 4, "zero", "silu", False),
    (2, 333, 64, 4, "continue", "silu", True), (40, 1, 520, 4, "continue", "silu", True),
])
def test_conv_batches(sdm, dt, B, T, C, K, init, act, bias):
    g = gen(B * 1000 + T)
    t = TYPES[dt]
    x, w = randn(g, B, T, C, dtype=t), randn(g, C, K)
    b = randn(g, C) if bias else None
    state = randn(g, B, K - 1, C, dtype=t)
    s0 = d64(state) if init == "continue" else torch.zeros(B, K - 1, C, device=DEV).double()
    y = sdm.sdm_conv_forward(x, w, state, bias=b, init=init, act=act)
    ry, rs, bound = ref.conv(d64(x).flatten(0, 1), d64(w), d64(b), s0, act, [T] * B)
    ref.check(y.flatten(0, 1), ry, bound, "y")
    assert torch.equal(state.double(), rs)
    # pitched rows, and without a kept state, give the same bits
    y2 = sdm.sdm_conv_forward(pitched(x, 2, 24), w, None if init == "zero" else rs.to(t), bias=b,
                              init="zero", act=act)
    if init == "zero":
        assert torch.equal(y, y2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[5, 0, 1, 30, 2, 0, 0, 16], [0, 0, 0], [1] * 37,
                                  [15, 1, 1, 1, 1, 15], [0, 100, 3, 64, 0], [2, 2, 2, 200, 0]])
@pytest.mark.parametrize("init", ["zero", "continue"])
def test_conv_packed(sdm, dt, lens, init):
    """Empty and single-token sequences, sequences that begin next to a thread's last row, rows
    before and behind the sequences (NaN, and left as they were in y)."""
    t, C, K, B = TYPES[dt], 40, 4, len(lens)
    g = gen(sum(lens) + B)
    n, before, behind = sum(lens), 3, 5
    x = torch.full((before + n + behind, C), float("nan"), dtype=t, device=DEV)
    x[before:before + n] = randn(g, n, C, dtype=t)
    w, b = randn(g, C, K), randn(g, C)
    state = randn(g, B, K - 1, C, dtype=t)
    s0 = d64(state) if init == "continue" else torch.zeros_like(d64(state))
    y = torch.full_like(x, 7.0)
    sdm.sdm_conv_forward(x, w, state, bias=b, init=init, cu=cu_of(lens, before), y=y)
    ry, rs, bound = ref.conv(d64(x[before:before + n]), d64(w), d64(b), s0, "silu", lens)
    ref.check(y[before:before + n], ry, bound, "y")
    assert torch.equal(state.double(), rs)
    assert (y[:before] == 7).all() and (y[before + n:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,C,K", [(1, 8, 2), (3, 200, 3), (65, 1288, 4)])
def test_conv_step_continues_a_prompt_bit_for_bit(sdm, dt, B, C, K):
    t = TYPES[dt]
    g = gen(B + C)
    T = 9
    x, w, b = randn(g, B, T, C, dtype=t), randn(g, C, K), randn(g, C)
    whole = torch.zeros(B, K - 1, C, dtype=t, device=DEV)
    y = sdm.sdm_conv_forward(x, w, whole, bias=b)
    state = torch.empty_like(whole)
    ys = [sdm.sdm_conv_forward(x[:, :4].contiguous(), w, state, bias=b)]
    for i in range(4, T):
        ys.append(sdm.sdm_conv_step(x[:, i], w, state, bias=b)[:, None])
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(state, whole)


def test_conv_neighbours_do_not_mix(sdm):
    """A sequence of NaN and infinity next to others changes no bit of theirs."""
    g = gen(3)
    lens = [20, 33, 7]
    x, w = randn(g, 60, 64, dtype=torch.bfloat16), randn(g, 64, 4)
    y = sdm.sdm_conv_forward(x, w, cu=cu_of(lens))
    x2 = x.clone()
    x2[20:53] = float("nan")
    x2[30:40] = float("inf")
    y2 = sdm.sdm_conv_forward(x2, w, cu=cu_of(lens))
    assert torch.equal(y[:20], y2[:20]) and torch.equal(y[53:], y2[53:])


# ------------------------------------------------------------------------------------- scan
def ssm_inputs(g, lead, H, G, N, P, t, gate, D, B, dt_by=1.0):
    i = dict(k=randn(g, *lead, G, N, dtype=t, by=0.5), q=randn(g, *lead, G, N, dtype=t, by=0.5),
             v=randn(g, *lead, H, P, dtype=t), dt=randn(g, *lead, H, dtype=t, by=dt_by),
             A=-(0.5 + 15 * torch.rand(H, generator=g, device=DEV)),
             dt_bias=randn(g, H, by=0.5) - 3.0,
             D=randn(g, H) if D else None,
             gate=randn(g, *lead, H, P, dtype=t) if gate else None)
    return i, randn(g, B, H, N, P)


def ssm_ref(i, M, lens, dt, softplus=True, act="silu"):
    flat = {n: d64(x).reshape((-1,) + x.shape[-1 if n == "dt" else -2:]) for n, x in i.items()
            if n in ("k", "q", "v", "dt", "gate") and x is not None}
    return ref.ssm(flat["k"], flat["q"], flat["v"], flat["dt"], d64(i["A"]), M, d64(i["D"]),
                   d64(i["dt_bias"]), softplus, flat.get("gate"), act, lens,
                   weights=WEIGHTS[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,G,N,P,init,gate,D", [
    (1, 1, 1, 1, 8, 8, "zero", False, False), (2, 3, 2, 1, 16, 32, "continue", True, True),
    (1, 127, 3, 3, 128, 64, "zero", True, True), (2, 128, 2, 1, 128, 64, "continue", False, True),
    (1, 129, 4, 2, 64, 64, "continue", True, False), (2, 300, 2, 2, 72, 48, "zero", True, True),
    (1, 257, 2, 1, 128, 128, "continue", True, True), (1, 200, 2, 1, 256, 256, "zero", False, True),
    (3, 140, 2, 1, 24, 80, "continue", True, True), (1, 1000, 2, 1, 128, 64, "continue", False,
                                                     False),
    (1, 400, 1, 1, 136, 64, "continue", True, True), (2, 513, 1, 1, 40, 136, "zero", False, False),
])
def test_ssm_batches(sdm, dt, B, T, H, G, N, P, init, gate, D):
    t = TYPES[dt]
    i, M = ssm_inputs(gen(T + N), (B, T), H, G, N, P, t, gate, D, B)
    M0 = d64(M) if init == "continue" else torch.zeros_like(d64(M))
    y = sdm.sdm_ssm_forward(M=M, init=init, **i)
    ry, rM, yb, Mb = ssm_ref(i, M0, [T] * B, dt)
    ref.check(y.reshape(B * T, H, P), ry, yb, "y")
    ref.check(M, rM, Mb, "M")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[5, 0, 1, 130, 128, 0, 0, 16], [0, 0, 0], [1] * 9,
                                  [127, 1, 129], [0, 400, 3, 64, 0], [256, 255, 257]])
@pytest.mark.parametrize("init", ["zero", "continue"])
def test_ssm_packed(sdm, dt, lens, init):
    """Rows in no sequence are NaN on input and stay as they were in y."""
    t, B, H, G, N, P = TYPES[dt], len(lens), 4, 2, 64, 64
    n, before, behind = sum(lens), 3, 5
    i, M = ssm_inputs(gen(n + B), (before + n + behind,), H, G, N, P, t, True, True, B)
    for x in ("k", "q", "v", "dt", "gate"):
        i[x][:before] = float("nan")
        i[x][before + n:] = float("nan")
    M0 = d64(M) if init == "continue" else torch.zeros_like(d64(M))
    y = torch.full_like(i["v"], 7.0)
    sdm.sdm_ssm_forward(M=M, init=init, cu=cu_of(lens, before), y=y, **i)
    own = {x: (z[before:before + n] if x in ("k", "q", "v", "dt", "gate") else z)
           for x, z in i.items()}
    ry, rM, yb, Mb = ssm_ref(own, M0, lens, dt)
    ref.check(y[before:before + n], ry, yb, "y")
    ref.check(M, rM, Mb, "M")
    assert (y[:before] == 7).all() and (y[before + n:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,N,P,init", [
    (1, 5000, 2, 128, 64, "continue"), (2, 2437, 3, 64, 128, "zero"),
    (1, 4096, 1, 16, 40, "continue"), (1, 1500, 1, 200, 24, "continue"),
])
def test_ssm_long(sdm, dt, B, T, H, N, P, init):
    """Prompts that are cut into segments (few heads, many blocks)."""
    i, M = ssm_inputs(gen(T), (B, T), H, 1, N, P, TYPES[dt], True, True, B)
    M0 = d64(M) if init == "continue" else torch.zeros_like(d64(M))
    y = sdm.sdm_ssm_forward(M=M, init=init, **i)
    ry, rM, yb, Mb = ssm_ref(i, M0, [T] * B, dt)
    ref.check(y.reshape(B * T, H, P), ry, yb, "y")
    ref.check(M, rM, Mb, "M")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("init", ["zero", "continue"])
@pytest.mark.parametrize("lens", [[3000, 1, 0, 700, 1280, 128, 129], [0, 6000]])
def test_ssm_long_packed(sdm, dt, lens, init):
    """Packed batches with sequences of several segments next to short and empty ones."""
    B, H, N, P, n = len(lens), 2, 128, 64, sum(lens)
    i, M = ssm_inputs(gen(n), (n + 3,), H, 2, N, P, TYPES[dt], True, True, B)
    M0 = d64(M) if init == "continue" else torch.zeros_like(d64(M))
    y = torch.full_like(i["v"], 7.0)
    sdm.sdm_ssm_forward(M=M, init=init, cu=cu_of(lens), y=y, **i)
    own = {x: (z[:n] if x in ("k", "q", "v", "dt", "gate") else z) for x, z in i.items()}
    ry, rM, yb, Mb = ssm_ref(own, M0, lens, dt)
    ref.check(y[:n], ry, yb, "y")
    ref.check(M, rM, Mb, "M")
    assert (y[n:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ssm_views_of_one_row(sdm, dt):
    """k, q, v, dt and the gate as slices of one projected row give the bits of copies."""
    t, B, T, H, G, N, P = TYPES[dt], 2, 150, 4, 2, 64, 64
    g = gen(9)
    row = randn(g, B, T, 2 * H * P + 2 * G * N + H + 12, dtype=t, by=0.6)
    cut = row.split([H * P, G * N, H * P, G * N, H, 12], -1)
    v, k, z, q = (x.unflatten(-1, (-1, w)) for x, w in zip(cut, (P, N, P, N)))
    A, bias, D = -1 - torch.rand(H, generator=g, device=DEV), randn(g, H) - 2, randn(g, H)
    M, M2 = torch.empty(B, H, N, P, device=DEV), torch.empty(B, H, N, P, device=DEV)
    y = sdm.sdm_ssm_forward(k, q, v, cut[4], A, M, D=D, dt_bias=bias, gate=z)
    c = [x.contiguous() for x in (k, q, v, cut[4])]
    y2 = sdm.sdm_ssm_forward(*c, A, M2, D=D, dt_bias=bias, gate=z.contiguous())
    assert torch.equal(y, y2) and torch.equal(M, M2)
    # and a token of them
    y = sdm.sdm_ssm_step(k[:, 5], q[:, 5], v[:, 5], cut[4][:, 5], A, M, D=D, dt_bias=bias,
                         gate=z[:, 5])
    c = [x[:, 5].contiguous() for x in (k, q, v, cut[4])]
    y2 = sdm.sdm_ssm_step(*c, A, M2, D=D, dt_bias=bias, gate=z[:, 5].contiguous())
    assert torch.equal(y, y2) and torch.equal(M, M2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,N,P,gate,D", [
    (1, 1, 1, 8, 8, False, False), (2, 8, 1, 128, 128, True, True), (3, 4, 2, 64, 64, True, False),
    (5, 3, 3, 72, 80, False, True), (2, 2, 1, 256, 256, True, True), (33, 24, 8, 128, 64, True,
                                                                      True),
])
def test_ssm_step(sdm, dt, B, H, G, N, P, gate, D):
    t = TYPES[dt]
    i, M = ssm_inputs(gen(N + P), (B,), H, G, N, P, t, gate, D, B)
    M0 = d64(M)
    y = sdm.sdm_ssm_step(M=M, **i)
    ry, rM, yb, Mb = ssm_ref(i, M0, [1] * B, dt)
    ref.check(y, ry, yb, "y")
    ref.check(M, rM, Mb, "M")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("init", ["zero", "continue"])
def test_ssm_prompt_of_one_token_equals_the_step(sdm, dt, init):
    B, H, G, N, P = 3, 4, 2, 72, 80
    i, M = ssm_inputs(gen(31), (B, 1), H, G, N, P, TYPES[dt], True, True, B)
    Ms = M.clone() if init == "continue" else torch.zeros_like(M)
    y = sdm.sdm_ssm_forward(M=M, init=init, **i)
    one = {k: (x[:, 0] if k in ("k", "q", "v", "dt", "gate") else x) for k, x in i.items()}
    ys = sdm.sdm_ssm_step(M=Ms, **one)
    assert torch.equal(y[:, 0], ys) and torch.equal(M, Ms)


def test_ssm_more_pieces_than_multiprocessors(sdm):
    """Many (sequence, head) pieces of unequal lengths: each CTA walks several."""
    lens = [300, 40, 0, 129, 700, 25, 128, 64, 1, 511]
    B, H, G, N, P = len(lens), 48, 4, 40, 72
    i, M = ssm_inputs(gen(32), (sum(lens),), H, G, N, P, torch.bfloat16, True, True, B)
    M0 = d64(M)
    y = sdm.sdm_ssm_forward(M=M, init="continue", cu=cu_of(lens), **i)
    ry, rM, yb, Mb = ssm_ref(i, M0, lens, "bf16")
    ref.check(y, ry, yb, "y")
    ref.check(M, rM, Mb, "M")


def test_ssm_repeats_bit_for_bit(sdm):
    """No sum depends on the order in which CTAs run."""
    for lead, cu in (((2, 3000), None), ((3000,), cu_of([2100, 900]))):
        i, M = ssm_inputs(gen(33), lead, 3, 1, 128, 64, torch.bfloat16, True, True, 2)
        Ms = [M.clone() for _ in range(3)]
        ys = [sdm.sdm_ssm_forward(M=m, init="continue", cu=cu, **i) for m in Ms]
        for y, m in zip(ys[1:], Ms[1:]):
            assert torch.equal(y, ys[0]) and torch.equal(m, Ms[0])


@pytest.mark.parametrize("softplus,act", [(False, "identity"), (False, "sigmoid"), (True, "silu")])
def test_ssm_step_sizes(sdm, softplus, act):
    """Step sizes without softplus (negative ones are 0: the token leaves the state as it is),
    large ones that erase the state, tiny ones; A = 0 (no decay) among the heads."""
    B, T, H, N, P = 1, 200, 4, 64, 64
    g = gen(12)
    i, M = ssm_inputs(g, (B, T), H, 1, N, P, torch.bfloat16, True, True, B)
    i["A"][0] = 0.0
    i["dt_bias"] = None if not softplus else i["dt_bias"]
    i["dt"] = (i["dt"] * 0.1).contiguous()
    i["dt"][:, 10] = -3.0
    i["dt"][:, 50:60] = 90.0
    i["dt"][:, 60:] -= 0.05
    i["dt"][0, 100:130, 1] = -80.0
    M0 = d64(M)
    y = sdm.sdm_ssm_forward(M=M, init="continue", softplus=softplus, act=act, **i)
    ry, rM, yb, Mb = ssm_ref(i, M0, [T], "bf16", softplus, act)
    ref.check(y.reshape(T, H, P), ry, yb, "y")
    ref.check(M, rM, Mb, "M")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_far_apart(sdm, dt):
    """Pitched rows that reach past 2^31 elements: the same bits as contiguous rows."""
    t, H, N, P, T, pitch = TYPES[dt], 2, 32, 24, 40, 1 << 26
    i, M = ssm_inputs(gen(42), (1, T), H, 1, N, P, t, False, True, 1)
    far = torch.empty((T, pitch), dtype=t, device="cuda")
    views, at = {}, 0
    for name in ("k", "q", "v", "dt"):
        x = i[name]
        width = x[0, 0].numel()
        far[:, at:at + width] = x.reshape(T, width)
        views[name] = far[:, at:at + width].view((1, T) + x.shape[2:])
        at += (width + 7) // 8 * 8
    M1, M2 = M.clone(), M.clone()
    y1 = sdm.sdm_ssm_forward(M=M1, init="continue", **i)
    y2 = sdm.sdm_ssm_forward(M=M2, init="continue", **{**i, **views})
    assert torch.equal(y1, y2) and torch.equal(M1, M2)
    one = {n: x[0] for n, x in i.items() if n in views}
    rest = {n: x for n, x in i.items() if n not in views}
    B = T  # the same rows as one token of each of T sequences
    M1 = M.expand(B, -1, -1, -1).contiguous()
    M2 = M1.clone()
    y1 = sdm.sdm_ssm_step(M=M1, **one, **rest)
    y2 = sdm.sdm_ssm_step(M=M2, **{n: x[0] for n, x in views.items()}, **rest)
    assert torch.equal(y1, y2) and torch.equal(M1, M2)
    w = torch.randn(P * H, 4, device="cuda")
    x, xf = i["v"].reshape(1, T, -1), views["v"].view(1, T, -1)
    assert torch.equal(sdm.sdm_conv_forward(x, w), sdm.sdm_conv_forward(xf, w))


def test_ssm_large_state(sdm):
    """A batch whose state has more than 2^31 values: its last sequences are as on their own."""
    B, N, P = 33000, 256, 256
    M = torch.zeros((B, 1, N, P), device="cuda")
    for T in (1, 3):
        i, Ms = ssm_inputs(gen(43), (B, T), 1, 1, N, P, torch.bfloat16, False, True, 1)
        M[-1:] = Ms
        y = sdm.sdm_ssm_forward(M=M, init="continue", **i)
        own = {n: (x[-1:].contiguous() if n in ("k", "q", "v", "dt") else x) for n, x in i.items()}
        yo = sdm.sdm_ssm_forward(M=Ms, init="continue", **own)
        assert torch.equal(y[-1:], yo) and torch.equal(M[-1:], Ms)
    M[-1:] = Ms
    one = {n: (x[:, 0].contiguous() if n in ("k", "q", "v", "dt") else x) for n, x in i.items()}
    y = sdm.sdm_ssm_step(M=M, **one)
    own = {n: (x[-1:].contiguous() if n in ("k", "q", "v", "dt") else x) for n, x in one.items()}
    yo = sdm.sdm_ssm_step(M=Ms, **own)
    assert torch.equal(y[-1:], yo) and torch.equal(M[-1:], Ms)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("low", [float("-inf"), "lowest"])
def test_ssm_padding_by_the_step_size(sdm, dt, low):
    """Tokens whose dt is -infinity or the type's lowest value leave the state as it is: left and
    right padding of a batch gives the states of the sequences without it."""
    t, H, N, P = TYPES[dt], 2, 64, 64
    low = torch.finfo(t).min if low == "lowest" else low
    i, M = ssm_inputs(gen(41), (1, 400), H, 1, N, P, t, False, True, 1)
    own = {k: (x[:, 37:300].contiguous() if k in ("k", "q", "v", "dt") and x is not None else x)
           for k, x in i.items()}
    Mo = M.clone()
    yo = sdm.sdm_ssm_forward(M=Mo, init="continue", **own)
    i["dt"][:, :37] = low
    i["dt"][:, 300:] = low
    y = sdm.sdm_ssm_forward(M=M, init="continue", **i)
    # the same terms in other blocks: fp32 rounding of the state, one bf16 weight and y's own
    assert (M - Mo).norm() <= 2e-6 * Mo.norm()
    tol = 4 * 2.0 ** -8 if dt == "bf16" else 2e-6
    assert (y[:, 37:300].float() - yo.float()).norm() <= tol * yo.float().norm()
    assert torch.isfinite(y).all()


def test_ssm_neighbours_do_not_mix(sdm):
    """A sequence of NaN and infinity next to others changes no bit of theirs."""
    lens = [200, 133, 270]
    i, M = ssm_inputs(gen(5), (603,), 2, 1, 128, 64, torch.bfloat16, True, True, 3)
    Ma, Mb = M.clone(), M.clone()
    y = sdm.sdm_ssm_forward(M=Ma, init="continue", cu=cu_of(lens), **i)
    for x in ("k", "q", "v", "dt", "gate"):
        i[x][200:333] = float("nan")
        i[x][250:260] = float("inf")
    Mb[1] = float("inf")
    y2 = sdm.sdm_ssm_forward(M=Mb, init="continue", cu=cu_of(lens), **i)
    assert torch.equal(y[:200], y2[:200]) and torch.equal(y[333:], y2[333:])
    assert torch.equal(Ma[[0, 2]], Mb[[0, 2]])


def test_ssm_bad_offsets_are_reported(sdm):
    """Offsets out of range or not ascending: clamped, reported in the status word, rows in no
    sequence left as they were."""
    i, M = ssm_inputs(gen(6), (40,), 2, 1, 16, 32, torch.bfloat16, False, False, 3)
    x, w = randn(gen(7), 40, 64, dtype=torch.bfloat16), randn(gen(8), 64, 4)
    for cu in ([0, 10, 5, 20], [-7, 3, 9, 20], [0, 10, 20, 999]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        sdm.sdm_ssm_forward(M=M, cu=c, **i)
        assert sdm.sdm_get_device_status() == 4
        y = torch.full_like(x, 7.0)
        sdm.sdm_conv_forward(x, w, cu=c, y=y)
        assert sdm.sdm_get_device_status() == 4
        if max(cu) <= 20:
            assert (y[20:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 64])
def test_ssm_bad_offsets_of_long_sequences(sdm, dt, H):
    """Offsets that make up more rows than there are, in a batch that is cut into segments: every
    access stays in the buffers (canaries around scratch, state and y), and it is reported."""
    T, B, N, P = 3000, 6, 64, 64
    i, _ = ssm_inputs(gen(8), (T,), H, 1, N, P, TYPES[dt], False, False, B)
    for cu in ([0, T, 0, T, 0, T, 0], [0, 2 * T, -5, T, 7, T, T], [T, 0, T, 0, T, 0, T]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        shape = sdm.SdmSsmShape(B, T, H, 1, N, P, 1 if dt == "bf16" else 0, 1, 0, 0, 0, 0, 0)
        need = sdm.sdm_ssm_workspace_size(shape)
        big = torch.full((need + (1 << 22),), 0x5a, dtype=torch.uint8, device=DEV)
        M = torch.full((B + 2, H, N, P), 3.0, device=DEV)
        y = torch.full((T + 256, H, P), 7.0, dtype=TYPES[dt], device=DEV)
        sdm.sdm_ssm_forward(M=M[1:-1], cu=c, y=y[128:-128], ws=big[:need] if need else None, **i)
        assert sdm.sdm_get_device_status() == 4
        assert (big[need:] == 0x5a).all() and (M[0] == 3).all() and (M[-1] == 3).all()
        assert (y[:128] == 7).all() and (y[-128:] == 7).all()


# ------------------------------------------------------------------------------- block norm
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,post,gate,scale,act", [
    (1, 8, True, True, True, "silu"), (5, 64, True, False, False, "silu"),
    (37, 264, False, True, False, "sigmoid"), (300, 520, True, True, True, "silu"),
    (9, 1032, False, False, True, "silu"), (700, 2048, True, True, True, "silu"),
    (17, 4096, True, False, True, "silu"), (3, 8200, True, True, False, "identity"),
    (2, 16384, True, True, True, "silu"),
])
def test_block_norm(sdm, dt, res, rows, D, post, gate, scale, act):
    g = gen(rows + D)
    t = TYPES[dt]
    u, r = randn(g, rows, D, dtype=t, by=2), randn(g, rows, D, dtype=TYPES[res], by=3)
    z = randn(g, rows, D, dtype=t) if gate else None
    pg, sc, qg = (1 + randn(g, D, by=0.2) for _ in range(3))
    sc = sc if scale else None
    if rows > 2:
        u[1] = 0
        r[1] = 0  # a row of zeros stays zero: eps keeps the roots finite
    kw = dict(post_norm=post, post_gamma=pg, gate=z, act=act, scale=sc, pre_gamma=qg, eps=1e-5)
    ro, n = sdm.sdm_block_norm(u, r, **kw)
    rr, rn, re, ne = ref.block_norm(d64(u), d64(r), post, d64(pg), d64(z), act, d64(sc), d64(qg),
                                    1e-5)
    ref.check(ro, rr, re, "r")
    ref.check(n, rn, ne, "n")
    # in place: the residual into itself, the norm into the block's output
    u2, r2 = u.clone(), r.clone()
    sdm.sdm_block_norm(u2, r2, r_out=r2, n=u2, **kw)
    assert torch.equal(r2, ro) and torch.equal(u2, n)
    if gate:
        z2 = z.clone()
        sdm.sdm_block_norm(u, r, n=z2, **{**kw, "gate": z2})
        assert torch.equal(z2, n)
    ro2, none = sdm.sdm_block_norm(u, r, want_n=False, **kw)
    assert none is None and torch.equal(ro2, ro)


def test_block_norm_without_gammas(sdm):
    g = gen(1)
    u, r = randn(g, 6, 96), randn(g, 6, 96)
    ro, n = sdm.sdm_block_norm(u, r)
    rr, rn, re, ne = ref.block_norm(d64(u), d64(r), True, None, None, "silu", None, None, 1e-6)
    ref.check(ro, rr, re, "r")
    ref.check(n, rn, ne, "n")


# ---------------------------------------------------------------------------- used together
def layer(sdm, p, x, r, conv_state, M, cu=None, init="zero", step=False):
    """One dense-state layer: convolution over [v | k | q], scan, norms around the block."""
    H, G, N, P = p["H"], p["G"], p["N"], p["P"]
    if step:
        row = sdm.sdm_conv_step(x["row"], p["w"], conv_state, bias=p["bias"])
    else:
        row = sdm.sdm_conv_forward(x["row"], p["w"], conv_state, bias=p["bias"], cu=cu, init=init)
    v, k, q = row.split([H * P, G * N, G * N], -1)
    args = (k.unflatten(-1, (G, N)), q.unflatten(-1, (G, N)), v.unflatten(-1, (H, P)), x["dt"],
            p["A"], M)
    kw = dict(D=p["D"], dt_bias=p["dt_bias"], gate=x["gate"])
    y = sdm.sdm_ssm_step(*args, **kw) if step else sdm.sdm_ssm_forward(*args, cu=cu, init=init,
                                                                      **kw)
    return sdm.sdm_block_norm(y.flatten(-2), r, post_gamma=p["pg"], scale=p["sc"],
                              pre_gamma=p["qg"])


def layer_setup(seed, lead, H=4, G=2, N=64, P=64):
    g = gen(seed)
    bf = torch.bfloat16
    C = H * P + 2 * G * N
    p = dict(H=H, G=G, N=N, P=P, w=randn(g, C, 4, by=0.5), bias=randn(g, C, by=0.1),
             A=-1 - 15 * torch.rand(H, generator=g, device=DEV), D=randn(g, H),
             dt_bias=randn(g, H) - 3, pg=1 + randn(g, H * P, by=0.1),
             sc=randn(g, H * P, by=0.5), qg=1 + randn(g, H * P, by=0.1))
    x = dict(row=randn(g, *lead, C, dtype=bf), dt=randn(g, *lead, H, dtype=bf),
             gate=randn(g, *lead, H, P, dtype=bf))
    return p, x, randn(g, *lead, H * P)


def test_layer_prompt_then_tokens_matches_the_whole_prompt(sdm):
    """A prompt of 150 tokens and 8 single tokens, against the prompt of 158: both follow the
    same formulas, so each lies within its own bound of the 64-bit layer.  Compared here end
    to end: a bf16 y differs by at most the two roundings and the bf16 weights of the scan, and
    the norm's output by the same relative to the row's norm."""
    B, T, n = 2, 158, 8
    p, x, r = layer_setup(21, (B, T))
    C = x["row"].shape[-1]
    cs, M = torch.empty(B, 3, C, dtype=torch.bfloat16, device=DEV), torch.empty(B, 4, 64, 64,
                                                                              device=DEV)
    r1, n1 = layer(sdm, p, x, r, cs, M)
    cs2, M2 = torch.empty_like(cs), torch.empty_like(M)
    cut = lambda a, b: {k: v[:, a:b].contiguous() for k, v in x.items()}  # noqa: E731
    ra, na = layer(sdm, p, cut(0, T - n), r[:, :T - n].contiguous(), cs2, M2)
    got_r, got_n = [ra], [na]
    for i in range(T - n, T):
        one = {k: v[:, i] for k, v in x.items()}
        ri, ni = layer(sdm, p, one, r[:, i].contiguous(), cs2, M2, step=True)
        got_r.append(ri[:, None])
        got_n.append(ni[:, None])
    assert torch.equal(cs, cs2)
    # the states: fp32 sums of the same terms in another order
    assert (M - M2).norm() <= 2e-6 * M.norm()
    a, b = torch.cat(got_r, 1), r1
    assert (a - b).norm() <= 4 * 2.0 ** -8 * (b - r).norm()
    a, b = torch.cat(got_n, 1).float(), n1.float()
    assert (a - b).norm() <= 4 * 2.0 ** -8 * b.norm()


def test_layer_packed_equals_separate(sdm):
    """A packed batch gives every sequence what it gets alone."""
    lens = [140, 1, 260]
    p, x, r = layer_setup(22, (sum(lens),))
    C = x["row"].shape[-1]
    cs = torch.empty(3, 3, C, dtype=torch.bfloat16, device=DEV)
    M = torch.empty(3, 4, 64, 64, device=DEV)
    rr, nn = layer(sdm, p, x, r, cs, M, cu=cu_of(lens))
    at = 0
    for b, n in enumerate(lens):
        one = {k: v[None, at:at + n].contiguous() for k, v in x.items()}
        cs1, M1 = torch.empty_like(cs[:1]), torch.empty_like(M[:1])
        r1, n1 = layer(sdm, p, one, r[None, at:at + n].contiguous(), cs1, M1)
        assert torch.equal(cs1[0], cs[b])
        assert (M1[0] - M[b]).norm() <= 2e-6 * M[b].norm()
        assert (r1[0] - rr[at:at + n]).norm() <= 4 * 2.0 ** -8 * (rr - r)[at:at + n].norm()
        at += n


def test_layer_in_graphs_and_streams(sdm):
    """The layer captured into two graphs, replayed in turn with new inputs, and on a side
    stream, gives the eager bits."""
    B, T = 2, 200
    p, x, r = layer_setup(23, (B, T))
    C = x["row"].shape[-1]

    def fresh():
        return (torch.empty(B, 3, C, dtype=torch.bfloat16, device=DEV),
                torch.empty(B, 4, 64, 64, device=DEV))

    cs, M = fresh()
    want = layer(sdm, p, x, r, cs, M)
    one = {k: v[:, 3].contiguous() for k, v in x.items()}
    r1 = r[:, 3].contiguous()
    cs_s, M_s = cs.clone(), M.clone()
    want_s = layer(sdm, p, one, r1, cs_s, M_s, step=True)
    torch.cuda.synchronize()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    csb, Mb = fresh()
    with torch.cuda.stream(side):
        got = layer(sdm, p, x, r, csb, Mb)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(Mb, M)

    # the same by a stream argument, a torch stream's and a raw handle
    for handle in (side, side.cuda_stream):
        csb, Mb = fresh()
        side.wait_stream(torch.cuda.current_stream())
        row = sdm.sdm_conv_forward(x["row"], p["w"], csb, bias=p["bias"], stream=handle)
        side.synchronize()
        assert torch.equal(csb, cs)
        H, G, N, P = p["H"], p["G"], p["N"], p["P"]
        v, k, q = row.split([H * P, G * N, G * N], -1)
        y = sdm.sdm_ssm_forward(k.unflatten(-1, (G, N)), q.unflatten(-1, (G, N)),
                                v.unflatten(-1, (H, P)), x["dt"], p["A"], Mb, D=p["D"],
                                dt_bias=p["dt_bias"], gate=x["gate"], stream=handle)
        out = sdm.sdm_block_norm(y.flatten(-2), r, post_gamma=p["pg"], scale=p["sc"],
                                 pre_gamma=p["qg"], stream=handle)
        side.synchronize()
        assert torch.equal(Mb, M) and all(torch.equal(a, b) for a, b in zip(out, want))

    graphs, outs, states = [], [], []
    xs = [{k: torch.zeros_like(v) for k, v in d.items()} for d in (x, one)]
    for which in range(2):
        st = fresh()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = layer(sdm, p, xs[which], (r, r1)[which], *st, step=which == 1)
        graphs.append(gr)
        outs.append(o)
        states.append(st)
    for _ in range(2):
        for which, src in enumerate((x, one)):
            for k in src:
                xs[which][k].copy_(src[k])
        states[1][0].copy_(cs)
        states[1][1].copy_(M)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[0], want))
        assert all(torch.equal(a, b) for a, b in zip(outs[1], want_s))
        assert torch.equal(states[0][1], M) and torch.equal(states[1][1], M_s)


# -------------------------------------------------------------------------------- refusals
def test_binding_refuses(sdm):
    g = gen(2)
    n0 = sdm.sdm_launch_count()
    i, M = ssm_inputs(g, (2, 16), 4, 2, 64, 64, torch.bfloat16, True, True, 2)

    def bad(exc=(ValueError, TypeError, sdm.SdmError), **over):
        with pytest.raises(exc):
            sdm.sdm_ssm_forward(**{**i, "M": M, **over})

    bad(k=i["k"].float())
    bad(k=i["k"][:, :, :, :32])
    bad(q=i["q"][:, :8])
    bad(v=i["v"].transpose(2, 3))
    bad(dt=i["dt"].float())
    bad(A=i["A"][:2])
    bad(A=i["A"].double())
    bad(M=M[:1])
    bad(M=M.to(torch.bfloat16))
    bad(init="m0")
    bad(act="gelu", exc=KeyError)
    bad(k=i["k"][:, :, :1].expand(2, 16, 2, 64))
    bad(v=i["v"][:1].expand(2, 16, 4, 64))
    bad(cu=torch.zeros(3, dtype=torch.int32, device=DEV))
    bad(y=i["v"])            # y over an input
    bad(gate=i["gate"].cpu())
    bad(ws=torch.empty(1, dtype=torch.int32, device=DEV))
    long, M8 = ssm_inputs(g, (2, 8192), 4, 2, 64, 64, torch.bfloat16, False, False, 2)
    with pytest.raises(sdm.SdmError):  # scratch too small for the states between segments
        sdm.sdm_ssm_forward(M=M8, ws=torch.empty(1024, dtype=torch.uint8, device=DEV), **long)
    x, w = randn(g, 2, 9, 64), randn(g, 64, 4)
    for args, kw in (((x, w[:, :3]), dict(init="continue")), ((x.half(), w), {}),
                     ((x, w.to(torch.bfloat16)), {}), ((x, randn(g, 64, 5)), {}),
                     ((x, w, randn(g, 2, 4, 64)), {}), ((x, w), dict(y=x)),
                     ((x[..., :60], w[:60]), {}), ((x[:, :, ::2], w[:32]), {}),
                     ((x[0], w), {})):
        with pytest.raises((ValueError, TypeError, sdm.SdmError)):
            sdm.sdm_conv_forward(*args, **kw)
    u, r = randn(g, 4, 64), randn(g, 4, 64)
    for args, kw in (((u, r[:2]), {}), ((u[:, :60], r[:, :60]), {}), ((u, r), dict(n=r)),
                     ((u, r), dict(r_out=u)), ((u, r), dict(post_gamma=u[0, :8])),
                     ((u, r), dict(eps=-1.0)), ((u.double(), r), {}), ((u.cpu(), r), {})):
        with pytest.raises((ValueError, TypeError, sdm.SdmError)):
            sdm.sdm_block_norm(*args, **kw)
    assert sdm.sdm_launch_count() == n0


def test_nothing_to_do(sdm):
    """T = 0: only the initialisation happens; rows = 0: nothing."""
    bf = torch.bfloat16
    i, M = ssm_inputs(gen(2), (2, 0), 4, 2, 64, 64, bf, False, False, 2)
    keep = M.clone()
    sdm.sdm_ssm_forward(M=M, init="continue", **i)
    assert torch.equal(M, keep)
    sdm.sdm_ssm_forward(M=M, init="zero", **i)
    assert not M.any()
    state = torch.ones(2, 3, 64, device=DEV)
    x, w = torch.empty(2, 0, 64, device=DEV), torch.ones(64, 4, device=DEV)
    sdm.sdm_conv_forward(x, w, state, init="continue")
    assert (state == 1).all()
    sdm.sdm_conv_forward(x, w, state)
    assert not state.any()
    ro, n = sdm.sdm_block_norm(torch.empty(0, 64, device=DEV), torch.empty(0, 64, device=DEV))
    assert ro.shape == n.shape == (0, 64)
