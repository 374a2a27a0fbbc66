"""Measured cases of the dense-state layer's operators: what runs next to the sparse memory pass
in a stack of recurrent layers.

  conv   causal short convolution over the projected channels, for prompts (whole batches and
         packed sequences) and for single tokens (sdm_conv_forward, sdm_conv_step)
  ssm    selective state-space scan, the dense counterpart of the sparse memory pass, for
         prompts and for single tokens (sdm_ssm_forward, sdm_ssm_step)
  norm   norms after and before a block, fused with the block's gate, its residual scale and
         the residual sum (sdm_block_norm)

`own` chooses between the plain form (elementary torch operations in 32 bits, angles and long
sums in 64, rounded once) and the package's calls.  `exact` follows the definitions token by
token in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 128   # tokens of one block of the plain scan: its token-token matrices are BLOCK^2
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the convolution in front of a layer of 8 heads of 128 values, 4 prompts of 8192 tokens
        # (the batch, heads, width and length of the 1.4B-like layer), k, q and v channels as one row
        dict(name="conv prompt 4x8192", op="conv", B=4, T=8192, C=1280, K=4, dtype="bf16",
             act="silu", bias=True, init="zero", packed=False),
        # prompts of unequal lengths packed one after another, continuing from kept states
        dict(name="conv packed 23 seqs", op="conv", B=23, T=20011, C=2568, K=3, dtype="f32",
             act="silu", bias=False, init="continue", packed=True),
        # serving: one token for each of 64 sequences, and a single sequence
        dict(name="conv step 64", op="conv_step", B=64, C=4352, K=4, dtype="bf16", act="silu",
             bias=True),
        dict(name="conv step 1", op="conv_step", B=1, C=1280, K=4, dtype="bf16", act="silu",
             bias=True),
        # the scan of that layer over the same 4 prompts, reading views of the convolution's rows
        dict(name="ssm prompt 4x8192", op="ssm", B=4, T=8192, H=8, G=1, N=128, P=128,
             dtype="bf16", gate=False, skip=True, init="zero", packed=False, views=True),
        # one long prompt with an odd length and a gate
        dict(name="ssm long 1x65437", op="ssm", B=1, T=65437, H=16, G=1, N=128, P=64,
             dtype="bf16", gate=True, skip=True, init="zero", packed=False, views=False),
        # packed ragged prompts on many heads, states kept from earlier calls
        dict(name="ssm packed 23 seqs", op="ssm", B=23, T=9973, H=64, G=8, N=64, P=64,
             dtype="bf16", gate=True, skip=False, init="continue", packed=True, views=True),
        # the small workload's batch, heads, width and length with 32-bit inputs
        dict(name="ssm f32 2x2048", op="ssm", B=2, T=2048, H=4, G=4, N=16, P=64, dtype="f32",
             gate=False, skip=True, init="continue", packed=False, views=False),
        # serving: the state is read and written once per token
        dict(name="ssm step 64x64", op="ssm_step", B=64, H=64, G=8, N=128, P=64, dtype="bf16",
             gate=True, skip=True),
        dict(name="ssm step 1x8", op="ssm_step", B=1, H=8, G=1, N=128, P=128, dtype="bf16",
             gate=False, skip=True),
        # between two blocks of a prompt: 4 x 8192 rows of the layer's channels, 32-bit residual
        dict(name="norm 32768x2048", op="norm", rows=32768, D=2048, dtype="bf16", res="f32",
             post=True, gate=True, scale=True),
        # between two blocks of a decode step: 64 rows
        dict(name="norm 64x4096", op="norm", rows=64, D=4096, dtype="bf16", res="bf16",
             post=True, gate=False, scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "ssm", "ssm", "ssm", "ssm_step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("conv", "conv_step"):
        C = 8 * _log(rng, 8, 640)
        K = rng.choice([2, 3, 4, 4])
        if op == "conv_step":
            return dict(op=op, B=_log(rng, 1, 256), C=C, K=K, dtype=dtype,
                        act=rng.choice(["silu", "identity"]), bias=yes())
        packed = yes()
        T = _log(rng, 1, min(32768, (1 << 25) // C))
        B = rng.randint(1, 40) if packed else _log(rng, 1, max(1, (1 << 25) // (C * T)) if T > 1
                                                   else 64)
        return dict(op=op, B=min(B, 64), T=T, C=C, K=K, dtype=dtype,
                    act=rng.choice(["silu", "identity"]), bias=yes(),
                    init=rng.choice(["zero", "continue"]), packed=packed)
    if op in ("ssm", "ssm_step"):
        G = rng.choice([1, 1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4, 8])
        N = rng.choice([16, 24, 32, 64, 64, 96, 128, 128])
        P = rng.choice([32, 64, 64, 80, 128, 128])
        if op == "ssm_step":
            return dict(op=op, B=_log(rng, 1, min(256, (1 << 25) // (H * N * P))), H=H, G=G, N=N,
                        P=P, dtype=dtype, gate=yes(), skip=yes())
        most = (1 << 25) // (H * P) if dtype == "bf16" else (1 << 22) // (H * P)
        packed = yes()
        T = _log(rng, 1, min(32768, most))
        B = rng.randint(1, 24) if packed else min(16, _log(rng, 1, max(1, most // T)))
        return dict(op=op, B=B, T=T, H=H, G=G, N=N, P=P, dtype=dtype, gate=yes(), skip=yes(),
                    init=rng.choice(["zero", "continue"]), packed=packed, views=yes())
    D = 8 * _log(rng, 8, 1024)
    return dict(op="norm", rows=_log(rng, 1, min(65536, (1 << 26) // D)), D=D, dtype=dtype,
                res=rng.choice(["bf16", "f32"]), post=yes(), gate=yes(), scale=yes())


# ------------------------------------------------------------------------------ the inputs
def _lengths(case):
    """Lengths of a packed batch: unequal, one sequence empty and one of a single token where
    there are enough, all T tokens used."""
    B, T = case["B"], case["T"]
    r = random.Random(1000 * B + T)
    cuts = sorted(r.randint(0, T) for _ in range(B - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    if B >= 4:
        lens[1], lens[0] = 0, lens[0] + lens[1]
        if lens[2] > 1:
            lens[2], lens[0] = 1, lens[0] + lens[2] - 1
    return lens


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    t = TYPES[case["dtype"]]

    def rand(*shape, to=t, by=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * by).to(to)

    f32 = torch.float32
    s = dict(case)
    op = case["op"]
    if op in ("conv", "conv_step"):
        B, C, K = case["B"], case["C"], case["K"]
        lead = (B,) if op == "conv_step" else (case["T"],) if case["packed"] else (B, case["T"])
        s["x"] = rand(*lead, C)
        s["w"] = rand(C, K, to=f32, by=K ** -0.5)
        s["bias_t"] = rand(C, to=f32, by=0.1) if case["bias"] else None
        s["state"] = rand(B, K - 1, C)
        if op == "conv" and case["packed"]:
            s["lens"] = _lengths(case)
            s["cu"] = _cu(s["lens"])
        return s
    if op in ("ssm", "ssm_step"):
        B, H, G, N, P = (case[k] for k in ("B", "H", "G", "N", "P"))
        lead = (B,) if op == "ssm_step" else (case["T"],) if case["packed"] else (B, case["T"])
        if case.get("views"):  # k, q and v are slices of one row, as the convolution leaves them
            row = torch.nn.functional.silu(rand(*lead, H * P + 2 * G * N, to=f32)).to(t)
            s["v"] = row[..., :H * P].unflatten(-1, (H, P))
            s["k"] = row[..., H * P:H * P + G * N].unflatten(-1, (G, N))
            s["q"] = row[..., H * P + G * N:].unflatten(-1, (G, N))
        else:
            s["v"] = rand(*lead, H, P)
            s["k"] = rand(*lead, G, N, by=0.5)
            s["q"] = rand(*lead, G, N, by=0.5)
        s["dt"] = rand(*lead, H)
        # softplus(bias) between 0.001 and 0.1 and decay rates between 1 and 16, as such layers start
        u = torch.rand(H, generator=g, device=DEV)
        step = torch.exp(u * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -(1.0 + 15.0 * torch.rand(H, generator=g, device=DEV))
        s["D"] = rand(H, to=f32) if case["skip"] else None
        s["z"] = rand(*lead, H, P) if case["gate"] else None
        s["M"] = rand(B, H, N, P, to=f32, by=0.3)
        if op == "ssm" and case["packed"]:
            s["lens"] = _lengths(case)
            s["cu"] = _cu(s["lens"])
        return s
    rows, D = case["rows"], case["D"]
    s["u"] = rand(rows, D, by=2.0)
    s["r"] = rand(rows, D, to=TYPES[case["res"]], by=3.0)
    s["z"] = rand(rows, D) if case["gate"] else None
    s["post_gamma"] = 1.0 + rand(D, to=f32, by=0.1) if case["post"] else None
    s["scale_t"] = rand(D, to=f32, by=0.3) if case["scale"] else None
    s["pre_gamma"] = 1.0 + rand(D, to=f32, by=0.1)
    return s


# ------------------------------------------------------------------------- the package's calls
def _own(s):
    import sparse_memory_linear_b200 as sdm
    op = s["op"]
    if op == "conv":
        y = sdm.sdm_conv_forward(s["x"], s["w"], s["state"], bias=s["bias_t"], init=s["init"],
                                 act=s["act"], cu=s.get("cu"))
        return {"y": y, "state": s["state"]}
    if op == "conv_step":
        y = sdm.sdm_conv_step(s["x"], s["w"], s["state"], bias=s["bias_t"], act=s["act"])
        return {"y": y, "state": s["state"]}
    if op == "ssm":
        y = sdm.sdm_ssm_forward(s["k"], s["q"], s["v"], s["dt"], s["A"], s["M"], D=s["D"],
                                dt_bias=s["dt_bias"], gate=s["z"], init=s["init"],
                                cu=s.get("cu"))
        return {"y": y, "M": s["M"]}
    if op == "ssm_step":
        y = sdm.sdm_ssm_step(s["k"], s["q"], s["v"], s["dt"], s["A"], s["M"], D=s["D"],
                             dt_bias=s["dt_bias"], gate=s["z"])
        return {"y": y, "M": s["M"]}
    r, n = sdm.sdm_block_norm(s["u"], s["r"], post_norm=s["post"], post_gamma=s["post_gamma"],
                              gate=s["z"], scale=s["scale_t"], pre_gamma=s["pre_gamma"])
    return {"r": r, "n": n}


# ---------------------------------------------------------------------------- the plain forms
def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _places(s):
    """For a packed batch, padded to its longest sequence: the row of each (sequence, step), and
    whether there is one; and for each row its sequence and step."""
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    step = torch.arange(max(1, max(s["lens"])), device=DEV)
    here = step[None, :] < lens[:, None]
    row = torch.where(here, cu[:-1, None] + step[None, :], torch.zeros_like(cu[:-1, None]))
    at = torch.arange(s["T"], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    return row, here, seq, at - cu[seq]


def _padded(s, x, row, here):
    """[B, longest, ...] rows of a packed tensor, zeros where there is none."""
    w = here.reshape(here.shape + (1,) * (x.dim() - 1))
    return torch.where(w, x[row], torch.zeros((), dtype=x.dtype, device=DEV))


def _plain_conv(s):
    x, K = s["x"].float(), s["K"]
    B = s["B"]
    if s["packed"]:
        row, here, seq, at = _places(s)
        x = _padded(s, x, row, here)
        lens = here.sum(1)
    else:
        lens = torch.full((B,), s["T"], device=DEV)
    old = s["state"].float() if s["init"] == "continue" else torch.zeros_like(s["state"]).float()
    full = torch.cat([old, x], 1)                               # [B, K - 1 + T, C]
    T = x.shape[1]
    y = sum(full[:, j:j + T] * s["w"][:, j] for j in range(K))
    if s["bias_t"] is not None:
        y = y + s["bias_t"]
    if s["act"] == "silu":
        y = _silu(y)
    if s["packed"]:
        y = y[seq, at]
    last = lens[:, None] + torch.arange(K - 1, device=DEV)      # the last K - 1 inputs
    new = torch.gather(full, 1, last[..., None].expand(-1, -1, full.shape[2]))
    s["state"].copy_(new)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _plain_conv_step(s):
    full = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    y = (full * s["w"].t()).sum(1)
    if s["bias_t"] is not None:
        y = y + s["bias_t"]
    if s["act"] == "silu":
        y = _silu(y)
    s["state"].copy_(full[:, 1:])
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _plain_ssm(s):
    """In blocks of BLOCK tokens: inside a block the token-token matrix of decayed inner products,
    between blocks the decayed states."""
    H, G, N, P = s["H"], s["G"], s["N"], s["P"]
    names = ("k", "q", "v", "dt")
    k, q, v, dt = (s[n].float() for n in names)
    dt = _softplus(dt + s["dt_bias"])
    if s["packed"]:
        row, here, seq, at = _places(s)
        k, q, v, dt = (_padded(s, x, row, here) for x in (k, q, v, dt))  # a step of 0 keeps the state
    B, T = dt.shape[:2]
    nb = -(-T // BLOCK)
    more = nb * BLOCK - T

    def blocks(x):
        x = torch.cat([x, torch.zeros((B, more) + x.shape[2:], device=DEV)], 1) if more else x
        return x.reshape((B, nb, BLOCK) + x.shape[2:])

    kb, qb, vb, db = (blocks(x) for x in (k, q, v, dt))
    R = H // G
    sums = torch.cumsum((db * s["A"]).double(), 2)                   # [B, nb, L, H]
    ends = sums[:, :, -1]                                            # [B, nb, H]
    back = torch.exp((ends[:, :, None] - sums)).float() * db         # a token's weight at the block's end
    wv = vb * back[..., None]
    made = torch.einsum("bclgn,bclgrp->bcgrnp", kb, wv.unflatten(3, (G, R)))
    made = made.flatten(2, 3)                                        # [B, nb, H, N, P]
    M0 = s["M"] if s["init"] == "continue" else torch.zeros_like(s["M"])
    made = torch.cat([M0[:, None], made], 1)                         # [B, nb + 1, H, N, P]
    run_ = torch.cat([torch.zeros_like(ends[:, :1]), torch.cumsum(ends, 1)], 1)   # [B, nb + 1, H]
    between = run_[:, :, None] - run_[:, None]                       # [B, to, from, H]
    low = torch.tril(torch.ones(nb + 1, nb + 1, dtype=torch.bool, device=DEV))[None, :, :, None]
    between = torch.exp(torch.where(low, between, torch.full_like(between, -math.inf))).float()
    states = torch.einsum("bijh,bjhnp->bihnp", between, made)        # before each block, and the last
    diff = sums[:, :, :, None] - sums[:, :, None]                    # [B, nb, t, s, H]
    low = torch.tril(torch.ones(BLOCK, BLOCK, dtype=torch.bool, device=DEV))[None, None, :, :, None]
    diff = torch.exp(torch.where(low, diff, torch.full_like(diff, -math.inf)).float())
    qk = torch.einsum("bctgn,bcsgn->bctsg", qb, kb).repeat_interleave(R, 4)
    y = torch.einsum("bctsh,bcshp->bcthp", qk * diff * db[:, :, None], vb)
    on = torch.einsum("bctgn,bcgrnp->bctgrp", qb, states[:, :-1].unflatten(2, (G, R))).flatten(3, 4)
    y = y + on * torch.exp(sums).float()[..., None]
    y = y.reshape(B, nb * BLOCK, H, P)[:, :T]
    if s["packed"]:
        y = y[seq, at]
    if s["D"] is not None:
        y = y + s["D"][:, None] * s["v"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["M"].copy_(states[:, -1])
    return {"y": y.to(s["v"].dtype), "M": s["M"]}


def _plain_ssm_step(s):
    R = s["H"] // s["G"]
    k, q = (s[n].float().repeat_interleave(R, 1) for n in ("k", "q"))
    v = s["v"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    M = s["M"] * torch.exp(dt * s["A"])[..., None, None] + k[..., None] * (dt[..., None] * v)[:, :, None]
    y = (q[..., None] * M).sum(2)
    if s["D"] is not None:
        y = y + s["D"][:, None] * v
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["M"].copy_(M)
    return {"y": y.to(s["v"].dtype), "M": s["M"]}


def _plain_norm(s):
    f = s["u"].float()
    if s["post"]:
        f = f / torch.sqrt((f * f).mean(-1, keepdim=True) + 1e-6) * s["post_gamma"]
    if s["z"] is not None:
        f = f * _silu(s["z"].float())
    if s["scale_t"] is not None:
        f = f * s["scale_t"]
    r = s["r"].float() + f
    n = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6) * s["pre_gamma"]
    return {"r": r.to(s["r"].dtype), "n": n.to(s["u"].dtype)}


def run(state):
    if own:
        return _own(state)
    return {"conv": _plain_conv, "conv_step": _plain_conv_step, "ssm": _plain_ssm,
            "ssm_step": _plain_ssm_step, "norm": _plain_norm}[state["op"]](state)


# ------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: x.double() for k, x in s.items() if torch.is_tensor(x) and x.is_floating_point()}
    sig = torch.sigmoid
    if op == "conv_step":
        win = torch.cat([d["state"], d["x"].unsqueeze(1)], 1)
        y = torch.einsum("bjc,cj->bc", win, d["w"])
        y = y + d["bias_t"] if "bias_t" in d else y
        y = y * sig(y) if case["act"] == "silu" else y
        return {"y": y, "state": win[:, 1:]}
    if op == "conv":
        K, B = case["K"], case["B"]
        x = d["x"] if case["packed"] else d["x"].flatten(0, 1)
        lens = s["lens"] if case["packed"] else [case["T"]] * B
        ys, new, at = [], [], 0
        for b, n in enumerate(lens):
            old = d["state"][b] if case["init"] == "continue" else torch.zeros_like(d["state"][b])
            whole = torch.cat([old, x[at:at + n]])
            y = torch.einsum("tcj,cj->tc", whole.unfold(0, K, 1), d["w"]) if n else whole[:0]
            y = y + d["bias_t"] if "bias_t" in d else y
            ys.append(y * sig(y) if case["act"] == "silu" else y)
            new.append(whole[n:])
            at += n
        y = torch.cat(ys)
        return {"y": y if case["packed"] else y.reshape(B, case["T"], -1), "state": torch.stack(new)}
    if op in ("ssm", "ssm_step"):
        B, H, G, N, P = (case[k] for k in ("B", "H", "G", "N", "P"))
        lens = s["lens"] if case.get("packed") else [case.get("T", 1)] * B
        first = [sum(lens[:b]) for b in range(B)]
        flat = {n: d[n].reshape((-1,) + d[n].shape[-1 if n == "dt" else -2:])
                for n in ("k", "q", "v", "dt")}
        head = torch.arange(H, device=DEV) // (H // G)
        raw = flat["dt"] + d["dt_bias"]
        step = torch.logaddexp(raw, torch.zeros_like(raw))
        keep = torch.exp(step * d["A"])
        M = d["M"].clone() if op == "ssm_step" or case["init"] == "continue" else torch.zeros_like(d["M"])
        y = torch.zeros_like(flat["v"])
        order = sorted(range(B), key=lambda b: -lens[b])            # those still running come first
        M = M[order]
        starts = torch.tensor([first[b] for b in order], device=DEV)
        for t in range(max(lens)):
            n = sum(m > t for m in lens)
            i = starts[:n] + t
            M[:n] *= keep[i][:, :, None, None]
            M[:n] += flat["k"][i][:, head][..., None] * (step[i][..., None] * flat["v"][i])[:, :, None]
            y[i] = torch.matmul(flat["q"][i][:, head].unsqueeze(2), M[:n]).squeeze(2)
        back = torch.empty_like(M)
        back[order] = M
        y = y.reshape(d["v"].shape)
        if "D" in d:
            y = y + d["D"][:, None] * d["v"]
        if "z" in d:
            y = y * d["z"] * sig(d["z"])
        return {"y": y, "M": back}
    f = d["u"]
    if case["post"]:
        f = f * torch.rsqrt(f.square().mean(1, keepdim=True) + 1e-6) * d["post_gamma"]
    f = f * d["z"] * sig(d["z"]) if "z" in d else f
    f = f * d["scale_t"] if "scale_t" in d else f
    r = d["r"] + f
    return {"r": r, "n": r * torch.rsqrt(r.square().mean(1, keepdim=True) + 1e-6) * d["pre_gamma"]}


# -------------------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("conv", "conv_step"):
        B, C, K = case["B"], case["C"], case["K"]
        rows = B if op == "conv_step" else case["T"] if case["packed"] else B * case["T"]
        kept = B * (K - 1) * C * e
        read = kept if op == "conv_step" or case["init"] == "continue" else 0
        par = C * K * 4 + (C * 4 if case["bias"] else 0)
        return {"bytes": 2 * rows * C * e + read + kept + par, "flops": rows * C * (2 * K + 4)}
    if op in ("ssm", "ssm_step"):
        B, H, G, N, P = (case[k] for k in ("B", "H", "G", "N", "P"))
        rows = B if op == "ssm_step" else case["T"] if case["packed"] else B * case["T"]
        state = B * H * N * P * 4
        read = state if op == "ssm_step" or case["init"] == "continue" else 0
        row = (2 + (1 if case["gate"] else 0)) * H * P * e + 2 * G * N * e + H * e
        # per token and head: decay, rank-one update and read of an N x P state
        return {"bytes": rows * row + read + state + 12 * H, "flops": rows * H * 5 * N * P}
    rows, D = case["rows"], case["D"]
    re = 2 if case["res"] == "bf16" else 4
    cols = 4 * D * (1 + (1 if case["post"] else 0) + (1 if case["scale"] else 0))
    return {"bytes": rows * D * ((2 + (1 if case["gate"] else 0)) * e + 2 * re) + cols,
            "flops": rows * D * 14}
