"""Which row layouts the dense-state layer's calls accept, without a GPU: the binding's view of a
tensor's strides, and that a call with rows it cannot describe ends before the library is reached."""

import pytest
import torch

from sparse_memory_linear_b200 import _binding as b

CPU = torch.device("cpu")


def pitch(t, lead):
    return b._pitch(t, "t", t.shape, lead, t.dtype, t.device)


@pytest.mark.parametrize("tail", [(64,), (2, 32), (4, 8), (8,), (1,)])
@pytest.mark.parametrize("B,T", [(4, 100), (2, 2), (1, 7), (7, 1), (3, 1000)])
def test_rows_shared_by_tokens_or_sequences_are_refused(tail, B, T):
    """A tensor broadcast over its tokens, its sequences or both holds fewer rows than a pitch can
    describe: with token stride 0 and B > 1 rows b T + t would be read behind the last one."""
    one = torch.zeros(1, 1, *tail)
    cases = [one.expand(B, T, *tail)]
    if T > 1:
        cases.append(torch.zeros(B, 1, *tail).expand(B, T, *tail))
    if B > 1:
        cases.append(torch.zeros(1, T, *tail).expand(B, T, *tail))
    for t in cases:
        with pytest.raises(ValueError):
            pitch(t, 2)
    # packed rows, and the rows of a step
    with pytest.raises(ValueError):
        pitch(torch.zeros(1, *tail).expand(B * T, *tail), 1)


def test_rows_that_a_pitch_describes():
    row = torch.zeros(3, 5, 96)
    assert pitch(row, 2) == 0
    assert pitch(row[..., 8:72], 2) == 96
    assert pitch(row[..., 8:72].unflatten(-1, (2, 32)), 2) == 96
    assert pitch(row[:, 2, 8:72], 1) == 5 * 96       # a token of each sequence
    assert pitch(row[:, 2:3, 8:72], 2) == 5 * 96
    assert pitch(row[1:2, :, 8:72], 2) == 96
    assert pitch(row[1:2, 2:3, 8:72], 2) == 0        # one row
    for t, lead in ((row.transpose(0, 1), 2), (row[:, :4], 2), (row[..., ::2], 2),
                    (torch.zeros(4096).as_strided((3, 5, 96), (5 * 64, 64, 1)), 2),
                    (torch.zeros(4096).as_strided((3, 5, 96), (96, 3 * 96, 1)), 2)):
        with pytest.raises(ValueError):
            pitch(t, lead)


@pytest.fixture
def calls(monkeypatch):
    """The calls on CPU tensors up to the library, with a list of what would have reached it."""
    made = []
    monkeypatch.setattr(b, "_cuda", lambda t, name: (t.device, t.dtype))
    monkeypatch.setattr(b, "_call", lambda name, dev, *args: made.append(name))
    monkeypatch.setattr(b, "_ssm_scratch", lambda *fields: 0)
    return made


def test_calls_refuse_broadcast_rows(calls):
    B, T, H, G, N, P = 4, 100, 8, 2, 32, 16
    i = dict(k=torch.zeros(B, T, G, N), q=torch.zeros(B, T, G, N), v=torch.zeros(B, T, H, P),
             dt=torch.zeros(B, T, H), gate=torch.zeros(B, T, H, P))
    rest = dict(A=torch.zeros(H), M=torch.zeros(B, H, N, P))
    b.sdm_ssm_forward(**i, **rest)
    assert calls == ["sdm_ssm_forward"]
    for name, t in i.items():
        for shared in (t[:, :1], t[:1], t[:1, :1]):
            with pytest.raises(ValueError):
                b.sdm_ssm_forward(**{**i, name: shared.expand(t.shape)}, **rest)
    x, w = torch.zeros(B, T, 64), torch.zeros(64, 4)
    b.sdm_conv_forward(x, w)
    assert calls == ["sdm_ssm_forward", "sdm_conv_forward"]
    for shared in (x[:, :1], x[:1], x[:1, :1]):
        with pytest.raises(ValueError):
            b.sdm_conv_forward(shared.expand(x.shape), w)
    with pytest.raises(ValueError):
        b.sdm_conv_step(x[:1, 0].expand(B, 64), w, torch.zeros(B, 3, 64))
    assert len(calls) == 2
