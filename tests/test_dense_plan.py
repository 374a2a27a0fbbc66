"""How the state-space scan is planned, without a GPU: which kernel takes a batch and what scratch
it needs, as far as sdm_ssm_workspace_size shows them (sizes for a B200 where there is no device)."""

import pytest

L = 128       # tokens of a block of the block-wise scan
SUMS = 2176   # bytes of a block's step sizes and decay sums, which only that scan keeps


@pytest.fixture(scope="module")
def sdm():
    from sparse_memory_linear_b200.build import build_library
    build_library()
    import sparse_memory_linear_b200 as m
    m.library()
    return m


def scratch(sdm, B, T, H=1, G=1, N=8, P=8, bf16=True):
    return sdm.sdm_ssm_workspace_size(sdm.SdmSsmShape(B, T, H, G, N, P, 1 if bf16 else 0, 1, 0, 0,
                                                      0, 0, 0))


@pytest.mark.parametrize("B", [1, 2, 1 << 12])
def test_block_wise_scan_keeps_its_row_numbers_in_32_bits(sdm, B):
    """Its last block's rows reach up to 127 rows behind the batch: batches whose rows would leave
    32 bits there are scanned token by token, with 64-bit rows."""
    most = 2 ** 31 - 1 - L
    for rows, blocks in ((most, True), (most + 1, False), (most + L - 1, False),
                         (most + L, False)):
        T = rows // B
        if B > 1 and not blocks:
            T += 1        # B T rows are then past the limit, and the packed reading too small
        got = scratch(sdm, B, T)
        assert (got >= rows // L * SUMS) == blocks, rows


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,T,H,P", [(1024, 8192, 32, 128), (4096, 512, 8, 64), (60000, 30, 4, 32),
                                     (512, 8192, 64, 64)])
def test_scratch_does_not_grow_with_the_states_of_whole_sequences(sdm, bf16, B, T, H, P):
    """Batches with enough sequences to fill the device are not cut into segments; read as packed
    (the size serves both), only sequences of several segments need room for states, two for
    every segment's worth of rows at most.  What is left are the blocks' sums and the items."""
    N = 128
    states = B * H * N * P * 4
    blocks = max(B * -(-T // L), T // L + B + 1) if bf16 else 0
    need = scratch(sdm, B, T, H, 1, N, P, bf16)
    assert need - blocks * H * SUMS - 20 * (blocks + B) <= states / 8
