"""Which form of the norms' gradients a size takes, seen on the host from the workspace that it asks for: partial
sums of several blocks, or none for few rows (one launch) and for rows that one block holds.
"""
import pytest

import moe_expert_dispatch_amd as moe


@pytest.mark.parametrize("H", [520, 1032, 2048, 2056, 4096, 8192])
def test_one_launch_where_it_takes_no_longer(H):
    for T in (1, 2, 3, 8, 15, 16):
        assert moe.norm_backward_workspace_size(T, H) == 0, T
    for T in (17, 24, 32, 63, 64, 65, 200):   # the columns' blocks would form every row's mean again
        assert moe.norm_backward_workspace_size(T, H) >= 2 * 2 * H * 4, T


def test_rows_wider_than_a_block_and_short_ones():
    for T in (2, 16, 64):
        assert moe.norm_backward_workspace_size(T, 8200) == T * 2 * 8200 * 4
    # short rows: up to 16, 8 or 4 to a block of waves' parts, whose sums need no second launch
    for T, H in ((16, 8), (16, 128), (8, 136), (8, 256), (4, 264), (4, 512)):
        assert moe.norm_backward_workspace_size(T, H) == 0
    assert moe.norm_backward_workspace_size(17, 128) > 0 and moe.norm_backward_workspace_size(64, 512) > 0
