"""Sizes beyond the library's 32-bit ints are refused; their low 32 bits are not taken for them."""
import pytest
import torch

import momentum_delta_rule_mdn_b200 as mdn
from momentum_delta_rule_mdn_b200 import build_lib

BIG = (1 << 32) + 5


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib.build()


@pytest.mark.parametrize("shape", [(1, BIG, 1), (BIG, 1, 1), (1, 1, BIG), (1, (1 << 31) + 1, 1)])
def test_norm_refuses(shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="below 2"):
        mdn.group_norm_fwd(x, 1)
    m = torch.empty(shape[0], 1, device="meta")
    with pytest.raises(ValueError, match="below 2"):
        mdn.group_norm_bwd(x, 1, m, m, x)


def test_workspace_sizes_are_zero():
    assert mdn.group_norm_workspace_size(3, 5, 64, 4) > 0
    assert mdn.gdr_chunk_workspace_size(1, 5, 1, 1, 64) > 0
    for big in (BIG, 1 << 31, -BIG):
        for sizes in ((big, 5, 64, 4), (3, big, 64, 4), (3, 5, big, 1), (3, 5, 64, big)):
            assert mdn.group_norm_workspace_size(*sizes) == 0, sizes
            assert mdn.group_norm_workspace_size(*sizes, backward=True) == 0, sizes
        for sizes in ((big, 5, 1, 1, 64), (1, big, 1, 1, 64), (1, 5, big, big, 64), (1, 5, 1, 1, big)):
            for packed in (False, True):
                assert mdn.gdr_chunk_workspace_size(*sizes, packed=packed) == 0, sizes
