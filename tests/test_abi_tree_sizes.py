"""CPU check of dspark_tree_attention's workspace: the running tile counts of 1,024 requests, then for every slot of the launch
that the sizes lead to - two a block - rows of head_dim float32 sums and 16 bytes of statistics."""
import os

import pytest

SMS = 148                                                    # what the library takes without a device; with one, its SMs


@pytest.fixture(scope="module")
def ds():
    from dspark_draft_selection_gb300.build import LIB, build
    if not os.path.exists(LIB):
        build()
    import dspark_draft_selection_gb300 as ds
    return ds


@pytest.mark.parametrize("T", [1, 3, 16, 17, 64, 512])
@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 8), (32, 4), (12, 4), (64, 1), (1024, 1)])
@pytest.mark.parametrize("D", [8, 16, 72, 80, 128, 136, 256])
def test_every_partial_result_has_its_place(ds, T, Hq, H, D):
    n = ds.dspark_workspace_size(ds.OP_TREE_ATTENTION, 3, T, Hq * D, H)
    rows = T * Hq // H
    forms = []
    if D <= 128:                                             # tensor cores: one block an SM, row groups of 128 or 256
        forms.append((1, min(rows, 256 if rows > 128 else 128)))
    groups = -(-rows // 64)                                  # float32 arithmetic: even groups of at most 64 rows
    forms.append((2 if D <= 128 else 1, min(rows, -(-rows // (groups * 16)) * 16)))
    for blocks, kept in forms:
        assert n >= 4352 + 2 * blocks * SMS * kept * (D * 4 + 16), (blocks, kept)
    assert ds.dspark_workspace_size(ds.OP_TREE_ATTENTION, 0, T, Hq * D, H) == 0
