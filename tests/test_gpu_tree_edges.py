"""Edges of dspark_tree_attention."""
import pytest
import torch

from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


# --- a wait that ran out ---
@pytest.mark.parametrize("R,ctx,T", [(30, 100, 8), (60, 100, 8), (60, 200, 8), (20, 150, 80), (60, 900, 80)])
def test_a_wait_that_ran_out_leaves_nothing_in_flight(R, ctx, T):
    """Blocks with short shares have every copy under way when their first wait runs out. The calls right behind them, whose
    blocks get the same shared memory, are as ever."""
    import dspark_draft_selection_gb300 as ds
    c = Case(13, T, 4, 2, 128, 16, [ctx] * R, None, mask="chain")
    c.run()
    want, want_lse = c.out.clone(), c.lse.clone()
    lens = torch.tensor(c.ctx, dtype=torch.int32, device="cuda")
    ws, out = ds.workspace(ds.OP_TREE_ATTENTION, R, T, 4 * 128, 2), torch.empty_like(c.out)
    for _ in range(20):
        late, good = ds.new_status(), ds.new_status()
        try:
            ds.dspark_test_set_first_wait_polls(0)
            ds.dspark_tree_attention(c.q, c.k, c.v, c.table, lens, scale=c.scale, out=out, ws=ws, status=late)
        finally:
            ds.dspark_test_set_first_wait_polls(0xFFFFFFFF)
        _, lse, _ = ds.dspark_tree_attention(c.q, c.k, c.v, c.table, lens, scale=c.scale, out=out, ws=ws, status=good)
        assert int(late) == 6 and int(good) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
