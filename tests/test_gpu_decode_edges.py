"""tt_tree_decode_plan / tt_tree_decode_attn at the ends of what they take."""
import dataclasses

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held,said", [(1, 256), (0, 3), (300, 1), (2, 1000)])
def test_a_plan_of_another_number_of_segments_is_refused(tt, held, said):
    """The header of the plan, not the call, says how many segments there are to read. The buffer has room for both numbers
    and its rest holds bytes that would be a segment of every query."""
    B, rows = 4, 1000
    q, k, v = (torch.randn(s, device="cuda", dtype=torch.bfloat16) for s in ((B, 2, 64), (rows, 1, 64), (rows, 1, 64)))
    room = torch.ones(tt.lib().tt_tree_decode_plan_bytes(max(held, said)) // 4, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0], [3], [0], [B]], dtype=torch.int32, device="cuda").expand(4, held).contiguous()
    plan = tt.tree_decode_plan(table, B, rows, held * B, 2, 1, 64, out=room)
    plan.check()
    out = (torch.full_like(q, 7.0), torch.full((2, B), 7.0, device="cuda"))
    other = dataclasses.replace(plan, S=said, err=tt.new_err("cuda"))
    tt.tree_decode_attn(other, q, k, v, out=out)
    assert int(other.err.item()) == -1 and (out[0] == 7).all() and (out[1] == 7).all()
    tt.tree_decode_attn(plan, q, k, v, out=out)
    plan.check()
    assert (out[0] != 7).all() if held else (out[0] == 0).all()
