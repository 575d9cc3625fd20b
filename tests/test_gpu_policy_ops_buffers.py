"""Scratch that callers bring to the calls of the policy step: views with gaps are refused, and nothing is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def calls(tt):
    f = lambda *s: torch.randn(*s, device="cuda")
    q, k, v = f(4, 2, 64).bfloat16(), f(50, 1, 64).bfloat16(), f(50, 1, 64).bfloat16()
    table = torch.tensor([[0], [50], [0], [4]], dtype=torch.int32, device="cuda")
    plan = tt.tree_decode_plan(table, 4, 50, 4, 2, 1, 64)
    x, lp, z = f(9, 3, 64), -f(20000).abs(), f(3, 100)
    y = torch.zeros(3, dtype=torch.int32, device="cuda")
    return {"decode": (plan.ws_bytes, lambda ws: tt.tree_decode_attn(plan, q, k, v, ws=ws)),
            "plan": (plan.plan.numel(), lambda out: tt.tree_decode_plan(table, 4, 50, 4, 2, 1, 64, out=out)),
            "norm": (tt.lib().tt_qk_norm_rope_bwd_workspace_bytes(64),
                     lambda ws: tt.qk_norm_rope_bwd(x, None, x, None, None, rot_dim=0, ws=ws)),
            "policy": (tt.lib().tt_policy_loss_workspace_bytes(20000), lambda ws: tt.policy_loss(lp, lp, lp, ws=ws)),
            "logits": (tt.lib().tt_policy_loss_logits_workspace_bytes(3),
                       lambda ws: tt.policy_loss_logits(z, y, z[:, 0].contiguous(), z[:, 1].contiguous(), ws=ws))}


@pytest.mark.parametrize("name", ["decode", "plan", "norm", "policy", "logits"])
def test_scratch_with_gaps_is_refused(calls, name):
    need, call = calls[name]
    rows = -(-need // 16)
    for buf, view in ((torch.full((rows, 48), 7, dtype=torch.uint8, device="cuda"), lambda b: b[:, :16]),
                      (torch.full((16,), 7, dtype=torch.uint8, device="cuda"), lambda b: b.expand(rows, 16))):
        with pytest.raises(ValueError):
            call(view(buf))
        assert (buf == 7).all()
    whole = torch.full((rows * 16 + 16,), 7, dtype=torch.uint8, device="cuda")
    call(whole[:rows * 16])
    assert (whole[rows * 16:] == 7).all()
