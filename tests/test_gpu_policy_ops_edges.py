"""Calls of the policy step at the ends of what they take: inputs that are infinite or tiny, steps too large to count."""
import numpy as np
import pytest
import torch

from oracle import norm_rope as NR
from oracle import policy as P
from oracle import token_logprob as TL
from tests._util import dev_to_f64, rel_l2

pytestmark = pytest.mark.gpu


def test_a_step_whose_work_wraps_64_bits_is_refused(tt):
    """65,536 segments of 2^48 units of work each: their sum is 2^64."""
    S, B, rows = 1 << 16, 1 << 20, (1 << 30) - 1
    table = torch.tensor([[0], [((1 << 23) - 3) * 128], [0], [B]], dtype=torch.int32, device="cuda").expand(4, S).contiguous()
    plan = tt.tree_decode_plan(table, B, rows, 1, 1024, 1024, 64)
    with pytest.raises(tt.TTError) as e:
        plan.check()
    assert e.value.code == -3


@pytest.mark.parametrize("V", [50, 40_000])
def test_infinite_log_probs_of_the_sampler_give_what_the_formulas_give(tt, V):
    rng = np.random.default_rng(V)
    z = rng.standard_normal((5, V)).astype(np.float32)
    y = rng.integers(0, V, 5).astype(np.int32)
    inf = np.inf
    old = np.array([-inf, inf, inf, -12.0, -12.0], np.float32)  # ratios inf, 0, 0
    adv = np.array([1.0, 1.0, -1.0, 0.5, -0.5], np.float32)
    ref = np.array([-12.0, -12.0, -12.0, -inf, -12.0], np.float32)  # e^x − 1 − x = inf, its slope kl
    dev = lambda a: torch.tensor(a, device="cuda")
    sums, logp, h, dz = tt.policy_loss_logits(dev(z), dev(y), dev(old), dev(adv), ref_logp=dev(ref), kl_coef=0.1)
    zd = z.astype(np.float64)
    r_logp, r_h, _, _, _ = TL.token_logprob(zd, y)
    r_sums, r_dl, _ = P.objective(r_logp, old, adv, None, ref, r_h, None, kl=0.1)
    assert np.isfinite(r_dl).all() and r_sums[2] == inf and np.isfinite(r_sums[1])
    got = dev_to_f64(sums)
    # the last token's ratio of some e^8, without an upper bound for its advantage, makes the sum thousands: its rounding
    # to fp32 alone is 2^-24 of it (3.6e-4 of 5978), the ratio's exponential within 2^-22 of it
    near = 5e-5 * max(1.0, abs(r_sums[1]) * 2.0 ** -7)
    assert got[2] == got[0] == inf and abs(got[1] - r_sums[1]) <= near
    r = TL.token_logprob_grad(zd, y, r_dl, np.zeros(5))
    assert np.abs(dev_to_f64(dz) - r).max() <= 1e-5 * max(1.0, np.abs(r).max())
    # and the call on log-probs
    s2, dl2, _ = tt.policy_loss(logp, dev(old), dev(adv), ref_logp=dev(ref), kl_coef=0.1)
    assert np.abs(dev_to_f64(dl2) - r_dl).max() <= 1e-5 * max(1.0, np.abs(r_dl).max())
    assert torch.isinf(s2[0]) and torch.isinf(s2[2]) and abs(float(s2[1]) - r_sums[1]) <= near + 5e-7 * abs(r_sums[1])  # (logp, about 8, is rounded)


@pytest.mark.parametrize("d,dtype", [(64, torch.float32), (62, torch.float32), (128, torch.bfloat16)])
@pytest.mark.parametrize("size", [1e-15, 1e-3, 1e15])
def test_norm_gradients_of_tiny_and_large_heads(tt, d, dtype, size):
    """Without eps the norm does not depend on the size: r³ leaves fp32's range long before r does. fp32: a sum of d
    products is off by less than d·2^-24 of its terms' sizes; bf16 outputs by 2^-8."""
    rng = np.random.default_rng(d)
    x = torch.tensor(rng.standard_normal((9, 3, d)) * size).to(dtype).cuda()
    g = torch.tensor(rng.standard_normal((9, 3, d))).to(dtype).cuda()
    dx, _, dw, _ = tt.qk_norm_rope_bwd(g, None, x, None, None, eps=0.0, rot_dim=0)
    f = lambda t: t.double().cpu().numpy()
    r, rw = NR.backward(f(g), f(x), None, 0.0)
    tol = 1e-5 if dtype == torch.float32 else 2.0 ** -8
    assert rel_l2(f(dx) * size, r * size) <= tol and rel_l2(f(dw), rw) <= 1e-5


def test_nan_keys_reach_the_queries_that_see_them(tt):
    q, k, v = (torch.randn(s, device="cuda", dtype=torch.bfloat16) for s in ((20, 2, 64), (300, 1, 64), (300, 1, 64)))
    k[100] = float("nan")
    table = torch.tensor([[0, 90, 110], [80, 20, 190], [0, 3, 0], [20, 4, 20]], dtype=torch.int32, device="cuda")
    o, lse = tt.tree_decode_attn(tt.tree_decode_plan(table, 20, 300, 41, 2, 1, 64), q, k, v)
    hit = torch.arange(20, device="cuda") == 3
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[:, hit]).all()
    assert torch.isfinite(o[~hit]).all() and torch.isfinite(lse[:, ~hit]).all()


@pytest.mark.parametrize("N", [3000, 100_000])
def test_terms_of_both_signs_cancel_and_their_roundings_do_not(tt, N):
    """The policy term's sum over advantages that add up to nearly nothing: ratios, products and sums are pairs of floats (a
    ratio to 2^-34, with twice that for the rest), so that what is left of the sum is rounded once."""
    rng = np.random.default_rng(N)
    lp = (-rng.exponential(2.0, N)).astype(np.float32)
    old = (lp + 0.2 * rng.standard_normal(N)).astype(np.float32)
    adv = rng.standard_normal(N).astype(np.float32)
    w = np.ones(N, np.float32)
    whole = P.objective(lp, old, adv, None, None, None, w, lo=float(np.float32(0.2)), hi=float(np.float32(0.2)))[0][1]
    r = np.exp(lp.astype(np.float64) - old)
    adv[0] = np.float32(adv[0] + whole / max(1.0, min(r[0], 1.2)))  # nearly nothing is left
    ref = P.objective(lp, old, adv, None, None, None, w, lo=float(np.float32(0.2)), hi=float(np.float32(0.2)))[0][1]
    dev = lambda a: torch.tensor(a, device="cuda")
    sums, _, _ = tt.policy_loss(dev(lp), dev(old), dev(adv), weights=dev(w), clip=0.2)
    size = (np.abs(adv.astype(np.float64)) * np.maximum(r, 0.8)).sum()
    assert abs(float(sums[1]) - ref) <= 2.0 ** -24 * abs(ref) + 2.0 ** -32 * size
    assert abs(ref) < 0.05 * size


@pytest.mark.parametrize("move", [-100.0, -79.5, -20.3, -1.1, -0.3466, -1e-3, 0.0, 3e-5, 0.3466, 0.7, 15.9, 79.9])
def test_ratios_of_all_sizes(tt, move):
    """One token with an unbounded advantage: the term is the ratio itself, or 1 − clip below; from |move| = 80 on its
    exponential is fp32's (2^-22)."""
    lp, old = torch.full((1,), -3.0, device="cuda"), torch.full((1,), -3.0 - move, device="cuda")
    sums, dlogp, _ = tt.policy_loss(lp, old, torch.full((1,), -1.0, device="cuda"), clip=(1.0, 0.2))
    r = np.exp(-3.0 - old.double().item())
    assert abs(float(sums[1]) - r) <= 2.0 ** (-22 if abs(move) >= 79 else -24) * r * 1.001 + (2.0 ** -148 if r < 2.0 ** -126 else 0)
    assert abs(float(dlogp[0]) - r) <= 2.0 ** -22 * r + (2.0 ** -148 if r < 2.0 ** -126 else 0)
