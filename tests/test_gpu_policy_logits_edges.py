"""tt_policy_loss_logits at the ends of what it takes."""
import math

import numpy as np
import pytest
import torch

from oracle import policy as P
from oracle import token_logprob as TL
from tests.test_gpu_policy import DT, ENT, HOW, _args, _check_logits, _dev, _f64, _inputs, _logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,N,V,ld", [
    ("bf16", 400, 9001, 9003), ("bf16", 40, 4099, 4103), ("bf16", 40, 9001, 9001),  # 1, 2 and 4 CTAs to a row
    ("bf16", 40, 40003, 40007), ("fp32", 20, 20001, 20003), ("fp32", 400, 30001, 30001)])  # 8, 8, 2
def test_masked_rows_among_others_whose_lanes_do_not_end_together(tt, dtype, N, V, ld):
    """Every second row masked, rows of odd lengths at all alignments: a masked row's lanes store different numbers of
    vectors and elements before they wait for the row's other CTAs."""
    rng = np.random.default_rng(V)
    z = _logits(rng, N, V, ld, DT[dtype])
    y = rng.integers(0, V, N)
    s = _inputs(rng, TL.token_logprob(_f64(z), y)[0], True, True, False)
    s["weights"] = np.where(np.arange(N) % 2, 0.75, 0.0).astype(np.float32)
    want = _check_logits(tt, rng, z, s, y)
    pos, kw = _args(s)
    for fill in (math.nan, math.inf):
        z[::2] = fill
        got = tt.policy_loss_logits(z, _dev(y, np.int32), *pos, **kw, entropy_coef=ENT, **HOW)
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and (got[3][::2] == 0).all()


@pytest.mark.parametrize("dtype,tops", [
    ("fp16", [-63968, -64000, -64032, -64480, -64512, -64544, -64768, -64960, -64992, -65024, -65472, -65504, 65504]),
    ("bf16", [-1e29, -1e30, -2e30, -1e36, -9.9e37, -1e38, -1.2e38, -3e38, 1e29, 2e30, 9e35, 1.1e36, 3e38])])
@pytest.mark.parametrize("times,V,weight", [(1, 700, 1.0), (100, 130, 8.0), (100, 5000, 1.0), (1, 12000, 1e6), (1, 40000, 0.5)])
def test_masked_logits_beside_a_far_maximum(tt, dtype, times, V, weight, tops):
    """Rows whose largest logits (four of them, the target among them: log-prob -log 4 exactly) lie near the ends of the
    type's range, with masked logits and lower finite ones (p = 0) beside them. The weight scales the gradient's line."""
    rng = np.random.default_rng(V)
    tops = tops * times
    t, N, weight = DT[dtype], len(tops), min(weight, 1e6 if dtype == "bf16" else 100.0)  # (fp16 gradients end at 65,504)
    z = torch.full((N, V), -math.inf, dtype=t, device="cuda")
    top = torch.tensor(tops, dtype=torch.float64).to(t).cuda()
    at = torch.from_numpy(np.argsort(rng.random((N, V)), axis=1)[:, :5].copy()).cuda()
    y = at[:, 0].cpu().numpy()
    z.scatter_(1, at[:, :4], top[:, None].expand(N, 4))
    lower = (torch.arange(N, device="cuda") % 2 == 1) & (top != torch.finfo(t).min)
    z[lower, at[lower, 4]] = torch.finfo(t).min
    s = _inputs(rng, np.full(N, -math.log(4.0)), True, True, False)
    s["weights"] = np.full(N, weight, np.float32)
    _check_logits(tt, rng, z, s, y)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,V", [(4, 300), (1300, 100), (1300, 5000), (4, 9000), (4, 60000)])
def test_a_bad_target_of_a_row_without_a_distribution(tt, dtype, N, V):
    """The row's log-prob, and with it the loss, is NaN, as with any other row; entropy 0 and dlogits zeros."""
    rng = np.random.default_rng(V)
    z = _logits(rng, N, V, V, DT[dtype])
    z[1:3] = -math.inf
    y = rng.integers(0, V, N)
    for bad in (V, -1, 2 ** 31 - 1, -2 ** 31):
        y[1] = bad
        err = tt.new_err("cuda")
        sums, logp, h, dz = tt.policy_loss_logits(z, _dev(y, np.int32), _dev(np.zeros(N)), _dev(np.ones(N)), err=err)
        assert int(err.item()) == -1 and torch.isnan(sums[:2]).all()
        assert torch.isnan(logp).tolist() == [i == 1 for i in range(N)] and logp[2] == -math.inf
        assert (h[1:3] == 0).all() and (dz[1:3] == 0).all() and torch.isfinite(dz).all()


@pytest.mark.parametrize("N,V", [(400, 64), (1300, 64), (1300, 6000), (400, 9000), (30, 5000), (120, 90000)])
@pytest.mark.parametrize("seed", range(4))
def test_terms_of_both_signs_cancel_and_their_roundings_do_not(tt, N, V, seed):
    """Rows of 2^j equal logits and masked ones: the sum of exponentials is 2^j and the log-prob -j·log 2, so that nothing is
    off but what the objective itself rounds. The policy term's sum is brought down to nearly nothing by one advantage; a ratio
    is within 2^-34, log 2^j and the products add less than twice that, and the sum is rounded once."""
    rng = np.random.default_rng(seed)
    t = [torch.bfloat16, torch.float16, torch.float32][seed % 3]
    j = rng.integers(0, int(math.log2(V)) + 1, N)
    rank = torch.from_numpy(np.argsort(np.argsort(rng.random((N, V)), axis=1), axis=1)).cuda()
    top = torch.from_numpy(rng.integers(-40, 40, N) / 8).cuda()
    z = torch.where(rank < torch.from_numpy(2 ** j).cuda()[:, None], top[:, None], -math.inf).to(t)
    y = (rank == 0).int().argmax(1).int()
    logp = -j * math.log(2.0)
    old = (logp + 0.2 * rng.standard_normal(N)).astype(np.float32)
    old[0] = np.float32(logp[0])
    adv, w = rng.standard_normal(N).astype(np.float32), (rng.integers(1, 17, N) / 16).astype(np.float32)
    how = dict(lo=float(np.float32(0.2)), hi=float(np.float32(0.2)))
    for _ in range(2):  # the first token's ratio is 1, its slope -weight on either side
        adv[0] = np.float32(adv[0] + P.objective(logp, old, adv, weights=w, **how)[0][1] / w[0])
    ref = P.objective(logp, old, adv, weights=w, **how)[0][1]
    size = (w * np.abs(adv.astype(np.float64)) * np.maximum(np.exp(logp - old), 0.8)).sum()
    assert abs(ref) < 1e-4 * size
    sums, got, h, _ = tt.policy_loss_logits(z, y, _dev(old), _dev(adv), weights=_dev(w), clip=0.2)
    assert abs(float(sums[1]) - ref) <= 2.0 ** -24 * abs(ref) + 2.0 ** -32 * size
    assert float(sums[0]) == float(sums[1])
    assert (np.abs(_f64(got) - logp) <= 2.0 ** -23 * np.abs(logp)).all() and (np.abs(_f64(h) + logp) <= 2.0 ** -22 * np.abs(logp)).all()


@pytest.mark.parametrize("dtype,V,ld", [("bf16", 900_000, 900_003), ("fp16", 899_999, 899_999), ("fp32", 450_000, 450_001)])
def test_widest_rows(tt, dtype, V, ld):
    rng = np.random.default_rng(V)
    z = _logits(rng, 5, V, ld, DT[dtype], 0.1)
    ids = np.flatnonzero(np.isfinite(_f64(z[0])))
    y = ids[rng.integers(0, len(ids), 5)]
    s = _inputs(rng, TL.token_logprob(_f64(z), y)[0], True, True, True)
    s["weights"][:3] = [1.0, 0.0, 0.5]
    _check_logits(tt, rng, z, s, y)
