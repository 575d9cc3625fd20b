"""tt_policy_loss_logits at the ends of what it takes."""
import math

import numpy as np
import pytest
import torch

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
