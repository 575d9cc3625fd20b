"""tt_policy_loss and tt_policy_loss_logits against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import policy as P
from oracle import token_logprob as TL

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CLIP, DUAL, KL, ENT, G = (0.2, 0.28), 3.0, 0.3, 0.1, 0.7
HOW = dict(clip=CLIP, dual_clip=DUAL, kl_coef=KL, g=G)
ORACLE = dict(lo=CLIP[0], hi=CLIP[1], dual=DUAL, kl=KL, g=G)


def _dev(a, dtype=np.float32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _inputs(rng, logp, two_sided, ref, weights):
    """fp32 inputs around logp, none within 1e-4 of a border of the ratio (the gradient jumps there)."""
    N = len(logp)
    move = 0.3 * rng.standard_normal(N)
    for edge in (math.log1p(-CLIP[0]), math.log1p(CLIP[1]), math.log(DUAL)):
        move = np.where(np.abs(move - edge) < 1e-4, move + 3e-4, move)
    s = {"old": (logp - move).astype(np.float32), "adv": rng.standard_normal(N).astype(np.float32)}
    if two_sided:
        s["adv"], s["adv_neg"] = np.abs(s["adv"]), rng.random(N).astype(np.float32)
    if ref:
        s["ref"] = (logp + 0.2 * rng.standard_normal(N)).astype(np.float32)
    if weights:
        s["weights"] = (rng.integers(0, 5, N) / 4).astype(np.float32)
    return s


def _args(s):
    return (_dev(s["old"]), _dev(s["adv"])), dict(adv_neg=_dev(s.get("adv_neg")), ref_logp=_dev(s.get("ref")),
                                                  weights=_dev(s.get("weights")))


def _oracle(logp, s, **more):
    return P.objective(logp, s["old"], s["adv"], s.get("adv_neg"), s.get("ref"), weights=s.get("weights"), **ORACLE, **more)


def _slope_error(logp, s, err):
    """Error of w·slope·g and of the token's terms, where logp − old and ref − logp are off by err (abs) and e^x by 2^-22:
    the slope's error is r·err·(gain + cost), and of the KL term β·e^x·err."""
    w = np.ones(len(logp)) if "weights" not in s else s["weights"].astype(np.float64)
    r = np.exp(logp - s["old"])
    a = np.abs(s["adv"].astype(np.float64)) + s.get("adv_neg", np.float32(0))
    e = err + 2.0 ** -22
    x = np.exp(np.abs(s["ref"] - logp)) if "ref" in s else 0.0
    return w * (a * r * e + KL * x * e) * 1.01


@pytest.mark.parametrize("two_sided", [False, True])
@pytest.mark.parametrize("ref", [False, True])
@pytest.mark.parametrize("N,shift", [(1, 0), (31, 1), (1024, 0), (1025, 0), (8192, 0), (8193, 0), (8193, 3), (70000, 0)])
def test_from_log_probs(tt, N, shift, ref, two_sided):
    rng = np.random.default_rng(N + shift)
    logp = (-3 * rng.random(N)).astype(np.float32)
    h = rng.random(N).astype(np.float32)
    for weights in (False, True):
        s = _inputs(rng, logp.astype(np.float64), two_sided, ref, weights)
        for entropy in (None, h):
            more = {} if entropy is None else dict(entropy=h.astype(np.float64), ent=ENT)
            want, dlogp, dent = _oracle(logp.astype(np.float64), s, **more)
            pos, kw = _args(s)

            def at(t):  # the same values behind an odd number of elements
                return None if t is None else torch.cat((t.new_zeros(shift), t))[shift:]
            sums, dl, dh = tt.policy_loss(at(_dev(logp)), *map(at, pos), entropy=at(_dev(entropy)),
                                          entropy_coef=0.0 if entropy is None else ENT,
                                          **{n: at(t) for n, t in kw.items()}, **HOW)
            # logp − old in fp32: half a step of at most 4
            err = _slope_error(logp.astype(np.float64), s, 2.0 ** -23)
            assert (np.abs(_f64(dl) - dlogp) <= G * err + 3 * 2.0 ** -24 * np.abs(dlogp) + 1e-30).all()
            if entropy is None:
                assert dh is None
            else:
                assert (np.abs(_f64(dh) - dent) <= 3 * 2.0 ** -24 * np.abs(dent)).all()
            # the terms' errors add up at worst; each has two roundings of its own, and the sums one
            w = np.ones(N) if "weights" not in s else s["weights"]
            size = (w * 8 * (np.abs(s["adv"]) + s.get("adv_neg", 0) + 1)).sum()
            tol = (err / KL).sum() + 2.0 ** -22 * size + 1e-30
            assert (np.abs(_f64(sums) - want) <= tol).all(), (sums, want, tol)


def test_loss_sum_is_tight(tt):
    """The sums' own precision: 500,000 equal terms, exact in fp32, of which an fp32 running sum would lose 1e-3."""
    N = 500_000
    one = torch.ones(N, device="cuda")
    adv = torch.full((N,), 1 + 2.0 ** -20, device="cuda")
    sums, dl, _ = tt.policy_loss(-one, -one, adv)
    assert abs(sums[1].item() + N * (1 + 2.0 ** -20)) <= 2.0 ** -24 * N * 1.01
    assert torch.equal(dl, -adv)


def test_borders_belong_to_the_range(tt):
    """A ratio of exactly 1 with an empty range [1, 1] keeps its slope on both sides; one of exactly dual too."""
    z = torch.zeros(2, device="cuda")
    adv = torch.tensor([2.0, -2.0], device="cuda")
    sums, dl, _ = tt.policy_loss(z, z, adv, clip=0.0)
    assert dl.tolist() == [-2.0, 2.0] and sums[0].item() == 0.0
    sums, dl, _ = tt.policy_loss(z, z, adv, clip=0.5, dual_clip=1.0)
    assert dl.tolist() == [-2.0, 2.0]
    far = torch.tensor([5.0, 5.0, -5.0, -5.0], device="cuda")
    sums, dl, _ = tt.policy_loss(far, torch.zeros(4, device="cuda"), torch.tensor([1.0, -1.0, 1.0, -1.0], device="cuda"),
                                 clip=0.2, dual_clip=2.0)
    assert dl[0] == 0 and dl[1] == 0 and dl[3] == 0 and abs(dl[2].item() + math.exp(-5)) < 1e-8


@pytest.mark.parametrize("N", [40, 9000])
def test_masked_tokens_and_infinities(tt, N):
    """Tokens of weight 0 add nothing whatever they hold; a NaN elsewhere shows in the loss and in its own gradient."""
    rng = np.random.default_rng(1)
    logp = (-rng.random(N)).astype(np.float32)
    s = _inputs(rng, logp.astype(np.float64), True, True, False)
    s["weights"] = np.ones(N, np.float32)
    s["weights"][::3] = 0
    want, dlogp, _ = _oracle(logp.astype(np.float64), s)
    bad = np.resize(np.array([np.nan, np.inf, -np.inf, 3e38], np.float32), len(logp[::3]))
    noisy = {k: v.copy() for k, v in s.items()}
    lp = logp.copy()
    lp[::3] = bad
    for k in ("old", "adv", "adv_neg", "ref"):
        noisy[k][::3] = bad
    pos, kw = _args(noisy)
    sums, dl, _ = tt.policy_loss(_dev(lp), *pos, **kw, **HOW)
    clean = tt.policy_loss(_dev(logp), *_args(s)[0], **_args(s)[1], **HOW)
    assert torch.equal(sums, clean[0]) and torch.equal(dl, clean[1]) and (dl[::3] == 0).all()
    lp[1] = np.nan
    sums, dl, _ = tt.policy_loss(_dev(lp), *pos, **kw, **HOW)
    assert torch.isnan(sums[0]) and torch.isnan(dl[1]) and torch.isfinite(dl[2:]).all()
    # no probability left: the ratio is 0
    sums, dl, _ = tt.policy_loss(_dev([-np.inf]), _dev([-1.0]), _dev([1.0]), clip=0.2)
    assert sums[0] == 0 and dl[0] == 0


def _logits(rng, N, V, ld, t, masked=0.0):
    z = torch.from_numpy((2 * rng.standard_normal((N, ld))).astype(np.float32)).to("cuda").to(t)[:, :V]
    if masked:
        m = rng.random(V) < masked
        m[0] = False
        z[:, torch.from_numpy(m).cuda()] = -math.inf
    return z


def _lp_error(V):
    """Error of logp: an exponential 2^-22 and its argument |d|·(2^-24 + 2^-25 + 2^-24), |d| <= 20 at logits of deviation
    2; a thread adds up at most V/32/2 of a pair's sums in a row (rows up to 2048 by a warp) or 160; joins 2^-21."""
    return 2.0 ** -22 + 20 * 2.5 * 2.0 ** -24 + min(160, V / 64 + 16) * 2.0 ** -24 + 2.0 ** -21


def _check_logits(tt, rng, z, s, y, entropy_coef=ENT, **call):
    t, (N, V) = z.dtype, z.shape
    zf = _f64(z)
    logp, h, lse, _, _ = TL.token_logprob(zf, y)
    want, dlogp, dent = _oracle(logp, s, entropy=h, ent=entropy_coef)
    dz = TL.token_logprob_grad(zf, y, dlogp=dlogp, dentropy=dent)
    pos, kw = _args(s)
    err = tt.new_err("cuda")
    sums, glp, gh, gdz = tt.policy_loss_logits(z, _dev(y, np.int32), *pos, **kw, entropy_coef=entropy_coef, err=err, **HOW,
                                               **call)
    tt.check_err(err)
    on = np.ones(N, bool) if "weights" not in s else s["weights"] != 0
    e = _lp_error(V)
    assert (np.abs(_f64(glp) - np.where(on, logp, 0)) <= e + 2.0 ** -24 * np.abs(logp)).all()
    assert (np.abs(_f64(gh) - np.where(on, h, 0)) <= 4 * e + 2.0 ** -22 * h).all()
    slope = _slope_error(logp, s, e + 2.0 ** -23)
    w = np.ones(N) if "weights" not in s else s["weights"].astype(np.float64)
    size = (w * 8 * (np.abs(s["adv"]) + s.get("adv_neg", 0) + 1 + ENT * h)).sum()
    assert (np.abs(_f64(sums) - want) <= (slope / KL).sum() + (w * 8 * e).sum() + 2.0 ** -22 * size + 1e-30).all()
    if gdz is None:
        return sums, glp, gh, gdz
    lp = zf - lse[:, None]
    p = np.exp(lp)
    lp = np.where(p > 0, lp, 0.0)
    one = np.zeros_like(p)
    one[np.arange(N), y] = 1
    # p: its argument's roundings and log S; the line in log p: its own roundings; the slope's error with both
    line = np.abs(dlogp)[:, None] + np.abs(dent)[:, None] * (np.abs(lp) + h[:, None])
    tol = torch.finfo(t).eps / 2 * np.abs(dz) * (1 + 1e-5) + p * line * (e + 2.0 ** -21 + 4 * np.abs(lp) * 2.0 ** -24) + \
        (p + one) * (G * slope + 3 * 2.0 ** -24 * np.abs(dlogp))[:, None] + \
        p * np.abs(dent)[:, None] * (8 * e) + {torch.float16: 2.0 ** -25}.get(t, 1e-38)
    off = np.abs(_f64(gdz) - dz)
    assert (off <= tol).all(), (off.max(), int((off > tol).sum()))
    return sums, glp, gh, gdz


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,V,pad,masked", [
    (1, 1, 0, 0.0), (1, 5, 3, 0.0), (3, 1000, 0, 0.4), (5, 1003, 0, 0.0), (2, 32003, 61, 0.2), (1300, 1001, 0, 0.0),
    (1300, 130, 6, 0.3), (1300, 7000, 1, 0.0), (700, 8200, 0, 0.0), (61, 40000, 0, 0.0), (1, 151936, 0, 0.0),
    (1400, 16000, 0, 0.0)])
def test_from_logits(tt, dtype, N, V, pad, masked):
    rng = np.random.default_rng(N + V)
    z = _logits(rng, N, V, V + pad, DT[dtype], masked)
    y = rng.integers(0, V, N)
    if masked:
        ids = np.flatnonzero(np.isfinite(_f64(z[0])))
        y = ids[rng.integers(0, len(ids), N)]
    logp = TL.token_logprob(_f64(z), y)[0]
    s = _inputs(rng, logp, N % 2 == 1, V % 2 == 0 or N > 1000, N > 2)
    if N > 2:
        s["weights"][0] = 1.0
    _check_logits(tt, rng, z, s, y)


def test_from_logits_options(tt):
    rng = np.random.default_rng(3)
    z = _logits(rng, 9, 1500, 1500, torch.bfloat16)
    y = rng.integers(0, 1500, 9)
    s = _inputs(rng, TL.token_logprob(_f64(z), y)[0], False, False, True)
    full = _check_logits(tt, rng, z, s, y)
    none = _check_logits(tt, rng, z, s, y, want_dlogits=False)
    assert none[3] is None and all(torch.equal(a, b) for a, b in zip(full[:3], none[:3]))
    _check_logits(tt, rng, z, s, y, entropy_coef=0.0)
    # in place
    pos, kw = _args(s)
    z2 = z.clone()
    out = (torch.empty(4, device="cuda"), torch.empty(9, device="cuda"), torch.empty(9, device="cuda"), z2)
    tt.policy_loss_logits(z2, _dev(y, np.int32), *pos, **kw, entropy_coef=ENT, out=out, **HOW)
    assert all(torch.equal(a, b) for a, b in zip(full, out))
    # another alignment of the gradient than the logits'
    odd = torch.empty(9 * 1500 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(9, 1500)
    out = (*out[:3], odd)
    tt.policy_loss_logits(z, _dev(y, np.int32), *pos, **kw, entropy_coef=ENT, out=out, **HOW)
    assert torch.equal(odd, full[3])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [600, 20000, 60000])
def test_padding_masked_rows_and_neighbours_stay(tt, dtype, V):
    """Rows of weight 0 are not read (NaN there stays there) and get zeros; columns behind V stay as they were."""
    rng = np.random.default_rng(V)
    N, ld = 12, V + 7
    z = _logits(rng, N, V, ld, DT[dtype])
    y = rng.integers(0, V, N)
    s = _inputs(rng, TL.token_logprob(_f64(z), y)[0], True, True, False)
    s["weights"] = np.ones(N, np.float32)
    s["weights"][[0, 5, 11]] = 0
    want = _check_logits(tt, rng, z, s, y)
    z[torch.tensor([0, 5, 11])] = math.nan
    y[5] = -7  # not regarded either
    buf = torch.full((N + 1, ld), 3.0, dtype=z.dtype, device="cuda")
    out = (torch.empty(4, device="cuda"), torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), buf[:N, :V])
    pos, kw = _args(s)
    err = tt.new_err("cuda")
    tt.policy_loss_logits(z, _dev(y, np.int32), *pos, **kw, entropy_coef=ENT, out=out, err=err, **HOW)
    tt.check_err(err)
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert (buf[:N, V:] == 3).all() and (buf[N] == 3).all() and (out[3][5] == 0).all()


@pytest.mark.parametrize("N", [6, 1300])
def test_bad_targets_and_rows(tt, N):
    rng = np.random.default_rng(5)
    V = 900
    z = _logits(rng, N, V, V, torch.bfloat16)
    y = rng.integers(0, V, N)
    s = _inputs(rng, TL.token_logprob(_f64(z), y)[0], False, True, False)
    pos, kw = _args(s)
    ref = tt.policy_loss_logits(z, _dev(y, np.int32), *pos, **kw, entropy_coef=ENT, **HOW)
    y2, z2 = y.copy(), z.clone()
    y2[0], y2[1] = V, -1
    z2[2] = -math.inf
    z2[3, 7] = math.nan
    z2[4, int(y[4])] = -math.inf
    err = tt.new_err("cuda")
    sums, logp, h, dz = tt.policy_loss_logits(z2, _dev(y2, np.int32), *pos, **kw, entropy_coef=ENT, err=err, **HOW)
    assert int(err.item()) == -1 and torch.isnan(sums[0])
    assert torch.isnan(logp[:2]).all() and (dz[:3] == 0).all() and torch.isfinite(h[:2]).all()
    assert logp[2] == -math.inf and h[2] == 0 and logp[4] == -math.inf
    assert torch.isnan(logp[3]) and torch.isnan(h[3]) and torch.isnan(dz[3]).all()
    assert torch.equal(dz[5:], ref[3][5:]) and torch.equal(logp[5:], ref[1][5:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_extreme_rows(tt, dtype):
    """Rows at the type's lowest and highest values, far offsets, and one token far above the rest."""
    t, V, N = DT[dtype], 2000, 5
    low, high = torch.finfo(t).min, torch.finfo(t).max
    rng = np.random.default_rng(6)
    z = _logits(rng, N, V, V, t)
    z[0] = low
    z[1] = high
    z[2, 1:] = low
    z[3] = (z[3].float() + 3000).to(t)
    z[4, 17] = 100.0
    y = np.array([3, 4, 0, 9, 17])
    zf = _f64(z)
    logp, h, _, _, _ = TL.token_logprob(zf, y)
    s = {"old": (logp - 0.1).astype(np.float32), "adv": np.array([1, -1, 1, -1, 1], np.float32)}
    pos, kw = _args(s)
    _, glp, gh, dz = tt.policy_loss_logits(z, _dev(y, np.int32), *pos, **kw, entropy_coef=ENT, **HOW)
    assert (np.abs(_f64(glp) - logp) <= 4e-6).all() and (np.abs(_f64(gh) - h) <= 2e-5).all()
    _, dlogp, dent = P.objective(logp, s["old"], s["adv"], entropy=h, ent=ENT, **ORACLE)
    ref = TL.token_logprob_grad(zf, y, dlogp=dlogp, dentropy=dent)
    assert (np.abs(_f64(dz) - ref) <= torch.finfo(t).eps / 2 * np.abs(ref) * 1.001 + 2e-5 * np.abs(ref).max() + 1e-7).all()


def test_gradient_against_differences_of_the_loss(tt):
    """The kernel's dlogits against central differences of its own loss in fp32 logits: step 2e-2; third derivatives
    below 1 give 1e-4, the loss's rounding 2^-24·4/2e-2 = 2e-5."""
    rng = np.random.default_rng(7)
    N, V = 4, 50
    z = _logits(rng, N, V, V, torch.float32)
    y = rng.integers(0, V, N)
    logp = TL.token_logprob(_f64(z), y)[0]
    s = {"old": (logp - np.array([0.1, 0.1, 1.0, -1.0])).astype(np.float32),
         "adv": np.array([1.0, -1.0, 1.0, -1.0], np.float32), "ref": (logp + 0.3).astype(np.float32)}
    pos, kw = _args(s)
    how = dict(kl_coef=0.5, entropy_coef=0.2, clip=0.2)
    f = lambda x: tt.policy_loss_logits(x, _dev(y, np.int32), *pos, **kw, want_dlogits=False, **how)[0][0].item()
    dz = tt.policy_loss_logits(z, _dev(y, np.int32), *pos, **kw, **how)[3]
    for _ in range(20):
        v = torch.from_numpy(rng.standard_normal((N, V)).astype(np.float32)).cuda()
        v /= v.norm()
        num = (f(z + 2e-2 * v) - f(z - 2e-2 * v)) / 4e-2
        assert abs(num - (dz * v).sum().item()) < 3e-4


def test_streams_graphs_and_repeated_calls(tt):
    rng = np.random.default_rng(8)
    for N, V in ((1300, 700), (40, 20000), (3, 151936)):
        z = _logits(rng, N, V, V, torch.bfloat16)
        y = _dev(rng.integers(0, V, N), np.int32)
        logp = tt.token_logprob(z, y)[0]
        s = _inputs(rng, _f64(logp), True, True, True)
        pos, kw = _args(s)
        calls = [lambda: tt.policy_loss_logits(z, y, *pos, **kw, entropy_coef=ENT, **HOW),
                 lambda: tt.policy_loss(logp, *pos, **kw, **HOW)[:2]]
        long = [torch.cat([t] * 8) if t is not None else None for t in (logp, *pos)]
        calls.append(lambda: tt.policy_loss(long[0], long[1], long[2], **HOW)[:2])
        for call in calls:
            ref = call()
            for _ in range(3):
                assert all(torch.equal(a, b) for a, b in zip(ref, call()))
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                got = call()
            torch.cuda.current_stream().wait_stream(side)
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = call()
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_no_tokens(tt):
    none = torch.zeros(0, device="cuda")
    sums, dl, _ = tt.policy_loss(none, none, none)
    assert (sums == 0).all() and dl.numel() == 0
    sums, lp, h, dz = tt.policy_loss_logits(torch.zeros(0, 8, device="cuda"), none.int(), none, none)
    assert (sums == 0).all() and dz.shape == (0, 8)
