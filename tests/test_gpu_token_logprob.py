"""tt_token_logprob and tt_token_logprob_bwd against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import token_logprob as TL

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INF = float("inf")


def _logits(x, dtype, ld=None, offset=0):
    """x [N, V] as a CUDA tensor of rows ld apart that starts `offset` elements into its buffer (NaN around it)."""
    N, V = x.shape
    ld = V if ld is None else ld
    buf = torch.full((offset + N * ld,), float("nan"), dtype=DT[dtype], device="cuda")
    z = buf[offset:].view(N, ld)[:, :V]
    z.copy_(torch.from_numpy(np.ascontiguousarray(x, np.float32)))
    return z


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, ref, tol):
    got = _f64(got)
    fin = np.isfinite(ref)
    np.testing.assert_array_equal(got[~fin], ref[~fin])
    off = np.abs(got[fin] - ref[fin])
    assert (off <= np.broadcast_to(tol, ref.shape)[fin]).all(), off.max()


def _check_fwd(tt, z, y, k):
    """Sums of at most 1024 fp32 terms a thread and 2^8 partial sums: 2^10·2^-24 = 6.1e-5 relative at worst; the
    exponentials (ex2 2^-22, argument 2·2^-24·|d| with weight e^d) below 2e-6: S within 7e-5, log S and with it lse
    and log-probs within 1e-4 (lse adds a rounding of its own size). U/S is off by as much relatively, twice."""
    err = tt.new_err("cuda")
    logp, h, lse, ids, top = tt.token_logprob(z, None if y is None else torch.tensor(y, dtype=torch.int32,
                                                                                    device="cuda"), top_k=k, err=err)
    assert int(err.item()) == 0
    r_logp, r_h, r_lse, r_ids, r_top = TL.token_logprob(_f64(z), y, k)
    big = 2.0 ** -23 * np.where(np.isfinite(r_lse), np.abs(r_lse), 0)
    _close(lse, r_lse, 1e-4 + big)
    m = np.where(np.isfinite(_f64(z)), _f64(z), -np.inf).max(1)
    with np.errstate(invalid="ignore"):
        us = np.nan_to_num(r_lse - m - r_h)
    _close(h, r_h, 1e-4 + 1.5e-4 * np.abs(us))
    if y is None:
        assert logp is None
    else:
        _close(logp, r_logp, 1e-4 + 2.0 ** -23 * np.abs(np.where(np.isfinite(r_logp), r_logp, 0)))
    if k:
        np.testing.assert_array_equal(ids.cpu().numpy(), r_ids)
        _close(top, r_top, 1e-4 + 2.0 ** -23 * np.abs(np.where(np.isfinite(r_top), r_top, 0)))
    else:
        assert ids is None and top is None
    return logp, h, lse, ids, top


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,V,k", [(1, 1, 1), (3, 2, 2), (5, 7, 7), (9, 31, 3), (4, 32, 32), (2, 33, 32), (17, 257, 20),
                                   (64, 1000, 8), (33, 2049, 32), (3, 32003, 20), (700, 515, 5), (40, 4096, 1),
                                   (1, 151936, 20), (2, 200003, 32), (20, 30011, 0)])
def test_against_oracle(tt, dtype, N, V, k):
    rng = np.random.default_rng(N * 31 + V)
    x = rng.standard_normal((N, V)) * 2
    y = rng.integers(0, V, N)
    _check_fwd(tt, _logits(x, dtype), y, k)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
@pytest.mark.parametrize("pad", [0, 1, 6, 8])
def test_alignments_and_padded_rows(tt, dtype, offset, pad):
    """Rows that start at every place of a 16-byte block; what lies around the rows is NaN and must not matter."""
    rng = np.random.default_rng(offset * 10 + pad)
    for N, V, k in ((5, 1003, 9), (3, 13, 13), (2, 5, 2)):
        x = rng.standard_normal((N, V)) * 3
        _check_fwd(tt, _logits(x, dtype, V + pad, offset), rng.integers(0, V, N), k)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_ties_go_to_the_lower_index(tt, dtype):
    rng = np.random.default_rng(0)
    N, V = 12, 9001
    x = rng.integers(-2, 3, (N, V)).astype(np.float64)  # five values: thousands of ties
    x[0] = 0.0                                          # one value
    x[1] = np.where(rng.random(V) < 0.5, 0.0, -0.0)     # both zeros are one value
    x[2] = np.sort(x[2])                                # ascending
    x[3] = np.arange(V) // 40                           # ascending in steps: the best come last
    x[4] = -(np.arange(V) // 40)
    x[5, :] = -3.0
    x[5, -3:] = 7.0                                     # the best in the ragged end
    _check_fwd(tt, _logits(x, dtype), rng.integers(0, V, N), 32)
    _check_fwd(tt, _logits(x[:, :1500], dtype), None, 20)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,V,stride", [(4, 40009, 256), (700, 4003, 32)])
def test_best_logits_in_few_places(tt, dtype, N, V, stride):
    """The best logits crowd into a few 16-byte vectors of every `stride`-th, in ascending, descending and random
    order: far more candidates than alternatives."""
    rng = np.random.default_rng(V)
    vn = 4 if dtype == "fp32" else 8
    vec = np.arange(V) // vn
    x = -1.0 - rng.random((N, V))
    crowd = vec % stride < 3
    n = int(crowd.sum())
    for i in range(min(N, 8)):
        v = rng.permutation(n) if i % 3 == 0 else np.arange(n) if i % 3 == 1 else np.arange(n)[::-1]
        x[i, crowd] = v // (1 + i // 3)
    x[N - 1] = -5.0
    x[N - 1, crowd] = 1.0
    _check_fwd(tt, _logits(x, dtype), None, 32)
    _check_fwd(tt, _logits(x[:5], dtype), None, 5)


def test_very_long_rows(tt):
    """More vectors to a slice than 16 bits count, one CTA to a row: ties, and two rows against the oracle."""
    N, V = 153, 530003
    g = torch.Generator(device="cuda").manual_seed(0)
    z = torch.randn(N, V, generator=g, device="cuda").to(torch.bfloat16)
    z[1] = 0.25
    z[1, V - 1] = 0.5
    z[N - 1, 500000:] = 9.0
    logp, h, lse, ids, top = tt.token_logprob(z, top_k=20)
    for r in (0, 1, N - 1):
        _, rh, rl, ri, rt = TL.token_logprob(_f64(z[r:r + 1]), None, 20)
        assert ids[r].tolist() == ri[0].tolist()
        # 2071 terms a thread instead of 1024 (see _check_fwd)
        assert abs(lse[r].item() - rl[0]) <= 2e-4 and np.abs(_f64(top[r]) - rt[0]).max() <= 2e-4
        assert abs(h[r].item() - rh[0]) <= 2e-4 * (1 + abs(rl[0] - z[r].float().max().item() - rh[0]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_masks_and_extremes(tt, dtype):
    rng = np.random.default_rng(1)
    N, V = 12, 3001
    low, high = float(torch.finfo(DT[dtype]).min), float(torch.finfo(DT[dtype]).max)
    x = rng.standard_normal((N, V)) * 2
    x[0] = -INF                          # nothing left
    x[1] = -INF
    x[1, 2000] = 3.0                     # one token left
    x[2, rng.random(V) < 0.9] = -INF
    x[3] = low                           # masked with the type's lowest value throughout: uniform
    x[4] = low
    x[4, 77] = 1.0
    x[5] = low
    x[5, ::2] = -INF
    x[6] = high                          # uniform at the other end
    x[7, 5] = high
    x[8, :1024] = -INF                   # whole vectors and threads masked
    x[9, 1024:] = -INF
    x[10] = 0.0
    x[10, 17] = 80.0                     # one dominant token
    x[11] = np.linspace(-60, 60, V)
    y = np.array([5, 2000, 1, 9, 77, 4, 0, 5, 2000, 3, 17, V - 1])
    x[2, 1] = 0.5
    z = _logits(x, dtype)
    logp, h, lse, ids, top = _check_fwd(tt, z, y, 20)
    assert logp[0] == -INF and lse[0] == -INF and h[0] == 0 and (top[0] == -INF).all()
    assert ids[0].tolist() == list(range(20))
    assert logp[1] == 0 and h[1] == 0


def test_nan_and_infinity(tt):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 700))
    x[0, 13] = np.nan
    x[1, 650] = INF
    x[2] = np.nan
    x[3, 0] = x[3, 699] = INF
    for dtype in DT:
        logp, h, lse, ids, top = tt.token_logprob(_logits(x, dtype), torch.zeros(5, dtype=torch.int32, device="cuda"),
                                                  top_k=4)
        for t in (logp, h, lse, top):
            assert torch.isnan(t[:4]).all() and torch.isfinite(t[4]).all()
        assert ((ids >= 0) & (ids < 700)).all()
        assert ids[1, 0] == 650 and ids[3, :2].tolist() == [0, 699]


def test_bad_targets(tt):
    z = torch.randn(6, 100, device="cuda")
    y = torch.tensor([0, -1, 99, 100, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    err = tt.new_err("cuda")
    logp, h, lse, ids, top = tt.token_logprob(z, y, top_k=2, err=err)
    assert int(err.item()) == -1
    assert torch.isnan(logp).tolist() == [False, True, False, True, False, True]
    assert torch.isfinite(h).all() and torch.isfinite(lse).all() and torch.isfinite(top).all()


def test_repeatable_streams_graphs_and_empty(tt):
    z = torch.randn(77, 5003, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, 5003, (77,), device="cuda", dtype=torch.int32)
    err = tt.new_err("cuda")
    a = tt.token_logprob(z, y, top_k=9, err=err)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = tt.token_logprob(z, y, top_k=9, err=err)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dz = torch.empty_like(z)
    args = dict(dlogp=torch.randn(77, device="cuda"), dentropy=torch.randn(77, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tt.token_logprob(z, y, top_k=9, out=b, err=err)
        tt.token_logprob_bwd(z, b[2], b[1], y, out=dz, err=err, **args)
    z.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    a = tt.token_logprob(z, y, top_k=9)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(dz, tt.token_logprob_bwd(z, a[2], a[1], y, **args))
    e = tt.token_logprob(z[:0], y[:0], top_k=3)
    assert e[0].shape == (0,) and e[3].shape == (0, 3)
    assert tt.token_logprob_bwd(z[:0], e[2]).shape == (0, 5003)


def _check_bwd(tt, z, y, k, seed, inplace=False, terms=("dlogp", "dentropy", "dlse", "dtop"), ids=None):
    rng = np.random.default_rng(seed)
    N, V = z.shape
    dev = dict(device="cuda")
    g = {n: rng.standard_normal(N).astype(np.float32) for n in ("dlogp", "dentropy", "dlse") if n in terms}
    if k and "dtop" in terms:
        g["dtop"] = rng.standard_normal((N, k)).astype(np.float32)
        g["top_ids"] = rng.integers(0, V, (N, k)).astype(np.int32) if ids is None else ids
    z64 = _f64(z)
    _, h, lse, _, _ = tt.token_logprob(z)
    err = tt.new_err("cuda")
    dz = tt.token_logprob_bwd(z, lse, h, torch.tensor(y, dtype=torch.int32, **dev), out=z if inplace else None, err=err,
                              **{n: torch.tensor(v, **dev) for n, v in g.items()})
    assert int(err.item()) == 0 and dz.dtype == z.dtype and dz.stride() == z.stride()
    ref = TL.token_logprob_grad(z64, y, **g)
    # p from an lse within 1e-4 (see _check_fwd) and an exponential within 2e-6: 1.1e-4 relative of each summand
    # p·g; the entropy (within 1e-4 + 1.5e-4·|U/S|, |U/S| < 70 here) enters times p·dentropy; half a step of the
    # output type and its smallest step
    _, rh, rlse, _, _ = TL.token_logprob(z64)
    with np.errstate(invalid="ignore"):
        lp = np.where(np.isfinite(z64), z64 - np.where(np.isfinite(rlse), rlse, 0)[:, None], 0)
        p = np.where(np.isfinite(z64), np.exp(np.minimum(lp, 0)), 0)
    absd = sum(np.abs(g[n]) for n in ("dlogp", "dlse") if n in g) + (np.abs(g["dtop"]).sum(1) if "dtop" in g else 0)
    dh = np.abs(g["dentropy"]) if "dentropy" in g else np.zeros(N)
    add = np.zeros((N, V))
    if "dlogp" in g:
        np.add.at(add, (np.arange(N), y), np.abs(g["dlogp"]))
    if "dtop" in g:
        np.add.at(add, (np.arange(N)[:, None], g["top_ids"]), np.abs(g["dtop"]))
    mx = np.where(np.isfinite(z64), z64, -np.inf).max(1)
    with np.errstate(invalid="ignore"):
        us = np.nan_to_num(rlse - mx - rh)
    tol = 1.1e-4 * p * ((absd + dh * rh)[:, None] + dh[:, None] * np.abs(lp)) \
        + p * (dh * (2e-4 + 1.5e-4 * np.abs(us)))[:, None] + 2.0 ** -20 * add
    tiny = {torch.float16: 2.0 ** -25}.get(z.dtype, 1e-37)
    tol = tol + torch.finfo(z.dtype).eps / 2 * (np.abs(ref) + tol) + tiny
    bad = ~(np.abs(_f64(dz) - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], _f64(dz)[bad][:3], ref[bad][:3])
    return dz


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("N,V,k,pad", [(1, 1, 1, 0), (4, 5, 3, 1), (33, 257, 0, 0), (9, 1000, 8, 24), (5, 32003, 32, 0),
                                       (700, 130, 2, 6), (2, 151936, 5, 0)])
def test_gradient_against_oracle(tt, dtype, inplace, N, V, k, pad):
    rng = np.random.default_rng(N + V)
    z = _logits(rng.standard_normal((N, V)) * 2, dtype, V + pad, offset=pad % 8)
    _check_bwd(tt, z, rng.integers(0, V, N), k, N, inplace)


@pytest.mark.parametrize("terms", [(), ("dlogp",), ("dentropy",), ("dlse",), ("dtop",), ("dlogp", "dentropy")])
def test_gradient_terms(tt, terms):
    rng = np.random.default_rng(4)
    z = _logits(rng.standard_normal((6, 900)) * 2, "fp32")
    dz = _check_bwd(tt, z, rng.integers(0, 900, 6), 4, 5, terms=terms)
    if not terms:
        assert (dz == 0).all()


def test_gradient_repeated_ids(tt):
    """The target among the alternatives, and one id several times: the terms add up."""
    rng = np.random.default_rng(6)
    N, V = 8, 4099
    z = _logits(rng.standard_normal((N, V)), "bf16")
    y = rng.integers(0, V, N)
    ids = np.repeat(y[:, None], 6, 1).astype(np.int32)
    ids[:, 3:5] = (y[:, None] + 1) % V
    ids[:, 5] = V - 1
    _check_bwd(tt, z, y, 6, 7, ids=ids)
    _check_bwd(tt, z, y, 6, 7, inplace=True, ids=ids)


def test_gradient_masks(tt):
    rng = np.random.default_rng(8)
    N, V = 6, 2500
    x = rng.standard_normal((N, V)) * 2
    x[0] = -INF
    x[1] = -INF
    x[1, 100] = 1.0
    x[2, rng.random(V) < 0.8] = -INF
    x[2, 7] = 0.0
    x[3] = -10000.0
    x[3, 50:60] = 0.0
    y = np.array([3, 100, 7, 55, 1, 2])
    for dtype in DT:
        dz = _check_bwd(tt, _logits(x, dtype), y, 3, 9, ids=np.repeat(y[:, None], 3, 1).astype(np.int32))
        assert (dz[0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_gradient_where_lse_is_too_wide_for_fp32(tt, dtype):
    """Rows at the type's lowest or highest value throughout, and rows far from 0: e^(z − lse) with lse rounded to
    fp32 would be off by |lse|·2^-24; in closed form they are uniform, or an ordinary row moved by a constant."""
    N, V = 5, 3001
    low, high = float(torch.finfo(DT[dtype]).min), float(torch.finfo(DT[dtype]).max)
    x = np.full((N, V), low)
    x[1] = high
    x[2] = 4096.0
    x[2, ::3] -= 32.0
    x[3, 1::2] = -INF
    x[4] = np.where(np.arange(V) % 7, -2048.0, -2040.0)
    y = np.arange(N) * 500
    for n in (N, 1):  # N = 1: several CTAs to a row
        z = _logits(x[:n], dtype)
        _, h, lse, _, _ = tt.token_logprob(z)
        d = torch.arange(1, n + 1, dtype=torch.float32, device="cuda")
        dz = _f64(tt.token_logprob_bwd(z, lse, h, torch.tensor(y[:n], dtype=torch.int32, device="cuda"), dlogp=d,
                                       dentropy=d, dlse=d))
        ref = TL.token_logprob_grad(_f64(z), y[:n], _f64(d), _f64(d), _f64(d))
        # p within 1e-4 (its sum, as in _check_fwd), entropy within 1e-4·(1 + |U/S|) <= 1e-3 here
        tol = 1e-3 * _f64(d)[:, None] / V + torch.finfo(DT[dtype]).eps / 2 * np.abs(ref) + 2e-6 * (np.abs(ref) > 0.1)
        tol = tol * 3 + {torch.float16: 2.0 ** -25}.get(DT[dtype], 0)
        assert (np.abs(dz - ref) <= tol).all(), np.abs(dz - ref).max()


def test_gradient_against_differences_of_the_forward(tt):
    """d/dz of Σ a·logp + b·entropy by central differences of the fp32 forward: the forward is within 2e-6 here
    (V = 40), so a step of 0.05 leaves 2e-6·(|a| + |b|)·2/0.1 + O(step²)·third derivative (< 2)/6."""
    rng = np.random.default_rng(11)
    V = 40
    base = torch.tensor(rng.standard_normal(V), dtype=torch.float32, device="cuda")
    y = torch.zeros(2 * V, dtype=torch.int32, device="cuda")
    a, b, step = 1.3, -0.7, 0.05
    pts = torch.cat([base + step * torch.eye(V, device="cuda"), base - step * torch.eye(V, device="cuda")])
    logp, h, _, _, _ = tt.token_logprob(pts, y)
    f = a * logp + b * h
    diff = (f[:V] - f[V:]) / (2 * step)
    _, h0, lse0, _, _ = tt.token_logprob(base[None])
    one = torch.ones(1, device="cuda")
    dz = tt.token_logprob_bwd(base[None], lse0, h0, y[:1], dlogp=a * one, dentropy=b * one)[0]
    assert (dz - diff).abs().max().item() <= 2e-6 * 2 * 20 + step ** 2 * 2 / 6


def test_gradient_bad_ids(tt):
    rng = np.random.default_rng(12)
    z = _logits(rng.standard_normal((3, 200)), "fp32")
    _, h, lse, _, _ = tt.token_logprob(z)
    y = torch.tensor([5, 200, -1], dtype=torch.int32, device="cuda")
    one = torch.ones(3, device="cuda")
    err = tt.new_err("cuda")
    dz = tt.token_logprob_bwd(z, lse, h, y, dlogp=one, err=err)
    assert int(err.item()) == -1
    p = torch.softmax(z, 1)
    p[0, 5] -= 1
    assert (dz + p).abs().max().item() < 1e-5
    ids = torch.tensor([[1, 200], [-7, 3], [2, 2]], dtype=torch.int32, device="cuda")
    err = tt.new_err("cuda")
    tt.token_logprob_bwd(z, lse, h, top_ids=ids, dtop=torch.ones(3, 2, device="cuda"), err=err)
    assert int(err.item()) == -1


def test_offsets_past_32_bits(tt):
    """More than 2^31 logits before the last rows: these equal the same rows alone, forward, backward and in place."""
    N, V = 14_200, 151_936
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    z[-3:] = torch.randn(3, V, device="cuda") * 2
    y = torch.arange(N, dtype=torch.int32, device="cuda")
    g = torch.randn(N, device="cuda")
    last = z[-3:].clone()
    logp, h, lse, ids, top = tt.token_logprob(z, y, top_k=3)
    r_logp, r_h, r_lse, r_ids, r_top = TL.token_logprob(_f64(last), y[-3:].cpu().numpy(), 3)
    _close(logp[-3:], r_logp, 2e-4)
    _close(lse[-3:], r_lse, 2e-4)
    np.testing.assert_array_equal(ids[-3:].cpu().numpy(), r_ids)
    dz = tt.token_logprob_bwd(last, lse[-3:], h[-3:], y[-3:], dlogp=g[-3:], dentropy=g[-3:])
    tt.token_logprob_bwd(z, lse, h, y, dlogp=g, dentropy=g, out=z)
    assert torch.equal(z[-3:], dz)


def test_two_streams_at_once(tt):
    """Calls that overlap share nothing."""
    zs = [torch.randn(200, 20003, device="cuda").to(torch.bfloat16) for _ in range(4)]
    ref = [tt.token_logprob(z, top_k=12) for z in zs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in zs]
    got = [None] * 4
    for _ in range(5):
        for i, (s, z) in enumerate(zip(streams, zs)):
            with torch.cuda.stream(s):
                got[i] = tt.token_logprob(z, top_k=12)
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert all(torch.equal(x, w) for x, w in zip(a[1:], b[1:]))


def test_rows_around_the_batch_stay(tt):
    """Columns from V on and rows outside the view are neither read into the results nor written."""
    buf = torch.full((7, 130), float("nan"), device="cuda", dtype=torch.bfloat16)
    z = buf[2:5, 3:104]
    z.copy_(torch.randn(3, 101, device="cuda"))
    was = buf.clone()
    logp, h, lse, ids, top = tt.token_logprob(z, torch.zeros(3, dtype=torch.int32, device="cuda"), top_k=5)
    assert torch.isfinite(logp).all() and torch.isfinite(h).all() and torch.isfinite(top).all()
    out = torch.full((7, 130), 9.0, device="cuda", dtype=torch.bfloat16)
    tt.token_logprob_bwd(z, lse, h, dentropy=torch.ones(3, device="cuda"), out=out[2:5, 3:104])
    mask = torch.ones_like(out, dtype=torch.bool)
    mask[2:5, 3:104] = False
    assert (out[mask] == 9).all() and torch.isfinite(out).all()
    assert torch.equal(buf.view(torch.int16), was.view(torch.int16))


def test_refusals(tt):
    z = torch.randn(4, 64, device="cuda")
    y = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, device="cuda")
    for bad in (lambda: tt.token_logprob(z.double()), lambda: tt.token_logprob(z, y.long()),
                lambda: tt.token_logprob_bwd(z, f.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: tt.token_logprob(z, y[:3]), lambda: tt.token_logprob(z.T),
                lambda: tt.token_logprob_bwd(z, f[:3]), lambda: tt.token_logprob_bwd(z, f, dtop=z[:, :2]),
                lambda: tt.token_logprob_bwd(z, f, out=z.T), lambda: tt.token_logprob_bwd(z, f, out=z[:, :63])):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: tt.token_logprob(z, top_k=33), -3), (lambda: tt.token_logprob(z[:, :3], top_k=4), -1),
                      (lambda: tt.token_logprob(z, top_k=-1), -1), (lambda: tt.token_logprob_bwd(z, f, dlogp=f), -1),
                      (lambda: tt.token_logprob_bwd(z, f, dentropy=f), -1),
                      (lambda: tt.token_logprob(z[:1].expand(4, 64)), None)):
        with pytest.raises((tt.TTError, ValueError)) as e:
            bad()
        assert code is None or e.value.code == code


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,V", [(1, 70_003), (2, 40_001), (9, 131_072)])
def test_masks_and_extremes_with_several_ctas_to_a_row(tt, dtype, N, V):
    """Few long rows are cut into slices, one to a CTA of a cluster: whole slices masked, rows at the type's lowest and
    highest value, one token left, one dominant, NaN and infinity in one slice alone, each forward and backward."""
    rng = np.random.default_rng(V)
    low, high = float(torch.finfo(DT[dtype]).min), float(torch.finfo(DT[dtype]).max)
    half, rows = V // 2, []
    x = np.full(V, -INF)                          # nothing left
    rows.append(x)
    x = np.full(V, -INF)
    x[V - 2] = 3.0                                # one token, in the last slice
    rows.append(x)
    x = rng.standard_normal(V) * 2
    x[:half + 5] = -INF                           # the first slices masked
    rows.append(x)
    x = rng.standard_normal(V) * 2
    x[half - 5:] = -INF                           # the last ones
    rows.append(x)
    rows.append(np.full(V, low))                  # masked with the lowest value throughout: uniform
    x = np.full(V, low)
    x[half:] = -INF                               # the lowest value in some slices, -inf in the others
    rows.append(x)
    x = np.full(V, low)
    x[7] = 1.0                                    # one plain logit among lowest ones
    rows.append(x)
    x = rng.standard_normal(V)
    x[half] = high                                # one slice far above the others
    rows.append(x)
    x = np.zeros(V)
    x[V - 1] = 60.0
    rows.append(x)
    for i in range(0, len(rows), N):
        part = np.stack((rows[i:i + N] + rows)[:N])
        y = np.array([V - 2 if np.isneginf(r[7]) or r[7] == 1.0 else 7 for r in part])
        z = _logits(part, dtype)
        logp, h, lse, ids, top = _check_fwd(tt, z, y, 20)
        for r in range(N):
            if np.isneginf(part[r]).all():
                assert lse[r] == -INF and h[r] == 0 and ids[r].tolist() == list(range(20))
        one = torch.ones(N, device="cuda")
        dz = tt.token_logprob_bwd(z, lse, h, torch.tensor(y, dtype=torch.int32, device="cuda"), dlogp=one, dentropy=one)
        ref = TL.token_logprob_grad(_f64(z), y, np.ones(N), np.ones(N))
        # p off by 1.1e-4 and the entropy by 1e-4·(1 + 1.5·|U/S|), |U/S| <= log V < 12 here, both times p <= 1 (see
        # _check_bwd); p·|log p + H| < 12
        assert (np.abs(_f64(dz) - ref) <= 1.1e-4 * 13 + 2e-3 + torch.finfo(DT[dtype]).eps / 2 * np.abs(ref)).all()
        assert (dz[np.isneginf(part) & (np.arange(V) != y[:, None])] == 0).all()
    for bad, where in ((np.nan, 3), (np.nan, V - 1), (INF, half), (np.nan, None)):
        x = rng.standard_normal((N, V))
        if where is None:
            x[0] = bad
        else:
            x[0, where] = bad
            if where == V - 1:
                x[0, :half] = -INF
        z = _logits(x, dtype)
        y = torch.full((N,), 5, dtype=torch.int32, device="cuda")
        logp, h, lse, ids, top = tt.token_logprob(z, y, top_k=4)
        for t in (logp, h, lse, top):
            assert torch.isnan(t[0]).all() and torch.isfinite(t[1:]).all()
        assert ((ids >= 0) & (ids < V)).all()
        dz = tt.token_logprob_bwd(z, lse, h, y, dlogp=torch.ones(N, device="cuda"))
        assert torch.isnan(dz[0]).all() and torch.isfinite(dz[1:]).all()
