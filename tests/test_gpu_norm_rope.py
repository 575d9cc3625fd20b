"""tt_qk_norm_rope and its backward against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import norm_rope as NR
from oracle import rope as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rand(rng, shape, t, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to("cuda").to(t)


def _f64(t):
    return t.double().cpu().numpy()


def _tiny(t):
    return {torch.float16: 2.0 ** -25}.get(t, 1e-38)


# fp32 arithmetic in front of the output's rounding. A lane adds 16 squares in a row and the lanes 5 times more:
# 21·2^-24 of the sum, half of it in r; rsqrtf 2^-22; two products 2^-23; the turn 7.5e-7 (angle) + 3·2^-24. In all
# 2.1e-6, of the largest entry of the head times sqrt 2 (a pair's length).
FWD = 2.1e-6 * 2 ** 0.5


def _check_fwd(got, x, w, eps, how, pos_far=0.0):
    ref = NR.forward(x, w, eps, how)
    n = np.abs(NR.forward(x, w, eps)).max(-1, keepdims=True)
    bad = np.abs(_f64(got) - ref) > torch.finfo(got.dtype).eps / 2 * np.abs(ref) * (1 + 1e-5) + (FWD + pos_far) * n + \
        _tiny(got.dtype)
    assert not bad.any(), (int(bad.sum()), np.abs(_f64(got) - ref).max())


def _check_bwd(got, got_w, dy, x, w, eps, how, pos_far=0.0):
    """dx: h = w·g has the turn's error (1.2e-6 of a pair's length) and a rounding; the head's sum Σ h·x has that and
    21·2^-24 of Σ |h·x|; r to the third power has 3·9e-7. dw: each term as g·x·r, and the additions: at most 64 in a row
    of a block's own (the tokens of its turns), 8 warps, 64 rows of parts and 8 warps again."""
    dx, dw = NR.backward(dy, x, w, eps, how)
    wf = np.ones(x.shape[-1]) if w is None else w
    g = np.abs(R.rope(dy, *how["tables"], how["adjacent"], True) if how else dy)
    size = np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    top = 2 ** 0.5 * g.max(-1, keepdims=True)
    h = np.abs(wf) * top
    along = np.abs(x) / size ** 3 * (h * np.abs(x)).mean(-1, keepdims=True)
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(dx) * (1 + 1e-5) + (3e-6 + pos_far) * h / size + \
        (6e-6 + pos_far) * along + _tiny(got.dtype)
    bad = np.abs(_f64(got) - dx) > tol
    assert not bad.any(), (int(bad.sum()), np.abs(_f64(got) - dx).max())
    if got_w is not None:
        tol_w = (3.3e-6 + pos_far + 144 * 2.0 ** -24) * (top * np.abs(x) / size).sum((0, 1)) + 1e-30
        assert (np.abs(_f64(got_w) - dw) <= tol_w).all(), np.abs(_f64(got_w) - dw).max()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("N,hq,hkv,d,rot,sections,w32", [
    (1, 1, 1, 64, 64, (32,), False), (1, 16, 8, 128, 128, (64,), True), (7, 5, 1, 128, 128, (16, 24, 24), False),
    (130, 4, 2, 64, 32, (6, 10), False),             # part of the head
    (33, 3, 3, 80, 80, (20, 20), True),              # d no power of two
    (9, 2, 1, 36, 20, (10,), False),                 # no 16-byte vectors
    (5, 10, 2, 256, 256, (32, 32, 32, 32), False), (3, 2, 1, 512, 256, (128,), False),
    (2500, 2, 1, 16, 16, (8,), False),               # several turns of a block
    (3, 7, 0, 2, 2, (1,), False), (11, 3, 2, 96, 0, (), False)])  # one pair, no k; the norm alone
def test_against_oracle(tt, dtype, adjacent, N, hq, hkv, d, rot, sections, w32):
    rng = np.random.default_rng(N * 100 + d + rot)
    t, eps = DT[dtype], 1e-6
    q, k = _rand(rng, (N, hq, d), t, 1.5), (_rand(rng, (N, hkv, d), t, 0.02) if hkv else None)
    dq, dk = _rand(rng, (N, hq, d), t), (_rand(rng, (N, hkv, d), t) if hkv else None)
    wt = torch.float32 if w32 else t
    wq, wk = (_rand(rng, (d,), wt, 0.3) + 1 for _ in range(2))
    pos = rng.integers(-1000, 100000, (max(1, len(sections)), N)).astype(np.int32)
    args = dict(eps=eps, rot_dim=rot, adjacent=adjacent)
    how, far = None, 0.0
    if rot:
        args["sections"] = sections
        freq = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
        how = {"tables": (pos, R.axis_of(sections), freq), "adjacent": adjacent}
        far = 1e5 * 2.0 ** -52  # the oracle's own angle
    pt = torch.from_numpy(pos).cuda() if rot else None
    got = tt.qk_norm_rope(q, k, pt, wq, wk if hkv else None, **args)
    grads = tt.qk_norm_rope_bwd(dq, dk, q, k, pt, wq, wk if hkv else None, **args)
    for x, dy, w, y, dx, dw in ((q, dq, wq, got[0], grads[0], grads[2]), (k, dk, wk, got[1], grads[1], grads[3])):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        _check_fwd(y, _f64(x), _f64(w), eps, how, far)
        _check_bwd(dx, dw, _f64(dy), _f64(x), _f64(w), eps, how, far)
    # in place: the same values
    q2, k2 = q.clone(), None if k is None else k.clone()
    tt.qk_norm_rope(q2, k2, pt, wq, wk if hkv else None, out=(q2, k2), **args)
    assert torch.equal(q2, got[0]) and (k is None or torch.equal(k2, got[1]))
    for over in ((dq.clone(), None if k is None else dk.clone()), (q.clone(), None if k is None else k.clone())):
        first = over[0].data_ptr()
        src = (over[0], over[1], q, k) if torch.equal(over[0], dq) else (dq, dk, over[0], over[1])
        r = tt.qk_norm_rope_bwd(*src, pt, wq, wk if hkv else None, out=over, **args)
        assert r[0].data_ptr() == first and torch.equal(r[0], grads[0]) and torch.equal(r[2], grads[2])
        assert k is None or (torch.equal(r[1], grads[1]) and torch.equal(r[3], grads[3]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_views_of_a_fused_projection(tt, dtype, pad):
    """q and k as slices of one buffer (with an odd row stride: element accesses), in place: the rest stays, and the
    results are those of contiguous tensors, up to the order of a head's sum."""
    rng = np.random.default_rng(pad)
    N, hq, hkv, d = 37, 6, 2, 64
    buf = _rand(rng, (N, (hq + 2 * hkv) * d + pad), DT[dtype])
    was = buf.clone()
    q = buf[:, :hq * d].unflatten(1, (hq, d))
    k = buf[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    how = {"tables": (np.arange(N)[None], np.zeros(32, int), 10000.0 ** (-np.arange(32) / 32)), "adjacent": False}
    qx, kx = _f64(q), _f64(k)
    tt.qk_norm_rope(q, k, pos, out=(q, k))
    _check_fwd(q, qx, None, 1e-6, how)
    _check_fwd(k, kx, None, 1e-6, how)
    assert torch.equal(buf[:, (hq + hkv) * d:], was[:, (hq + hkv) * d:])


def test_unaligned_base_and_zero_heads(tt):
    rng = np.random.default_rng(8)
    raw = _rand(rng, (1 + 5 * 2 * 64,), torch.bfloat16)
    q = raw[1:].view(5, 2, 64)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    how = {"tables": (np.arange(5)[None], np.zeros(32, int), 10000.0 ** (-np.arange(32) / 32)), "adjacent": False}
    y, _ = tt.qk_norm_rope(q, None, pos)
    _check_fwd(y, _f64(q), None, 1e-6, how)
    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    y, _ = tt.qk_norm_rope(z, None, pos[:4])
    assert (y == 0).all()
    dx, _, dw, _ = tt.qk_norm_rope_bwd(torch.ones_like(z), None, z, None, pos[:4])
    assert torch.isfinite(dx.float()).all() and (dw == 0).all()


def test_gradients_against_differences_of_the_forward(tt):
    """The backward against central differences of the kernel's own fp32 forward: step 1e-2, curvature 1e-4·|y|, and the
    forward's own error 2e-6·|y|/1e-2, over 64 entries."""
    rng = np.random.default_rng(9)
    q, dy = _rand(rng, (2, 1, 64), torch.float32), _rand(rng, (2, 1, 64), torch.float32)
    w = _rand(rng, (64,), torch.float32, 0.2) + 1
    pos = torch.tensor([3, 1000], dtype=torch.int32, device="cuda")
    dx, _, dw, _ = tt.qk_norm_rope_bwd(dy, None, q, None, pos, w, None)
    f = lambda x, w: (tt.qk_norm_rope(x, None, pos, w, None)[0].double() * dy.double()).sum().item()
    for _ in range(20):
        v, u = _rand(rng, (2, 1, 64), torch.float32), _rand(rng, (64,), torch.float32)
        v, u = v / v.norm(), u / u.norm()
        num = (f(q + 1e-2 * v, w) - f(q - 1e-2 * v, w)) / 2e-2
        assert abs(num - (dx.double() * v.double()).sum().item()) < 1e-4 * 12 + 2e-4 * 12
        num = (f(q, w + 1e-2 * u) - f(q, w - 1e-2 * u)) / 2e-2
        assert abs(num - (dw.double() * u.double()).sum().item()) < 2e-4 * 12


def test_empty_streams_and_graphs(tt):
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    a, b = tt.qk_norm_rope(z, z, none)
    assert a.shape == b.shape == z.shape
    _, _, dwq, dwk = tt.qk_norm_rope_bwd(z, z, z, z, none)
    assert (dwq == 0).all() and (dwk == 0).all()
    rng = np.random.default_rng(2)
    q, k = _rand(rng, (50, 4, 64), torch.bfloat16), _rand(rng, (50, 2, 64), torch.bfloat16)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    fwd = lambda: tt.qk_norm_rope(q, k, pos)
    bwd = lambda: tt.qk_norm_rope_bwd(q, k, q, k, pos)
    ref = [*fwd(), *bwd()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [*fwd(), *bwd()]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*fwd(), *bwd()]
    for x in got:
        x.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))


def test_repeated_calls_agree_bitwise_and_weights_are_optional(tt):
    rng = np.random.default_rng(4)
    q, k = _rand(rng, (3001, 5, 128), torch.bfloat16), _rand(rng, (3001, 1, 128), torch.bfloat16)
    pos = torch.arange(3001, dtype=torch.int32, device="cuda")
    ones = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    a = tt.qk_norm_rope_bwd(k.expand(3001, 5, 128).contiguous(), k, q, k, pos, ones, ones)
    for _ in range(3):
        b = tt.qk_norm_rope_bwd(k.expand(3001, 5, 128).contiguous(), k, q, k, pos)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = tt.qk_norm_rope_bwd(k.expand(3001, 5, 128).contiguous(), k, q, k, pos, want_dw=False)
    assert torch.equal(a[0], c[0]) and c[2] is None and c[3] is None
