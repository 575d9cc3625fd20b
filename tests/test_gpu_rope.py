"""tt_rope (rotary positions, several axes, and the inverse) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import synth
from oracle import rope as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rand(rng, shape, t):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to("cuda").to(t)


def _f64(t):
    return t.double().cpu().numpy()


def _check(got, x, ref, pos, freq):
    """Output rounding (half a step) + fp32 arithmetic: the angle is off by at most 2^-23 of a turn (7.5e-7) plus
    the oracle's own rounding of the fp64 product |pos·f|·2^-53; sincospif and the two products add 3·2^-24."""
    n2 = np.abs(x).max(axis=-1, keepdims=True) * 2
    far = np.abs(np.asarray(pos, np.float64)).max() * np.abs(freq).max() * 2.0 ** -52
    eps = torch.finfo(got.dtype).eps / 2
    tiny = {torch.float16: 2.0 ** -25}.get(got.dtype, 1e-38)
    bad = np.abs(_f64(got) - ref) > eps * np.abs(ref) * (1 + 1e-5) + (1e-6 + far) * n2 + tiny
    assert not bad.any(), (int(bad.sum()), np.abs(_f64(got) - ref).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("N,hq,hkv,d,rot,sections,interleaved", [
    (1, 1, 1, 64, 64, (32,), False), (1, 16, 8, 128, 128, (64,), False), (7, 5, 1, 128, 128, (16, 24, 24), False),
    (130, 4, 2, 64, 32, (6, 5, 5), True),           # part of the head
    (33, 3, 3, 80, 80, (20, 20), True),             # d and rot not powers of two
    (9, 2, 1, 36, 20, (10,), False),                # no 16-byte vectors
    (5, 40, 8, 256, 256, (32, 32, 32, 32), False),  # the largest table
    (3, 7, 0, 2, 2, (1,), False)])                  # one pair, no k
def test_against_oracle(tt, dtype, adjacent, N, hq, hkv, d, rot, sections, interleaved):
    rng = np.random.default_rng(N * 100 + d + rot)
    t = DT[dtype]
    q, k = _rand(rng, (N, hq, d), t), (_rand(rng, (N, hkv, d), t) if hkv else None)
    pos = rng.integers(-1000, 100000, (len(sections), N)).astype(np.int32)
    pt = torch.from_numpy(pos).cuda()
    freq = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    axis = R.axis_of(sections, interleaved)
    how = dict(rot_dim=rot, sections=sections, interleaved=interleaved, adjacent=adjacent)
    for inverse in (False, True):
        call = tt.rope_bwd if inverse else tt.rope
        got = call(q, k, pt, **how)
        for x, y in zip((q, k), got):
            if x is None:
                assert y is None
                continue
            _check(y, _f64(x), R.rope(_f64(x), pos, axis, freq, adjacent, inverse), pos, freq)
            assert torch.equal(y[..., rot:], x[..., rot:])
        # in place: the same values
        q2, k2 = q.clone(), None if k is None else k.clone()
        r = call(q2, k2, pt, out=(q2, k2), **how)
        assert r[0] is q2 and torch.equal(q2, got[0]) and (k is None or torch.equal(k2, got[1]))


def test_far_positions_and_given_frequencies(tt):
    """Positions over the whole int32 range: the fp64 oracle's own angle is known to |pos·f|·2^-53."""
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 123456789], np.int32)
    freq = np.concatenate([[1.0, 0.0, -0.5, 6.283185307179586, 7.0], 10000.0 ** (-np.arange(11) / 11)])
    q = _rand(rng, (7, 2, 32), torch.float32)
    got, _ = tt.rope(q, None, torch.from_numpy(pos).cuda(), inv_freq=freq)
    _check(got, _f64(q), R.rope(_f64(q), pos[None], np.zeros(16, int), freq), pos, freq)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_views_of_a_fused_projection(tt, dtype, pad):
    """q and k as slices of one [N, (Hq + 2·Hkv)·d + pad] buffer, rotated in place: the rest of the buffer stays."""
    rng = np.random.default_rng(pad)
    N, hq, hkv, d = 37, 6, 2, 64
    buf = _rand(rng, (N, (hq + 2 * hkv) * d + pad), DT[dtype])
    was = buf.clone()
    q = buf[:, :hq * d].unflatten(1, (hq, d))
    k = buf[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    rq, rk = tt.rope(q.contiguous(), k.contiguous(), pos)
    tt.rope(q, k, pos, out=(q, k))
    assert torch.equal(q, rq) and torch.equal(k, rk)
    assert torch.equal(buf[:, (hq + hkv) * d:], was[:, (hq + hkv) * d:])


def test_shared_and_strided_positions(tt):
    rng = np.random.default_rng(1)
    N = 21
    q, k = _rand(rng, (N, 4, 64), torch.bfloat16), _rand(rng, (N, 2, 64), torch.bfloat16)
    one = torch.arange(100, 100 + N, dtype=torch.int32, device="cuda")
    ref = tt.rope(q, k, one)
    same = tt.rope(q, k, one.expand(3, N), sections=(10, 11, 11))
    assert all(torch.equal(a, b) for a, b in zip(ref, same))
    wide = torch.zeros(3, N + 5, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + N] = one
    cut = tt.rope(q, k, wide[:, 2:2 + N], sections=(10, 11, 11), interleaved=True)
    assert all(torch.equal(a, b) for a, b in zip(ref, cut))


def test_empty_streams_and_graphs(tt):
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    a, b = tt.rope(z, z, torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert a.shape == b.shape == z.shape
    rng = np.random.default_rng(2)
    q, k = _rand(rng, (50, 4, 64), torch.bfloat16), _rand(rng, (50, 2, 64), torch.bfloat16)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    out = (torch.empty_like(q), torch.empty_like(k))
    ref = tt.rope(q, k, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tt.rope(q, k, pos, out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(ref, out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tt.rope(q, k, pos, out=out)
    q.mul_(-1)
    pos.add_(3)
    g.replay()
    torch.cuda.synchronize()
    ref = tt.rope(q, k, pos)
    assert all(torch.equal(x, y) for x, y in zip(ref, out))


def test_positions_of_a_tree(tt):
    """A token's rotation depends on its depth along its path alone: the tree's Q rows equal each branch's own."""
    sh = synth.tree_shape(0)
    tree = tt.tree_build(torch.tensor(sh.seg_parent, device="cuda"), torch.tensor(sh.seg_len, device="cuda"))
    tree.check()
    rng = np.random.default_rng(0)
    q = _rand(rng, (sh.N, 2, 64), torch.bfloat16)
    got, _ = tt.rope(q, None, tree.tok_pos)
    from oracle import tree as T
    for br in T.branches(T.tables(sh.seg_parent, sh.seg_len)):
        rows = torch.tensor(np.asarray(br), device="cuda")
        alone, _ = tt.rope(q[rows], None, torch.arange(len(rows), dtype=torch.int32, device="cuda"))
        assert torch.equal(got[rows], alone)


def test_offsets_past_32_bits(tt):
    """More than 2^31 elements before the last tokens: these equal the same tokens alone."""
    N, hq, d = 420_001, 40, 128
    q = torch.zeros(N, hq, d, dtype=torch.bfloat16, device="cuda")
    q[-5:] = torch.randn(5, hq, d, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    ref, _ = tt.rope(q[-5:].clone(), None, pos[-5:])
    tt.rope(q, None, pos, out=(q, None))
    assert torch.equal(q[-5:], ref) and not q[:100].any()


def test_one_tensor_twice(tt):
    """q and k the same tensor: fine into new tensors, refused in place (one would be turned twice)."""
    q = torch.randn(9, 2, 64, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    a, b = tt.rope(q, q, pos)
    assert torch.equal(a, b)
    with pytest.raises(tt.TTError) as e:
        tt.rope(q, q, pos, out=(q, q))
    assert e.value.code == -1


def test_refusals(tt):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: tt.rope(q.double(), None, pos), lambda: tt.rope(q, None, pos.long()),
                lambda: tt.rope(q[0], None, pos)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: tt.rope(q, q.float(), pos), lambda: tt.rope(q, None, pos[:3]),
                lambda: tt.rope(q, None, pos, rot_dim=63), lambda: tt.rope(q, None, pos, rot_dim=66),
                lambda: tt.rope(q, None, pos.expand(2, 4)), lambda: tt.rope(q, None, pos, sections=(31,)),
                lambda: tt.rope(q[..., ::2], None, pos), lambda: tt.rope(q.transpose(0, 1), None, pos[:2]),
                lambda: tt.rope(q, None, pos, out=(q[:3], None)), lambda: tt.rope(q, None, pos, inv_freq=[1.0])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tt.TTError) as e:
        tt.rope(q[:1].expand(4, 2, 64), None, pos)  # rows on top of each other
    assert e.value.code == -1


def test_angles_of_any_frequency_at_far_positions(tt):
    """(1, 0) turned is (cos θ, sin θ), against angles reduced in whole numbers. θ is within 2^-24 of a turn: the
    fraction of a turn is cut off at 2^-64 (times a position up to 2^31) and at 2^-32, and rounded to fp32 (2^-25 of a
    turn at half a turn); sincospif is within 2^-23."""
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 123456789, -987654321], np.int32)
    freq = np.array([1.0, 0.0, -0.5, 2 * np.pi, 7.0, -7.0, 100.0, 1000.0, 0.1, 3e-5, 1e6 + 0.1, 1e17, -1e300, 1.7e308,
                     5e-324, 1e-12])
    q = torch.zeros(8, 1, 32, device="cuda")
    q[..., :16] = 1
    got, _ = tt.rope(q, None, torch.from_numpy(pos).cuda(), inv_freq=freq)
    back, _ = tt.rope_bwd(q, None, torch.from_numpy(pos).cuda(), inv_freq=freq)
    theta = np.array([[R.angle(p, f) for f in freq] for p in pos])
    tol = 2 * np.pi * 2.0 ** -24 + 2.0 ** -23
    for x, sign in ((got, 1), (back, -1)):
        x = _f64(x)[:, 0]
        assert np.abs(x[:, :16] - np.cos(theta)).max() <= tol
        assert np.abs(x[:, 16:] - sign * np.sin(theta)).max() <= tol


def test_frequencies_on_the_device_are_refused(tt):
    q = torch.randn(4, 2, 8, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    f = torch.tensor([1.0, 0.1, 0.01, 0.001])
    with pytest.raises(TypeError):
        tt.rope(q, None, pos, inv_freq=f.cuda())
    a, b = tt.rope(q, None, pos, inv_freq=f)[0], tt.rope(q, None, pos, inv_freq=f.tolist())[0]
    assert torch.equal(a, b)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        tt.rope(q, None, pos, inv_freq=f, out=(out, None))
    graph.replay()
    assert torch.equal(out, a)
