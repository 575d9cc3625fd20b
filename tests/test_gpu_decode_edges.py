"""tt_tree_decode_plan / tt_tree_decode_attn at the ends of what they take."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_decode import _check, _rand, _run, _tree

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


def _attention64(q, k, v, segs, scale):
    """O and Σ p·|v| of queries with one segment each or all with the same, in 64 bits on the device."""
    O, A = torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    G = q.shape[1] // k.shape[1]
    for s, n, q0, q1 in segs:
        for h in range(k.shape[1]):
            x = q[q0:q1, h * G:(h + 1) * G].double() @ k[s:s + n, h].double().T * scale
            p = torch.softmax(x, -1)
            O[q0:q1, h * G:(h + 1) * G] = p @ v[s:s + n, h].double()
            A[q0:q1, h * G:(h + 1) * G] = p @ v[s:s + n, h].double().abs()
    return O, A


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n,hq,hkv", [(32, 8192, 16, 4), (1, 131072, 160, 8)])  # rows of 4 and of 20 queries' heads
@pytest.mark.parametrize("far", [20.0, 26.0, 28.0])
def test_many_far_keys_beside_a_near_one(tt, dtype, d, B, n, hq, hkv, far):
    """One key some 2^far times as likely as each of the thousands behind it, whose values are large: together they are a good
    part of O. A weight's rounding: half a step of its type, or half of fp16's last step: 2^-32 of the largest weight."""
    g = torch.Generator(device="cuda").manual_seed(int(far))
    q, k, v = (torch.randn(s, device="cuda", generator=g) for s in ((B, hq, d), (B * n, hkv, d), (B * n, hkv, d)))
    q[..., 0], k[..., 0] = 8.0, 0.0
    q[..., 1:] *= 0.1
    k[::n, :, 0] = far * math.log(2.0) / 8
    k[..., 1:] *= 0.1
    v += 2.0 ** (far - 14)
    v[::n] = torch.randn(B, hkv, d, device="cuda", generator=g)
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    segs = [(i * n, n, i, i + 1) for i in range(B)]
    table = torch.tensor(segs, dtype=torch.int32).T.contiguous().cuda()
    plan = tt.tree_decode_plan(table, B, B * n, B, hq, hkv, d)
    o, lse = tt.tree_decode_attn(plan, q, k, v, scale=1.0)
    plan.check()
    O, A = _attention64(q, k, v, segs, 1.0)
    half = torch.finfo(dtype).eps / 2
    tol = half * O.abs() + (half + 1e-4) * A * 1.01
    if dtype == torch.float16:
        tol += n * 2.0 ** -32 * 1.01 * v.double().abs().max() + 2.0 ** -24
    off = (o.double() - O).abs()
    assert (off <= tol).all(), (off.max(), (off / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 64, 16), (6, 1, 128, 64), (20, 1, 64, 64), (4, 4, 128, 1)])
def test_pages_in_any_order(tt, dtype, hq, hkv, d, page):
    """A prompt and the rollouts' own rows in pages anywhere in the pool, the last of each partly filled (what lies behind its
    keys was never written): many hundreds of segments, so that the parts of a query are joined in several goes."""
    rng = np.random.default_rng(page)
    whole, B, _ = _tree(rng, [(1, 700, 700), (3, 50, 200), (6, 0, 300)])
    if page == 1:
        whole = [(s, min(n, 60), a, b) for s, n, a, b in whole]
    pages = [(min(page, n - i), a, b) for _, n, a, b in whole for i in range(0, n, page)]
    rows = len(pages) * page
    at = rng.permutation(len(pages)) * page
    segs = [(int(x), n, a, b) for x, (n, a, b) in zip(at, pages)]
    segs = [segs[i] for i in rng.permutation(len(segs))]
    q, k, v = _rand(rng, (B, hq, d), dtype, 1.5), _rand(rng, (rows, hkv, d), dtype), _rand(rng, (rows, hkv, d), dtype)
    held = np.zeros(rows, bool)
    for s, n, _, _ in segs:
        held[s:s + n] = True
    for t in (k, v):
        t[torch.from_numpy(~held).cuda()] = math.nan
    got = _run(tt, q, k, v, segs)
    _check(got, q, torch.nan_to_num(k), torch.nan_to_num(v), segs)


@pytest.mark.parametrize("hq,hkv,d", [(1024, 1, 64), (1024, 1024, 64), (1024, 8, 128), (1020, 60, 128)])
def test_most_heads(tt, hq, hkv, d):
    rng = np.random.default_rng(hkv)
    segs, B, rows = _tree(rng, [(1, 150, 150), (3, 0, 140)])
    q, k, v = _rand(rng, (B, hq, d), torch.bfloat16), *(_rand(rng, (rows, hkv, d), torch.bfloat16) for _ in range(2))
    _check(_run(tt, q, k, v, segs), q, k, v, segs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq", [4, 40])  # narrow and wide tiles
@pytest.mark.parametrize("scale", [0.125, 0.1, -0.0625, 0.03, 0.005, 1.0, 3.0, 300.0, -1e5, 1e20])
def test_scores_whose_steps_are_whole_powers_of_two(tt, dtype, hq, scale):
    """Scores of 2^30·scale, some of fp32's steps apart and growing along the keys: weights stay within their type, and O a mean of
    the values (of which all are 1: a weight is off by half a step of its type)."""
    g = torch.Generator(device="cuda").manual_seed(int(1000 * abs(scale)) % 2 ** 31)
    n, d, B = 3000, 64, 6
    q, k = torch.zeros(B, hq, d, device="cuda"), torch.zeros(n * B, 1, d, device="cuda")
    q[..., 0], q[..., 1] = 32768.0, 128.0
    k[..., 0] = 32768.0
    steps = torch.randint(0, 2, (B, n), device="cuda", generator=g).cumsum(1) % torch.tensor([[3], [7], [20], [128], [200], [256]]).cuda()
    k[..., 1] = steps.reshape(-1, 1) * (1.0 if scale > 0 else -1.0)
    v = torch.ones(n * B, 1, d, device="cuda", dtype=dtype)
    table = torch.tensor([[i * n, n, i, i + 1] for i in range(B)], dtype=torch.int32).T.contiguous().cuda()
    plan = tt.tree_decode_plan(table, B, n * B, B, hq, 1, d)
    o, lse = tt.tree_decode_attn(plan, q.to(dtype), k.to(dtype), v, scale=scale)
    assert ((o.double() - 1).abs() <= 2 * torch.finfo(dtype).eps / 2 + 1e-4).all() and torch.isfinite(lse).all()
