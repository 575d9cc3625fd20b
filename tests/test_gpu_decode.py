"""tt_tree_decode_plan / tt_tree_decode_attn against the fp64 oracle, one softmax per query."""
import math

import numpy as np
import pytest
import torch

from oracle import decode as D

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _rand(rng, shape, t, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to("cuda").to(t)


def _f64(t):
    return t.double().cpu().numpy()


def _table(segs):
    return torch.tensor(np.array(segs, np.int32).reshape(-1, 4).T.copy(), device="cuda")


def _tree(rng, levels):
    """Segments (rows, first query, past the last) of a tree whose level [n, lo, hi] gives every segment above n children
    of lo .. hi rows; the pool has gaps between them."""
    total = math.prod(n for n, _, _ in levels)
    segs, above, row = [], 1, int(rng.integers(0, 5))
    for n, lo, hi in levels:
        above *= n
        for i in range(above):
            size = int(rng.integers(lo, hi + 1))
            segs.append((row, size, i * (total // above), (i + 1) * (total // above)))
            row += size + int(rng.integers(0, 9))
    return segs, total, row


def _run(tt, q, k, v, segs, scale=None, **more):
    plan = tt.tree_decode_plan(_table(segs), q.shape[0], k.shape[0], sum(s[3] - s[2] for s in segs), q.shape[1],
                               k.shape[1], q.shape[2])
    got = tt.tree_decode_attn(plan, q, k, v, scale=scale, **more)
    plan.check()
    return got


def _check(got, q, k, v, segs, scale=None):
    """O: its rounding (half a step), and the weights' rounding to the type in front of the second product: each term
    p·v by half a step of its own, and the sum of weights is that of the unrounded ones; fp32 sums (a score's dot product
    of d terms by d·2^-24 of Σ|q·k|, below 1.3e-5·d^1/2 here) and ex2 below 2e-5. LSE: 1e-5·(1 + |scores|)."""
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    O, LSE = D.attention(_f64(q), _f64(k), _f64(v), segs, scale)
    A, _ = D.attention(_f64(q), _f64(k), np.abs(_f64(v)), segs, scale)  # Σ p·|v|
    half = torch.finfo(q.dtype).eps / 2
    tiny = 2.0 ** -24 if q.dtype == torch.float16 else 1e-38
    off = np.abs(_f64(got[0]) - O)
    assert (off <= half * np.abs(O) + (half + 1e-4) * A * 1.01 + tiny).all(), off.max()
    none = np.isneginf(LSE)
    assert (np.isneginf(_f64(got[1])) == none).all() and (_f64(got[0]).transpose(1, 0, 2)[none] == 0).all()
    top = np.abs(scale) * np.abs(_f64(q)).sum(-1).max() * max(1e-30, np.abs(_f64(k)[np.isfinite(_f64(k))]).max(initial=0))
    assert (np.abs(_f64(got[1])[~none] - LSE[~none]) <= 4e-6 + 2.0 ** -22 * (np.abs(LSE[~none]) + min(top, 200))).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (16, 8, 128), (5, 1, 128), (14, 2, 64), (4, 4, 128), (32, 1, 64)])
@pytest.mark.parametrize("levels", [
    [(1, 1, 1)], [(1, 127, 127)], [(1, 128, 128)], [(1, 129, 129)],       # one rollout
    [(1, 500, 500), (4, 1, 40)], [(3, 0, 300), (3, 0, 2)],                # just left the prompt; some segments empty
    [(1, 1000, 1000), (2, 100, 300), (9, 0, 200)],                        # two levels of shared turns
    [(1, 130, 130), (40, 1, 260)], [(33, 5, 90)]])                        # many rollouts; unrelated ones
def test_against_oracle(tt, dtype, hq, hkv, d, levels):
    rng = np.random.default_rng(hq * 100 + d + len(levels))
    t = DT[dtype]
    segs, B, rows = _tree(rng, levels)
    q, k, v = _rand(rng, (B, hq, d), t, 1.5), _rand(rng, (rows, hkv, d), t), _rand(rng, (rows, hkv, d), t)
    # rows that no segment holds: never written
    held = np.zeros(rows, bool)
    for s, n, _, _ in segs:
        held[s:s + n] = True
    k[torch.from_numpy(~held).cuda()] = math.nan
    v[torch.from_numpy(~held).cuda()] = math.nan
    got = _run(tt, q, k, v, segs)
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)
    _check(got, q, k, v, segs)


@pytest.mark.parametrize("shared", [6, 16, 17, 31, 64, 100])
def test_numbers_of_rollouts_to_a_prompt(tt, shared):
    """Rows of a tile from a few to more than one tile of 128 (six query heads to a key head)."""
    rng = np.random.default_rng(shared)
    segs, B, rows = _tree(rng, [(1, 700, 700), (shared, 1, 20)])
    q, k, v = (_rand(rng, s, torch.bfloat16) for s in ((B, 12, 64), (rows, 2, 64), (rows, 2, 64)))
    _check(_run(tt, q, k, v, segs), q, k, v, segs)


def test_any_set_of_segments(tt):
    """Pages of one rollout in any order, a segment twice, segments inside one another, queries without keys, segments
    without queries, and scales of either sign."""
    rng = np.random.default_rng(1)
    rows, B = 900, 7
    segs = [(640, 64, 1, 2), (0, 64, 1, 2), (320, 37, 1, 2), (100, 200, 0, 3), (100, 200, 2, 3), (150, 10, 2, 5),
            (0, 900, 4, 4), (5, 0, 0, 7), (899, 1, 6, 7), (0, 900, 4, 5)]
    q, k, v = (_rand(rng, s, torch.bfloat16) for s in ((B, 6, 128), (rows, 2, 128), (rows, 2, 128)))
    for scale in (None, 0.3, -0.1, 0.0):
        _check(_run(tt, q, k, v, segs, scale=scale), q, k, v, segs, scale)
    order = [segs[i] for i in rng.permutation(len(segs))]
    _check(_run(tt, q, k, v, order), q, k, v, order)


def test_no_segments_and_no_queries(tt):
    rng = np.random.default_rng(2)
    q, k, v = (_rand(rng, s, torch.bfloat16) for s in ((3, 2, 64), (10, 1, 64), (10, 1, 64)))
    o, lse = _run(tt, q, k, v, [])
    assert (o == 0).all() and (lse == -math.inf).all()
    o, lse = _run(tt, q, k[:0], v[:0], [(0, 0, 0, 3)])
    assert (o == 0).all() and (lse == -math.inf).all()
    o, lse = _run(tt, q[:0], k, v, [(0, 5, 0, 0)])
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_pool_of_interleaved_rows_and_strided_queries(tt, dtype):
    rng = np.random.default_rng(3)
    segs, B, rows = _tree(rng, [(1, 300, 300), (6, 1, 200)])
    pool = _rand(rng, (rows, 2, 2, 128), DT[dtype])
    k, v = pool[:, 0], pool[:, 1]
    q = _rand(rng, (B, 4 * 3 * 128), DT[dtype])[:, :4 * 128].unflatten(1, (4, 128))
    _check(_run(tt, q, k, v, segs), q, k, v, segs)


def test_large_scores(tt):
    """Scores of several hundred, the largest in another block than the first: maxima move, small weights vanish."""
    rng = np.random.default_rng(4)
    segs, B, rows = _tree(rng, [(1, 2000, 2000), (3, 300, 300)])
    q, k, v = (_rand(rng, s, torch.bfloat16, 6.0) for s in ((B, 2, 64), (rows, 1, 64), (rows, 1, 64)))
    got = _run(tt, q, k, v, segs)
    O, LSE = D.attention(_f64(q), _f64(k), _f64(v), segs, 0.125)
    A, _ = D.attention(_f64(q), _f64(k), np.abs(_f64(v)), segs, 0.125)
    # a score up to 600 in fp32: 64 additions' worth of 2^-24 of Σ|q·k| <= 5000 is 3e-4, in e^s as much
    assert (np.abs(_f64(got[0]) - O) <= 2.0 ** -9 * np.abs(O) + (2.0 ** -8 + 2e-3) * A).all()
    assert (np.abs(_f64(got[1]) - LSE) <= 1e-3).all()


def test_bad_segments_are_reported_and_nothing_is_written(tt):
    rng = np.random.default_rng(5)
    q, k, v = (_rand(rng, s, torch.bfloat16) for s in ((4, 2, 64), (100, 1, 64), (100, 1, 64)))
    good = (0, 50, 0, 4)
    for bad, code in (((-1, 5, 0, 1), -1), ((0, -1, 0, 1), -1), ((90, 11, 0, 1), -1), ((0, 5, -1, 1), -1),
                      ((0, 5, 3, 2), -1), ((0, 5, 0, 5), -1), ((2 ** 31 - 1, 2 ** 31 - 1, 0, 1), -1)):
        plan = tt.tree_decode_plan(_table([good, bad]), 4, 100, 8, 2, 1, 64)
        out = (torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device="cuda"))
        tt.tree_decode_attn(plan, q, k, v, out=out)
        with pytest.raises(tt.TTError) as e:
            plan.check()
        assert e.value.code == code and (out[0] == 7).all() and (out[1] == 7).all()
    plan = tt.tree_decode_plan(_table([good, good]), 4, 100, 7, 2, 1, 64)  # 8 pairs
    out = (torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device="cuda"))
    err = tt.new_err("cuda")
    tt.tree_decode_attn(plan, q, k, v, out=out, err=err)
    assert int(plan.err.item()) == int(err.item()) == -4 and (out[0] == 7).all()
    # bytes that are no plan
    fake = tt.DecodePlan(torch.zeros_like(plan.plan), *(getattr(plan, n) for n in ("S", "B", "rows", "pairs", "hq", "hkv",
                                                                                 "d", "ws_bytes")), tt.new_err("cuda"))
    tt.tree_decode_attn(fake, q, k, v, out=out)
    assert int(fake.err.item()) == -1 and (out[0] == 7).all()
    with pytest.raises(ValueError):
        tt.tree_decode_attn(plan, q[:3], k, v)
    with pytest.raises(ValueError):
        tt.tree_decode_attn(plan, q, k, v.half())


def test_repeated_calls_streams_and_a_growing_step_in_a_graph(tt):
    """A captured step reads the lengths at every replay; eager calls on other streams give the same bits."""
    rng = np.random.default_rng(6)
    segs, B, rows = _tree(rng, [(1, 400, 400), (5, 20, 30)])
    segs = [(s, n, a, b) for s, n, a, b in segs]
    pool = 2000
    for i in range(1, len(segs)):  # room to grow behind each
        segs[i] = (500 + 250 * i, segs[i][1], *segs[i][2:])
    q, k, v = (_rand(rng, s, torch.bfloat16) for s in ((B, 8, 128), (pool, 2, 128), (pool, 2, 128)))
    table, pairs = _table(segs), sum(s[3] - s[2] for s in segs)

    def step():
        return tt.tree_decode_attn(tt.tree_decode_plan(table, B, pool, pairs, 8, 2, 128, err=err), q, k, v)

    err = tt.new_err("cuda")
    ref = step()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(ref, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for grow in (0, 1, 150):
        table[1, 1:] = torch.tensor([s[1] + grow for s in segs[1:]], dtype=torch.int32)
        graph.replay()
        torch.cuda.synchronize()
        now = [segs[0]] + [(s, n + grow, a, b) for s, n, a, b in segs[1:]]
        _check(out, q, k, v, now)
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
    assert int(err.item()) == 0


def test_two_calls_at_once(tt):
    """Two layers of one plan on two streams, each with its own scratch."""
    rng = np.random.default_rng(7)
    segs, B, rows = _tree(rng, [(1, 3000, 3000), (20, 100, 400)])
    a = [_rand(rng, s, torch.bfloat16) for s in ((B, 8, 128), (rows, 2, 128), (rows, 2, 128))]
    b = [_rand(rng, s, torch.bfloat16) for s in ((B, 8, 128), (rows, 2, 128), (rows, 2, 128))]
    plan = tt.tree_decode_plan(_table(segs), B, rows, sum(s[3] - s[2] for s in segs), 8, 2, 128)
    ra, rb = tt.tree_decode_attn(plan, *a), tt.tree_decode_attn(plan, *b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            ga = tt.tree_decode_attn(plan, *a)
        with torch.cuda.stream(s2):
            gb = tt.tree_decode_attn(plan, *b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*ra, *rb), (*ga, *gb)))
    plan.check()


def test_as_the_chunk_call_on_a_path(tt):
    """One rollout: the last query of a chunk against its path, by the training attention."""
    rng = np.random.default_rng(8)
    q, k, v = (_rand(rng, s, torch.bfloat16) for s in ((1, 16, 128), (777, 8, 128), (777, 8, 128)))
    o, lse = _run(tt, q, k, v, [(0, 512, 0, 1), (512, 265, 0, 1)])
    o2, lse2 = tt.tree_attn_chunk_fwd(q, 776, k, v)
    assert (o.float() - o2.float()).abs().max().item() <= 2e-2 and (lse - lse2).abs().max().item() <= 1e-4


def test_far_rows_of_a_large_pool(tt):
    """Offsets past 2^31 elements: a segment at the end of a pool of 2.2e9 elements."""
    rows, hkv, d = 2_200_000, 8, 128
    k = torch.empty(rows, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(rows, hkv, d, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(9)
    n = 333
    for t in (k, v):
        t[rows - n:] = _rand(rng, (n, hkv, d), torch.bfloat16)
    q = _rand(rng, (2, 16, d), torch.bfloat16)
    got = _run(tt, q, k, v, [(rows - n, n, 0, 2)])
    kt, vt = k[rows - n:].clone(), v[rows - n:].clone()
    _check(got, q, kt, vt, [(0, n, 0, 2)])
