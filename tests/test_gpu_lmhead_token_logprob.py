"""tt_lmhead_token_logprob and its backward (LM head fused with log-prob and entropy) against the fp64 oracle, and a
policy-optimisation step over a tree through all the calls."""
import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import lmhead as LH
from oracle import rope as R
from oracle import token_logprob as TL
from oracle import tree as T
from tests._util import GRAD_RL2, LOGP_ATOL, dev_to_f64, f64, rel_l2, to_dev_bf16

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 64), (77, 1000, 64), (300, 3001, 128), (129, 256, 192), (513, 4099, 256), (256, 511, 64)]


def _inputs(N, V, Hd):
    d = synth.lmhead_inputs(N + V + Hd, n_rows=N, vocab=V, hidden=Hd)
    y = torch.tensor(d["targets"], dtype=torch.int32, device="cuda")
    return d, to_dev_bf16(d["H"]), to_dev_bf16(d["W"]), y


@pytest.mark.parametrize("N,V,Hd", SHAPES)
def test_forward(tt, N, V, Hd):
    """log-probs and lse within 1e-4 (as the log-prob fused with the head); the entropy adds U/S, off by as much
    relative to |U/S| = max z + ... = lse − max z − H."""
    d, H, W, y = _inputs(N, V, Hd)
    err = tt.new_err("cuda")
    logp, h, lse = tt.lmhead_token_logprob(H, W, y, err=err)
    assert int(err.item()) == 0
    z = LH.logits(f64(d["H"]), f64(d["W"]))
    r_logp, r_h, r_lse, _, _ = TL.token_logprob(z, d["targets"])
    assert np.abs(dev_to_f64(logp) - r_logp).max() <= LOGP_ATOL
    assert np.abs(dev_to_f64(lse) - r_lse).max() <= LOGP_ATOL
    us = np.abs(r_lse - z.max(1) - r_h)
    assert (np.abs(dev_to_f64(h) - r_h) <= LOGP_ATOL * (1 + us)).all()
    # bitwise repeatable; the log-prob call's values up to rounding
    again = tt.lmhead_token_logprob(H, W, y)
    assert all(torch.equal(a, b) for a, b in zip((logp, h, lse), again))
    old, old_lse, _ = tt.lmhead_logprob(H, W, y)
    assert (old - logp).abs().max().item() <= 2e-5 and (old_lse - lse).abs().max().item() <= 2e-5


@pytest.mark.parametrize("N,V,Hd", SHAPES[1:])
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
def test_backward(tt, N, V, Hd, dw_dtype):
    """Relative L2 1e-2 as for the gradients of the log-prob (bf16 inputs and dz, fp32 sums)."""
    d, H, W, y = _inputs(N, V, Hd)
    rng = np.random.default_rng(N)
    g = {n: rng.standard_normal(N).astype(np.float32) for n in ("dlogp", "dentropy", "dlse")}
    gt = {n: torch.tensor(v, device="cuda") for n, v in g.items()}
    z = LH.logits(f64(d["H"]), f64(d["W"]))
    _, h, lse = tt.lmhead_token_logprob(H, W, y)
    for names in (("dlogp",), ("dentropy",), ("dlse",), ("dlogp", "dentropy", "dlse")):
        err = tt.new_err("cuda")
        dh, dw = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, **{n: gt[n] for n in names}, err=err, dw_dtype=dw_dtype)
        assert int(err.item()) == 0 and dh.dtype == torch.bfloat16 and dw.dtype == dw_dtype
        dz = TL.token_logprob_grad(z, d["targets"], **{n: g[n] for n in names})
        assert rel_l2(dev_to_f64(dh), dz @ f64(d["W"])) <= GRAD_RL2, names
        assert rel_l2(dev_to_f64(dw), dz.T @ f64(d["H"])) <= GRAD_RL2, names
    again = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, **gt, dw_dtype=dw_dtype)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


@pytest.mark.parametrize("N", [1, 5, 8, 31, 32])
def test_few_rows_of_a_large_head(tt, N):
    """Where W is large and the rows few (up to 31), the rows are laid out apart for the product: against fp64, and the
    backward's two products against the dz of the definition; repeatable, with a workspace exactly as large as asked."""
    V, Hd = 70_001, 1024
    g = torch.Generator(device="cuda").manual_seed(N)
    H = torch.randn(N, Hd, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, Hd, generator=g, device="cuda") * (2 / 32)).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    ws = torch.empty(tt.lib().tt_lmhead_token_logprob_workspace_bytes(N, V, Hd), dtype=torch.uint8, device="cuda")
    logp, h, lse = tt.lmhead_token_logprob(H, W, y, ws=ws)
    z = (H.double() @ W.double().T).cpu().numpy()
    r_logp, r_h, r_lse, _, _ = TL.token_logprob(z, y.cpu().numpy())
    assert np.abs(dev_to_f64(logp) - r_logp).max() <= LOGP_ATOL and np.abs(dev_to_f64(lse) - r_lse).max() <= LOGP_ATOL
    assert (np.abs(dev_to_f64(h) - r_h) <= LOGP_ATOL * (1 + np.abs(r_lse - z.max(1) - r_h))).all()
    dl, de = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    dh, dw = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, dentropy=de)
    dz = torch.from_numpy(TL.token_logprob_grad(z, y.cpu().numpy(), dev_to_f64(dl), dev_to_f64(de))).cuda()
    assert rel_l2(dev_to_f64(dh), (dz @ W.double()).cpu().numpy()) <= GRAD_RL2
    r_dw = dz.T @ H.double()
    assert ((dw.double() - r_dw).norm() / r_dw.norm()).item() <= GRAD_RL2
    again = tt.lmhead_token_logprob(H, W, y) + tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, dentropy=de)
    assert all(torch.equal(a, b) for a, b in zip(again, (logp, h, lse, dh, dw)))


@pytest.mark.parametrize("N,V,Hd", [(1, 9000, 64), (61, 32003, 512), (129, 5003, 1024), (130, 20001, 256)])
def test_backward_of_few_rows(tt, N, V, Hd):
    """Few tiles of d_hidden: its sum over the vocabulary is split over the SMs. Tolerance as test_backward; a
    workspace one byte short is refused."""
    d, H, W, y = _inputs(N, V, Hd)
    rng = np.random.default_rng(N)
    dl, de = (rng.standard_normal(N).astype(np.float32) for _ in range(2))
    _, h, lse = tt.lmhead_token_logprob(H, W, y)
    args = dict(dlogp=torch.tensor(dl, device="cuda"), dentropy=torch.tensor(de, device="cuda"))
    dh, dw = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, **args)
    dz = TL.token_logprob_grad(LH.logits(f64(d["H"]), f64(d["W"])), d["targets"], dlogp=dl, dentropy=de)
    assert rel_l2(dev_to_f64(dh), dz @ f64(d["W"])) <= GRAD_RL2
    assert rel_l2(dev_to_f64(dw), dz.T @ f64(d["H"])) <= GRAD_RL2
    again = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, **args)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
    n = tt.lib().tt_lmhead_token_logprob_bwd_workspace_bytes(N, V, Hd)
    with pytest.raises(tt.TTError) as e:
        tt.lmhead_token_logprob_bwd(H, W, y, lse, h, ws=torch.empty(n - 1, dtype=torch.uint8, device="cuda"), **args)
    assert e.value.code == -4
    # a workspace and outputs on 16-byte boundaries only: 16-byte stores, the same values
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")[16:]
    out = (torch.empty(N * Hd + 8, dtype=torch.bfloat16, device="cuda")[8:].view(N, Hd),
           torch.empty(V * Hd + 8, dtype=torch.bfloat16, device="cuda")[8:].view(V, Hd))
    dh2, dw2 = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, out=out, ws=ws, **args)
    assert torch.equal(dh2, dh) and torch.equal(dw2, dw.to(torch.bfloat16))


@pytest.mark.parametrize("N,V,Hd", [(6001, 2401, 512), (4129, 9999, 1024), (2100, 3001, 1088)])
def test_backward_of_many_rows(tt, N, V, Hd):
    """Long sums, which pairs of CTAs take by tiles of 256 rows: an odd number of 128-row tiles, a ragged vocabulary, one
    wave of tiles and several. Tolerance as test_backward, every row and column by itself too: the roundings to bf16
    of dz and of the sum are each 2^-8 of a row at most, its terms being independent, the fp32 sums under 1e-4; 1e-2 again. In a captured
    graph, replayed, and from the weighted call over the same kernels."""
    g = torch.Generator(device="cuda").manual_seed(N)
    H = torch.randn(N, Hd, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, Hd, generator=g, device="cuda") * (2 / Hd ** 0.5)).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    dl, de = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    z = H.double() @ W.double().T
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    p = lp.exp()
    h = -(p * lp).sum(1)
    dz = -p * (dl.double()[:, None] + de.double()[:, None] * (lp + h[:, None]))
    dz[torch.arange(N, device="cuda"), y.long()] += dl.double()
    r_dh, r_dw = dz @ W.double(), dz.T @ H.double()
    for dw_dtype in (torch.float32, torch.bfloat16):
        args = dict(dlogp=dl, dentropy=de, dw_dtype=dw_dtype)
        err = tt.new_err("cuda")
        dh, dw = tt.lmhead_token_logprob_bwd(H, W, y, lse.float(), h.float(), err=err, **args)
        assert int(err.item()) == 0
        for x, r in ((dh, r_dh), (dw, r_dw)):
            e = (x.double() - r).norm(dim=1)
            assert (e <= GRAD_RL2 * r.norm(dim=1)).all()
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                gh, gw = tt.lmhead_token_logprob_bwd(H, W, y, lse.float(), h.float(), **args)
            for _ in range(2):
                gh.zero_(), gw.zero_()
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gh, dh) and torch.equal(gw, dw)
    w = torch.rand(N, generator=g, device="cuda")
    a = tt.lmhead_logprob_bwd(H, W, y, lse.float(), w, g=0.5)
    b = tt.lmhead_token_logprob_bwd(H, W, y, lse.float(), dlogp=-0.5 * w)
    for x, t in zip(a, b):
        assert ((x.double() - t.double()).norm() / t.double().norm()).item() <= 2.0 ** -8


def test_log_prob_gradient_equals_the_weighted_call(tt):
    """dlogp = −g·w is the weighted loss: the two calls form dz in another order of two products, then round to bf16."""
    d, H, W, y = _inputs(300, 3001, 128)
    w = torch.rand(300, device="cuda")
    _, lse, _ = tt.lmhead_logprob(H, W, y, w)
    a = tt.lmhead_logprob_bwd(H, W, y, lse, w, g=0.5)
    b = tt.lmhead_token_logprob_bwd(H, W, y, lse, dlogp=-0.5 * w)
    for x, z in zip(a, b):
        assert rel_l2(dev_to_f64(x), dev_to_f64(z)) <= 2.0 ** -8


def test_bad_target_and_arguments(tt):
    d, H, W, y = _inputs(40, 700, 64)
    y[5], y[6] = 700, -1
    err = tt.new_err("cuda")
    logp, h, lse = tt.lmhead_token_logprob(H, W, y, err=err)
    assert int(err.item()) == -1
    assert torch.isnan(logp).nonzero().flatten().tolist() == [5, 6]
    assert torch.isfinite(h).all() and torch.isfinite(lse).all()
    err = tt.new_err("cuda")
    dh, dw = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=torch.ones(40, device="cuda"), err=err)
    assert int(err.item()) == -1 and torch.isfinite(dh).all() and torch.isfinite(dw).all()
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    for bad, code in ((lambda: tt.lmhead_token_logprob(H[:, :32].contiguous(), W[:, :32].contiguous(), y), -3),
                      (lambda: tt.lmhead_token_logprob(H, W, y, ws=small), -4),
                      (lambda: tt.lmhead_token_logprob_bwd(H, W, y, lse, ws=small), -4),
                      (lambda: tt.lmhead_token_logprob_bwd(H, W, y, lse, dentropy=lse), -1)):
        with pytest.raises(tt.TTError) as e:
            bad()
        assert e.value.code == code
    for bad in (lambda: tt.lmhead_token_logprob(H, W, y[:3]), lambda: tt.lmhead_token_logprob(H, W[:, :32], y),
                lambda: tt.lmhead_token_logprob_bwd(H, W, y, lse[:3])):
        with pytest.raises(ValueError):
            bad()


def test_captured_step(tt):
    """Forward and backward captured into one graph, replayed on new inputs."""
    d, H, W, y = _inputs(129, 1000, 128)
    dev = "cuda"
    out, grads = tuple(torch.empty(3, 129, device=dev)), (torch.empty_like(H), torch.empty(1000, 128, device=dev))
    dl, de, err = torch.randn(129, device=dev), torch.randn(129, device=dev), tt.new_err(dev)

    def step(out, grads):
        logp, h, lse = tt.lmhead_token_logprob(H, W, y, out=out, err=err)
        return (logp, h, lse) + tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, dentropy=de, out=grads, err=err)

    step(None, None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out, grads)
    H.mul_(0.5)
    y.copy_(y.flip(0))
    g.replay()
    torch.cuda.synchronize()
    ref = step(None, None)
    assert all(torch.equal(a, b) for a, b in zip(ref, out + grads))
    assert int(err.item()) == 0


@pytest.mark.parametrize("axes", [1, 3])
def test_policy_step_over_a_tree(tt, axes):
    """Rotary -> tree attention -> head with log-prob and entropy -> backward of all of it, against the fp64 oracle
    of the same chain on the bf16 values that each call receives."""
    sh = synth.tree_shape(0)
    tab = T.tables(sh.seg_parent, sh.seg_len)
    N, hq, hkv, d, V = sh.N, 4, 2, 64, 1000
    rng = np.random.default_rng(axes)
    qr, kr, v = (to_dev_bf16(synth.normal_bf16(rng, (N, n, d))) for n in (hq, hkv, hkv))
    W = to_dev_bf16(synth.normal_bf16(rng, (V, hq * d), 0.1))
    y = torch.tensor(rng.integers(0, V, N), dtype=torch.int32, device="cuda")
    tree = tt.tree_build(torch.tensor(sh.seg_parent, device="cuda"), torch.tensor(sh.seg_len, device="cuda"))
    pos = tree.tok_pos if axes == 1 else torch.stack([tree.tok_pos, tree.tok_pos // 4, tree.tok_pos % 4])
    how = {} if axes == 1 else dict(sections=(12, 10, 10))
    w = torch.tensor(tab.tok_weight, device="cuda")
    dlogp, dent = -w, -0.01 * w
    err = tt.new_err("cuda")
    # forward
    q, k = tt.rope(qr, kr, pos, **how)
    O, LSE = tt.tree_attn_fwd(tree, q, k, v, err=err)
    hid = O.view(N, hq * d)
    logp, ent, lse = tt.lmhead_token_logprob(hid, W, y, err=err)
    # backward
    dh, dw = tt.lmhead_token_logprob_bwd(hid, W, y, lse, ent, dlogp=dlogp, dentropy=dent, err=err)
    dO = dh.view(N, hq, d)
    dq, dk, dv = tt.tree_attn_bwd(tree, q, k, v, O, LSE, dO, err=err)
    dqr, dkr = tt.rope_bwd(dq, dk, pos, **how)
    torch.cuda.synchronize()
    tree.check()
    assert int(err.item()) == 0

    pn = pos.cpu().numpy().reshape(axes, N)
    axis = np.zeros(32, int) if axes == 1 else R.axis_of((12, 10, 10))
    freq = 10000.0 ** (-np.arange(32) / 32)
    rq, rk = R.rope(dev_to_f64(qr), pn, axis, freq), R.rope(dev_to_f64(kr), pn, axis, freq)
    rO, _, _, _, _ = A.tree_attention_branches(tab, rq, rk, dev_to_f64(v), np.zeros((N, hq, d)))
    z = LH.logits(rO.reshape(N, -1), dev_to_f64(W))
    r_logp, r_ent, _, _, _ = TL.token_logprob(z, y.cpu().numpy())
    # O is within 2^-8 of its size (bf16 Q, K and O): z, a sum over 256 such terms with |W| ~ 0.1, within 0.02
    assert np.abs(dev_to_f64(logp) - r_logp).max() <= 0.04 and np.abs(dev_to_f64(ent) - r_ent).max() <= 0.04
    dz = TL.token_logprob_grad(z, y.cpu().numpy(), dev_to_f64(dlogp), dev_to_f64(dent))
    r_dh = dz @ dev_to_f64(W)
    _, _, r_dq, r_dk, r_dv = A.tree_attention_branches(tab, rq, rk, dev_to_f64(v), r_dh.reshape(N, hq, d))
    # each stage rounds to bf16 (2^-8): four of them lie between the inputs and dq, dk
    for got, ref in ((dh, r_dh), (dw, dz.T @ rO.reshape(N, -1)), (dv, r_dv),
                     (dqr, R.rope(r_dq, pn, axis, freq, inverse=True)), (dkr, R.rope(r_dk, pn, axis, freq, inverse=True))):
        got = dev_to_f64(got).reshape(ref.shape)
        assert rel_l2(got, ref) <= 2 * GRAD_RL2, rel_l2(got, ref)
    # the same objective on stored logits: the fused gradient rounds dz to bf16 as this call does
    zb = (hid.float() @ W.float().T)
    lp2, e2, lse2, ids, top = tt.token_logprob(zb, y, top_k=5, err=err)
    assert (lp2 - logp).abs().max().item() <= 1e-4 and (e2 - ent).abs().max().item() <= 2e-4
    dzb = tt.token_logprob_bwd(zb, lse2, e2, y, dlogp=dlogp, dentropy=dent, err=err)
    assert rel_l2(dev_to_f64(dh), dev_to_f64(dzb) @ dev_to_f64(W)) <= GRAD_RL2
    assert int(err.item()) == 0


@pytest.mark.parametrize("N,V,Hd", [(513, 4099, 256), (61, 32003, 512), (4129, 9999, 1024)])
def test_backward_rounds_dz_and_outputs_only(tt, N, V, Hd):
    """The gradients' error is that of dz's rounding to bf16 and of the outputs' own. A rounding error is spread evenly
    over at most half a step, 2^-8 of the value: its root mean square is at most 2^-8/sqrt(3). Against 64 bits, with
    terms of random signs and independent roundings, fp32 dW has one such error and bf16 dH and dW have two: their
    relative L2 is at most 2^-8/sqrt(3) and sqrt(2) times that. 5 % above for the spread over the few thousand sums
    that share a row of dz and for the fp32 arithmetic (< 2e-4: see test_backward_of_many_rows)."""
    g = torch.Generator(device="cuda").manual_seed(N + V)
    H = torch.randn(N, Hd, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, Hd, generator=g, device="cuda") * (2 / Hd ** 0.5)).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    dl, de = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    z = H.double() @ W.double().T
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    p = lp.exp()
    h = -(p * lp).sum(1)
    dz = -p * (dl.double()[:, None] + de.double()[:, None] * (lp + h[:, None]))
    dz[torch.arange(N, device="cuda"), y.long()] += dl.double()
    r_dh, r_dw = dz @ W.double(), dz.T @ H.double()
    one = 2.0 ** -8 / 3 ** 0.5 * 1.05
    for dw_dtype, tol in ((torch.float32, one), (torch.bfloat16, 2 ** 0.5 * one)):
        dh, dw = tt.lmhead_token_logprob_bwd(H, W, y, lse.float(), h.float(), dlogp=dl, dentropy=de, dw_dtype=dw_dtype)
        assert ((dh.double() - r_dh).norm() / r_dh.norm()).item() <= 2 ** 0.5 * one
        assert ((dw.double() - r_dw).norm() / r_dw.norm()).item() <= tol


@pytest.mark.parametrize("N,V,Hd", [
    (1025, 3900, 512),    # 9 tiles of 128 rows, 31 of 128 vocabulary entries; no more than a tile to a CTA
    (4129, 9999, 1024),   # tiles claimed from counters, dH and dW on two streams
    (2100, 3001, 1088)])  # Hd no multiple of 256: pairs for dz alone
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
def test_pairs_of_ctas_give_the_same_bits(tt, N, V, Hd, dw_dtype):
    """Every product by single CTAs, by pairs, and as the call chooses: equal bit for bit, on any number of SMs."""
    from tests.test_gpu_timeout import _head_inputs, _head_path_test
    H, W, y, dl, de = _head_inputs(N, V, Hd)
    _, h, lse = tt.lmhead_token_logprob(H, W, y)
    ref = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, dentropy=de, dw_dtype=dw_dtype)
    for path in (1, 2):
        rc, err, dh, dw = _head_path_test(tt, H, W, y, lse, h, dl, de, path, dw_dtype=dw_dtype)
        assert rc == 0 and err == 0
        assert torch.equal(dh, ref[0]) and torch.equal(dw, ref[1]), path


@pytest.mark.parametrize("N,V,Hd,claims", [
    (40, 700, 64, False),       # a tile or less to a CTA in all three products
    (19000, 256, 8192, True),   # dH alone has several waves of tiles
    (2100, 3001, 1088, True)])  # 108 pair tiles of dz, of which one to two SMs run at a time
def test_tiles_are_claimed_where_a_product_has_several_waves(tt, N, V, Hd, claims):
    """Tiles are claimed from counters, behind dz in the workspace, where any of the three products has more tiles than
    run at once; each counter ends at its product's tiles or above, and is not touched otherwise."""
    g = torch.Generator(device="cuda").manual_seed(N)
    H = torch.randn(N, Hd, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, Hd, generator=g, device="cuda") * (2 / Hd ** 0.5)).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    _, h, lse = tt.lmhead_token_logprob(H, W, y)
    dl = torch.randn(N, generator=g, device="cuda")
    ws = torch.full((tt.lib().tt_lmhead_token_logprob_bwd_workspace_bytes(N, V, Hd),), 0xff, dtype=torch.uint8,
                    device="cuda")
    dh, dw = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, ws=ws)
    at = (N * ((V + 15) // 16 * 16) * 2 + 255) // 256 * 256
    counters = ws[at:at + 12].clone().view(torch.int32).tolist()
    assert all(c > 0 for c in counters) if claims else counters == [-1] * 3
    z = H.float() @ W.float().T
    dz = -torch.softmax(z, 1) * dl[:, None]
    dz[torch.arange(N, device="cuda"), y.long()] += dl
    for x, r in ((dh, dz @ W.float()), (dw, dz.T @ H.float())):
        assert ((x.float() - r).norm() / r.norm()).item() <= GRAD_RL2


@pytest.mark.parametrize("N,V,Hd", [(3, 1, 64), (77, 1000, 64), (300, 3001, 128), (40, 70_001, 1024), (2000, 20_001, 256)])
def test_nan_in_hidden_and_in_the_vocabulary(tt, N, V, Hd):
    """A row of hidden with a NaN has nothing but NaN logits: its three outputs are NaN (an lse of -inf would say that
    the row has no distribution); the other rows keep their bits. A row of W with a NaN gives NaN in every row, alone or with the whole vector of
    columns that an epilogue step takes."""
    from tests.test_gpu_timeout import _head_inputs
    H, W, y, _, _ = _head_inputs(N, V, Hd)
    ref = tt.lmhead_token_logprob(H, W, y)
    rows = sorted({0, N // 2, N - 1})
    bad = H.clone()
    for i, r in enumerate(rows):
        bad[r, (17 * i) % Hd] = float("nan")
    bad[rows[-1]] = float("nan")
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[rows] = False
    err = tt.new_err("cuda")
    for t, r in zip(tt.lmhead_token_logprob(bad, W, y, err=err), ref):
        assert torch.isnan(t[rows]).all() and torch.equal(t[keep], r[keep])
    assert int(err.item()) == 0
    for lo, hi in ((V - 1, V), (0, min(V, 32)), (V // 64 * 32, V // 64 * 32 + 32)):
        w = W.clone()
        w[lo:hi, 3] = float("nan")
        for t in tt.lmhead_token_logprob(H, w, y):
            assert torch.isnan(t).all(), (lo, hi)
