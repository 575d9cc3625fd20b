"""A policy step through all its calls: rollouts sampled token by token over a shared prompt, then their tree trained with
the clipped objective; and tensors whose offsets pass 2^31 elements."""
import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import lmhead as LH
from oracle import norm_rope as NR
from oracle import policy as P
from oracle import token_logprob as TL
from oracle import tree as T
from tests._util import GRAD_RL2, LSE_RTOL, O_ATOL, dev_to_f64, rel_l2, to_dev_bf16

pytestmark = pytest.mark.gpu

HQ, HKV, D, V = 4, 2, 64, 1000


def _model(rng, N):
    """Q, K, V before their norms for N tokens, the norms' weights, the head."""
    q, k, v = (to_dev_bf16(synth.normal_bf16(rng, (N, n, D))) for n in (HQ, HKV, HKV))
    wq, wk = (to_dev_bf16(synth.normal_bf16(rng, (D,), 0.2)) + 1 for _ in range(2))
    return q, k, v, wq, wk, to_dev_bf16(synth.normal_bf16(rng, (V, HQ * D), 0.1))


def test_training_step_over_a_tree(tt):
    """Norm with rotary positions -> tree attention -> fused head -> objective -> backward of all of it, against the fp64
    oracles of the same chain."""
    sh = synth.tree_shape(0)
    tab = T.tables(sh.seg_parent, sh.seg_len)
    N, rng = sh.N, np.random.default_rng(1)
    q0, k0, v, wq, wk, W = _model(rng, N)
    y = torch.tensor(rng.integers(0, V, N), dtype=torch.int32, device="cuda")
    tree = tt.tree_build(torch.tensor(sh.seg_parent, device="cuda"), torch.tensor(sh.seg_len, device="cuda"))
    err = tt.new_err("cuda")
    # forward
    q, k = tt.qk_norm_rope(q0, k0, tree.tok_pos, wq, wk)
    O, LSE = tt.tree_attn_fwd(tree, q, k, v, err=err)
    hid = O.view(N, HQ * D)
    logp, ent, lse = tt.lmhead_token_logprob(hid, W, y, err=err)
    # what the sampler and the rollouts' scores left: advantages of the branches, summed by sign at every token
    leaves, at = np.flatnonzero(tab.tok_send == np.arange(N) + 1), np.arange(N)
    through = ((at <= leaves[:, None]) & (leaves[:, None] < tab.tok_send)).astype(float)
    B = len(leaves)
    assert (through.sum(0) == tab.tok_leafcnt).all()
    adv = rng.standard_normal(B)
    gain, cost = np.maximum(adv, 0) @ through / B, np.maximum(-adv, 0) @ through / B
    w = (tab.tok_pos >= 16).astype(np.float32)  # the first tokens are the prompt
    lp = dev_to_f64(logp)
    move = rng.uniform(-0.15, 0.15, N)
    far = rng.random(N) < 0.1
    move[far] = np.where(rng.random(N) < 0.5, 0.5, -0.5)[far]
    old, ref = (lp - move).astype(np.float32), (lp + 0.1 * rng.standard_normal(N)).astype(np.float32)
    dev = lambda a: torch.tensor(np.asarray(a, np.float32), device="cuda")
    how = dict(clip=(0.2, 0.3), kl_coef=0.1, entropy_coef=0.01)
    args = dict(adv_neg=dev(cost), ref_logp=dev(ref), weights=dev(w))
    sums, dlogp, dent = tt.policy_loss(logp, dev(old), dev(gain), entropy=ent, **args, **how)
    # backward
    dh, dw = tt.lmhead_token_logprob_bwd(hid, W, y, lse, ent, dlogp=dlogp, dentropy=dent, err=err)
    dq, dk, dv = tt.tree_attn_bwd(tree, q, k, v, O, LSE, dh.view(N, HQ, D), err=err)
    dq0, dk0, dwq, dwk = tt.qk_norm_rope_bwd(dq, dk, q0, k0, tree.tok_pos, wq, wk)
    torch.cuda.synchronize()
    tree.check()
    assert int(err.item()) == 0

    nr = {"tables": (tab.tok_pos[None], np.zeros(D // 2, int), 10000.0 ** (-np.arange(D // 2) / (D // 2))),
          "adjacent": False}
    f = dev_to_f64
    rq, rk = NR.forward(f(q0), f(wq), 1e-6, nr), NR.forward(f(k0), f(wk), 1e-6, nr)
    rO = A.tree_attention_branches(tab, rq, rk, f(v), np.zeros((N, HQ, D)))[0]
    z = LH.logits(rO.reshape(N, -1), f(W))
    yn = y.cpu().numpy()
    r_logp, r_ent, _, _, _ = TL.token_logprob(z, yn)
    # as in the chain of the fused head: bf16 Q, K and O lie in front of the logits
    assert np.abs(lp - r_logp).max() <= 0.04 and np.abs(f(ent) - r_ent).max() <= 0.04
    # the objective itself at the log-probs that it got
    r_sums, r_dlogp, r_dent = P.objective(lp, old, gain, cost, ref, f(ent), w, lo=0.2, hi=0.3, kl=0.1, ent=0.01)
    # fp32: log r = logp − old is exact (both near), exp within 2^-22 and four roundings behind it, of values below 4
    assert np.abs(f(sums) - r_sums).max() <= 1e-5 * np.abs(r_sums).max() and np.abs(f(dlogp) - r_dlogp).max() <= 2e-6
    assert (np.abs(f(dent) - r_dent) <= 1e-8).all() and (f(dlogp)[w == 0] == 0).all()
    dz = TL.token_logprob_grad(z, yn, f(dlogp), f(dent))
    r_dh = dz @ f(W)
    _, _, r_dq, r_dk, r_dv = A.tree_attention_branches(tab, rq, rk, f(v), r_dh.reshape(N, HQ, D))
    r_dq0, r_dwq = NR.backward(r_dq, f(q0), f(wq), 1e-6, nr)
    r_dk0, r_dwk = NR.backward(r_dk, f(k0), f(wk), 1e-6, nr)
    # each stage rounds to bf16 (2^-8): five of them lie between the inputs and dq0, dk0
    for got, want in ((dh, r_dh), (dw, dz.T @ rO.reshape(N, -1)), (dv, r_dv), (dq0, r_dq0), (dk0, r_dk0), (dwq, r_dwq),
                      (dwk, r_dwk)):
        assert rel_l2(f(got).reshape(want.shape), want) <= 2.5 * GRAD_RL2, rel_l2(f(got).reshape(want.shape), want)

    # the same step on stored logits, in one call: the head's own log-probs up to the order of their sums
    zb = hid.float() @ W.float().T
    s2, lp2, e2, dz2 = tt.policy_loss_logits(zb, y, dev(old), dev(gain), err=err, **args, **how)
    on = torch.tensor(w > 0, device="cuda")
    assert (lp2 - logp)[on].abs().max().item() <= 1e-4 and (e2 - ent)[on].abs().max().item() <= 2e-4
    assert (lp2[~on] == 0).all() and (dz2[~on] == 0).all()
    assert (s2 - sums).abs().max().item() <= 3e-4 * float(w.sum())
    assert rel_l2(f(dh), f(dz2) @ f(W)) <= GRAD_RL2
    # and as three calls
    lp3, e3, lse3, _, _ = tt.token_logprob(zb, y, err=err)
    s3, dl3, de3 = tt.policy_loss(lp3, dev(old), dev(gain), entropy=e3, **args, **how)
    dz3 = tt.token_logprob_bwd(zb, lse3, e3, y, dlogp=dl3, dentropy=de3, err=err)
    # log-probs to 2^-22 of their rounding apart: the gradients, of size <= 1, by as much times the slopes
    assert (s2 - s3).abs().max().item() <= 2e-5 * float(w.sum()) and (dz2 - dz3).abs().max().item() <= 2e-5
    assert int(err.item()) == 0


def test_sampled_rollouts_see_what_training_sees(tt):
    """Five rollouts of one prompt grow token by token: norm with rotary positions into the pool's rows, attention over
    prompt and own rows. Every step's attention is the row that the training attention gives that token in the tree."""
    rng = np.random.default_rng(2)
    prompt, steps, R = 150, 9, 5
    lens = [steps] * R
    N = prompt + R * steps
    q0, k0, v0, wq, wk, _ = _model(rng, N)  # tokens in DFS order: the prompt, then rollout after rollout
    tree = tt.tree_build(torch.tensor([-1] + [0] * R, dtype=torch.int32, device="cuda"),
                         torch.tensor([prompt] + lens, dtype=torch.int32, device="cuda"))
    q, k = tt.qk_norm_rope(q0, k0, tree.tok_pos, wq, wk)
    O, LSE = tt.tree_attn_fwd(tree, q, k, v0)
    # the pool: the prompt's rows, then room for every rollout
    room = 64
    pool_k = torch.full((prompt + R * room, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool_v = pool_k.clone()
    pos = torch.arange(prompt, dtype=torch.int32, device="cuda")
    tt.qk_norm_rope(q0[:prompt], k0[:prompt], pos, wq, wk, out=(torch.empty_like(q0[:prompt]), pool_k[:prompt]))
    pool_v[:prompt] = v0[:prompt]
    table = torch.tensor([[0] + [prompt + r * room for r in range(R)], [prompt] + [0] * R, [0] + list(range(R)),
                          [R] + list(range(1, R + 1))], dtype=torch.int32, device="cuda")
    err = tt.new_err("cuda")
    for t in range(steps):
        rows = torch.tensor([prompt + r * steps + t for r in range(R)], device="cuda")
        at = torch.full((R,), prompt + t, dtype=torch.int32, device="cuda")
        qn, kn = tt.qk_norm_rope(q0[rows].contiguous(), k0[rows].contiguous(), at, wq, wk)
        assert torch.equal(qn, q[rows]) and torch.equal(kn, k[rows])  # one token or many: the same bits
        into = torch.tensor([prompt + r * room + t for r in range(R)], device="cuda")
        pool_k[into], pool_v[into] = kn, v0[rows]
        table[1, 1:] += 1
        plan = tt.tree_decode_plan(table, R, pool_k.shape[0], 2 * R, HQ, HKV, D, err=err)
        o, lse = tt.tree_decode_attn(plan, qn, pool_k, pool_v)
        assert (o.float() - O[rows].float()).abs().max().item() <= O_ATOL
        assert ((lse - LSE[:, rows]).abs() <= 2 * LSE_RTOL * LSE[:, rows].abs().clamp(min=1)).all()
    assert int(err.item()) == 0


def test_offsets_past_32_bits(tt):
    """Logits and heads of more than 2^31 elements: the last rows as in a small call of their own."""
    N, Vb = 16_500, 131_072
    z = torch.empty(N, Vb, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = slice(N - 5, N)
    z[:] = 0
    z[tail] = torch.randn(5, Vb, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, Vb, (N,), generator=g, device="cuda", dtype=torch.int32)
    old, adv = torch.full((N,), -12.0, device="cuda"), torch.randn(N, generator=g, device="cuda")
    w = torch.zeros(N, device="cuda")
    w[tail] = 1
    _, lp, h, dz = tt.policy_loss_logits(z, y, old, adv, weights=w, clip=0.1)
    _, lp2, h2, dz2 = tt.policy_loss_logits(z[tail].clone(), y[tail].clone(), old[tail].clone(), adv[tail].clone(),
                                            weights=w[tail].clone(), clip=0.1)
    # (how many CTAs share a row may differ: the order of its sums)
    assert (lp[tail] - lp2).abs().max().item() <= 2e-6 and (h[tail] - h2).abs().max().item() <= 2e-5
    assert (dz[tail].float() - dz2.float()).abs().max().item() <= 2.0 ** -7 * dz2.float().abs().max().item()
    assert (dz[:N - 5].view(torch.int16) == 0).all()
    del z, dz
    n, hq, d = 1_100_000, 16, 128
    q = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    q[-5:] = torch.randn(5, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    yq, _ = tt.qk_norm_rope(q, None, pos)
    y5, _ = tt.qk_norm_rope(q[-5:].clone(), None, pos[-5:].clone())
    assert torch.equal(yq[-5:], y5)
    dq, _, _, _ = tt.qk_norm_rope_bwd(yq, None, q, None, pos)
    d5, _, _, _ = tt.qk_norm_rope_bwd(y5, None, q[-5:].clone(), None, pos[-5:].clone())
    assert torch.equal(dq[-5:], d5)
