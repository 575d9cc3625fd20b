"""Workloads of the per-token operators: rotary positions, token log-probabilities with entropy and top
alternatives (on logits and fused with the LM head), and their gradients.

A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` is one pass of it (the library's
calls where `own` is true, elementary torch operations where it is false) and `exact` its result in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # ---- log-prob, entropy and top alternatives of given logits
        # one token of a running rollout: the call's latency
        {"name": "score_one_token", "op": "token_logprob", "N": 1, "V": 151936, "ld": 151936, "dtype": "bf16", "k": 20,
         "masked": 0.0},
        # the next tokens of a batch of rollouts, fp32 logits, part of the vocabulary masked out
        {"name": "score_batch_fp32", "op": "token_logprob", "N": 64, "V": 151936, "ld": 151936, "dtype": "fp32",
         "k": 8, "masked": 0.3},
        # odd vocabulary, rows packed without padding (no row but the first aligned)
        {"name": "score_odd_rows_fp16", "op": "token_logprob", "N": 1537, "V": 32003, "ld": 32003, "dtype": "fp16",
         "k": 5, "masked": 0.0},
        # every token of a rollout tree, log-prob and entropy with the 8 best alternatives
        {"name": "score_tree", "op": "token_logprob", "N": 12669, "V": 151936, "ld": 151936, "dtype": "bf16", "k": 8,
         "masked": 0.0},
        # ---- gradient of those with respect to the logits
        # every token of a rollout tree, objective of log-prob and entropy
        {"name": "grad_tree", "op": "token_logprob_bwd", "N": 12669, "V": 151936, "ld": 151936, "dtype": "bf16",
         "k": 0, "masked": 0.0},
        # distillation on the top alternatives, odd vocabulary in padded fp32 rows
        {"name": "grad_top_odd_fp32", "op": "token_logprob_bwd", "N": 511, "V": 32003, "ld": 32064, "dtype": "fp32",
         "k": 16, "masked": 0.1},
        # ---- rotary positions of Q and K
        # one token of a running rollout
        {"name": "rope_one_token", "op": "rope", "N": 1, "Hq": 16, "Hkv": 8, "d": 128, "rot": 128, "axes": 1,
         "interleaved": False, "adjacent": False, "far": 4096, "dtype": "bf16"},
        # a deep agentic tree with image segments: three axes
        {"name": "rope_tree_3_axes", "op": "rope", "N": 65536, "Hq": 40, "Hkv": 8, "d": 128, "rot": 128, "axes": 3,
         "interleaved": False, "adjacent": False, "far": 65536, "dtype": "bf16"},
        # gradients of Q and K: adjacent pairs, half of each head rotated, far positions, an odd number of tokens
        {"name": "rope_bwd_partial_far", "op": "rope_bwd", "N": 12669, "Hq": 32, "Hkv": 8, "d": 128, "rot": 64,
         "axes": 2, "interleaved": True, "adjacent": True, "far": 1000000, "dtype": "fp32"},
        # ---- LM head fused with log-prob and entropy
        # a few rows: bound by reading the vocabulary matrix
        {"name": "head_few_rows", "op": "lmhead", "N": 61, "V": 151936, "Hd": 2048},
        # every token of a rollout tree
        {"name": "head_tree", "op": "lmhead", "N": 12669, "V": 151936, "Hd": 2048},
        # a training step: forward and backward, ragged sizes
        {"name": "head_step_ragged", "op": "lmhead_step", "N": 4001, "V": 32003, "Hd": 1024},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["token_logprob", "token_logprob", "token_logprob_bwd", "rope", "rope_bwd", "lmhead",
                     "lmhead_step"])
    if op in ("token_logprob", "token_logprob_bwd"):
        V = _log_uniform(rng, 1000, 160000)
        N = _log_uniform(rng, 1, max(2, min(20000, 400000000 // V)))
        pad = rng.choice([0, 0, -V % 64, 1 + rng.randrange(100)])
        return {"op": op, "N": N, "V": V, "ld": V + pad, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "k": rng.choice([0, 1, rng.randrange(2, 33)]), "masked": rng.choice([0.0, 0.0, rng.uniform(0.0, 0.9)])}
    if op in ("rope", "rope_bwd"):
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        rot = rng.choice([d, d, d // 2])
        return {"op": op, "N": _log_uniform(rng, 1, 30000), "Hq": hkv * rng.choice([1, 2, 4, 5, 7]), "Hkv": hkv, "d": d,
                "rot": rot, "axes": rng.choice([1, 2, 3]), "interleaved": rng.random() < 0.5,
                "adjacent": rng.random() < 0.3, "far": _log_uniform(rng, 64, 2000000),
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    V = _log_uniform(rng, 1000, 160000)
    Hd = 64 * _log_uniform(rng, 1, 32)
    N = _log_uniform(rng, 1, max(2, min(6000, int(3e11 / V / Hd))))
    return {"op": op, "N": N, "V": V, "Hd": Hd}


# ------------------------------------------------------------------ inputs
def _logits(case, g):
    """Normal logits of deviation 2, a share of them masked with -inf (token 0 never)."""
    N, V, ld = case["N"], case["V"], case["ld"]
    z = torch.randn(N, ld, generator=g, device=DEV, dtype=DTYPES[case["dtype"]]).mul_(2)[:, :V]
    if case["masked"] > 0:
        m = torch.rand(V, generator=g, device=DEV) < case["masked"]
        m[0] = False
        z[:, m] = -math.inf
    return z


def _visible_targets(z, g):
    """Targets among the unmasked tokens."""
    ids = torch.nonzero(z[0] > -math.inf)[:, 0]
    return ids[torch.randint(0, ids.numel(), (z.shape[0],), generator=g, device=DEV)].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    N = case["N"]
    if case["op"] in ("token_logprob", "token_logprob_bwd"):
        s["z"] = _logits(case, g)
        s["y"] = _visible_targets(s["z"], g)
        if case["op"] == "token_logprob_bwd":
            # what the forward pass left, and the gradients of an objective with respect to it
            z = s["z"].float()
            s["lse"] = torch.logsumexp(z, 1)
            z = z.sub_(s["lse"][:, None])
            s["entropy"] = -torch.where(z > -math.inf, z * z.exp(), 0.0).sum(1)
            s["dlogp"] = torch.randn(N, generator=g, device=DEV)
            s["dentropy"] = 0.1 * torch.randn(N, generator=g, device=DEV)
            if case["k"]:
                k = case["k"]
                s["top_ids"] = torch.topk(z, k, dim=1)[1].to(torch.int32)
                s["dtop"] = torch.randn(N, k, generator=g, device=DEV) / k
    elif case["op"] in ("rope", "rope_bwd"):
        t = DTYPES[case["dtype"]]
        s["q"] = torch.randn(N, case["Hq"], case["d"], generator=g, device=DEV, dtype=t)
        s["k"] = torch.randn(N, case["Hkv"], case["d"], generator=g, device=DEV, dtype=t)
        s["pos"] = torch.randint(0, case["far"], (case["axes"], N), generator=g, device=DEV, dtype=torch.int32)
        # the tables a program keeps: each frequency's axis and its value
        half = case["rot"] // 2
        s["axis"] = torch.tensor(_axis_of(case), device=DEV)
        s["freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    else:
        V, Hd = case["V"], case["Hd"]
        s["h"] = torch.randn(N, Hd, generator=g, device=DEV, dtype=torch.bfloat16)
        s["w"] = (torch.randn(V, Hd, generator=g, device=DEV) * (2 / math.sqrt(Hd))).to(torch.bfloat16)
        s["y"] = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
        if case["op"] == "lmhead_step":
            s["dlogp"] = torch.randn(N, generator=g, device=DEV)
            s["dentropy"] = 0.1 * torch.randn(N, generator=g, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def _sections(case):
    """Frequencies of each axis: half of them the first axis's, the rest shared."""
    half, axes = case["rot"] // 2, case["axes"]
    rest = [half // (2 * axes)] * (axes - 1)
    return [half - sum(rest)] + rest


def _axis_of(case):
    """Axis of each frequency: whole sections, or the axes in turn until a section is used up."""
    sec = _sections(case)
    if not case["interleaved"]:
        return [a for a, n in enumerate(sec) for _ in range(n)]
    return [a for i in range(max(sec)) for a, n in enumerate(sec) if i < n]


def _token_logprob(z, y, k):
    z = z.float()
    m = z.amax(1, keepdim=True)
    d = z - m
    e = d.exp()
    total = e.sum(1)
    lse = m[:, 0] + total.log()
    entropy = total.log() - (e * torch.where(e > 0, d, 0.0)).sum(1) / total
    logp = z.gather(1, y.long()[:, None])[:, 0] - lse
    out = {"logp": logp, "entropy": entropy, "lse": lse}
    if k:
        # one integer per element that orders by value, then by the lower index
        bits = (z + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7fffffff)).long() << 32
        key |= 0x7fffffff - torch.arange(z.shape[1], device=z.device)
        ids = 0x7fffffff - (torch.topk(key, k, dim=1)[0] & 0x7fffffff)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logp"] = z.gather(1, ids) - lse[:, None]
    return out


def _dlogits(z, lse, entropy, y, dlogp, dentropy, top_ids=None, dtop=None):
    lp = z.float() - lse[:, None]
    p = lp.exp()
    lp = torch.where(p > 0, lp, 0.0)
    whole = dlogp if dtop is None else dlogp + dtop.sum(1)
    dz = -p * (whole[:, None] + dentropy[:, None] * (lp + entropy[:, None]))
    dz.scatter_add_(1, y.long()[:, None], dlogp[:, None])
    if dtop is not None:
        dz.scatter_add_(1, top_ids.long(), dtop)
    return dz.to(z.dtype)


def _rotate(case, x, c, s):
    rot, half = case["rot"], case["rot"] // 2
    a = x[..., 0:rot:2] if case["adjacent"] else x[..., :half]
    b = x[..., 1:rot:2] if case["adjacent"] else x[..., half:rot]
    a, b = a.float(), b.float()
    u, v = a * c - b * s, b * c + a * s
    turned = torch.stack((u, v), -1).flatten(-2) if case["adjacent"] else torch.cat((u, v), -1)
    return torch.cat((turned.to(x.dtype), x[..., rot:]), -1)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import prefix_tree_gb300 as tt
        if op == "token_logprob":
            logp, entropy, lse, ids, top = tt.token_logprob(s["z"], s["y"], top_k=case["k"], err=s["err"])
            out = {"logp": logp, "entropy": entropy, "lse": lse}
            return out | {"top_ids": ids, "top_logp": top} if case["k"] else out
        if op == "token_logprob_bwd":
            return tt.token_logprob_bwd(s["z"], s["lse"], s["entropy"], s["y"], dlogp=s["dlogp"],
                                        dentropy=s["dentropy"], top_ids=s.get("top_ids"), dtop=s.get("dtop"),
                                        err=s["err"])
        if op in ("rope", "rope_bwd"):
            call = tt.rope if op == "rope" else tt.rope_bwd
            return call(s["q"], s["k"], s["pos"], rot_dim=case["rot"], sections=_sections(case),
                        interleaved=case["interleaved"], adjacent=case["adjacent"], base=10000.0)
        logp, entropy, lse = tt.lmhead_token_logprob(s["h"], s["w"], s["y"], err=s["err"])
        out = {"logp": logp, "entropy": entropy, "lse": lse}
        if op == "lmhead_step":
            out["dh"], out["dw"] = tt.lmhead_token_logprob_bwd(s["h"], s["w"], s["y"], lse, entropy, dlogp=s["dlogp"],
                                                               dentropy=s["dentropy"], dw_dtype=torch.bfloat16,
                                                               err=s["err"])
        return out
    if op == "token_logprob":
        return _token_logprob(s["z"], s["y"], case["k"])
    if op == "token_logprob_bwd":
        return _dlogits(s["z"], s["lse"], s["entropy"], s["y"], s["dlogp"], s["dentropy"], s.get("top_ids"),
                        s.get("dtop"))
    if op in ("rope", "rope_bwd"):
        at = (s["pos"][s["axis"]].T.double() * s["freq"])[:, None] * (1 if op == "rope" else -1)
        c, sn = at.cos().float(), at.sin().float()
        return _rotate(case, s["q"], c, sn), _rotate(case, s["k"], c, sn)
    z = s["h"].float() @ s["w"].float().T
    out = _token_logprob(z, s["y"], 0)
    if op == "lmhead_step":
        dz = _dlogits(z, out["lse"], out["entropy"], s["y"], s["dlogp"], s["dentropy"])
        out["dh"] = (dz @ s["w"].float()).to(torch.bfloat16)
        out["dw"] = (dz.T @ s["h"].float()).to(torch.bfloat16)
    return out


def work(case):
    N = case["N"]
    if case["op"] == "token_logprob":
        es = DTYPES[case["dtype"]].itemsize
        return {"bytes": N * (case["V"] * es + 4 + 12 + 8 * case["k"]), "flops": 5 * N * case["V"]}
    if case["op"] == "token_logprob_bwd":
        es = DTYPES[case["dtype"]].itemsize
        return {"bytes": N * (2 * case["V"] * es + 20 + 8 * case["k"]), "flops": 6 * N * case["V"]}
    if case["op"] in ("rope", "rope_bwd"):
        es = DTYPES[case["dtype"]].itemsize
        heads = case["Hq"] + case["Hkv"]
        return {"bytes": N * (2 * heads * case["d"] * es + 4 * case["axes"]), "flops": 3 * N * heads * case["rot"]}
    V, Hd = case["V"], case["Hd"]
    if case["op"] == "lmhead":
        return {"bytes": 2 * (N + V) * Hd + 16 * N, "flops": 2 * N * V * Hd}
    return {"bytes": 4 * (N + V) * Hd + 24 * N, "flops": 6 * N * V * Hd}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rows(z, y, k):
    """Definition on the rows of z: p = softmax(z), logp = log p_y, entropy = -Σ p log p."""
    z = z.double()
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    out = [lp[torch.arange(z.shape[0], device=z.device), y.long()], -torch.special.xlogy(lp.exp(), lp.exp()).sum(1), lse]
    return out + [torch.topk(lp, k, dim=1)[0]] if k else out


def _exact_dz(z, lse, entropy, y, dlogp, dentropy, ids, dtop):
    """dz_v = Σ over the outputs of their gradient times d output / d z_v."""
    lp = z.double() - lse.double()[:, None]
    p = lp.exp()
    rows = torch.arange(z.shape[0], device=z.device)
    dz = -dentropy.double()[:, None] * (torch.special.xlogy(p, p) + p * entropy.double()[:, None])
    dz -= dlogp.double()[:, None] * p
    dz[rows, y.long()] += dlogp.double()
    if ids is not None:
        dz -= dtop.double().sum(1, keepdim=True) * p
        dz[rows[:, None], ids.long()] += dtop.double()
    return dz


def exact(case, seed):
    s = prepare(case, seed)
    op, N = case["op"], case["N"]
    step = 512
    parts = [slice(i, min(N, i + step)) for i in range(0, N, step)]
    if op == "token_logprob":
        cols = [torch.cat(c) for c in zip(*[_exact_rows(s["z"][i], s["y"][i], case["k"]) for i in parts])]
        out = {"logp": cols[0], "entropy": cols[1], "lse": cols[2]}
        return out | {"top_ids": None, "top_logp": cols[3]} if case["k"] else out
    if op == "token_logprob_bwd":
        got = torch.empty(N, case["V"], dtype=torch.float64, device=DEV)
        for i in parts:
            got[i] = _exact_dz(s["z"][i], s["lse"][i], s["entropy"][i], s["y"][i], s["dlogp"][i], s["dentropy"][i],
                               s["top_ids"][i] if case["k"] else None, s["dtop"][i] if case["k"] else None)
        return got
    if op in ("rope", "rope_bwd"):
        half = case["rot"] // 2
        out = []
        axis = _axis_of(case)
        for x in (s["q"], s["k"]):
            x = x.double()
            y = x.clone()
            for i in range(half):
                at = s["pos"][axis[i]].double() * 10000.0 ** (-i / half) * (1 if op == "rope" else -1)
                at = at[:, None]
                j, l = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + half)
                turn = torch.polar(torch.ones_like(at), at) * torch.complex(x[..., j], x[..., l])
                y[..., j], y[..., l] = turn.real, turn.imag
            out.append(y)
        return out
    V, Hd = case["V"], case["Hd"]
    if 2 * N * V * Hd * (1 if op == "lmhead" else 3) > 12e12:
        return None
    w = s["w"].double()
    rows, dh, dw = [], [], torch.zeros(V, Hd, dtype=torch.float64, device=DEV) if op == "lmhead_step" else None
    for i in parts:
        h = s["h"][i].double()
        z = h @ w.T
        rows.append(_exact_rows(z, s["y"][i], 0))
        if op == "lmhead_step":
            dz = _exact_dz(z, rows[-1][2], rows[-1][1], s["y"][i], s["dlogp"][i], s["dentropy"][i], None, None)
            dh.append(dz @ w)
            dw += dz.T @ h
    cols = [torch.cat(c) for c in zip(*rows)]
    out = {"logp": cols[0], "entropy": cols[1], "lse": cols[2]}
    return out | {"dh": torch.cat(dh), "dw": dw} if op == "lmhead_step" else out
