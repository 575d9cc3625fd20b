"""Workloads of the operators around a policy step over rollout trees: the norm of every head of Q and K with the
rotary positions (forward and backward), the clipped policy objective (from log-probs, and from logits with their
gradient), and the attention of the next token of every running rollout over shared and own segments.

A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` is one pass of it (the library's
calls where `own` is true, elementary torch operations where it is false) and `exact` its result in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"
EPS = 1e-6
CLIP_LO, CLIP_HI, DUAL = 0.2, 0.28, 3.0


def listed():
    return [
        # ---- norm of the heads of Q and K with the rotary positions
        # the next token of one rollout: the call's latency
        {"name": "norm_rope_one_token", "op": "norm_rope", "N": 1, "Hq": 16, "Hkv": 8, "d": 128, "rot": 128,
         "axes": 1, "adjacent": False, "far": 4096, "dtype": "bf16"},
        # every token of a deep agentic tree
        {"name": "norm_rope_deep_tree", "op": "norm_rope", "N": 65536, "Hq": 40, "Hkv": 8, "d": 128, "rot": 128,
         "axes": 1, "adjacent": False, "far": 65536, "dtype": "bf16"},
        # gradients over a rollout tree
        {"name": "norm_rope_bwd_tree", "op": "norm_rope_bwd", "N": 12669, "Hq": 16, "Hkv": 8, "d": 128, "rot": 128,
         "axes": 1, "adjacent": False, "far": 8192, "dtype": "bf16"},
        # gradients, fp32, an odd number of tokens and heads, half of each head turned, two axes, adjacent pairs
        {"name": "norm_rope_bwd_odd_fp32", "op": "norm_rope_bwd", "N": 4001, "Hq": 5, "Hkv": 1, "d": 64, "rot": 32,
         "axes": 2, "adjacent": True, "far": 100000, "dtype": "fp32"},
        # ---- clipped policy objective from log-probs (as the fused head gives them)
        # the tokens of a short rollout
        {"name": "policy_short", "op": "policy", "N": 500, "entropy": False, "ref": False, "two_sided": False,
         "masked": 0.2},
        # eight packs of 65,536 tree tokens, every term
        {"name": "policy_packs", "op": "policy", "N": 524288, "entropy": True, "ref": True, "two_sided": True,
         "masked": 0.1},
        # ---- the same from logits, with their gradient
        # few rows: the end of one rollout
        {"name": "policy_logits_few", "op": "policy_logits", "N": 61, "V": 151936, "ld": 151936, "dtype": "bf16",
         "ref": True, "two_sided": False, "masked": 0.0},
        # every token of a rollout tree whose prompt is masked
        {"name": "policy_logits_tree", "op": "policy_logits", "N": 12669, "V": 151936, "ld": 151936, "dtype": "bf16",
         "ref": True, "two_sided": True, "masked": 0.16},
        # odd vocabulary in unpadded fp32 rows
        {"name": "policy_logits_odd_fp32", "op": "policy_logits", "N": 1537, "V": 32003, "ld": 32003, "dtype": "fp32",
         "ref": False, "two_sided": False, "masked": 0.1},
        # ---- attention of the next token of every running rollout (a step: the plan, then each layer)
        # four rollouts that have just left a short prompt
        {"name": "decode_few_short", "op": "decode", "levels": "1x509-509 4x1-40", "Hq": 16, "Hkv": 8,
         "d": 128, "layers": 4, "dtype": "bf16"},
        # a group of 64 rollouts of one prompt
        {"name": "decode_group_64", "op": "decode", "levels": "1x8192-8192 64x100-2048", "Hq": 32, "Hkv": 8,
         "d": 128, "layers": 4, "dtype": "bf16"},
        # a deep tree: a long prompt, common turns, 120 rollouts; five query heads to a key head
        {"name": "decode_deep_tree", "op": "decode", "levels": "1x16001-16001 6x500-4000 20x0-2999", "Hq": 40,
         "Hkv": 8, "d": 128, "layers": 4, "dtype": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "policy", "policy_logits", "policy_logits", "decode", "decode"])
    if op in ("norm_rope", "norm_rope_bwd"):
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "N": _log_uniform(rng, 1, 30000), "Hq": hkv * rng.choice([1, 2, 4, 5, 7]), "Hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2]), "axes": rng.choice([1, 1, 2, 3]), "adjacent": rng.random() < 0.3,
                "far": _log_uniform(rng, 64, 2000000), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    if op == "policy":
        return {"op": op, "N": _log_uniform(rng, 1, 500000), "entropy": rng.random() < 0.5, "ref": rng.random() < 0.5,
                "two_sided": rng.random() < 0.5, "masked": rng.choice([0.0, rng.uniform(0.0, 0.9)])}
    if op == "policy_logits":
        V = _log_uniform(rng, 1000, 160000)
        N = _log_uniform(rng, 1, max(2, min(20000, 400000000 // V)))
        pad = rng.choice([0, 0, -V % 64, 1 + rng.randrange(100)])
        return {"op": op, "N": N, "V": V, "ld": V + pad, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "ref": rng.random() < 0.5, "two_sided": rng.random() < 0.5,
                "masked": rng.choice([0.0, rng.uniform(0.0, 0.9)])}
    hkv = rng.choice([1, 2, 4, 8])
    prompt = _log_uniform(rng, 1, 16000)
    levels = [[1, prompt, prompt]]
    if rng.random() < 0.4:
        levels.append([rng.randrange(2, 7), 1, _log_uniform(rng, 10, 4000)])
    groups = 1 if len(levels) == 1 else levels[1][0]
    levels.append([_log_uniform(rng, 1, 120 // groups), rng.choice([0, 1, 50]), _log_uniform(rng, 60, 2000)])
    return {"op": op, "levels": " ".join("%dx%d-%d" % tuple(x) for x in levels), "Hq": hkv * rng.choice([1, 2, 4, 5, 7]), "Hkv": hkv, "d": rng.choice([64, 128]), "layers": rng.choice([1, 2, 4]),
            "dtype": rng.choice(["bf16", "bf16", "fp16"])}


# ------------------------------------------------------------------ inputs
def _tree_of(case):
    """Segments of a decode case, levels after one another: (rows, first query, one past the last query) each. A level
    "nxlo-hi" gives every segment of the level above n children of lo .. hi rows; a rollout ends at every segment of
    the last level. Lengths come from the case alone: they are part of its size."""
    levels = [tuple(int(x) for x in level.replace("x", "-").split("-")) for level in case["levels"].split()]
    total = math.prod(n for n, _, _ in levels)
    segs, above, x = [], 1, 12345
    for n, lo, hi in levels:
        above *= n
        for i in range(above):
            x = (x * 1103515245 + 12345) % 2147483648  # a small generator of its own
            segs.append((lo + (x >> 8) % (hi - lo + 1), i * (total // above), (i + 1) * (total // above)))
    return segs, total


def _logits(case, g):
    return torch.randn(case["N"], case["ld"], generator=g, device=DEV, dtype=DTYPES[case["dtype"]]).mul_(2)[:, :case["V"]]


def _log_probs(z, y):
    """Log-probs of y in 64 bits, some rows at a time."""
    out = torch.empty(z.shape[0], dtype=torch.float64, device=DEV)
    for i in range(0, z.shape[0], 256):
        x = z[i:i + 256].double()
        out[i:i + 256] = x.gather(1, y[i:i + 256].long()[:, None])[:, 0] - torch.logsumexp(x, 1)
    return out


def _objective_inputs(case, s, logp, g):
    """What a trainer holds beside the policy's log-probs: the sampler's, the reference's, advantages, weights."""
    N = case["N"]
    # how far the policy has moved since sampling; not within 1e-4 of a clip border, where the gradient jumps
    move = 0.15 * torch.randn(N, generator=g, device=DEV, dtype=torch.float64)
    for edge in (math.log1p(-CLIP_LO), math.log1p(CLIP_HI), math.log(DUAL)):
        near = (move - edge).abs() < 1e-4
        move = torch.where(near, move + 3e-4, move)
    s["old_logp"] = (logp - move).float()
    s["adv"] = torch.randn(N, generator=g, device=DEV)
    if case["two_sided"]:  # a shared token has rollouts of both signs behind it
        s["adv_neg"] = 0.5 * torch.rand(N, generator=g, device=DEV)
        s["adv"] = s["adv"].abs()
    if case["ref"]:
        s["ref_logp"] = (logp + 0.1 * torch.randn(N, generator=g, device=DEV, dtype=torch.float64)).float()
    s["weights"] = torch.randint(1, 17, (N,), generator=g, device=DEV).float() / 16
    s["weights"][torch.rand(N, generator=g, device=DEV) < case["masked"]] = 0  # prompt tokens


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        t, N, d = DTYPES[case["dtype"]], case["N"], case["d"]
        for name, h in (("q", case["Hq"]), ("k", case["Hkv"])):
            s[name] = torch.randn(N, h, d, generator=g, device=DEV, dtype=t).mul_(1.5)
            s["w" + name] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t)
            if case["op"] == "norm_rope_bwd":
                s["d" + name] = torch.randn(N, h, d, generator=g, device=DEV, dtype=t)
        s["pos"] = torch.randint(0, case["far"], (case["axes"], N), generator=g, device=DEV, dtype=torch.int32)
        half = case["rot"] // 2
        s["axis"] = torch.tensor(_axis_of(case), device=DEV)
        s["freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    elif case["op"] == "policy":
        s["logp"] = -(2 * torch.randn(case["N"], generator=g, device=DEV)).abs() - 1e-3
        if case["entropy"]:
            s["entropy"] = 3 * torch.rand(case["N"], generator=g, device=DEV)
        _objective_inputs(case, s, s["logp"].double(), g)
    elif case["op"] == "policy_logits":
        s["z"] = _logits(case, g)
        s["y"] = torch.randint(0, case["V"], (case["N"],), generator=g, device=DEV, dtype=torch.int32)
        _objective_inputs(case, s, _log_probs(s["z"], s["y"]), g)
    else:
        t = DTYPES[case["dtype"]]
        segs, B = _tree_of(case)
        # a pool of key and value rows for every layer; segments lie in it with room to grow behind each
        begin, rows = [], 0
        for n, _, _ in segs:
            begin.append(rows)
            rows += n + 32
        s["segs"] = [(b, n, q0, q1) for b, (n, q0, q1) in zip(begin, segs)]
        s["B"] = B
        s["table"] = torch.tensor(s["segs"], dtype=torch.int32, device=DEV).T.contiguous()
        s["pairs"] = sum(q1 - q0 for _, q0, q1 in segs)
        s["q"], s["k"], s["v"] = [], [], []
        for _ in range(case["layers"]):
            s["q"].append(torch.randn(B, case["Hq"], case["d"], generator=g, device=DEV, dtype=t))
            s["k"].append(torch.randn(rows, case["Hkv"], case["d"], generator=g, device=DEV, dtype=t))
            s["v"].append(torch.randn(rows, case["Hkv"], case["d"], generator=g, device=DEV, dtype=t))
    return s


# ------------------------------------------------------------------ one pass
def _sections(case):
    """Frequencies of each axis, one section after the other."""
    half, axes = case["rot"] // 2, case["axes"]
    rest = [half // (2 * axes)] * (axes - 1)
    return [half - sum(rest)] + rest


def _axis_of(case):
    return [a for a, n in enumerate(_sections(case)) for _ in range(n)]


def _rotate(case, x, c, s):
    """fp32 x turned, in the pairs' own places."""
    rot, half = case["rot"], case["rot"] // 2
    a = x[..., 0:rot:2] if case["adjacent"] else x[..., :half]
    b = x[..., 1:rot:2] if case["adjacent"] else x[..., half:rot]
    u, v = a * c - b * s, b * c + a * s
    turned = torch.stack((u, v), -1).flatten(-2) if case["adjacent"] else torch.cat((u, v), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _norm_rope_plain(s):
    case = s["case"]
    at = (s["pos"][s["axis"]].T.double() * s["freq"])[:, None]
    c, sn = at.cos().float(), at.sin().float()
    out = []
    for name in ("q", "k"):
        x = s[name].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        w = s["w" + name].float()
        if case["op"] == "norm_rope":
            out.append(_rotate(case, x * r * w, c, sn).to(s[name].dtype))
            continue
        dn = _rotate(case, s["d" + name].float(), c, -sn)
        h = dn * w
        dx = r * (h - x * r * r * (h * x).mean(-1, keepdim=True))
        out += [dx.to(s[name].dtype), (dn * x * r).sum((0, 1))]
    return out


def _objective(logp, entropy, s):
    """Sums (loss, policy, KL, entropy) and the gradients with respect to logp and entropy; logp in 64 bits."""
    w = s["weights"].double()
    gain, cost = (s["adv"], s["adv_neg"]) if "adv_neg" in s else (s["adv"].clamp(min=0), (-s["adv"]).clamp(min=0))
    gain, cost = gain.double(), cost.double()
    ratio = (logp - s["old_logp"].double()).exp()
    policy = -gain * ratio.clamp(max=1 + CLIP_HI) + cost * ratio.clamp(1 - CLIP_LO, DUAL)
    dlogp = -gain * ratio * (ratio <= 1 + CLIP_HI) + cost * ratio * ((ratio >= 1 - CLIP_LO) & (ratio <= DUAL))
    kl = torch.zeros_like(logp)
    if "ref_logp" in s:
        x = s["ref_logp"].double() - logp
        kl = x.exp() - 1 - x
        dlogp = dlogp - KL * (x.exp() - 1)
    on = w > 0
    ent = torch.zeros_like(logp) if entropy is None else entropy.double()
    sums = torch.stack([torch.where(on, w * t, 0.0).sum() for t in (policy, kl, ent)])
    loss = sums[0] + KL * sums[1] - ENTROPY * sums[2]
    return torch.cat((loss[None], sums)).float(), torch.where(on, w * dlogp, 0.0), torch.where(on, -w * ENTROPY, 0.0)


KL, ENTROPY = 0.05, 0.01  # coefficients of the KL and entropy terms


def _policy_logits_plain(s):
    z = s["z"].float()
    m = z.amax(1, keepdim=True)
    d = z - m
    e = d.exp()
    total = e.sum(1)
    log_total = total.double().log()
    ent = (log_total - ((e * d).sum(1) / total).double())
    logp = (z.gather(1, s["y"].long()[:, None]) - m)[:, 0].double() - log_total
    sums, dlogp, dent = _objective(logp, ent, s)
    dlogp, dent = dlogp.float()[:, None], dent.float()[:, None]
    lp = d - log_total.float()[:, None]
    dz = (e / total[:, None]) * (-dlogp - dent * (lp + ent.float()[:, None]))
    dz.scatter_add_(1, s["y"].long()[:, None], dlogp)
    on = s["weights"] > 0
    return {"sums": sums, "logp": torch.where(on, logp.float(), 0.0), "entropy": torch.where(on, ent.float(), 0.0),
            "dlogits": dz.to(s["z"].dtype)}


def _decode_layer_plain(s, q, k, v):
    """Each shared segment against all its queries at once; the rollouts' own segments as one padded batch."""
    case = s["case"]
    B, Hq, Hkv, d = s["B"], case["Hq"], case["Hkv"], case["d"]
    q = q.float().view(B, Hkv, Hq // Hkv, d) / math.sqrt(d)
    m = torch.full((B, Hkv, Hq // Hkv), -math.inf, device=DEV)
    l, o = torch.zeros_like(m), torch.zeros_like(q)

    def join(q0, q1, sc, value):
        sm = torch.maximum(m[q0:q1], sc.amax(-1))
        safe = torch.where(sm > -math.inf, sm, 0.0)
        p = (sc - safe[..., None]).exp()
        f = torch.where(m[q0:q1] > -math.inf, (m[q0:q1] - safe).exp(), 0.0)
        m[q0:q1], l[q0:q1] = sm, l[q0:q1] * f + p.sum(-1)
        o[q0:q1] = o[q0:q1] * f[..., None] + value(p)

    single = [x for x in s["segs"] if x[3] - x[2] == 1 and x[1] > 0]
    for b, n, q0, q1 in s["segs"]:
        if n == 0 or q1 - q0 == 1:
            continue
        ks, vs = k[b:b + n].float(), v[b:b + n].float()
        join(q0, q1, torch.einsum("bhgd,nhd->bhgn", q[q0:q1], ks), lambda p: torch.einsum("bhgn,nhd->bhgd", p, vs))
    done = 0
    while done < len(single):  # segments of different queries together
        part = []
        while done < len(single) and (not part or single[done][2] > part[-1][2]):
            part.append(single[done])
            done += 1
        longest = max(n for _, n, _, _ in part)
        at = torch.zeros(B, 2, dtype=torch.long)
        for b, n, q0, _ in part:
            at[q0, 0], at[q0, 1] = b, n
        at = at.to(DEV)
        col = torch.arange(longest, device=DEV)
        here = col < at[:, 1:]
        idx = torch.where(here, at[:, :1] + col, 0)
        ks, vs = k[idx].float(), v[idx].float()
        sc = torch.einsum("bhgd,bnhd->bhgn", q, ks).masked_fill(~here[:, None, None], -math.inf)
        join(0, B, sc, lambda p: torch.einsum("bhgn,bnhd->bhgd", p, vs))
    out = torch.where(l[..., None] > 0, o / l[..., None].clamp(min=1e-30), 0.0)
    lse = torch.where(l > 0, m + l.clamp(min=1e-30).log(), -math.inf)
    return out.view(B, Hq, d).to(k.dtype), lse.view(B, Hq).T.contiguous()


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import prefix_tree_gb300 as tt
        if op == "norm_rope":
            return list(tt.qk_norm_rope(s["q"], s["k"], s["pos"], s["wq"], s["wk"], eps=EPS, rot_dim=case["rot"],
                                        sections=_sections(case), adjacent=case["adjacent"]))
        if op == "norm_rope_bwd":
            dq, dk, dwq, dwk = tt.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["wq"], s["wk"],
                                                   eps=EPS, rot_dim=case["rot"], sections=_sections(case),
                                                   adjacent=case["adjacent"])
            return [dq, dwq, dk, dwk]
        how = dict(adv_neg=s.get("adv_neg"), ref_logp=s.get("ref_logp"), weights=s.get("weights"),
                   clip=(CLIP_LO, CLIP_HI), dual_clip=DUAL, kl_coef=KL)
        if op == "policy":
            sums, dlogp, dent = tt.policy_loss(s["logp"], s["old_logp"], s["adv"], entropy=s.get("entropy"),
                                               entropy_coef=ENTROPY if "entropy" in s else 0.0, **how)
            out = {"sums": sums, "dlogp": dlogp}
            return out | {"dentropy": dent} if "entropy" in s else out
        if op == "policy_logits":
            sums, logp, ent, dz = tt.policy_loss_logits(s["z"], s["y"], s["old_logp"], s["adv"], entropy_coef=ENTROPY,
                                                        err=s["err"], **how)
            return {"sums": sums, "logp": logp, "entropy": ent, "dlogits": dz}
        plan = tt.tree_decode_plan(s["table"], s["B"], s["k"][0].shape[0], s["pairs"], case["Hq"], case["Hkv"],
                                   case["d"], err=s["err"])
        out = []
        for q, k, v in zip(s["q"], s["k"], s["v"]):
            out += tt.tree_decode_attn(plan, q, k, v)
        return out
    if op in ("norm_rope", "norm_rope_bwd"):
        return _norm_rope_plain(s)
    if op == "policy":
        sums, dlogp, dent = _objective(s["logp"].double(), s.get("entropy"), s)
        out = {"sums": sums, "dlogp": dlogp.float()}
        return out | {"dentropy": dent.float()} if "entropy" in s else out
    if op == "policy_logits":
        return _policy_logits_plain(s)
    out = []
    for q, k, v in zip(s["q"], s["k"], s["v"]):
        out += _decode_layer_plain(s, q, k, v)
    return out


def work(case):
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        N, d, es = case["N"], case["d"], DTYPES[case["dtype"]].itemsize
        heads = case["Hq"] + case["Hkv"]
        if case["op"] == "norm_rope":
            return {"bytes": N * (2 * heads * d * es + 4 * case["axes"]) + 2 * d * es,
                    "flops": N * heads * (4 * d + 3 * case["rot"])}
        return {"bytes": N * (3 * heads * d * es + 4 * case["axes"]) + 2 * d * (es + 4),
                "flops": N * heads * (12 * d + 3 * case["rot"])}
    if case["op"] == "policy":
        arrays = 5 + 2 * case["entropy"] + case["ref"] + case["two_sided"]
        return {"bytes": 4 * case["N"] * arrays + 16, "flops": 30 * case["N"]}
    if case["op"] == "policy_logits":
        N, V, es = case["N"], case["V"], DTYPES[case["dtype"]].itemsize
        # a masked row's logits are not needed, its gradient is written all the same
        read = int(N * (1 - case["masked"])) * V * es
        return {"bytes": read + N * V * es + N * (24 + 4 * (case["ref"] + case["two_sided"])), "flops": 11 * N * V}
    segs, B = _tree_of(case)
    es, d, L = DTYPES[case["dtype"]].itemsize, case["d"], case["layers"]
    rows = sum(n for n, _, _ in segs)
    pairs = sum(n * (q1 - q0) for n, q0, q1 in segs)
    return {"bytes": L * (2 * rows * case["Hkv"] * d * es + B * case["Hq"] * (2 * d * es + 4)),
            "flops": L * 4 * pairs * case["Hq"] * d}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_norm_rope(case, s):
    half = case["rot"] // 2
    axis = _axis_of(case)
    out = []
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        size = torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["d"] + EPS)
        unit = x / size
        y = unit * w if case["op"] == "norm_rope" else s["d" + name].double().clone()
        for i in range(half):
            at = s["pos"][axis[i]].double() * 10000.0 ** (-i / half) * (1 if case["op"] == "norm_rope" else -1)
            j, l = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + half)
            turn = torch.polar(torch.ones_like(at), at)[:, None] * torch.complex(y[..., j], y[..., l])
            y[..., j], y[..., l] = turn.real, turn.imag
        if case["op"] == "norm_rope":
            out.append(y)
        else:  # y: the gradient of unit·w; d unit / d x projects on what is orthogonal to x (up to eps)
            out.append((y * w - unit * (y * w * unit).sum(-1, keepdim=True) / case["d"]) / size)
            out.append(torch.einsum("nhd,nhd->d", y, unit))
    return out


def _exact_objective(logp, entropy, s):
    w = s["weights"].double()
    adv = s["adv"].double()
    parts = [(adv, 1)] if "adv_neg" not in s else [(adv, 1), (-s["adv_neg"].double(), 1)]
    ratio = torch.exp(logp - s["old_logp"].double())
    bounded = torch.minimum(torch.maximum(ratio, torch.full_like(ratio, 1 - CLIP_LO)), torch.full_like(ratio, 1 + CLIP_HI))
    value, slope = torch.zeros_like(logp), torch.zeros_like(logp)
    for a, _ in parts:
        kept = torch.minimum(ratio * a, bounded * a)          # the pessimistic one of both
        moves = ratio * a <= bounded * a
        floor = torch.where(a < 0, DUAL * a, -math.inf)        # at most DUAL times a negative advantage
        moves &= kept >= floor
        kept = torch.maximum(kept, floor)
        value -= kept
        slope -= torch.where(moves, ratio * a, 0.0)
    kl = torch.zeros_like(logp)
    if "ref_logp" in s:
        x = s["ref_logp"].double() - logp
        kl = torch.expm1(x) - x
        slope -= KL * torch.expm1(x)
    ent = torch.zeros_like(logp) if entropy is None else entropy.double()
    on = w != 0
    value, kl, ent, slope = (torch.where(on, t, 0.0) for t in (value, kl, ent, slope))
    sums = torch.stack([(w * (value + KL * kl - ENTROPY * ent)).sum(), w @ value, w @ kl, w @ ent])
    return sums, w * slope, -ENTROPY * w


def _exact_decode(case, s):
    """Query by query: the rows of its segments, one softmax over them."""
    G = case["Hq"] // case["Hkv"]
    out = []
    for q, k, v in zip(s["q"], s["k"], s["v"]):
        o = torch.zeros(s["B"], case["Hq"], case["d"], dtype=torch.float64, device=DEV)
        lse = torch.full((case["Hq"], s["B"]), -math.inf, dtype=torch.float64, device=DEV)
        for b in range(s["B"]):
            spans = [(at, at + n) for at, n, q0, q1 in s["segs"] if q0 <= b < q1 and n]
            if not spans:
                continue
            ks = torch.cat([k[i:j] for i, j in spans]).double().transpose(0, 1)
            vs = torch.cat([v[i:j] for i, j in spans]).double().transpose(0, 1)
            sc = q[b].double().view(case["Hkv"], G, -1) @ ks.transpose(1, 2) / math.sqrt(case["d"])
            o[b] = (torch.softmax(sc, -1) @ vs).reshape(case["Hq"], -1)
            lse[:, b] = torch.logsumexp(sc, -1).reshape(-1)
        out += [o, lse]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        return _exact_norm_rope(case, s)
    if case["op"] == "policy":
        sums, dlogp, dent = _exact_objective(s["logp"].double(), s.get("entropy"), s)
        out = {"sums": sums, "dlogp": dlogp}
        return out | {"dentropy": dent} if "entropy" in s else out
    if case["op"] == "decode":
        return _exact_decode(case, s)
    N, V = case["N"], case["V"]
    logp = _log_probs(s["z"], s["y"])
    ent = torch.empty(N, dtype=torch.float64, device=DEV)
    for i in range(0, N, 256):
        lp = torch.log_softmax(s["z"][i:i + 256].double(), 1)
        ent[i:i + 256] = -torch.special.xlogy(lp.exp(), lp.exp()).sum(1)
    sums, dlogp, dent = _exact_objective(logp, ent, s)
    dz = torch.empty(N, V, dtype=torch.float64, device=DEV)
    for i in range(0, N, 256):
        j = slice(i, min(N, i + 256))
        lp = torch.log_softmax(s["z"][j].double(), 1)
        p = lp.exp()
        dz[j] = -dent[j, None] * (torch.special.xlogy(p, p) + p * ent[j, None]) - dlogp[j, None] * p
        rows = torch.arange(dz[j].shape[0], device=DEV)
        dz[j][rows, s["y"][j].long()] += dlogp[j]
    on = s["weights"] > 0
    return {"sums": sums, "logp": torch.where(on, logp, 0.0), "entropy": torch.where(on, ent, 0.0), "dlogits": dz}
