"""The calls of the policy step reject bad arguments on the host, before any GPU work (C ABI and binding; CPU)."""
import ctypes

import pytest
import torch

BAD, UNSUPPORTED, WS, OK = -1, -3, -4, 0
fake, fake2, fake3, fake4 = (ctypes.c_void_p(1 << s) for s in (12, 20, 22, 24))  # never dereferenced
odd = ctypes.c_void_p(4097)
big = 1 << 30


@pytest.fixture(scope="module")
def L():
    from prefix_tree_gb300 import build, lib
    build.build()
    return lib()


def _norm(L, **over):
    a = dict(q=fake, qo=fake, q_ld=256, qo_ld=256, k=fake2, ko=fake2, k_ld=128, ko_ld=128, dt=0, N=5, hq=4, hkv=2, d=64,
             wq=fake, wk=fake, wdt=0, eps=1e-6, rot=64, pos=fake, pos_ld=5, axes=1, axis=(ctypes.c_uint8 * 128)(),
             freq=(ctypes.c_double * 128)(), adj=0, st=None)
    a.update(over)
    return L.tt_qk_norm_rope(*a.values())


COMMON = [(dict(N=-1), BAD), (dict(d=0), BAD), (dict(rot=-2), BAD), (dict(rot=66), BAD), (dict(axes=0), BAD),
          (dict(dt=3), BAD), (dict(axis=None), BAD), (dict(freq=None), BAD), (dict(rot=63), UNSUPPORTED),
          (dict(d=65), UNSUPPORTED), (dict(axes=5), UNSUPPORTED), (dict(rot=258, d=512), UNSUPPORTED),
          (dict(d=514), UNSUPPORTED), (dict(hq=1025), UNSUPPORTED), (dict(hkv=-1), BAD), (dict(q=None), BAD),
          (dict(q_ld=255), BAD), (dict(q=odd), BAD), (dict(pos=None), BAD), (dict(axes=3, pos_ld=4), BAD),
          (dict(axis=(ctypes.c_uint8 * 128)(*[1] * 128)), BAD),
          (dict(freq=(ctypes.c_double * 128)(float("nan"))), BAD), (dict(wdt=1), BAD), (dict(wdt=7), BAD),
          (dict(wq=odd), BAD), (dict(wdt=2, wk=ctypes.c_void_p(4098)), BAD), (dict(eps=-1e-6), BAD),
          (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD)]


@pytest.mark.parametrize("over,code", COMMON + [
    (dict(ko=None), BAD), (dict(ko_ld=127), BAD), (dict(qo_ld=320), BAD), (dict(ko=fake), BAD), (dict(qo=fake2), BAD),
    (dict(N=0, q=None, k=None, qo=None, ko=None, pos=None), OK), (dict(hq=0, hkv=0, q=None, k=None), OK)])
def test_norm_rope_arguments(L, over, code):
    assert _norm(L, **over) == code


def _normb(L, **over):
    a = dict(dqo=fake3, dqo_ld=256, q=fake, q_ld=256, dq=fake3, dq_ld=256, dko=fake4, dko_ld=128, k=fake2, k_ld=128,
             dk=fake4, dk_ld=128, dt=0, N=5, hq=4, hkv=2, d=64, wq=fake, wk=fake, wdt=0, eps=1e-6, rot=64, pos=fake,
             pos_ld=5, axes=1, axis=(ctypes.c_uint8 * 128)(), freq=(ctypes.c_double * 128)(), adj=0, dwq=fake, dwk=fake,
             ws=fake, n=big, st=None)
    a.update(over)
    return L.tt_qk_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("over,code", COMMON + [
    (dict(dq=None), BAD), (dict(dko=None), BAD), (dict(dk_ld=127), BAD), (dict(dqo_ld=255), BAD),
    (dict(dq_ld=320), BAD),                            # in place with another stride
    (dict(dq=fake, q_ld=320), BAD), (dict(dk=fake3), BAD), (dict(dq=fake2), BAD), (dict(dq=fake4), BAD),
    (dict(ws=None), BAD), (dict(ws=ctypes.c_void_p(4104)), BAD), (dict(n=4096), WS), (dict(dwq=odd), BAD)])
def test_norm_rope_bwd_arguments(L, over, code):
    assert _normb(L, **over) == code


def test_norm_rope_workspace(L):
    assert L.tt_qk_norm_rope_bwd_workspace_bytes(128) > 0
    assert L.tt_qk_norm_rope_bwd_workspace_bytes(0) == L.tt_qk_norm_rope_bwd_workspace_bytes(514) == 0


class Policy(ctypes.Structure):
    _fields_ = [(n, ctypes.c_float) for n in ("clip_lo", "clip_hi", "dual_clip", "kl_coef", "entropy_coef", "g")]


def _pol(**over):
    a = dict(clip_lo=0.2, clip_hi=0.2, dual_clip=0.0, kl_coef=0.1, entropy_coef=0.1, g=1.0)
    a.update(over)
    return ctypes.byref(Policy(*a.values()))


POLICIES = [(dict(clip_lo=-0.1), BAD), (dict(clip_lo=1.1), BAD), (dict(clip_hi=-0.1), BAD), (dict(dual_clip=0.9), BAD),
            (dict(dual_clip=float("nan")), BAD), (dict(kl_coef=float("inf")), BAD), (dict(g=float("nan")), BAD),
            (dict(entropy_coef=float("nan")), BAD), (dict(clip_hi=float("inf")), BAD)]


def _loss(L, **over):
    a = dict(logp=fake, h=fake, old=fake, adv=fake, neg=fake, ref=fake, w=fake, N=10000, p=_pol(), sums=fake, dl=fake,
             dh=fake, ws=fake, n=big, st=None)
    a.update(over)
    return L.tt_policy_loss(*a.values())


@pytest.mark.parametrize("over,code", [(dict(p=_pol(**o)), c) for o, c in POLICIES] + [
    (dict(p=None), BAD), (dict(N=-1), BAD), (dict(N=1 << 31), BAD), (dict(logp=None), BAD), (dict(old=None), BAD),
    (dict(adv=None), BAD), (dict(h=None), BAD), (dict(sums=None), BAD), (dict(ref=odd), BAD), (dict(dl=odd), BAD),
    (dict(ws=None), BAD), (dict(ws=ctypes.c_void_p(4104)), BAD), (dict(n=16), WS)])
def test_policy_loss_arguments(L, over, code):
    assert _loss(L, **over) == code


def test_policy_loss_workspace(L):
    f = L.tt_policy_loss_workspace_bytes
    assert f(0) == f(-5) == f(8192) == 0 < f(8193)
    g = L.tt_policy_loss_logits_workspace_bytes
    assert g(0) == 0 and g(7) == 112


def _logits(L, **over):
    a = dict(z=fake, dt=0, N=3, V=100, ld=100, y=fake, old=fake, adv=fake, neg=fake, ref=fake, w=fake, p=_pol(), sums=fake,
             logp=fake, h=fake, dz=fake, ws=fake, n=big, err=fake, st=None)
    a.update(over)
    return L.tt_policy_loss_logits(*a.values())


@pytest.mark.parametrize("over,code", [(dict(p=_pol(**o)), c) for o, c in POLICIES] + [
    (dict(p=None), BAD), (dict(N=-1), BAD), (dict(V=0), BAD), (dict(ld=99), BAD), (dict(dt=5), BAD), (dict(z=None), BAD),
    (dict(z=odd), BAD), (dict(dz=odd), BAD), (dict(dt=2, z=ctypes.c_void_p(4098)), BAD), (dict(y=None), BAD),
    (dict(old=None), BAD), (dict(adv=None), BAD), (dict(sums=None), BAD), (dict(logp=None), BAD), (dict(h=None), BAD),
    (dict(err=None), BAD), (dict(ws=None), BAD), (dict(ws=ctypes.c_void_p(4104)), BAD), (dict(n=16), WS),
    (dict(N=1 << 31), BAD), (dict(V=1 << 20, ld=1 << 20), UNSUPPORTED), (dict(dt=2, V=500000, ld=500000), UNSUPPORTED)])
def test_policy_loss_logits_arguments(L, over, code):
    assert _logits(L, **over) == code


def test_binding_refuses_cpu_tensors_and_mixed_arguments():
    import prefix_tree_gb300 as tt
    x, r = torch.zeros(2, 1, 8), torch.zeros(2)
    pos = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: tt.qk_norm_rope(x, None, pos), lambda: tt.qk_norm_rope_bwd(x, None, x, None, pos),
                 lambda: tt.policy_loss(r, r, r), lambda: tt.policy_loss(None, r, r),
                 lambda: tt.policy_loss_logits(torch.zeros(2, 8), pos, r, r)):
        with pytest.raises(TypeError):
            call()
    from prefix_tree_gb300._native import _policy_of
    with pytest.raises(ValueError):
        _policy_of(0.2, 0.5, 0.0, 0.0, 1.0)


def _plan(L, **over):
    a = dict(kb=fake, kl=fake, qb=fake, qe=fake, S=3, B=4, rows=100, pairs=9, hq=4, hkv=2, d=64, plan=fake, n=big, err=fake,
             st=None)
    a.update(over)
    return L.tt_tree_decode_plan(*a.values())


DECODE_SIZES = [(dict(S=-1), BAD), (dict(B=-1), BAD), (dict(rows=-1), BAD), (dict(pairs=-1), BAD), (dict(hq=0), BAD),
                (dict(hkv=0), BAD), (dict(rows=1 << 31), BAD), (dict(pairs=1 << 31), BAD), (dict(d=96), UNSUPPORTED),
                (dict(hq=5), UNSUPPORTED), (dict(hq=1026), UNSUPPORTED), (dict(B=1 << 21), UNSUPPORTED),
                (dict(plan=None), BAD), (dict(plan=ctypes.c_void_p(4104)), BAD), (dict(err=None), BAD)]


@pytest.mark.parametrize("over,code", DECODE_SIZES + [(dict(kb=None), BAD), (dict(qe=None), BAD), (dict(n=64), WS)])
def test_decode_plan_arguments(L, over, code):
    assert _plan(L, **over) == code


def _decode(L, **over):
    a = dict(plan=fake, q=fake, q_ld=256, k=fake, v=fake, kv_ld=128, dt=0, S=3, B=4, rows=100, pairs=9, hq=4, hkv=2, d=64,
             scale=0.125, o=fake, lse=fake, ws=fake, n=big, err=fake, st=None)
    a.update(over)
    return L.tt_tree_decode_attn(*a.values())


@pytest.mark.parametrize("over,code", DECODE_SIZES + [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD),
    (dict(ws=None), BAD), (dict(n=64), WS), (dict(q=ctypes.c_void_p(4098)), BAD), (dict(k=ctypes.c_void_p(4104)), BAD),
    (dict(q_ld=255), BAD), (dict(q_ld=260), BAD), (dict(kv_ld=120), BAD), (dict(kv_ld=132), BAD), (dict(dt=2), UNSUPPORTED),
    (dict(dt=9), BAD), (dict(scale=float("nan")), BAD), (dict(B=0, q=None, o=None, lse=None, ws=None), OK)])
def test_decode_attn_arguments(L, over, code):
    assert _decode(L, **over) == code


def test_decode_workspaces(L):
    assert L.tt_tree_decode_plan_bytes(0) > 0 and L.tt_tree_decode_plan_bytes(-1) == 0
    assert L.tt_tree_decode_plan_bytes(65) == L.tt_tree_decode_plan_bytes(0) + 65 * 32
    f = L.tt_tree_decode_attn_workspace_bytes
    assert f(-1, 4, 64) == f(1, 0, 64) == f(1, 4, 80) == 0 < f(0, 4, 64) < f(10, 4, 64) < f(10, 4, 128)
