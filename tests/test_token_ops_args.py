"""The per-token operators reject bad arguments on the host, before any GPU work (C ABI and binding; CPU)."""
import ctypes

import pytest
import torch

BAD, UNSUPPORTED, WS, OK = -1, -3, -4, 0
fake = ctypes.c_void_p(4096)  # never dereferenced: validation fails first
odd = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    from prefix_tree_gb300 import build, lib
    build.build()
    return lib()


fake2 = ctypes.c_void_p(1 << 20)


def _rope(L, **over):
    a = dict(q=fake, qo=fake, q_ld=256, qo_ld=256, k=fake2, ko=fake2, k_ld=128, ko_ld=128, dt=0, N=5, hq=4, hkv=2, d=64,
             rot=64, pos=fake, pos_ld=5, axes=1, axis=(ctypes.c_uint8 * 128)(), freq=(ctypes.c_double * 128)(), adj=0,
             inv=0, st=None)
    a.update(over)
    return L.tt_rope(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(N=-1), BAD), (dict(d=0), BAD), (dict(rot=0), BAD), (dict(rot=66), BAD), (dict(axes=0), BAD),
    (dict(dt=3), BAD), (dict(dt=-1), BAD), (dict(axis=None), BAD), (dict(freq=None), BAD),
    (dict(rot=63), UNSUPPORTED), (dict(d=65), UNSUPPORTED), (dict(axes=5, pos_ld=5), UNSUPPORTED),
    (dict(d=1026, q_ld=9999, qo_ld=9999, k_ld=9999, ko_ld=9999), UNSUPPORTED), (dict(rot=258, d=512), UNSUPPORTED),
    (dict(hq=1025), UNSUPPORTED), (dict(hkv=-1), BAD), (dict(q=None), BAD), (dict(ko=None), BAD),
    (dict(q_ld=255), BAD), (dict(ko_ld=127), BAD), (dict(q=odd), BAD), (dict(ko=odd), BAD), (dict(pos=None), BAD),
    (dict(qo_ld=320), BAD),                     # in place with another stride
    (dict(ko=fake), BAD), (dict(qo=fake2), BAD), (dict(k=fake, ko=fake), BAD),  # one into the other
    (dict(axes=3, pos_ld=4), BAD),              # axes overlap
    (dict(axes=1, axis=(ctypes.c_uint8 * 128)(*[1] * 128)), BAD),
    (dict(freq=(ctypes.c_double * 128)(float("nan"))), BAD), (dict(freq=(ctypes.c_double * 128)(float("inf"))), BAD),
    (dict(N=0, q=None, k=None, qo=None, ko=None, pos=None), OK), (dict(hq=0, hkv=0, q=None, k=None), OK)])
def test_rope_arguments(L, over, code):
    assert _rope(L, **over) == code


def _tok(L, **over):
    a = dict(z=fake, dt=0, N=3, V=100, ld=100, y=fake, k=4, logp=fake, h=fake, lse=fake, ids=fake, top=fake, err=fake,
             st=None)
    a.update(over)
    return L.tt_token_logprob(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(z=None), BAD), (dict(z=odd), BAD), (dict(dt=7), BAD), (dict(N=-1), BAD), (dict(V=0, ld=4), BAD),
    (dict(ld=99), BAD), (dict(k=-1), BAD), (dict(k=101), BAD), (dict(k=33), UNSUPPORTED), (dict(logp=None), BAD),
    (dict(h=None), BAD), (dict(lse=None), BAD), (dict(ids=None), BAD), (dict(top=None), BAD), (dict(err=None), BAD),
    (dict(dt=2, z=ctypes.c_void_p(4098)), BAD), (dict(V=1 << 31, ld=1 << 31), BAD), (dict(N=1 << 31), BAD),
    (dict(N=0, z=None, logp=None, h=None), OK)])
def test_token_logprob_arguments(L, over, code):
    assert _tok(L, **over) == code


def _tokb(L, **over):
    a = dict(z=fake, dt=0, N=3, V=100, ld=100, lse=fake, h=fake, y=fake, dlogp=fake, dh=fake, dlse=fake, ids=fake,
             dtop=fake, k=4, dz=fake, err=fake, st=None)
    a.update(over)
    return L.tt_token_logprob_bwd(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(z=None), BAD), (dict(dz=None), BAD), (dict(dz=odd), BAD), (dict(lse=None), BAD), (dict(y=None), BAD),
    (dict(h=None), BAD), (dict(ids=None), BAD), (dict(dtop=None), BAD), (dict(k=-1), BAD), (dict(k=33), UNSUPPORTED),
    (dict(err=None), BAD), (dict(ld=99), BAD), (dict(N=0, z=None, dz=None, lse=None), OK)])
def test_token_logprob_bwd_arguments(L, over, code):
    assert _tokb(L, **over) == code


def test_lmhead_token_logprob_arguments(L):
    nb = L.tt_lmhead_token_logprob_workspace_bytes
    assert nb(0, 5, 64) == nb(5, 5, 0) == 0 and nb(300, 1000, 64) >= 12 * 300 * 4 + 4 * 300
    bwd_bytes = L.tt_lmhead_token_logprob_bwd_workspace_bytes
    assert bwd_bytes(0, 1000, 128) == 0 and bwd_bytes(300, 1000, 128) >= 300 * 1000 * 2
    big = 1 << 40

    def fwd(h=fake, w=fake, N=300, V=1000, Hd=128, y=fake, logp=fake, ent=fake, lse=fake, ws=fake, n=big, err=fake):
        return L.tt_lmhead_token_logprob(h, w, N, V, Hd, y, logp, ent, lse, ws, n, err, None)

    def bwd(h=fake, w=fake, N=300, V=1000, Hd=128, y=fake, lse=fake, ent=fake, dl=fake, dent=fake, ds=fake, dh=fake,
            dw=fake, dt=2, ws=fake, n=big, err=fake):
        return L.tt_lmhead_token_logprob_bwd(h, w, N, V, Hd, y, lse, ent, dl, dent, ds, dh, dw, dt, ws, n, err, None)

    for f in (fwd, bwd):
        for name in ("h", "w", "y", "lse", "ent", "ws", "err"):
            assert f(**{name: None}) == BAD, (f, name)
        assert f(N=0) == f(V=0) == f(Hd=0) == f(h=ctypes.c_void_p(4104)) == BAD
        assert f(Hd=96) == UNSUPPORTED and f(n=64) == WS
    assert fwd(logp=None) == BAD
    assert bwd(dh=None) == bwd(dw=None) == bwd(dt=1) == bwd(dw=ctypes.c_void_p(4104)) == BAD


def test_binding_refuses_cpu_tensors_and_bad_tables():
    import prefix_tree_gb300 as tt
    from prefix_tree_gb300._native import _rope_tables
    x, pos = torch.zeros(2, 1, 8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: tt.rope(x, None, pos), lambda: tt.token_logprob(torch.zeros(2, 8)),
                 lambda: tt.token_logprob_bwd(torch.zeros(2, 8), torch.zeros(2)),
                 lambda: tt.lmhead_token_logprob(torch.zeros(2, 64), torch.zeros(3, 64), pos)):
        with pytest.raises(TypeError):
            call()
    for bad in (((2, 1), None), ((5, -1), None), ((4,), (1.0, 2.0))):
        with pytest.raises(ValueError):
            _rope_tables(8, bad[0], False, 1e4, bad[1])
    axis, freq = _rope_tables(8, (2, 1, 1), True, 1e4, None)
    assert list(axis) == [0, 1, 2, 0] and list(freq) == [1e4 ** (-i / 4) for i in range(4)]


def test_frequencies_are_host_numbers():
    """A tensor on a device would be read back at every call; one on the host, an array or a list gives the same key."""
    from prefix_tree_gb300._native import _frequencies
    f = [1.0, 0.5, 0.25]
    want = tuple(f)
    assert _frequencies(None) is None
    assert _frequencies(f) == _frequencies(torch.tensor(f)) == _frequencies(torch.tensor(f).numpy()) == want
    for t in (torch.float32, torch.float64):
        with pytest.raises(TypeError, match="host"):
            _frequencies(torch.empty(3, dtype=t, device="meta"))
