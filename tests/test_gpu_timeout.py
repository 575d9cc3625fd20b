"""The bounded-wait timeout path of the tensor-memory forward, forced on purpose.

tt_tree_attn_fwd_stall_test makes the MMA-issuing thread of each CTA wait, in
the middle of its pipeline (before its second key block), on a barrier that
nothing arrives at, with a 10 ms limit. The wait expires; the kernel must then
stop its other roles, wait for every TMA copy and tensor-core operation it
already issued, free tensor memory and report TT_ERR_TIMEOUT in the error word,
leaving the context usable: the next normal calls on the same stream must
match the oracle. No wait here is unbounded and nothing faults on purpose.
"""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import tree as T
from tests._util import GRAD_RL2, LSE_RTOL, O_ATOL, dev_to_f64, f64, rel_l2, to_dev_bf16

pytestmark = pytest.mark.gpu

TT_ERR_TIMEOUT = -6


def _vp(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("tiles", [1, 2])
def test_forward_wait_expires_then_calls_recover(tt, tiles):
    sh = synth.random_tree(61, n_seg=9, len_range=(80, 300), max_children=3)
    inp = synth.attention_inputs(None, tree=sh, heads=(4, 2, 128))
    tab = T.tables(sh.seg_parent, sh.seg_len)
    tree = tt.tree_build(torch.tensor(sh.seg_parent, device="cuda"), torch.tensor(sh.seg_len, device="cuda")).check()
    Q, K, V, dO = (to_dev_bf16(inp[k]) for k in ("Q", "K", "V", "dO"))
    N, hq, d = Q.shape
    hkv = K.shape[1]
    O = torch.empty_like(Q)
    LSE = torch.empty(hq, N, dtype=torch.float32, device="cuda")
    err = tt.new_err("cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rc = tt.lib().tt_tree_attn_fwd_stall_test(_vp(tree.ws), _vp(Q), _vp(K), _vp(V), _vp(O), _vp(LSE), N, hq, hkv, d,
                                               ctypes.c_float(1.0 / np.sqrt(d)), tiles, 10_000_000, _vp(err), stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert int(err.item()) == TT_ERR_TIMEOUT
    # the same stream, the same buffers: normal forward and backward match the oracle
    err2 = tt.new_err("cuda")
    O2, LSE2 = tt.tree_attn_fwd(tree, Q, K, V, out=(O, LSE), err=err2, tiles=tiles)
    dQ, dK, dV = tt.tree_attn_bwd(tree, Q, K, V, O2, LSE2, dO, err=err2)
    torch.cuda.synchronize()
    assert int(err2.item()) == 0
    ref = A.tree_attention_segments(tab, *(f64(inp[k]) for k in ("Q", "K", "V", "dO")))
    assert np.abs(dev_to_f64(O2) - ref[0]).max() <= O_ATOL
    lse = LSE2.cpu().numpy().astype(np.float64)
    assert (np.abs(lse - ref[1]) <= LSE_RTOL * np.abs(ref[1]) + 1e-5).all()
    for got, r in ((dQ, ref[2]), (dK, ref[3]), (dV, ref[4])):
        assert rel_l2(dev_to_f64(got), r) <= GRAD_RL2


def test_stall_test_rejects_bad_limits(tt):
    fake = ctypes.c_void_p(4096)  # rejected before any pointer is used
    for ns in (0, -1, 10_000_000_001):
        rc = tt.lib().tt_tree_attn_fwd_stall_test(fake, fake, fake, fake, fake, fake, 128, 1, 1, 64,
                                                   ctypes.c_float(0.125), 1, ns, fake, None)
        assert rc == -1


def _head_path_test(tt, H, W, y, lse, h, dl, de, path, stall_ns=0, drain_ns=0, dw_dtype=torch.float32):
    """tt_lmhead_token_logprob_bwd_path_test: (return code, error word, d_hidden, d_w_vocab)."""
    N, Hd = H.shape
    V = W.shape[0]
    dh, dw = torch.empty_like(H), torch.empty((V, Hd), dtype=dw_dtype, device="cuda")
    n = tt.lib().tt_lmhead_token_logprob_bwd_workspace_bytes(N, V, Hd)
    ws, err = torch.zeros(n, dtype=torch.uint8, device="cuda"), tt.new_err("cuda")
    rc = tt.lib().tt_lmhead_token_logprob_bwd_path_test(
        _vp(H), _vp(W), N, V, Hd, _vp(y), _vp(lse), _vp(h), _vp(dl), _vp(de), None, _vp(dh), _vp(dw),
        2 if dw_dtype == torch.float32 else 0, _vp(ws), n, path, stall_ns, drain_ns, _vp(err),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    return rc, int(err.item()), dh, dw


def _head_inputs(N, V, Hd):
    g = torch.Generator(device="cuda").manual_seed(N + V)
    H = torch.randn(N, Hd, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, Hd, generator=g, device="cuda") * (2 / Hd ** 0.5)).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    return H, W, y, torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")


@pytest.mark.parametrize("N,V,Hd,path", [
    (300, 3001, 256, 1),    # half tiles, one to a CTA
    (1000, 4000, 256, 1),   # whole tiles, one to a CTA
    (1000, 4000, 256, 2),   # one to a pair of CTAs
    (4129, 9999, 256, 1), (4129, 9999, 256, 2)])  # several to a CTA, to a pair: claimed from a counter
def test_head_wait_expires_late_in_a_tile_then_calls_recover(tt, N, V, Hd, path):
    """The head's MMA thread gives up before the last K step of its first tile, when the CTA's producer has issued
    every copy of it: where a CTA has one tile only, the producer is done by then, and the error must be reported all
    the same. The next calls on the stream give what calls before gave."""
    H, W, y, dl, de = _head_inputs(N, V, Hd)
    _, h, lse = tt.lmhead_token_logprob(H, W, y)
    before = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, dentropy=de)
    rc, err, _, _ = _head_path_test(tt, H, W, y, lse, h, dl, de, path, 10_000_000)
    assert rc == 0 and err == TT_ERR_TIMEOUT
    err2 = tt.new_err("cuda")
    after = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, dentropy=de, err=err2)
    torch.cuda.synchronize()
    assert int(err2.item()) == 0 and all(torch.equal(a, b) for a, b in zip(before, after))


def test_head_path_test_rejects_bad_arguments(tt):
    f = ctypes.c_void_p(4096)  # rejected before any pointer is used
    for path, ns, drain in ((3, 0, 0), (-1, 0, 0), (0, -1, 0), (0, 10_000_000_001, 0), (0, 0, -1),
                            (0, 0, 10_000_000_001)):
        rc = tt.lib().tt_lmhead_token_logprob_bwd_path_test(f, f, 300, 1000, 128, f, f, f, f, f, f, f, f, 2, f, 1 << 40,
                                                           path, ns, drain, f, None)
        assert rc == -1


@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("heads", [(2, 1, 64), (4, 2, 128)])
def test_forward_wait_expires_at_the_last_block(tt, tiles, heads):
    """One segment of two key blocks: the stall comes before a tile's last block, when the producer may have nothing
    left to wait for. It is reported all the same."""
    hq, hkv, d = heads
    N = 256
    tree = tt.tree_build(torch.tensor([-1], dtype=torch.int32, device="cuda"),
                         torch.tensor([N], dtype=torch.int32, device="cuda")).check()
    g = torch.Generator(device="cuda").manual_seed(d)
    Q, K, V = (torch.randn(N, n, d, generator=g, device="cuda").to(torch.bfloat16) for n in (hq, hkv, hkv))
    before = tt.tree_attn_fwd(tree, Q, K, V, tiles=tiles)
    O, LSE, err = torch.empty_like(Q), torch.empty(hq, N, dtype=torch.float32, device="cuda"), tt.new_err("cuda")
    rc = tt.lib().tt_tree_attn_fwd_stall_test(_vp(tree.ws), _vp(Q), _vp(K), _vp(V), _vp(O), _vp(LSE), N, hq, hkv, d,
                                              ctypes.c_float(d ** -0.5), tiles, 10_000_000, _vp(err),
                                              ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert int(err.item()) == TT_ERR_TIMEOUT
    err2 = tt.new_err("cuda")
    after = tt.tree_attn_fwd(tree, Q, K, V, err=err2, tiles=tiles)
    torch.cuda.synchronize()
    assert int(err2.item()) == 0 and all(torch.equal(a, b) for a, b in zip(before, after))


def test_head_limit_of_the_last_wait_is_not_that_of_the_product(tt):
    """The wait of a pair's second CTA for the last MMAs begins when its own work has ended: 0.5 ms are enough for it in
    a product that cannot take less than 1.9 ms (4.4 TFLOP at the nominal 2.25 PFLOP/s)."""
    H, W, y, dl, de = _head_inputs(16384, 65536, 2048)
    _, h, lse = tt.lmhead_token_logprob(H, W, y)
    ref = tt.lmhead_token_logprob_bwd(H, W, y, lse, h, dlogp=dl, dentropy=de)
    rc, err, dh, dw = _head_path_test(tt, H, W, y, lse, h, dl, de, 2, drain_ns=500_000)
    assert rc == 0 and err == 0
    assert torch.equal(dh, ref[0]) and torch.equal(dw, ref[1])
