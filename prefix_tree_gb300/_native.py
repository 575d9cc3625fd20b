"""ctypes binding of libtt (include/tt.h): argument marshalling only.

Every computation runs in the CUDA library; this module allocates outputs and
workspaces with PyTorch on the tensors' device, passes raw pointers and the
current CUDA stream, and raises on a non-zero status. There is no fallback: a
missing libtt.so raises immediately.
"""
from __future__ import annotations

import ctypes
import functools
import math
import operator
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtt.so")

TT_OK = 0
_STATUS = {0: "TT_OK", -1: "TT_ERR_INVALID_ARG", -2: "TT_ERR_INVALID_TREE", -3: "TT_ERR_UNSUPPORTED",
           -4: "TT_ERR_WORKSPACE", -5: "TT_ERR_CUDA", -6: "TT_ERR_TIMEOUT"}

_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_int = ctypes.c_int


class TTError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = int(code)
        super().__init__(f"{what}: {_STATUS.get(self.code, self.code)} ({lib().tt_status_string(self.code).decode()})")


class _TreeOut(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("seg_start", "seg_subtree_end", "seg_depth", "seg_pathlen", "seg_leafcnt", "iv_ptr",
                                   "iv", "tok_seg", "tok_pos", "tok_send", "tok_leafcnt", "tok_weight", "stats")]


_SIGS = {
    "tt_tree_workspace_bytes": (_sz, [_i32, _i64]),
    "tt_tree_build": (_int, [_vp, _vp, _i32, _i64, ctypes.POINTER(_TreeOut), _i64, _vp, _sz, _vp, _vp]),
    "tt_tree_schedules": (_int, [_vp, _i64] + [_vp] * 7 + [_vp]),
    "tt_tree_attn_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _f32, _vp, _vp]),
    "tt_tree_attn_fwd_tiles": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _f32, _int, _vp, _vp]),
    "tt_tree_attn_fwd_stall_test": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _f32, _int, _i64, _vp,
                                           _vp]),
    "tt_tree_attn_bwd_workspace_bytes": (_sz, [_i64, _int]),
    "tt_tree_attn_bwd": (_int, [_vp] * 10 + [_i64, _int, _int, _int, _f32, _vp, _sz, _vp, _vp]),
    "tt_tree_attn_chunk_fwd": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _f32, _vp, _vp]),
    "tt_tree_attn_chunk_fwd_tiles": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _f32, _int,
                                            _vp, _vp]),
    "tt_tree_attn_chunk_fwd_split": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _f32, _int,
                                            _vp, _vp]),
    "tt_tree_attn_chunk_bwd_workspace_bytes": (_sz, [_i64, _int]),
    "tt_tree_attn_chunk_bwd": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _int, _int, _int,
                                      _f32, _vp, _sz, _vp, _vp]),
    "tt_tree_attn_chunk_fwd_packed": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int,
                                             _f32, _vp, _vp]),
    "tt_tree_attn_chunk_bwd_packed": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp,
                                             _vp, _int, _int, _int, _f32, _vp, _sz, _vp, _vp]),
    "tt_tree_attn_chunk_bwd_noalloc": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _int,
                                              _int, _int, _f32, _vp, _vp]),
    "tt_dta_workspace_bytes": (_sz, [_vp, _vp, _i32, _i64, _int, _int, _int]),
    "tt_dta_tree_attn": (_int, [_vp, _vp, _i32, _i64, _i64] + [_vp] * 9 + [_int, _int, _int, _f32, _vp, _sz, _vp, _vp]),
    "tt_dta_tree_attn_ordered": (_int, [_vp, _vp, _i32, _i64, _i64, _int] + [_vp] * 9
                                 + [_int, _int, _int, _f32, _vp, _sz, _vp, _vp]),
    "tt_tree_partition": (_int, [_vp, _vp, _i32, _i64, _int, _vp, _vp, _vp, _vp, _i32]),
    "tt_dta_leaf_order": (_int, [_vp, _vp, _i32, _int, _vp, _i32]),
    "tt_dta_plan_create": (_int, [_vp, _vp, _i32, _i64, _i64, _int, _int] + [_vp] * 9
                           + [_int, _int, _int, _f32, _vp, _sz, _vp, _vp]),
    "tt_dta_workspace_bytes_slots": (_sz, [_vp, _vp, _i32, _i64, _int, _int, _int, _int]),
    "tt_dta_tree_attn_slots": (_int, [_vp, _vp, _i32, _i64, _i64, _int, _int] + [_vp] * 9
                               + [_int, _int, _int, _f32, _vp, _sz, _vp, _vp]),
    "tt_dta_plan_launch": (_int, [_vp, _vp]),
    "tt_dta_plan_destroy": (_int, [_vp]),
    "tt_weighted_logprob": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _vp]),
    "tt_rope": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _int, _i64, _int, _int, _int, _int, _vp, _i64, _int,
                       _vp, _vp, _int, _int, _vp]),
    "tt_qk_norm_rope": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _int, _i64, _int, _int, _int, _vp, _vp, _int,
                               _f32, _int, _vp, _i64, _int, _vp, _vp, _int, _vp]),
    "tt_qk_norm_rope_bwd_workspace_bytes": (_sz, [_int]),
    "tt_qk_norm_rope_bwd": (_int, [_vp, _i64] * 6 + [_int, _i64, _int, _int, _int, _vp, _vp, _int, _f32, _int, _vp, _i64,
                                                     _int, _vp, _vp, _int, _vp, _vp, _vp, _sz, _vp]),
    "tt_tree_decode_plan_bytes": (_sz, [_i32]),
    "tt_tree_decode_plan": (_int, [_vp] * 4 + [_i32, _i32, _i64, _i64, _int, _int, _int, _vp, _sz, _vp, _vp]),
    "tt_tree_decode_attn_workspace_bytes": (_sz, [_i64, _int, _int]),
    "tt_tree_decode_attn": (_int, [_vp, _vp, _i64, _vp, _vp, _i64, _int, _i32, _i32, _i64, _i64, _int, _int, _int, _f32,
                                   _vp, _vp, _vp, _sz, _vp, _vp]),
    "tt_policy_loss_workspace_bytes": (_sz, [_i64]),
    "tt_policy_loss": (_int, [_vp] * 7 + [_i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "tt_policy_loss_logits_workspace_bytes": (_sz, [_i64]),
    "tt_policy_loss_logits": (_int, [_vp, _int, _i64, _i64, _i64] + [_vp] * 12 + [_sz, _vp, _vp]),
    "tt_token_logprob": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "tt_token_logprob_bwd": (_int, [_vp, _int, _i64, _i64, _i64] + [_vp] * 8 + [_int, _vp, _vp, _vp]),
    "tt_lmhead_logprob_workspace_bytes": (_sz, [_i64, _i64]),
    "tt_lmhead_logprob": (_int, [_vp, _vp, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "tt_lmhead_logprob_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "tt_lmhead_logprob_bwd": (_int, [_vp, _vp, _i64, _i64, _int, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "tt_lmhead_token_logprob_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "tt_lmhead_token_logprob": (_int, [_vp, _vp, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "tt_lmhead_token_logprob_bwd_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "tt_lmhead_token_logprob_bwd": (_int, [_vp, _vp, _i64, _i64, _int] + [_vp] * 8 + [_int, _vp, _sz, _vp, _vp]),
    "tt_lmhead_token_logprob_bwd_path_test": (_int, [_vp, _vp, _i64, _i64, _int] + [_vp] * 8 +
                                              [_int, _vp, _sz, _int, _i64, _i64, _vp, _vp]),
    "tt_status_string": (ctypes.c_char_p, [_int]),
    "tt_version": (_int, []),
    "tt_trie_build": (_int, [_vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp]),
    "tt_kernel_timing": (_int, [_int]),
    "tt_kernel_timing_read": (_int, [_vp, _vp, _int, _vp]),
}

_LIB = None


def lib():
    """The loaded libtt (raises if it was not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtt.so is not built ({LIB_PATH}); run prefix_tree_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def exported_symbols():
    return list(_SIGS)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev=None):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _check(rc, what):
    if rc != TT_OK:
        raise TTError(rc, what)


def _need(t, dtype, name, dims=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims")


def new_err(device):
    """A zeroed device error word (see tt.h)."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def check_err(err, what="device"):
    """Synchronise on the error word and raise if a kernel recorded an error."""
    code = int(err.item())
    if code != 0:
        raise TTError(code, what)


# --------------------------------------------------------------------------- tree build
@dataclass
class Tree:
    """Device tables of a DFS-serialised tree plus the attention workspace."""
    S: int
    N: int
    seg_start: torch.Tensor
    seg_subtree_end: torch.Tensor
    seg_depth: torch.Tensor
    seg_pathlen: torch.Tensor
    seg_leafcnt: torch.Tensor
    iv_ptr: torch.Tensor
    iv: torch.Tensor
    tok_seg: torch.Tensor
    tok_pos: torch.Tensor
    tok_send: torch.Tensor
    tok_leafcnt: torch.Tensor
    tok_weight: torch.Tensor
    stats: torch.Tensor
    ws: torch.Tensor
    err: torch.Tensor

    def check(self):
        check_err(self.err, "tt_tree_build")
        return self


def tree_build(seg_parent: torch.Tensor, seg_len: torch.Tensor, N: int | None = None, iv_capacity: int | None = None,
               err: torch.Tensor | None = None) -> Tree:
    _need(seg_parent, torch.int32, "seg_parent", 1)
    _need(seg_len, torch.int32, "seg_len", 1)
    S = seg_parent.numel()
    dev = seg_parent.device
    if N is None:
        N = int(seg_len.sum().item())
    if iv_capacity is None:
        iv_capacity = S * (S + 1) // 2
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(seg_start=torch.empty(S, **i32), seg_subtree_end=torch.empty(S, **i32),
               seg_depth=torch.empty(S, **i32), seg_pathlen=torch.empty(S, **i32),
               seg_leafcnt=torch.empty(S, **i32), iv_ptr=torch.empty(S + 1, **i32),
               iv=torch.empty(max(1, iv_capacity), 2, **i32), tok_seg=torch.empty(N, **i32),
               tok_pos=torch.empty(N, **i32), tok_send=torch.empty(N, **i32), tok_leafcnt=torch.empty(N, **i32),
               tok_weight=torch.empty(N, dtype=torch.float32, device=dev),
               stats=torch.zeros(8, dtype=torch.int64, device=dev))
    nbytes = lib().tt_tree_workspace_bytes(S, N)
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    err = new_err(dev) if err is None else err
    s = _TreeOut(**{k: _p(v).value for k, v in out.items()})
    rc = lib().tt_tree_build(_p(seg_parent), _p(seg_len), S, N, ctypes.byref(s), iv_capacity, _p(ws), nbytes,
                             _p(err), _stream(dev))
    _check(rc, "tt_tree_build")
    return Tree(S=S, N=N, ws=ws, err=err, **out)


def tree_schedules(tree: Tree) -> dict:
    """The tile schedules the tree build wrote (tt_tree_schedules), as int32 device tensors."""
    nT = (tree.N + 127) // 128
    dev = tree.ws.device
    names = ("send", "blk_min", "blk_max", "fwd_cnt", "fwd_order", "bwd_cnt", "bwd_order")
    out = {n: torch.empty(nT * 128 if n == "send" else nT, dtype=torch.int32, device=dev) for n in names}
    _check(lib().tt_tree_schedules(_p(tree.ws), tree.N, *(_p(out[n]) for n in names), _stream(dev)),
           "tt_tree_schedules")
    return out


# --------------------------------------------------------------------------- rotary positions
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # TT_DT_*


# The raw current stream of a device: a tenth of the cost of a torch.cuda.Stream object, which is
# a good part of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _room_of(t, name):
    """Bytes of a buffer that a call writes from its first one on (0 for None): one without gaps, which would hold others' data."""
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.numel() * t.element_size()


def _device_of(t, *others):
    """Ordinal of t's device; the other tensors must be on it."""
    index = t.get_device()
    for o in others:
        if o is not None and o.get_device() != index:
            raise ValueError(f"tensors on {t.device} and {o.device}")
    return index


def _call(what, index, *args):
    """A C call on the current stream (its last argument) of device `index`, with that device current."""
    fn = getattr(_LIB or lib(), what)
    if index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != TT_OK:
        raise TTError(rc, what)


@functools.lru_cache(maxsize=64)
def _rope_tables(rot, sections, interleaved, base, inv_freq):
    """Host tables of tt_rope: the axis and the frequency of each pair."""
    half = rot // 2
    if any(n < 0 for n in sections) or sum(sections) != half:
        raise ValueError(f"sections must be non-negative and add up to rot_dim / 2 = {half}")
    if interleaved:
        axis = [a for i in range(max(sections)) for a, n in enumerate(sections) if i < n]
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    freq = [base ** (-i / half) for i in range(half)] if inv_freq is None else list(inv_freq)
    if len(freq) != half:
        raise ValueError(f"inv_freq must hold rot_dim / 2 = {half} frequencies")
    return (ctypes.c_uint8 * half)(*axis), (ctypes.c_double * half)(*freq)


def _frequencies(inv_freq):
    """inv_freq as the key of _rope_tables. A tensor on a device is refused: to read it back would make every call wait
    for the stream, and fail in a capture."""
    if inv_freq is None:
        return None
    if isinstance(inv_freq, torch.Tensor):
        if inv_freq.device.type != "cpu":
            raise TypeError("inv_freq must be on the host: read it back once (inv_freq.tolist()) and keep the list")
        inv_freq = inv_freq.tolist()
    return tuple(float(f) for f in inv_freq)


def _section_sizes(sections):
    """sections as the key of _rope_tables: their values now, whatever holds them."""
    if any(isinstance(n, torch.Tensor) and n.device.type != "cpu" for n in sections):
        raise TypeError("sections must be numbers on the host")
    return tuple(operator.index(n) for n in sections)


def _rope_rows(t, name):
    """(N, heads, d, elements between tokens) of a tensor of heads."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DTYPES or t.dim() != 3:
        raise TypeError(f"{name} must be a 3-D bf16, fp16 or fp32 CUDA tensor [N, heads, d]")
    n, h, d = t.shape
    if t.is_contiguous():
        return n, h, d, h * d
    ld, hd, one = t.stride()
    if (d > 1 and one != 1) or (h > 1 and hd != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return n, h, d, ld if n > 1 else h * d


def _rope_how(positions, N, d, rot_dim, sections, interleaved, base, inv_freq):
    """Checked positions, their stride between axes, the axes, rot and the host tables of tt_rope."""
    if not isinstance(positions, torch.Tensor) or not positions.is_cuda or positions.dtype != torch.int32:
        raise TypeError("positions must be an int32 CUDA tensor")
    many = positions.dim() == 2
    axes = positions.shape[0] if many else 1
    if positions.dim() > 2 or positions.dim() == 0 or positions.shape[-1] != N or (N > 1 and positions.stride(-1) != 1):
        raise ValueError("positions must be [N] or [axes, N] with contiguous tokens")
    rot = d if rot_dim is None else int(rot_dim)
    if rot < 2 or rot > d or rot % 2:
        raise ValueError("rot_dim must be even and in 2 .. d")
    if sections is None:
        if axes != 1:
            raise ValueError("several axes need sections")
        sections = (rot // 2,)
    elif len(sections) != axes:
        raise ValueError("positions and sections must agree on the number of axes")
    axis, freq = _rope_tables(rot, _section_sizes(sections), bool(interleaved), float(base), _frequencies(inv_freq))
    return positions, positions.stride(0) if many else N, axes, rot, axis, freq


def rope(q, k, positions, rot_dim=None, sections=None, interleaved=False, adjacent=False, base=10000.0, inv_freq=None,
         out=None, inverse=False):
    """Rotary positions of q [N,Hq,d] and k [N,Hkv,d] (tt_rope; k may be None): returns (q_out, k_out).

    `positions`: int32 [N] (one axis, e.g. Tree.tok_pos) or [axes, N]. The first `rot_dim` (default d) dimensions turn,
    in the pairs (i, i + rot_dim/2) or, `adjacent`, (2i, 2i + 1), by positions times the frequencies base^(-2i/rot_dim)
    or `inv_freq` (rot_dim/2 numbers on the host). `sections`: how many frequencies each axis takes, one after the other or,
    `interleaved`, the axes in turn while their section lasts. q and k may be views of one buffer (tokens any stride
    apart); `out` = (q_out, k_out) may be (q, k). `inverse` turns back."""
    N, hq, d, q_ld = _rope_rows(q, "q")
    hkv = k_ld = 0
    if k is not None:
        nk, hkv, dk, k_ld = _rope_rows(k, "k")
        if k.dtype != q.dtype or nk != N or dk != d:
            raise ValueError("q and k must share type, tokens and head dimension")
    positions, pos_ld, axes, rot, axis, freq = _rope_how(positions, N, d, rot_dim, sections, interleaved, base, inv_freq)
    if out is None:
        qo = torch.empty_like(q, memory_format=torch.contiguous_format)
        ko = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
        qo_ld, ko_ld = hq * d, hkv * d
    else:
        qo, ko = out
        if qo.shape != q.shape or qo.dtype != q.dtype or (ko is None) != (k is None) or \
                (k is not None and (ko.shape != k.shape or ko.dtype != k.dtype)):
            raise ValueError("out must have the shapes and type of q and k")
        qo_ld = _rope_rows(qo, "q_out")[3]
        ko_ld = 0 if ko is None else _rope_rows(ko, "k_out")[3]
    _call("tt_rope", _device_of(q, k, positions, qo, ko), q.data_ptr(), qo.data_ptr(), q_ld, qo_ld, _ptr(k), _ptr(ko),
          k_ld, ko_ld, _DTYPES[q.dtype], N, hq, hkv, d, rot, positions.data_ptr(), pos_ld, axes, axis, freq,
          1 if adjacent else 0, 1 if inverse else 0)
    return qo, ko


def rope_bwd(dq, dk, positions, **how):
    """Gradients of the unrotated q and k from those of rope's outputs (the inverse rotation; arguments as rope's)."""
    return rope(dq, dk, positions, inverse=True, **how)


# --------------------------------------------------------------------------- norm of the heads with rotary positions
def _norm_pair(q, k):
    """Checked (N, hq, hkv, d, stride of q, stride of k)."""
    N, hq, d, q_ld = _rope_rows(q, "q")
    if k is None:
        return N, hq, 0, d, q_ld, 0
    nk, hkv, dk, k_ld = _rope_rows(k, "k")
    if k.dtype != q.dtype or nk != N or dk != d:
        raise ValueError("q and k must share type, tokens and head dimension")
    return N, hq, hkv, d, q_ld, k_ld


def _norm_weights(q, q_weight, k_weight, d):
    """TT_DT_* of the weights: one type for both, q's or fp32."""
    kind = None
    for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor) or not w.is_cuda or w.dtype not in (q.dtype, torch.float32) or \
                (kind is not None and w.dtype != kind):
            raise TypeError(f"{n} must be a CUDA tensor of q's type or fp32, one type for both weights")
        if w.shape != (d,) or not w.is_contiguous():
            raise ValueError(f"{n} must be contiguous and have shape ({d},)")
        kind = w.dtype
    return _DTYPES[q.dtype if kind is None else kind]


def _like_heads(t, like, name):
    """Stride between tokens of a tensor with the shape and type of `like`."""
    if not isinstance(t, torch.Tensor) or t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError(f"{name} must have the shape and type of its input")
    return _rope_rows(t, name)[3]


def _norm_how(positions, N, d, rot_dim, sections, interleaved, base, inv_freq):
    """As _rope_how; rot_dim = 0: no positions."""
    if rot_dim is not None and int(rot_dim) == 0:
        return None, 0, 1, 0, None, None
    return _rope_how(positions, N, d, rot_dim, sections, interleaved, base, inv_freq)


def qk_norm_rope(q, k, positions, q_weight=None, k_weight=None, eps=1e-6, rot_dim=None, sections=None,
                 interleaved=False, adjacent=False, base=10000.0, inv_freq=None, out=None):
    """RMS norm of every head of q [N,Hq,d] and k [N,Hkv,d] and their rotary positions in one pass (tt_qk_norm_rope; k
    may be None): returns (q_out, k_out). Weights [d] (q's type or fp32; None = ones) are shared by the heads. Positions
    and tables as in `rope`; rot_dim = 0 leaves the rotation out (positions may be None). `out` = (q_out, k_out) may be
    (q, k)."""
    N, hq, hkv, d, q_ld, k_ld = _norm_pair(q, k)
    w_dtype = _norm_weights(q, q_weight, k_weight, d)
    positions, pos_ld, axes, rot, axis, freq = _norm_how(positions, N, d, rot_dim, sections, interleaved, base, inv_freq)
    if out is None:
        qo = torch.empty_like(q, memory_format=torch.contiguous_format)
        ko = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
        qo_ld, ko_ld = hq * d, hkv * d
    else:
        qo, ko = out
        if (ko is None) != (k is None):
            raise ValueError("out must have the shapes and type of q and k")
        qo_ld = _like_heads(qo, q, "q_out")
        ko_ld = 0 if ko is None else _like_heads(ko, k, "k_out")
    _call("tt_qk_norm_rope", _device_of(q, k, positions, q_weight, k_weight, qo, ko), q.data_ptr(), qo.data_ptr(), q_ld,
          qo_ld, _ptr(k), _ptr(ko), k_ld, ko_ld, _DTYPES[q.dtype], N, hq, hkv, d, _ptr(q_weight), _ptr(k_weight), w_dtype,
          eps, rot, _ptr(positions), pos_ld, axes, axis, freq, 1 if adjacent else 0)
    return qo, ko


def qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, q_weight=None, k_weight=None, eps=1e-6, rot_dim=None,
                     sections=None, interleaved=False, adjacent=False, base=10000.0, inv_freq=None, out=None, ws=None,
                     want_dw=True):
    """Gradients of qk_norm_rope (tt_qk_norm_rope_bwd): from those of its outputs and its inputs q, k, returns (dq, dk,
    dq_weight, dk_weight), the last two fp32 [d] (None without `want_dw`, and dk_weight without k). `out` = (dq, dk) may
    be (dq_out, dk_out) or (q, k)."""
    N, hq, hkv, d, q_ld, k_ld = _norm_pair(q, k)
    w_dtype = _norm_weights(q, q_weight, k_weight, d)
    positions, pos_ld, axes, rot, axis, freq = _norm_how(positions, N, d, rot_dim, sections, interleaved, base, inv_freq)
    if (dk_out is None) != (k is None):
        raise ValueError("dk_out goes with k")
    dqo_ld = _like_heads(dq_out, q, "dq_out")
    dko_ld = 0 if k is None else _like_heads(dk_out, k, "dk_out")
    if out is None:
        dq = torch.empty_like(q, memory_format=torch.contiguous_format)
        dk = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
        dq_ld, dk_ld = hq * d, hkv * d
    else:
        dq, dk = out
        if (dk is None) != (k is None):
            raise ValueError("out must have the shapes and type of q and k")
        dq_ld = _like_heads(dq, q, "dq")
        dk_ld = 0 if dk is None else _like_heads(dk, k, "dk")
    dwq = dwk = None
    if want_dw:
        dwq = torch.empty(d, dtype=torch.float32, device=q.device)
        dwk = None if k is None else torch.empty(d, dtype=torch.float32, device=q.device)
        if ws is None:
            ws = torch.empty(lib().tt_qk_norm_rope_bwd_workspace_bytes(d), dtype=torch.uint8, device=q.device)
    _call("tt_qk_norm_rope_bwd", _device_of(q, k, dq_out, dk_out, positions, q_weight, k_weight, dq, dk, ws),
          dq_out.data_ptr(), dqo_ld, q.data_ptr(), q_ld, dq.data_ptr(), dq_ld, _ptr(dk_out), dko_ld, _ptr(k), k_ld,
          _ptr(dk), dk_ld, _DTYPES[q.dtype], N, hq, hkv, d, _ptr(q_weight), _ptr(k_weight), w_dtype, eps, rot,
          _ptr(positions), pos_ld, axes, axis, freq, 1 if adjacent else 0, _ptr(dwq), _ptr(dwk), _ptr(ws),
          _room_of(ws, "ws"))
    return dq, dk, dwq, dwk


# --------------------------------------------------------------------------- attention
def _heads(Q, K):
    N, hq, d = Q.shape
    return N, hq, K.shape[1], d


def tree_attn_fwd(tree: Tree, Q, K, V, scale=None, out=None, err=None, tiles=None):
    """O [N,Hq,d] bf16, LSE [Hq,N] fp32 of tree attention (tt_tree_attn_fwd; with `tiles` = 1 or 2 the
    forward schedule is fixed through tt_tree_attn_fwd_tiles)."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _need(t, torch.bfloat16, n, 3)
    N, hq, hkv, d = _heads(Q, K)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    O = torch.empty_like(Q) if out is None else out[0]
    LSE = torch.empty(hq, N, dtype=torch.float32, device=Q.device) if out is None else out[1]
    err = tree.err if err is None else err
    if tiles is None:
        rc = lib().tt_tree_attn_fwd(_p(tree.ws), _p(Q), _p(K), _p(V), _p(O), _p(LSE), N, hq, hkv, d, scale, _p(err),
                                    _stream(Q.device))
    else:
        rc = lib().tt_tree_attn_fwd_tiles(_p(tree.ws), _p(Q), _p(K), _p(V), _p(O), _p(LSE), N, hq, hkv, d, scale,
                                          int(tiles), _p(err), _stream(Q.device))
    _check(rc, "tt_tree_attn_fwd")
    return O, LSE


def tree_attn_bwd(tree: Tree, Q, K, V, O, LSE, dO, scale=None, out=None, ws=None, err=None):
    """dQ, dK, dV (bf16) of tree attention (tt_tree_attn_bwd)."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O"), (dO, "dO")):
        _need(t, torch.bfloat16, n, 3)
    _need(LSE, torch.float32, "LSE", 2)
    N, hq, hkv, d = _heads(Q, K)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dQ, dK, dV = (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)) if out is None else out
    nbytes = lib().tt_tree_attn_bwd_workspace_bytes(N, hq)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=Q.device)
    err = tree.err if err is None else err
    rc = lib().tt_tree_attn_bwd(_p(tree.ws), _p(Q), _p(K), _p(V), _p(O), _p(LSE), _p(dO), _p(dQ), _p(dK), _p(dV), N,
                                hq, hkv, d, scale, _p(ws), ws.numel(), _p(err), _stream(Q.device))
    _check(rc, "tt_tree_attn_bwd")
    return dQ, dK, dV


def tree_attn_chunk_fwd(q, s0, k_path, v_path, o=None, lse=None, lse_ld=None, scale=None, err=None, tiles=None,
                        splits=None, send=None, blk_max=None):
    """Chunk-vs-path forward: q [C,Hq,d] at path offset s0 against k/v_path [s0+C,Hkv,d] (`tiles` as in
    tree_attn_fwd; `splits` = key-range splits per tile on the one-tile schedule, 0 = chosen, 1..4 fixed).
    `send` and `blk_max` (int32 device tensors, tt_tree_attn_chunk_fwd_packed) make it a packed chunk of sibling
    subtrees."""
    C, hq, d = q.shape
    hkv = k_path.shape[1]
    if k_path.shape[0] < s0 + C:
        raise ValueError("k_path must hold s0 + C rows")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q) if o is None else o
    lse_ld = C if lse_ld is None else lse_ld
    lse = torch.empty(hq, lse_ld, dtype=torch.float32, device=q.device) if lse is None else lse
    err = new_err(q.device) if err is None else err
    if send is not None:
        if tiles is not None or splits is not None:
            raise ValueError("a packed chunk takes no tiles or splits")
        rc = lib().tt_tree_attn_chunk_fwd_packed(_p(q), C, s0, _p(k_path), _p(v_path), _p(send), _p(blk_max), _p(o),
                                                 _p(lse), lse_ld, hq, hkv, d, scale, _p(err), _stream(q.device))
    elif splits is not None:
        if tiles is not None:
            raise ValueError("give tiles or splits, not both")
        rc = lib().tt_tree_attn_chunk_fwd_split(_p(q), C, s0, _p(k_path), _p(v_path), _p(o), _p(lse), lse_ld, hq, hkv,
                                                d, scale, int(splits), _p(err), _stream(q.device))
    elif tiles is None:
        rc = lib().tt_tree_attn_chunk_fwd(_p(q), C, s0, _p(k_path), _p(v_path), _p(o), _p(lse), lse_ld, hq, hkv, d,
                                          scale, _p(err), _stream(q.device))
    else:
        rc = lib().tt_tree_attn_chunk_fwd_tiles(_p(q), C, s0, _p(k_path), _p(v_path), _p(o), _p(lse), lse_ld, hq, hkv,
                                                d, scale, int(tiles), _p(err), _stream(q.device))
    _check(rc, "tt_tree_attn_chunk_fwd")
    return o, lse


def tree_attn_chunk_bwd(q, s0, k_path, v_path, o, lse, dO, dk_acc, dv_acc, lse_ld=None, dq=None, scale=None,
                        err=None, ws=None, send=None, blk_max=None):
    """Chunk-vs-path backward: returns dq; accumulates fp32 dk_acc / dv_acc in place (`send`, `blk_max`: a packed
    chunk, tt_tree_attn_chunk_bwd_packed)."""
    C, hq, d = q.shape
    hkv = k_path.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    lse_ld = C if lse_ld is None else lse_ld
    nbytes = lib().tt_tree_attn_chunk_bwd_workspace_bytes(C, hq)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if ws is None else ws
    err = new_err(q.device) if err is None else err
    if send is not None:
        rc = lib().tt_tree_attn_chunk_bwd_packed(_p(q), C, s0, _p(k_path), _p(v_path), _p(send), _p(blk_max), _p(o),
                                                 _p(lse), lse_ld, _p(dO), _p(dq), _p(dk_acc), _p(dv_acc), hq, hkv, d,
                                                 scale, _p(ws), ws.numel(), _p(err), _stream(q.device))
    else:
        rc = lib().tt_tree_attn_chunk_bwd(_p(q), C, s0, _p(k_path), _p(v_path), _p(o), _p(lse), lse_ld, _p(dO),
                                          _p(dq), _p(dk_acc), _p(dv_acc), hq, hkv, d, scale, _p(ws), ws.numel(),
                                          _p(err), _stream(q.device))
    _check(rc, "tt_tree_attn_chunk_bwd")
    return dq


@dataclass
class DecodePlan:
    """How the attention of one step of running rollouts is shared out (tt_tree_decode_plan), for all layers' calls."""
    plan: torch.Tensor
    S: int
    B: int
    rows: int
    pairs: int
    hq: int
    hkv: int
    d: int
    ws_bytes: int
    err: torch.Tensor

    def check(self):
        check_err(self.err, "tt_tree_decode_plan")
        return self


def tree_decode_plan(segments, B, rows, pairs, hq, hkv, d, err=None, out=None):
    """The plan of one step of B running rollouts: segments int32 [4, S] on the device, its rows kv_begin, kv_len,
    q_begin, q_end: the pool's rows [kv_begin, kv_begin + kv_len) are seen by the queries q_begin <= b < q_end. rows: of
    the pool; pairs: at least the sum of q_end - q_begin. `out`: a plan's tensor to write into (of the same S)."""
    _need(segments, torch.int32, "segments", 2)
    if segments.shape[0] != 4:
        raise ValueError("segments must be [4, S]: kv_begin, kv_len, q_begin, q_end")
    S, L = segments.shape[1], lib()
    nbytes = L.tt_tree_decode_plan_bytes(S)
    plan = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=segments.device) if out is None else out
    err = new_err(segments.device) if err is None else err
    at, step = segments.data_ptr(), 4 * S
    _call("tt_tree_decode_plan", _device_of(segments, plan, err), at, at + step, at + 2 * step, at + 3 * step, S, B, rows,
          pairs, hq, hkv, d, plan.data_ptr(), _room_of(plan, "out"), err.data_ptr())
    return DecodePlan(plan, S, B, rows, pairs, hq, hkv, d, L.tt_tree_decode_attn_workspace_bytes(pairs, hq, d), err)


def tree_decode_attn(plan: DecodePlan, q, k, v, scale=None, out=None, ws=None, err=None):
    """O [B,Hq,d], LSE [Hq,B] fp32 of the queries q [B,Hq,d] over the pool's keys and values k, v [rows,Hkv,d] (bf16 or
    fp16; rows of the pool any stride apart) that the plan lists for them (tt_tree_decode_attn). `ws`: plan.ws_bytes of
    scratch, one for calls that may overlap."""
    B, hq, d, q_ld = _rope_rows(q, "q")
    rows, hkv, dk, k_ld = _rope_rows(k, "k")
    _, _, _, v_ld = _rope_rows(v, "v")
    if k.dtype != q.dtype or v.dtype != q.dtype or v.shape != k.shape or k_ld != v_ld or dk != d:
        raise ValueError("q, k and v must share type and head dimension, k and v shape and strides")
    if (B, rows, hq, hkv, d) != (plan.B, plan.rows, plan.hq, plan.hkv, plan.d):
        raise ValueError("the plan is of other sizes")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        O = torch.empty_like(q, memory_format=torch.contiguous_format)
        LSE = torch.empty((hq, B), dtype=torch.float32, device=q.device)
    else:
        O, LSE = out
        if O.dtype != q.dtype or O.shape != q.shape or not O.is_contiguous():
            raise ValueError("O must be contiguous, with the type and shape of q")
        _per_row(LSE, torch.float32, "LSE", (hq, B), True)
    if ws is None:
        ws = torch.empty(plan.ws_bytes, dtype=torch.uint8, device=q.device)
    err = plan.err if err is None else err
    _call("tt_tree_decode_attn", _device_of(q, k, v, plan.plan, O, LSE, ws, err), plan.plan.data_ptr(), q.data_ptr(), q_ld,
          k.data_ptr(), v.data_ptr(), k_ld, _DTYPES[q.dtype], plan.S, B, rows, plan.pairs, hq, hkv, d, scale, O.data_ptr(),
          LSE.data_ptr(), ws.data_ptr(), _room_of(ws, "ws"), err.data_ptr())
    return O, LSE


DTA_ORDER_INDEX, DTA_ORDER_GREEDY = 0, 1
DTA_DEFAULT_SLOTS = 2  # TT_DTA_DEFAULT_SLOTS


def dta_workspace_bytes(seg_parent_host, seg_len_host, chunk, hq, hkv, d, slots=DTA_DEFAULT_SLOTS):
    """Device scratch bytes of the path-at-a-time pass for this tree, chunk size and slot count
    (tt_dta_workspace_bytes_slots)."""
    import numpy as np
    par = np.ascontiguousarray(seg_parent_host, dtype=np.int32)
    ln = np.ascontiguousarray(seg_len_host, dtype=np.int32)
    n = lib().tt_dta_workspace_bytes_slots(par.ctypes.data_as(_vp), ln.ctypes.data_as(_vp), len(par), chunk, hq, hkv,
                                           d, slots)
    if n == 0:
        raise TTError(-2, "tt_dta_workspace_bytes")
    return n


def tree_partition(seg_parent_host, seg_len_host, budget, order=DTA_ORDER_GREEDY):
    """The partitions of the path-at-a-time traversal for a token budget (tt_tree_partition), in DFS layout order:
    numpy arrays (first row, rows, cached path rows, kind: 0 pack of sibling subtrees, 1 chunk of one segment)."""
    import numpy as np
    par = np.ascontiguousarray(seg_parent_host, dtype=np.int32)
    ln = np.ascontiguousarray(seg_len_host, dtype=np.int32)
    pp, lp = par.ctypes.data_as(_vp), ln.ctypes.data_as(_vp)
    n = lib().tt_tree_partition(pp, lp, len(par), int(budget), order, None, None, None, None, 0)
    _check(n if n < 0 else 0, "tt_tree_partition")
    first, rows, path = (np.zeros(n, np.int64) for _ in range(3))
    kind = np.zeros(n, np.int32)
    rc = lib().tt_tree_partition(pp, lp, len(par), int(budget), order, first.ctypes.data_as(_vp),
                                 rows.ctypes.data_as(_vp), path.ctypes.data_as(_vp), kind.ctypes.data_as(_vp), n)
    _check(rc if rc < 0 else 0, "tt_tree_partition")
    return first, rows, path, kind


def dta_leaf_order(seg_parent_host, seg_len_host, order=DTA_ORDER_GREEDY):
    """Leaves (segment ids) in the order the path-at-a-time traversal reaches them (tt_dta_leaf_order)."""
    import numpy as np
    par = np.ascontiguousarray(seg_parent_host, dtype=np.int32)
    ln = np.ascontiguousarray(seg_len_host, dtype=np.int32)
    out = np.empty(max(len(par), 1), np.int32)
    n = lib().tt_dta_leaf_order(par.ctypes.data_as(_vp), ln.ctypes.data_as(_vp), len(par), order,
                                out.ctypes.data_as(_vp), len(out))
    if n < 0:
        raise TTError(n, "tt_dta_leaf_order")
    return out[:n].copy()


def dta_tree_attn(seg_parent_host, seg_len_host, Q, K, V, dO, chunk=2048, scale=None, err=None, ws=None, out=None,
                  order=DTA_ORDER_GREEDY, slots=DTA_DEFAULT_SLOTS):
    """Whole-tree fwd+bwd by path-at-a-time traversal (tt_dta_tree_attn_slots): O, LSE, dQ, dK, dV
    (written into `out` = (O, LSE, dQ, dK, dV) when given); `order` = DTA_ORDER_GREEDY or DTA_ORDER_INDEX;
    `slots` = sibling leaves processed at once (1 = the one-path traversal)."""
    import numpy as np
    par = np.ascontiguousarray(seg_parent_host, dtype=np.int32)
    ln = np.ascontiguousarray(seg_len_host, dtype=np.int32)
    N, hq, hkv, d = _heads(Q, K)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    pp, lp = par.ctypes.data_as(_vp), ln.ctypes.data_as(_vp)
    if ws is None:
        nbytes = lib().tt_dta_workspace_bytes_slots(pp, lp, len(par), chunk, hq, hkv, d, slots)
        if nbytes == 0:
            raise TTError(-2, "tt_dta_workspace_bytes")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=Q.device)
    if out is None:
        O, dQ = torch.empty_like(Q), torch.empty_like(Q)
        dK, dV = torch.empty_like(K), torch.empty_like(V)
        LSE = torch.empty(hq, N, dtype=torch.float32, device=Q.device)
    else:
        O, LSE, dQ, dK, dV = out
    err = new_err(Q.device) if err is None else err
    rc = lib().tt_dta_tree_attn_slots(pp, lp, len(par), N, chunk, order, slots, _p(Q), _p(K), _p(V), _p(dO), _p(O),
                                      _p(LSE), _p(dQ), _p(dK), _p(dV), hq, hkv, d, scale, _p(ws), ws.numel(), _p(err),
                                      _stream(Q.device))
    _check(rc, "tt_dta_tree_attn")
    return O, LSE, dQ, dK, dV


class DtaPlan:
    """The path-at-a-time pass of one tree captured once into a CUDA graph (tt_dta_plan_create); launch() enqueues
    the whole pass with one call. The input and output tensors are bound at creation: write new inputs into them
    and keep them alive while the plan exists. `outputs` = (O, LSE, dQ, dK, dV)."""

    def __init__(self, seg_parent_host, seg_len_host, Q, K, V, dO, chunk=2048, scale=None, err=None, ws=None,
                 out=None, order=DTA_ORDER_GREEDY, slots=DTA_DEFAULT_SLOTS):
        import numpy as np
        self._plan = None
        par = np.ascontiguousarray(seg_parent_host, dtype=np.int32)
        ln = np.ascontiguousarray(seg_len_host, dtype=np.int32)
        N, hq, hkv, d = _heads(Q, K)
        scale = 1.0 / math.sqrt(d) if scale is None else scale
        pp, lp = par.ctypes.data_as(_vp), ln.ctypes.data_as(_vp)
        nbytes = lib().tt_dta_workspace_bytes_slots(pp, lp, len(par), chunk, hq, hkv, d, slots)
        if nbytes == 0:
            raise TTError(-2, "tt_dta_workspace_bytes")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=Q.device) if ws is None else ws
        if out is None:
            out = (torch.empty_like(Q), torch.empty(hq, N, dtype=torch.float32, device=Q.device), torch.empty_like(Q),
                   torch.empty_like(K), torch.empty_like(V))
        self.outputs = tuple(out)
        self.err = new_err(Q.device) if err is None else err
        self.device = Q.device
        self._keep = (Q, K, V, dO)
        O, LSE, dQ, dK, dV = self.outputs
        plan = ctypes.c_void_p(0)
        rc = lib().tt_dta_plan_create(pp, lp, len(par), N, chunk, order, slots, _p(Q), _p(K), _p(V), _p(dO), _p(O),
                                      _p(LSE),
                                      _p(dQ), _p(dK), _p(dV), hq, hkv, d, scale, _p(self.ws), self.ws.numel(),
                                      _p(self.err), ctypes.byref(plan))
        _check(rc, "tt_dta_plan_create")
        self._plan = plan

    def launch(self):
        """Enqueue the pass on the current stream; returns the output tensors."""
        _check(lib().tt_dta_plan_launch(self._plan, _stream(self.device)), "tt_dta_plan_launch")
        return self.outputs

    def close(self):
        if self._plan is not None and self._plan.value:
            _check(lib().tt_dta_plan_destroy(self._plan), "tt_dta_plan_destroy")
        self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------------------------- log-prob
def weighted_logprob(logits, targets, weights=None, g=1.0, want_dlogits=True, out=None, err=None):
    """logp fp32 [N], loss fp64 (device scalar), dlogits bf16 [N,V] or None (tt_weighted_logprob). `logits` may be a
    row-padded view (rows ld >= V elements apart, elements contiguous); dlogits then has the same row stride."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dtype != torch.bfloat16 or logits.dim() != 2:
        raise TypeError("logits must be a 2-D bf16 CUDA tensor")
    N, V = logits.shape
    ld = logits.stride(0) if N > 1 else V
    if logits.stride(1) != 1 or ld < V:
        raise ValueError("logits rows must be contiguous (stride(1) == 1, stride(0) >= V)")
    _need(targets, torch.int32, "targets", 1)
    if weights is not None:
        _need(weights, torch.float32, "weights", 1)
    dev = logits.device
    if out is None:
        logp = torch.empty(N, dtype=torch.float32, device=dev)
        loss = torch.empty(1, dtype=torch.float64, device=dev)
        dl = torch.empty(N, ld, dtype=torch.bfloat16, device=dev)[:, :V] if want_dlogits else None
    else:
        logp, loss, dl = out
    if dl is not None and (dl.shape != logits.shape or dl.stride() != logits.stride()):
        raise ValueError("dlogits must have the shape and strides of logits")
    err = new_err(dev) if err is None else err
    rc = lib().tt_weighted_logprob(_p(logits), N, V, ld, _p(targets), _p(weights), g, _p(logp), _p(loss), _p(dl),
                                   _p(err), _stream(dev))
    _check(rc, "tt_weighted_logprob")
    return logp, loss, dl


# --------------------------------------------------------------------------- log-prob, entropy, top alternatives
def _logit_rows(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DTYPES or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D bf16, fp16 or fp32 CUDA tensor")
    N, V = t.shape
    if t.is_contiguous():
        return N, V, V
    ld, one = t.stride()
    if N <= 1:
        ld = V
    if (V > 1 and one != 1) or ld < V:
        raise ValueError(f"{name} rows must be contiguous (stride(1) == 1, stride(0) >= V)")
    return N, V, ld


def _per_row(t, dtype, name, shape, required=False):
    if t is None:
        if required:
            raise TypeError(f"{name} must be a CUDA tensor")
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and have shape {tuple(shape)}")


def token_logprob(logits, targets=None, top_k=0, out=None, err=None):
    """Per row of logits [N,V] (bf16, fp16 or fp32; rows may be padded): (logp, entropy, lse, top_ids, top_logp) of
    tt_token_logprob: fp32 [N] each, and int32 / fp32 [N, top_k] of the top alternatives. logp is None without
    targets, top_ids and top_logp are None with top_k = 0."""
    N, V, ld = _logit_rows(logits, "logits")
    rows, dev, k = (N,), logits.device, int(top_k)
    _per_row(targets, torch.int32, "targets", rows)
    if out is None:
        logp = torch.empty(N, dtype=torch.float32, device=dev) if targets is not None else None
        entropy, lse = torch.empty(N, dtype=torch.float32, device=dev), torch.empty(N, dtype=torch.float32, device=dev)
        ids = torch.empty((N, k), dtype=torch.int32, device=dev) if k > 0 else None
        top = torch.empty((N, k), dtype=torch.float32, device=dev) if k > 0 else None
    else:
        logp, entropy, lse, ids, top = out
        for t, n in ((logp, "logp"), (entropy, "entropy"), (lse, "lse")):
            _per_row(t, torch.float32, n, rows)
        _per_row(ids, torch.int32, "top_ids", (N, k))
        _per_row(top, torch.float32, "top_logp", (N, k))
    err = new_err(dev) if err is None else err
    _call("tt_token_logprob", _device_of(logits, targets, logp, entropy, lse, ids, top, err), logits.data_ptr(),
          _DTYPES[logits.dtype], N, V, ld, _ptr(targets), k, _ptr(logp), _ptr(entropy), _ptr(lse), _ptr(ids), _ptr(top),
          err.data_ptr())
    return logp, entropy, lse, ids, top


def token_logprob_bwd(logits, lse, entropy=None, targets=None, dlogp=None, dentropy=None, dlse=None, top_ids=None,
                      dtop=None, out=None, err=None):
    """dlogits (type and row stride of logits) of an objective whose gradients with respect to token_logprob's outputs
    are dlogp, dentropy, dlse [N] and dtop [N, k] (log-probs of top_ids), each optional (tt_token_logprob_bwd). `out`
    may be logits itself, which is then overwritten."""
    N, V, ld = _logit_rows(logits, "logits")
    rows = (N,)
    _per_row(lse, torch.float32, "lse", rows, True)
    _per_row(targets, torch.int32, "targets", rows)
    for t, n in ((entropy, "entropy"), (dlogp, "dlogp"), (dentropy, "dentropy"), (dlse, "dlse")):
        _per_row(t, torch.float32, n, rows)
    if (top_ids is None) != (dtop is None):
        raise ValueError("top_ids and dtop go together")
    k = 0
    if dtop is not None:
        k = dtop.shape[-1]
        _per_row(top_ids, torch.int32, "top_ids", (N, k))
        _per_row(dtop, torch.float32, "dtop", (N, k))
    if out is None:
        out = torch.empty((N, ld), dtype=logits.dtype, device=logits.device)
        if ld != V:
            out = out[:, :V]
    elif out.dtype != logits.dtype or out.shape != logits.shape or (N > 1 and out.stride() != logits.stride()) or \
            (V > 1 and out.stride(1) != 1):
        raise ValueError("out must have the type, shape and strides of logits")
    err = new_err(logits.device) if err is None else err
    _call("tt_token_logprob_bwd", _device_of(logits, lse, entropy, targets, dlogp, dentropy, dlse, top_ids, dtop, out, err),
          logits.data_ptr(), _DTYPES[logits.dtype], N, V, ld, _ptr(lse), _ptr(entropy), _ptr(targets), _ptr(dlogp),
          _ptr(dentropy), _ptr(dlse), _ptr(top_ids), _ptr(dtop), k, out.data_ptr(), err.data_ptr())
    return out


def lmhead_logprob(hidden, w_vocab, targets, weights=None, out=None, ws=None, err=None):
    """LM head fused with the weighted log-prob (tt_lmhead_logprob): logits z = hidden·w_vocabᵀ are never stored.
    hidden [N,Hd] bf16, w_vocab [V,Hd] bf16 -> (logp fp32 [N], lse fp32 [N], loss fp64 device scalar)."""
    _need(hidden, torch.bfloat16, "hidden", 2)
    _need(w_vocab, torch.bfloat16, "w_vocab", 2)
    _need(targets, torch.int32, "targets", 1)
    if weights is not None:
        _need(weights, torch.float32, "weights", 1)
    N, Hd = hidden.shape
    V = w_vocab.shape[0]
    if w_vocab.shape[1] != Hd:
        raise ValueError("hidden and w_vocab must share Hd")
    dev = hidden.device
    if out is None:
        logp = torch.empty(N, dtype=torch.float32, device=dev)
        lse = torch.empty(N, dtype=torch.float32, device=dev)
        loss = torch.empty(1, dtype=torch.float64, device=dev)
    else:
        logp, lse, loss = out
    nbytes = lib().tt_lmhead_logprob_workspace_bytes(N, V)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if ws is None else ws
    err = new_err(dev) if err is None else err
    rc = lib().tt_lmhead_logprob(_p(hidden), _p(w_vocab), N, V, Hd, _p(targets), _p(weights), _p(logp), _p(lse),
                                 _p(loss), _p(ws), ws.numel(), _p(err), _stream(dev))
    _check(rc, "tt_lmhead_logprob")
    return logp, lse, loss


def lmhead_logprob_bwd(hidden, w_vocab, targets, lse, weights=None, g=1.0, out=None, ws=None, err=None):
    """Gradients of g·loss of lmhead_logprob (tt_lmhead_logprob_bwd): d_hidden bf16 [N,Hd], d_w_vocab fp32 [V,Hd]."""
    _need(hidden, torch.bfloat16, "hidden", 2)
    _need(w_vocab, torch.bfloat16, "w_vocab", 2)
    _need(targets, torch.int32, "targets", 1)
    _need(lse, torch.float32, "lse", 1)
    if weights is not None:
        _need(weights, torch.float32, "weights", 1)
    N, Hd = hidden.shape
    V = w_vocab.shape[0]
    dev = hidden.device
    if out is None:
        dh = torch.empty_like(hidden)
        dw = torch.empty(V, Hd, dtype=torch.float32, device=dev)
    else:
        dh, dw = out
    if ws is None:
        ws = torch.empty(lib().tt_lmhead_logprob_bwd_workspace_bytes(N, V), dtype=torch.uint8, device=dev)
    err = new_err(dev) if err is None else err
    rc = lib().tt_lmhead_logprob_bwd(_p(hidden), _p(w_vocab), N, V, Hd, _p(targets), _p(weights), g, _p(lse), _p(dh),
                                     _p(dw), _p(ws), ws.numel(), _p(err), _stream(dev))
    _check(rc, "tt_lmhead_logprob_bwd")
    return dh, dw


class _Policy(ctypes.Structure):
    _fields_ = [(n, _f32) for n in ("clip_lo", "clip_hi", "dual_clip", "kl_coef", "entropy_coef", "g")]


@functools.lru_cache(maxsize=64)
def _policy(clip, dual_clip, kl_coef, entropy_coef, g):
    lo, hi = clip
    return ctypes.byref(_Policy(lo, hi, 0.0 if dual_clip is None else dual_clip, kl_coef, entropy_coef, g))


def _coefficient(x, name):
    """x as a float: a tensor's value now, not the tensor, is what a cached struct may be kept by. One on a device is refused:
    to read it back would make every call wait for the stream, and fail in a capture."""
    if type(x) is float:
        return x
    if isinstance(x, torch.Tensor) and x.device.type != "cpu":
        raise TypeError(f"{name} must be a number on the host")
    return float(x)


def _policy_of(clip, dual_clip, kl_coef, entropy_coef, g):
    """The host struct tt_policy. clip: one number for both sides, or (below, above)."""
    lo, hi = clip if isinstance(clip, (tuple, list)) else (clip, clip)
    if dual_clip is not None:
        dual_clip = _coefficient(dual_clip, "dual_clip")
        if not dual_clip >= 1:
            raise ValueError("dual_clip must be at least 1 (None: no such bound)")
    return _policy((_coefficient(lo, "clip"), _coefficient(hi, "clip")), dual_clip, _coefficient(kl_coef, "kl_coef"),
                   _coefficient(entropy_coef, "entropy_coef"), _coefficient(g, "g"))


def policy_loss(logp, old_logp, adv, adv_neg=None, ref_logp=None, entropy=None, weights=None, clip=0.2, dual_clip=None,
                kl_coef=0.0, entropy_coef=0.0, g=1.0, out=None, ws=None):
    """Clipped policy objective from log-probs [N] (tt_policy_loss): (sums, dlogp, dentropy), all fp32: sums [4] = loss,
    policy, KL and entropy terms; dlogp [N] and dentropy [N] (None without `entropy`) the gradients of g·loss, which
    token_logprob_bwd and lmhead_token_logprob_bwd take. adv: a signed advantage per token, or with `adv_neg` the sums
    of the positive and of the negative advantages (magnitudes) of the rollouts through it. Tokens of weight 0 are
    masked."""
    _per_row(logp, torch.float32, "logp", (logp.numel(),) if isinstance(logp, torch.Tensor) else (0,), True)
    N = logp.numel()
    for t, n, need in ((old_logp, "old_logp", True), (adv, "adv", True), (adv_neg, "adv_neg", False),
                       (ref_logp, "ref_logp", False), (entropy, "entropy", False), (weights, "weights", False)):
        _per_row(t, torch.float32, n, (N,), need)
    dev = logp.device
    policy = _policy_of(clip, dual_clip, kl_coef, entropy_coef, g)
    if out is None:
        sums, dlogp = torch.empty(4, dtype=torch.float32, device=dev), torch.empty_like(logp)
        dent = None if entropy is None else torch.empty_like(logp)
    else:
        sums, dlogp, dent = out
        _per_row(sums, torch.float32, "sums", (4,), True)
        _per_row(dlogp, torch.float32, "dlogp", (N,))
        _per_row(dent, torch.float32, "dentropy", (N,))
    if ws is None:
        nbytes = lib().tt_policy_loss_workspace_bytes(N)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call("tt_policy_loss", _device_of(logp, old_logp, adv, adv_neg, ref_logp, entropy, weights, sums, dlogp, dent, ws),
          logp.data_ptr(), _ptr(entropy), old_logp.data_ptr(), adv.data_ptr(), _ptr(adv_neg), _ptr(ref_logp),
          _ptr(weights), N, policy, sums.data_ptr(), _ptr(dlogp), _ptr(dent), _ptr(ws), _room_of(ws, "ws"))
    return sums, dlogp, dent


def policy_loss_logits(logits, targets, old_logp, adv, adv_neg=None, ref_logp=None, weights=None, clip=0.2,
                       dual_clip=None, kl_coef=0.0, entropy_coef=0.0, g=1.0, want_dlogits=True, out=None, ws=None,
                       err=None):
    """Clipped policy objective from logits [N,V] (bf16, fp16 or fp32; rows may be padded) with the gradient with respect
    to them, in one read (tt_policy_loss_logits): (sums, logp, entropy, dlogits). Arguments as in policy_loss; `out` =
    (sums, logp, entropy, dlogits), whose dlogits may be logits itself. A masked row (weight 0) is not regarded: its
    logp, entropy and dlogits are 0."""
    N, V, ld = _logit_rows(logits, "logits")
    rows, dev = (N,), logits.device
    _per_row(targets, torch.int32, "targets", rows, True)
    for t, n, need in ((old_logp, "old_logp", True), (adv, "adv", True), (adv_neg, "adv_neg", False),
                       (ref_logp, "ref_logp", False), (weights, "weights", False)):
        _per_row(t, torch.float32, n, rows, need)
    policy = _policy_of(clip, dual_clip, kl_coef, entropy_coef, g)
    if out is None:
        sums, logp, entropy = (torch.empty(n, dtype=torch.float32, device=dev) for n in (4, N, N))
        dl = None
        if want_dlogits:
            dl = torch.empty((N, ld), dtype=logits.dtype, device=dev)
            if ld != V:
                dl = dl[:, :V]
    else:
        sums, logp, entropy, dl = out
        _per_row(sums, torch.float32, "sums", (4,), True)
        _per_row(logp, torch.float32, "logp", rows, True)
        _per_row(entropy, torch.float32, "entropy", rows, True)
        if dl is not None and (dl.dtype != logits.dtype or dl.shape != logits.shape or
                               (N > 1 and dl.stride() != logits.stride()) or (V > 1 and dl.stride(1) != 1)):
            raise ValueError("dlogits must have the type, shape and strides of logits")
    if ws is None:
        ws = torch.empty(max(1, lib().tt_policy_loss_logits_workspace_bytes(N)), dtype=torch.uint8, device=dev)
    err = new_err(dev) if err is None else err
    _call("tt_policy_loss_logits",
          _device_of(logits, targets, old_logp, adv, adv_neg, ref_logp, weights, sums, logp, entropy, dl, ws, err),
          logits.data_ptr(), _DTYPES[logits.dtype], N, V, ld, targets.data_ptr(), old_logp.data_ptr(), adv.data_ptr(),
          _ptr(adv_neg), _ptr(ref_logp), _ptr(weights), policy, sums.data_ptr(), logp.data_ptr(), entropy.data_ptr(),
          _ptr(dl), ws.data_ptr(), _room_of(ws, "ws"), err.data_ptr())
    return sums, logp, entropy, dl


def _lmhead_args(hidden, w_vocab, targets):
    _need(hidden, torch.bfloat16, "hidden", 2)
    _need(w_vocab, torch.bfloat16, "w_vocab", 2)
    N, Hd = hidden.shape
    if w_vocab.shape[1] != Hd:
        raise ValueError("hidden and w_vocab must share Hd")
    _per_row(targets, torch.int32, "targets", (N,), True)
    return N, w_vocab.shape[0], Hd


def lmhead_token_logprob(hidden, w_vocab, targets, out=None, ws=None, err=None):
    """LM head fused with the per-token log-prob and entropy (tt_lmhead_token_logprob): logits z = hidden·w_vocabᵀ are
    never stored. hidden [N,Hd] bf16, w_vocab [V,Hd] bf16 -> (logp, entropy, lse), fp32 [N] each."""
    N, V, Hd = _lmhead_args(hidden, w_vocab, targets)
    dev = hidden.device
    if out is None:
        logp, entropy, lse = (torch.empty(N, dtype=torch.float32, device=dev) for _ in range(3))
    else:
        logp, entropy, lse = out
        for t, n in ((logp, "logp"), (entropy, "entropy"), (lse, "lse")):
            _per_row(t, torch.float32, n, (N,), True)
    if ws is None:
        ws = torch.empty(lib().tt_lmhead_token_logprob_workspace_bytes(N, V, Hd), dtype=torch.uint8, device=dev)
    err = new_err(dev) if err is None else err
    _call("tt_lmhead_token_logprob", _device_of(hidden, w_vocab, targets, logp, entropy, lse, ws, err),
          hidden.data_ptr(), w_vocab.data_ptr(), N, V, Hd, targets.data_ptr(), logp.data_ptr(), entropy.data_ptr(),
          lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), err.data_ptr())
    return logp, entropy, lse


def lmhead_token_logprob_bwd(hidden, w_vocab, targets, lse, entropy=None, dlogp=None, dentropy=None, dlse=None,
                             out=None, ws=None, err=None, dw_dtype=torch.float32):
    """Gradients of an objective whose gradients with respect to lmhead_token_logprob's outputs are dlogp, dentropy and
    dlse [N] (each optional; tt_lmhead_token_logprob_bwd): d_hidden bf16 [N,Hd], d_w_vocab fp32 or bf16 [V,Hd]
    (`dw_dtype`, or the type of out[1])."""
    N, V, Hd = _lmhead_args(hidden, w_vocab, targets)
    dev = hidden.device
    _per_row(lse, torch.float32, "lse", (N,), True)
    for t, n in ((entropy, "entropy"), (dlogp, "dlogp"), (dentropy, "dentropy"), (dlse, "dlse")):
        _per_row(t, torch.float32, n, (N,))
    if out is None:
        if dw_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("dw_dtype must be torch.float32 or torch.bfloat16")
        dh, dw = torch.empty_like(hidden), torch.empty((V, Hd), dtype=dw_dtype, device=dev)
    else:
        dh, dw = out
        _per_row(dh, torch.bfloat16, "d_hidden", (N, Hd), True)
        if dw is None or dw.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("d_w_vocab must be an fp32 or bf16 CUDA tensor")
        _per_row(dw, dw.dtype, "d_w_vocab", (V, Hd))
    if ws is None:
        ws = torch.empty(lib().tt_lmhead_token_logprob_bwd_workspace_bytes(N, V, Hd), dtype=torch.uint8, device=dev)
    err = new_err(dev) if err is None else err
    _call("tt_lmhead_token_logprob_bwd",
          _device_of(hidden, w_vocab, targets, lse, entropy, dlogp, dentropy, dlse, dh, dw, ws, err), hidden.data_ptr(),
          w_vocab.data_ptr(), N, V, Hd, targets.data_ptr(), lse.data_ptr(), _ptr(entropy), _ptr(dlogp), _ptr(dentropy),
          _ptr(dlse), dh.data_ptr(), dw.data_ptr(), _DTYPES[dw.dtype], ws.data_ptr(), ws.numel() * ws.element_size(),
          err.data_ptr())
    return dh, dw


KERNEL_CLASSES = ("fwd", "bwd", "logprob", "lmhead")  # TT_KT_* order


def kernel_timing(on: bool):
    """Turn launch timing on (clearing earlier records) or off (tt_kernel_timing)."""
    _check(lib().tt_kernel_timing(1 if on else 0), "kernel_timing")


def kernel_timing_read():
    """{class: (milliseconds, launches)} of the launches timed since kernel_timing(True), and the
    number of launches that were not timed (tt_kernel_timing_read; waits for the recorded events)."""
    n = len(KERNEL_CLASSES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    dropped = ctypes.c_int64(0)
    _check(lib().tt_kernel_timing_read(ctypes.cast(ms, _vp), ctypes.cast(cnt, _vp), n, ctypes.byref(dropped)),
           "kernel_timing_read")
    return {c: (ms[i], cnt[i]) for i, c in enumerate(KERNEL_CLASSES)}, dropped.value


def trie_build(rollouts):
    """Prefix tree of rollouts given as sequences of token ids (tt_trie_build, host only).

    Returns a dict of numpy arrays: seg_parent [S], seg_len [S] (int32; valid tree_build inputs), tokens [N]
    (token ids in DFS order), rollout_end [R] (DFS index of each rollout's last token), and the counts
    total_tokens and leaf_tokens (compression = total_tokens / N; leaves-only = leaf_tokens / N)."""
    import numpy as np
    seqs = [np.asarray(r, dtype=np.int32).ravel() for r in rollouts]
    R = len(seqs)
    offsets = np.zeros(R + 1, np.int64)
    if R:
        offsets[1:] = np.cumsum([len(x) for x in seqs])
    toks = np.concatenate(seqs) if R else np.zeros(0, np.int32)
    cap = max(int(offsets[-1]), 1)
    par, ln, tok = (np.empty(cap, np.int32) for _ in range(3))
    ends = np.empty(max(R, 1), np.int64)
    counts = np.zeros(4, np.int64)
    vp = lambda a: a.ctypes.data_as(_vp)
    _check(lib().tt_trie_build(vp(toks), vp(offsets), R, cap, vp(par), vp(ln), vp(tok), vp(ends), vp(counts)),
           "trie_build")
    S, N = int(counts[0]), int(counts[1])
    return {"seg_parent": par[:S].copy(), "seg_len": ln[:S].copy(), "tokens": tok[:N].copy(),
            "rollout_end": ends[:R].copy(), "total_tokens": int(counts[2]), "leaf_tokens": int(counts[3])}
