"""The coefficients of the policy objective are taken by their values at the call (binding; CPU)."""
import numpy as np
import pytest
import torch

from prefix_tree_gb300._native import _policy_of

NAMES = ("clip", "dual_clip", "kl_coef", "entropy_coef", "g")
PLAIN = dict(clip=0.2, dual_clip=2.0, kl_coef=0.1, entropy_coef=0.01, g=1.0)


def _fields(p):
    return {n: getattr(p._obj, n) for n, _ in p._obj._fields_}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("make", [torch.tensor, lambda x: torch.tensor(x, dtype=torch.float64), np.array, np.float32])
def test_a_coefficient_that_changes_in_place(name, make):
    """An adaptive coefficient kept in a tensor or array: each call takes what it holds then."""
    c = make(PLAIN[name])
    for factor in (1.0, 1.5, 3.0):
        value = PLAIN[name] * factor
        if c.ndim == 0 and not isinstance(c, np.generic):
            c[...] = value
        else:
            c = make(value)
        got = _fields(_policy_of(**{**PLAIN, name: c}))
        assert got == _fields(_policy_of(**{**PLAIN, name: float(c)}))
        assert got[{"clip": "clip_hi"}.get(name, name)] == pytest.approx(value, rel=1e-6)


def test_both_sides_of_the_range():
    lo, hi = torch.tensor(0.1), torch.tensor(0.3)
    for clip in ((lo, hi), [lo, hi], (0.1, hi)):
        p = _fields(_policy_of(**{**PLAIN, "clip": clip}))
        assert p["clip_lo"] == pytest.approx(0.1) and p["clip_hi"] == pytest.approx(0.3)
    hi.mul_(2)
    assert _fields(_policy_of(**{**PLAIN, "clip": (lo, hi)}))["clip_hi"] == pytest.approx(0.6)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_that_are_not_on_the_host_are_refused(name):
    x = torch.empty((), device="meta")
    with pytest.raises(TypeError):
        _policy_of(**{**PLAIN, name: x})
    if name == "clip":
        with pytest.raises(TypeError):
            _policy_of(**{**PLAIN, "clip": (0.2, x)})


def test_refused_values():
    for bad in (0.5, torch.tensor(0.5), float("nan")):
        with pytest.raises(ValueError):
            _policy_of(**{**PLAIN, "dual_clip": bad})
    assert _fields(_policy_of(**{**PLAIN, "dual_clip": None}))["dual_clip"] == 0.0
