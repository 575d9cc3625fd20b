"""Sizes and addresses that the calls of the policy step refuse on the host (C ABI; CPU)."""
import ctypes

import pytest

from tests.test_policy_ops_args import BAD, L, _decode, _logits, _norm, _normb, _plan  # noqa: F401

odd = ctypes.c_void_p((1 << 12) + 2)


@pytest.mark.parametrize("S,ok", [(0, True), ((1 << 24) - 1, True), (1 << 24, False), (-1, False)])
def test_segments_fit_the_24_bits_that_count_them(L, S, ok):  # noqa: F811
    assert (L.tt_tree_decode_plan_bytes(S) > 0) == ok
    if not ok:
        assert _plan(L, S=S, n=1 << 40) == BAD


@pytest.mark.parametrize("name", ["kb", "kl", "qb", "qe"])
def test_plan_addresses(L, name):  # noqa: F811
    assert _plan(L, **{name: odd}) == BAD


@pytest.mark.parametrize("over", [dict(lse=odd), dict(scale=3e38), dict(scale=-3e38)])
def test_attention_addresses_and_scale(L, over):  # noqa: F811
    assert _decode(L, **over) == BAD


@pytest.mark.parametrize("name", ["y", "old", "adv", "neg", "ref", "w", "logp", "h", "err"])
def test_objective_addresses(L, name):  # noqa: F811
    assert _logits(L, **{name: odd}) == BAD


def test_norm_addresses(L):  # noqa: F811
    assert _norm(L, pos=odd) == _normb(L, pos=odd) == BAD
