"""The sections of the rotary positions are taken by their values at the call (binding; CPU and GPU)."""
import numpy as np
import pytest
import torch

from prefix_tree_gb300._native import _rope_tables, _section_sizes


@pytest.mark.parametrize("make", [torch.tensor, np.array, np.int32, int])
def test_sizes_are_kept_by_value(make):
    a, b = make(10), make(22)
    assert _section_sizes((a, b)) == _section_sizes([a, b]) == (10, 22)
    assert all(type(n) is int for n in _section_sizes((a, b)))
    tables = _rope_tables(64, _section_sizes((a, b)), False, 1e4, None)
    assert tables is _rope_tables(64, (10, 22), False, 1e4, None)


def test_other_numbers_are_refused():
    for bad in ((16.0, 16), (torch.tensor(16.0), 16), (torch.empty((), dtype=torch.int64, device="meta"), 16), ("16", 16)):
        with pytest.raises(TypeError):
            _section_sizes(bad)


@pytest.mark.gpu
def test_sections_that_change_in_place(tt):
    q = torch.randn(5, 2, 64, device="cuda")
    pos = torch.randint(0, 100, (2, 5), dtype=torch.int32, device="cuda")
    sizes = [torch.tensor(10), torch.tensor(22)]
    for first in (10, 20):
        sizes[0].fill_(first), sizes[1].fill_(32 - first)
        plain = (first, 32 - first)
        assert torch.equal(tt.rope(q, None, pos, sections=sizes)[0], tt.rope(q, None, pos, sections=plain)[0])
        assert torch.equal(tt.qk_norm_rope(q, None, pos, sections=sizes)[0], tt.qk_norm_rope(q, None, pos, sections=plain)[0])
