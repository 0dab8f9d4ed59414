"""Arguments that the paged attention's and the rotation's calls refuse, on the CPU."""
import ctypes

import pytest
import torch

from test_paged_abi import attn, lib, paged_desc  # noqa: F401


def test_scales_whose_power_of_two_is_out_of_range(lib):  # noqa: F811
    # scores are formed in powers of two: scale / ln 2 has to be finite as well
    for s in (2.4e38, 3.4e38):
        assert attn(lib, paged_desc(scale=s)) == -5, s
    n = ctypes.c_size_t()
    assert lib.kda_paged_attn_workspace_size(ctypes.byref(paged_desc(scale=2.4e38)), ctypes.byref(n)) == -5 and n.value == 0
    assert lib.kda_paged_attn_workspace_size(ctypes.byref(paged_desc(scale=2.3e38)), ctypes.byref(n)) == 0 and n.value > 0


def test_outputs_without_their_input_are_refused():
    from hybrid_linear_attention_chunk_gb300 import _lib
    t = torch.zeros(4, 2, 64)
    assert _lib._rows("k_out", None, None, torch.float32, -1) == (None, 0)
    with pytest.raises(ValueError, match="k_out"):
        _lib._rows("k_out", t, None, torch.float32, -1)
