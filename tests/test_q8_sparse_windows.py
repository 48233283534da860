"""The best- and sampled-team steps over an 8-bit cache take no window: their teams are chosen from the whole
sequence, and those of a window may not be among them (CPU)."""
import ctypes

import pytest
import torch

from sampled_sparse_decode_gb300 import binding
from sampled_sparse_decode_gb300.binding import SantaError
from test_cache_args import on
from test_q8_abi import cache_args, cpu_cache, lib, step_args  # noqa: F401

INVALID, UNSUPPORTED = 1, 2
I32 = torch.int32


@pytest.mark.parametrize("f", ["santa_q8_topk_decode", "santa_q8_decode"])
@pytest.mark.parametrize("window,expect", [(1, UNSUPPORTED), (4096, UNSUPPORTED), (2**31 - 1, UNSUPPORTED),
                                           (-1, INVALID)])
def test_entry_points_refuse_a_window(lib, f, window, expect):  # noqa: F811
    a, c = step_args(), cache_args(window=window)
    assert getattr(lib, f)(ctypes.addressof(a), ctypes.addressof(c), None) == expect


@pytest.mark.parametrize("name", ["santa_q8_topk_decode", "santa_q8_decode"])
def test_binding_refuses_a_window(name):
    with pytest.raises(SantaError, match="window"):
        binding._q8_sparse(name, q=on(torch.zeros(2, 4, 64)), cache=cpu_cache(), reps=on(torch.zeros(4, 2, 64)),
                           page_table=on(torch.zeros(2, 2, dtype=I32)),
                           seq_lens=on(torch.zeros(2, dtype=I32)), num_teams=3, softcap=0.0, window=64,
                           bufs=None, stream=None)
