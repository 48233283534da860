"""Numbers that a C field would hold as something else (a window of 33 bits, a cap below fp32's range)
are refused by the binding (CPU)."""
import math

import pytest
import torch

from sampled_sparse_decode_gb300 import binding
from sampled_sparse_decode_gb300.binding import SantaError
from test_cache_args import on
from test_q8_abi import call, cpu_cache

I32 = torch.int32


def sparse(**kw):
    base = dict(q=on(torch.zeros(2, 4, 64)), cache=cpu_cache(), reps=on(torch.zeros(4, 2, 64)),
                page_table=on(torch.zeros(2, 2, dtype=I32)), seq_lens=on(torch.zeros(2, dtype=I32)),
                num_teams=3, softcap=0.0, window=0, bufs=None, stream=None)
    return binding._q8_sparse("santa_q8_topk_decode", **dict(base, **kw))


@pytest.mark.parametrize("f", [call, sparse])
@pytest.mark.parametrize("window", [2**32 + 5, 2**31, -2**31 - 1, -2**32 + 7, 2**64, 5.5, 2.0**40, math.inf, math.nan, "5", None])
def test_windows_that_a_c_int_does_not_hold(f, window):
    with pytest.raises(SantaError, match="window"):
        f(window=window)


@pytest.mark.parametrize("f", [call, sparse])
@pytest.mark.parametrize("cap", [1e-50, -1e-50, 5e-324, 1e39, -1e300, "x", None])
def test_caps_that_fp32_does_not_hold(f, cap):
    with pytest.raises(SantaError, match="softcap"):
        f(softcap=cap)


@pytest.mark.parametrize("eps", [1e-50, 5e-324, 1e40, "x", None])
def test_eps_that_fp32_does_not_hold(eps):
    x = on(torch.zeros(3, 2, 64))
    with pytest.raises(SantaError, match="eps"):
        binding._append_norm(x, x, x, on(torch.zeros(2, dtype=I32)), cpu_cache(), on(torch.zeros(4, 2, 64)),
                             on(torch.zeros(1, 2, dtype=I32)), on(torch.zeros(1, dtype=I32)), None, None, None,
                             eps, None, None, False, None, None)


@pytest.mark.parametrize("x,want", [(0, 0.0), (0.0, 0.0), (-0.0, 0.0), (1e-6, 1e-6), (30, 30.0), (1e-40, 1e-40),
                                    (math.inf, math.inf)])
def test_what_fp32_holds_passes(x, want):
    assert binding._c_float(x, "x") == want


def test_what_an_int_holds_passes():
    for x in (0, 5, -1, 2**31 - 1, -2**31, torch.tensor(7), True, 12.0):
        assert binding._c_int(x, "x") == int(x)
    assert math.isnan(binding._c_float(math.nan, "x"))
