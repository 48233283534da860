"""Pages before a window may have been given back: their table entries are out of range, and neither a dense
call nor a list that still names their teams reads them or complains."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from q8_cases import E4M3, I8, Q8
from test_gpu_q8_attend import check_dense, check_listed, listed, queries, status_word

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def evicted(c, window):
    """The table with every page wholly before the window out of range."""
    t = c.table.clone()
    for b, L in enumerate(c.lens):
        n = max(0, L - window) // c.T
        t[b, :n] = torch.tensor([-1, 2**30, c.reps.shape[0]], dtype=torch.int32)[torch.arange(n) % 3].cuda()
    return t


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("window", [1, 64, 100, 700])
@pytest.mark.parametrize("lens,hq,hkv,d,T,dtype", [([1000, 65, 64, 2500], 8, 2, 128, 64, BF16),
                                                   ([3000] * 40, 4, 1, 64, 128, F32)])
def test_dense(kind, window, lens, hq, hkv, d, T, dtype):
    c = Q8(lens, hkv, d, T, kind, seed=window)
    q, status = queries(c, hq, dtype), status_word()
    out = santa.santa_q8_dense_decode(q, c.cache, evicted(c, window), c.seq_lens, window=window,
                                      device_status=status)
    assert int(status) == 0
    check_dense(c, q, out, window=window)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("window", [1, 64, 100, 700])
@pytest.mark.parametrize("lens,hq,hkv,d,T,M,dtype", [([1000, 65, 64, 2500], 8, 2, 128, 64, 9, BF16),
                                                     ([3000] * 40, 4, 1, 64, 128, 24, F32)])
def test_listed(kind, window, lens, hq, hkv, d, T, M, dtype):
    c = Q8(lens, hkv, d, T, kind, seed=window)
    q, status = queries(c, hq, dtype), status_word()
    ids, count, pi = listed(c, M, seed=2, order="any")
    out = santa.santa_q8_attend(q, c.cache, evicted(c, window), c.seq_lens, ids, count, pi, window=window,
                                device_status=status)
    assert int(status) == 0
    check_listed(c, q, out, ids, count, pi, window=window)
