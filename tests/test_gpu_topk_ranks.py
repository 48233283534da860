"""The order of teams without a finite score in santa_select_topk: -inf is a score and ranks below
every finite one; a NaN score and a page id out of range rank below that."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DEV_BAD_PAGE

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def ranked(scores, last):
    """Team indices from best to last: scores descending, then the teams of `last`, lower index
    first among equals."""
    return sorted(range(len(scores)),
                  key=lambda i: (i in last, 0.0 if i in last else -scores[i], i))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,finite", [(12, 3), (40, 0), (300, 100), (2000, 1)])
@pytest.mark.parametrize("pages", [False, True])
def test_minus_infinity_ranks_above_nan_and_bad_pages(n, finite, pages, dtype):
    d, T = 64, 64
    g = torch.Generator().manual_seed(n + finite)
    perm = torch.randperm(n, generator=g).tolist()
    last = set(perm[:n // 4]) | {0}
    rest = [i for i in perm if i not in last]
    # positive queries: an element of -inf makes the score of every head -inf, never NaN
    q = (torch.rand(1, 4, d, generator=g) + 0.5).to(dtype).cuda()
    reps = torch.randn(n, 1, d, generator=g)
    reps[rest[finite:], 0, 5] = -math.inf
    bad = [i for i in last if pages and i % 2 == 0]
    reps[[i for i in last if i not in bad], 0, 7] = math.nan
    reps = reps.cuda()
    table = torch.randperm(n, generator=g).int()
    pool = torch.zeros(n, 1, T, d, dtype=dtype, device="cuda")
    by_team = reps[:, 0].double()
    scores = (q[0].double() @ by_team.T).amax(0).tolist()
    placed = torch.empty_like(reps)
    placed[table.long().cuda()] = reps
    for i in bad:
        table[i] = [-1, n, 2 ** 31 - 1][i % 3]
    table = table[None].cuda()
    lens = torch.tensor([n * T], dtype=torch.int32, device="cuda")
    order = ranked(scores, last)
    for k in sorted({1, max(1, finite), finite + 1, len(rest), min(n, len(rest) + 1), n - 1}):
        bufs = santa.santa_select_topk(q, pool, pool, placed, table, lens, k)
        assert bufs.status() == (DEV_BAD_PAGE if bad else 0)
        assert bufs.sel_ids[0, 0].tolist() == sorted(order[:k])
