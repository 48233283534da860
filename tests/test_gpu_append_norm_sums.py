"""Representatives of normed keys are the means of the stored keys bit for bit: for every rotation, and
however the tokens were divided among calls."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import Cache, cu, rope_table
from test_gpu_append_norm import make

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

ROTATIONS = [(0, False), (64, False), (64, True), (16, True), (128, False)]


def append(sizes, lens, dtype, d, T, rope_dim, interleaved, total):
    c = Cache(lens, 2, d, T, dtype, seed=2, cap=max(lens) + total)
    q, k, v = make(3, total, 4, 2, d, dtype)
    w = torch.linspace(0.4, 1.7, d).cuda()
    rope = rope_table(1024, rope_dim) if rope_dim else None
    at, now = 0, c.seq_lens
    for m in sizes:
        nxt, sl = torch.empty_like(now), slice(at, at + m)
        santa.santa_append_norm(q[sl], k[sl], v[sl], cu([m]), (c.k, c.v), c.reps, c.table, now, rope,
                                q_norm=w, k_norm=w, seq_lens_next=nxt, interleaved=interleaved)
        at, now = at + m, nxt
    return c


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,T", [(64, 64), (128, 128), (128, 64), (64, 128)])
@pytest.mark.parametrize("rope_dim,interleaved", ROTATIONS)
def test_means_of_normed_keys_are_build_reps(dtype, d, T, rope_dim, interleaved):
    if rope_dim > d:
        rope_dim = d
    start, total = 37, 2 * T + 29
    one = append([total], [start], dtype, d, T, rope_dim, interleaved, total)
    fill = torch.zeros(one.k.shape[0], dtype=torch.int32, device="cuda")
    for i in range(-(-(start + total) // T)):
        fill[one.table[0, i]] = min(T, start + total - i * T)
    want = santa.santa_build_reps(one.k, fill)
    for p in (int(one.table[0, i]) for i in range(-(-(start + total) // T))):
        assert torch.equal(one.reps[p], want[p])
    many = append([1, 50, 2, total - 53], [start], dtype, d, T, rope_dim, interleaved, total)
    assert torch.equal(many.reps, one.reps)
    for a, b in ((many.k, one.k), (many.v, one.v)):
        assert torch.equal(a.nan_to_num(nan=5.0), b.nan_to_num(nan=5.0))
