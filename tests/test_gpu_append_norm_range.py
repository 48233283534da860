"""Norms of rows of every size that the sums of their squares allow in fp32."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import cu, rope_table
from test_gpu_append_norm import check, make, snapshot, target
from q8_cases import E4M3, I8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("kind", [None, I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,T,rope_dim,inter", [(128, 128, 128, False), (64, 64, 32, True), (128, 64, 0, False)])
@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_rows_of_every_size(kind, dtype, d, T, rope_dim, inter, eps):
    """Elements up to 2^3.9 times a power of two from 2^-54 to 2^55 for every (token, head): squares up to
    2^118, sums of 128 below 2^125, means above 2^-120."""
    lens, new, hq, hkv = [5, 0], [2 * T + 3, 40], 6, 2
    c, cache = target(lens, new, hkv, d, T, dtype, kind, seed=1)
    n = sum(new)
    q, k, v = make(2, n, hq, hkv, d, dtype, strided=False)
    for x, by in ((q, 7), (k, 5)):
        for h in range(x.shape[1]):
            e = (torch.arange(n, device="cuda") * by + 11 * h) % 110 - 54
            x[:, h] = (x[:, h].double().clamp(-15, 15) * torch.exp2(e.double())[:, None]).to(dtype)
    w = torch.linspace(0.5, 1.5, d).cuda()
    rope = rope_table(512, rope_dim) if rope_dim else None
    q_out = torch.zeros(n, hq, d, dtype=dtype, device="cuda")
    before = snapshot(c)
    santa.santa_append_norm(q, k, v, cu(new), cache, c.reps, c.table, c.seq_lens, rope, q_norm=w, k_norm=w,
                            eps=eps, q_out=q_out, interleaved=inter)
    # results are near 1 or, where eps = 1e-30 outweighs the row, above 2^-10: far from the rows' lower bound
    check(c, lens, new, q, k, v, rope, w, w, eps, inter, q_out, T, before)


def test_rows_of_zeros_without_eps_are_nan():
    """0 / 0, as the formula has it; other rows of the same warp are not concerned."""
    c, cache = target([0], [20], 1, 64, 64, F32, None, seed=1)
    q, k, v = make(2, 20, 2, 1, 64, F32, strided=False)
    q[3, 1], k[7] = 0.0, 0.0
    w = torch.ones(64, device="cuda")
    out = santa.santa_append_norm(q, k, v, cu([20]), cache, c.reps, c.table, c.seq_lens, q_norm=w, k_norm=w, eps=0.0)
    bad = torch.isnan(out).any(-1)
    assert bool(torch.isnan(out[3, 1]).all()) and int(bad.sum()) == 1
    stored = torch.isnan(c.k[int(c.table[0, 0]), 0, :20]).any(-1)
    assert stored.tolist() == [i == 7 for i in range(20)]
