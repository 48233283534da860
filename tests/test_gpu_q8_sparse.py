"""The sampled and best-team steps over 8-bit caches: every sampler and mixture, capped scores, groups and
types; the choice is santa_sample's or santa_select_topk's, the output the attention of 64 bits over it."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from q8_cases import E4M3, I8, Q8
from test_gpu_q8_attend import check_listed, queries

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def filled(lens, hkv, d, T, kind, seed):
    """A cache whose representatives are the means of its keys."""
    c = Q8(lens, hkv, d, T, kind, seed=seed)
    for b, L in enumerate(lens):
        for i in range(-(-L // T)):
            c.reps[int(c.table[b, i])] = c.tokens("k", b, min(L, (i + 1) * T), i * T).mean(1).float()
    return c


def pools(c, dtype):
    """santa_sample and santa_select_topk take a 16- or 32-bit cache of the same shape; they do not read it."""
    shape = tuple(c.cache.k.shape)
    return torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("sampler,mix", [("iid_ht", 0.0), ("iid_ht", 0.3), ("systematic", 0.0),
                                         ("systematic", 0.1), ("iid_hh", 0.0), ("iid_hh", 0.5)])
@pytest.mark.parametrize("cap", [0.0, 4.0])
@pytest.mark.parametrize("lens,hq,hkv,d,T,M,dtype,kind", [
    ([3000, 200, 64], 8, 2, 128, 128, 6, BF16, I8), ([1500, 1, 700, 333], 7, 1, 64, 64, 12, F32, E4M3),
    ([9000], 28, 4, 128, 128, 31, BF16, E4M3),
])
def test_sampled_steps(lens, hq, hkv, d, T, M, dtype, kind, sampler, mix, cap):
    c = filled(lens, hkv, d, T, kind, seed=hq)
    q = queries(c, hq, dtype, seed=2)
    bufs = santa.santa_q8_decode(q, c.cache, c.reps, c.table, c.seq_lens, M, seed=77, softcap=cap,
                                 sampler=sampler, mix_alpha=mix)
    drawn = santa.santa_sample(q, *pools(c, dtype), c.reps, c.table, c.seq_lens, M, 77, sampler=sampler,
                               mix_alpha=mix)
    assert bufs.status() == 0 and drawn.status() == 0
    for f in ("draw_ids", "sel_ids", "sel_count", "pi"):
        assert torch.equal(getattr(bufs, f), getattr(drawn, f))
    check_listed(c, q, bufs.out, bufs.sel_ids, bufs.sel_count, bufs.pi, cap)


@pytest.mark.parametrize("cap", [0.0, 4.0])
@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("lens,hq,hkv,d,T,M,dtype", [
    ([3000, 200, 0, 64], 8, 2, 128, 128, 6, BF16), ([1500, 1, 700, 333], 7, 1, 64, 64, 12, F32),
    ([500, 90], 8, 1, 64, 64, 4096, BF16), ([20000], 15, 3, 128, 64, 1, F32),
])
def test_best_teams(lens, hq, hkv, d, T, M, dtype, kind, cap):
    c = filled(lens, hkv, d, T, kind, seed=hq)
    q = queries(c, hq, dtype, seed=2)
    bufs = santa.santa_q8_topk_decode(q, c.cache, c.reps, c.table, c.seq_lens, M, softcap=cap)
    best = santa.santa_select_topk(q, *pools(c, dtype), c.reps, c.table, c.seq_lens, M)
    for f in ("sel_ids", "sel_count", "pi"):
        assert torch.equal(getattr(bufs, f), getattr(best, f))
    check_listed(c, q, bufs.out, bufs.sel_ids, bufs.sel_count, bufs.pi, cap)
