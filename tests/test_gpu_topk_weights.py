"""santa_topk_decode on bf16 caches: every bit of the weights enters the product with V (see
weight_pieces for the case and its bound), in both variants of the kernel."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from weight_pieces import BOUND, heads, result, weight

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("batch,hkv,G,d,T,teams", [
    (1, 1, 1, 64, 64, 1), (1, 4, 7, 128, 128, 9), (2, 2, 8, 64, 128, 40), (1, 8, 4, 128, 64, 33),
    (60, 8, 4, 128, 128, 2), (100, 4, 8, 64, 64, 3), (90, 8, 1, 128, 64, 4), (200, 3, 5, 64, 128, 2),
])
def test_every_bit_of_the_weights_counts(batch, hkv, G, d, T, teams):
    g = torch.Generator().manual_seed(batch + G)
    pages = batch * teams
    k = torch.zeros(pages, hkv, T, d)
    k[..., 0] = -8000.0
    v = torch.randn(pages, hkv, T, d, generator=g)
    # the group of 16 tokens that counts, and its four tokens, per unit
    for b in range(batch):
        for h in range(hkv):
            page = b * teams + int(torch.randint(teams, (1,), generator=g))
            at = 16 * int(torch.randint(T // 16, (1,), generator=g)) + torch.randperm(16, generator=g)[:4]
            k[page, h, at, 0] = torch.tensor([0.0, -1.0, -1.0, -1.0])
            v[page, h, at] = torch.tensor([0.0, 1.0, 1.0, 1.0])[:, None]
    all_b = heads(d)
    pick = all_b[torch.randint(len(all_b), (batch, hkv * G), generator=g)]
    q = torch.randn(batch, hkv * G, d, generator=g)
    q[..., 0] = pick.float()
    q, k, v = (x.to(BF16).cuda() for x in (q, k, v))
    table = torch.arange(pages, dtype=torch.int32).view(batch, teams).cuda()
    lens = torch.full((batch,), teams * T, dtype=torch.int32, device="cuda")
    reps = santa.santa_build_reps(k)
    bufs = santa.santa_topk_decode(q, k, v, reps, table, lens, teams)
    assert bufs.status() == 0 and (bufs.sel_count == teams).all()
    plan = santa.santa_decode_plan(q, k, table, teams, which="attend")
    assert plan["wide"] == (batch < 10)
    want = result(weight(pick, d))[..., None].cuda()
    err = ((bufs.out.double() - want).abs() / want).max().item()
    assert err <= BOUND, f"{err / BOUND:.3g} of the bound"
