"""Launches that follow one another without a pause and hand data on in memory that earlier launches
used too: partial results in one workspace, representatives and page tables rewritten in between."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import Cache, cu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_partial_results_of_calls_that_share_a_workspace(d, dtype):
    """Split tiles of two inputs, alternating in one workspace on one stream."""
    c = Cache([9000, 40], 2, d, 128, dtype, seed=d)
    g = torch.Generator().manual_seed(4)
    cu_q = cu([5, 3])
    qs = [torch.randn(8, 8, d, generator=g).to(dtype).cuda() for _ in range(2)]
    need = santa.santa_chunk_workspace_bytes(dtype, 2, 8, 8, 2, d, 128, c.table.shape[1])
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    outs = [[torch.zeros_like(q) for _ in range(40)] for q in qs]
    want = [santa.santa_chunk_attend(q, c.k, c.v, c.table, c.seq_lens, cu_q) for q in qs]
    torch.cuda.synchronize()
    handles = [[santa.santa_chunk_attend_prepared(q, c.k, c.v, c.table, c.seq_lens, cu_q, out=o,
                                                  workspace=ws) for o in row]
               for q, row in zip(qs, outs)]
    for a, b in zip(*handles):
        a.run()
        b.run()
    torch.cuda.synchronize()
    for row, w in zip(outs, want):
        assert all(torch.equal(o, w) for o in row)


@pytest.mark.parametrize("d", [64, 128])
def test_selection_behind_the_representatives_it_reads(d):
    """Representatives rebuilt from another cache directly before every selection."""
    g = torch.Generator().manual_seed(d)
    n, hkv, T, k = 500, 2, 64, 20
    pools = [torch.randn(n, hkv, T, d, generator=g).to(BF16).cuda() for _ in range(2)]
    q = torch.randn(1, 8, d, generator=g).to(BF16).cuda()
    table = torch.randperm(n, generator=g).int()[None].cuda()
    lens = torch.tensor([n * T], dtype=torch.int32, device="cuda")
    reps = torch.zeros(n, hkv, d, device="cuda")

    def step(i):
        santa.santa_build_reps(pools[i], None, reps)
        return santa.santa_select_topk(q, pools[i], pools[i], reps, table, lens, k)

    want = []
    for i in range(2):
        want.append(step(i).sel_ids.clone())
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    got = [step(j % 2).sel_ids for j in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(s, want[j % 2]) for j, s in enumerate(got))


def test_selection_behind_the_append_that_moves_its_page():
    """Appends of one token and selections in turn, on representatives that the append refreshes."""
    c = Cache([100, 640], 2, 64, 64, BF16, seed=5, cap=800)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(2, 4, 64, generator=g).to(BF16).cuda()
    kv = [(8 * torch.randn(2, 2, 64, generator=g)).to(BF16).cuda() for _ in range(40)]

    def steps(pause):
        k, v, reps = c.k.clone(), c.v.clone(), c.reps.clone()
        lens, sets = c.seq_lens, []
        for x in kv:
            nxt = torch.empty_like(lens)
            santa.santa_append_chunk(None, x, x, cu([1, 1]), k, v, reps, c.table, lens,
                                     seq_lens_next=nxt)
            if pause:
                torch.cuda.synchronize()
            sets.append(santa.santa_select_topk(q, k, v, reps, c.table, nxt, 2).sel_ids)
            if pause:
                torch.cuda.synchronize()
            lens = nxt
        return torch.stack(sets)

    want = steps(True)
    assert torch.equal(steps(False), want)
