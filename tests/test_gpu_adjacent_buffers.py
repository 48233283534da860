"""Buffers that lie against one another without overlapping, and the rotation in place of one
token's queries inside a fused row, are ordinary calls."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import Cache, cu, rope_table

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_with_results_against_its_inputs(dtype):
    """[rotated queries | fused rows | rotated queries], [lengths | new lengths] in one buffer each."""
    n, hq, hkv, d = 7, 6, 2, 64
    c = Cache([60, 5], hkv, d, 64, dtype, seed=1, cap=100)
    rope = rope_table(100, d)
    flat = torch.randn(n * (3 * hq + 2 * hkv) * d,
                       generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    size = n * hq * d
    before, after = flat[:size].view(n, hq, d), flat[-size:].view(n, hq, d)
    q, k, v = flat[size:-size].view(n, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    want = santa.santa_append_chunk(q, k, v, cu([3, 4]), c.k, c.v, c.reps, c.table, c.seq_lens, rope)
    both = torch.zeros(4, dtype=torch.int32, device="cuda")
    both[:2] = c.seq_lens
    for out in (before, after):
        got = santa.santa_append_chunk(q, k, v, cu([3, 4]), c.k, c.v, c.reps, c.table, both[:2], rope,
                                       seq_lens_next=both[2:], q_out=out)
        assert torch.equal(got, want) and both.tolist() == [60, 5, 63, 9]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_token_rotated_inside_its_fused_row(dtype):
    c = Cache([60], 2, 64, 64, dtype, seed=1, cap=100)
    rope = rope_table(100, 64)
    qkv = torch.randn(1, 10, 64, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    q, k, v = qkv.split([6, 2, 2], 1)
    args = (k, v, cu([1]), c.k, c.v, c.reps, c.table, c.seq_lens, rope)
    want = santa.santa_append_chunk(q, *args)
    santa.santa_append_chunk(q, *args, q_out=q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chunk_output_against_its_queries(dtype):
    c = Cache([200], 2, 64, 64, dtype, seed=1)
    flat = torch.randn(3, 50, 6, 64, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    want = santa.santa_chunk_attend(flat[1].clone(), c.k, c.v, c.table, c.seq_lens, cu([50]))
    for i in (0, 2):
        santa.santa_chunk_attend(flat[1], c.k, c.v, c.table, c.seq_lens, cu([50]), out=flat[i])
        assert torch.equal(flat[i], want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_overlapping_buffers_are_refused(dtype):
    c = Cache([200], 2, 64, 64, dtype, seed=1, cap=300)
    flat = torch.zeros(51, 6, 64, dtype=dtype, device="cuda")
    kv = torch.zeros(50, 2, 64, dtype=dtype, device="cuda")
    with pytest.raises(santa.SantaError):
        santa.santa_chunk_attend(flat[:50], c.k, c.v, c.table, c.seq_lens, cu([50]), out=flat[1:])
    with pytest.raises(santa.SantaError):
        santa.santa_append_chunk(flat[:50], kv, kv, cu([50]), c.k, c.v, c.reps, c.table,
                                 c.seq_lens, q_out=flat[1:])
