"""A workspace that serves calls over 8-bit and over 16- and 32-bit caches in turn: the arrival counters that
the latter keep in it stay as they are."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DecodeBuffers
from cache_cases import Cache
from q8_cases import E4M3, I8, Q8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
LENS, HQ, HKV, D, T, M = [40000], 4, 1, 128, 128, 4


def both(dtype, kind):
    g = torch.Generator().manual_seed(1)
    c, c8 = Cache(LENS, HKV, D, T, dtype, seed=1), Q8(LENS, HKV, D, T, kind, seed=2)
    q = torch.randn(1, HQ, D, generator=g).to(dtype).cuda()
    c8.reps += torch.randn(c8.reps.shape, generator=g).cuda()
    return c, c8, q


def calls(c8, q, ws=None, bufs=None):
    """Every call over the 8-bit cache, on the given buffers."""
    santa.santa_q8_dense_decode(q, c8.cache, c8.table, c8.seq_lens, workspace=ws)
    ids = torch.zeros(1, HKV, M, dtype=torch.int32, device="cuda")
    santa.santa_q8_attend(q, c8.cache, c8.table, c8.seq_lens, ids, torch.ones_like(ids[:, :, 0]),
                          torch.ones(ids.shape, device="cuda"), workspace=ws)
    args = (q, c8.cache, c8.reps, c8.table, c8.seq_lens, M)
    bufs = santa.santa_q8_topk_decode(*args, bufs=bufs)
    santa.santa_q8_decode(*args, seed=3, bufs=bufs)
    return bufs


def dense(c, q, bufs):
    """The dense step on these buffers' workspace, which several clusters of a unit share."""
    plan = santa.santa_decode_plan(q, c.k, c.table, 1, "dense", bufs.workspace.numel())
    assert plan["clusters_per_unit"] > 1
    bufs.out.fill_(7.0)
    return santa.santa_dense_decode(q, c.k, c.v, c.table, c.seq_lens, bufs=bufs).out.clone()


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_workspace_for_both_kinds_of_caches(dtype, kind):
    c, c8, q = both(dtype, kind)
    own = DecodeBuffers.allocate(dtype, 1, HQ, HKV, D, T, c.table.shape[1], 1, dense=True)
    want = dense(c, q, own)
    bytes8 = santa.santa_q8_workspace_bytes(1, HQ, HKV, D, T, c8.table.shape[1])
    shared = DecodeBuffers.allocate(dtype, 1, HQ, HKV, D, T, c.table.shape[1], M, dense=True)
    shared.workspace = torch.zeros(max(bytes8, own.workspace.numel()), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        calls(c8, q, shared.workspace, shared)
        assert not shared.workspace[:256].any()          # 256-byte aligned: the counters are the first bytes
        got = dense(c, q, shared)
        # the clusters' shares depend on the workspace's size: equal up to the order of sums in fp32
        assert bool(((got - want).abs() <= 2.0**-15 * want.abs().amax()).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_buffers_that_an_8_bit_step_made(dtype):
    c, c8, q = both(dtype, I8)
    want = dense(c, q, DecodeBuffers.allocate(dtype, 1, HQ, HKV, D, T, c.table.shape[1], 1, dense=True))
    noise = [torch.full((1 << 22,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(8)]
    del noise                                            # memory that is not zero by chance
    bufs = calls(c8, q)
    for _ in range(2):
        got = dense(c, q, bufs)
        assert bool(((got - want).abs() <= 2.0**-15 * want.abs().amax()).all())
        calls(c8, q, bufs.workspace, bufs)
