"""Non-finite values that only some rows of a chunk see: rows that see one hold it, the others keep
the bits of a clean cache.  Shapes where the last tile of a step's item sees further than the first."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import Cache, cu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("ctx,new,hq,hkv,d,T,token", [
    (95, 33, 4, 1, 128, 128, 110),     # 32 tokens per tile: the second tile holds one, at a step's end
    (95, 33, 8, 2, 64, 64, 127),       # the token itself, seen by the last row alone
    (127, 129, 1, 1, 128, 64, 200),    # one head per KV head: 128 tokens per tile
    (127, 129, 3, 3, 64, 128, 130),
    (2000, 256, 1, 1, 128, 128, 2010),  # one step per block: a run ends between the tiles' borders
    (2000, 256, 2, 2, 64, 64, 2040),
    (1900, 200, 2, 1, 128, 64, 1985),
    (100, 61, 8, 1, 128, 128, 120),
])
def test_value_seen_by_some_rows(ctx, new, hq, hkv, d, T, token, bad, dtype):
    c = Cache([ctx + new], hkv, d, T, dtype, seed=ctx + d)
    q = torch.randn(new, hq, d, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    args = (c.table, c.seq_lens, cu([new]))
    clean = santa.santa_chunk_attend(q, c.k, c.v, *args)
    assert clean.isfinite().all()
    h, col = hkv - 1, d - 3
    c.v[c.table[0, token // T].long(), h, token % T, col] = bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = santa.santa_chunk_attend(q, c.k, c.v, *args, device_status=status)
    assert int(status) == 0
    G, first = hq // hkv, max(0, token - ctx)
    got = out[first:, h * G:(h + 1) * G, col].clone()
    assert (got.isnan() if bad != bad else got == bad).all()
    # scores of a few units: no weight vanishes, so every row that sees the element holds it
    out[first:, h * G:(h + 1) * G, col] = clean[first:, h * G:(h + 1) * G, col]
    assert torch.equal(out, clean)
