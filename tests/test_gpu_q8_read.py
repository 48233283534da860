"""santa_q8_read: the values that codes and scales stand for, bit for bit, in the slots that the call
names and in no other."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DEV_BAD_PAGE, DEV_BAD_SEQLEN
from q8_cases import E4M3, I8, Q8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def destination(c, dtype, seed=1, spare=3):
    P = int((c.table < 2**30).sum()) + spare
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).int().cuda()
    table = torch.full_like(c.table, 2**30)
    table[c.table < 2**30] = perm[:P - spare]
    k = torch.full((P, c.hkv, c.T, c.d), 7.0, dtype=dtype, device="cuda")
    return k, k.clone(), table


def check(c, lens, first, k, v, table):
    for which, out in (("k", k), ("v", v)):
        want = torch.full_like(out, 7.0)
        codes, scale = getattr(c.cache, which), getattr(c.cache, which + "_scale")
        for b, (L, f) in enumerate(zip(lens, first)):
            for t in range(f, L):
                src, dst, slot = int(c.table[b, t // c.T]), int(table[b, t // c.T]), t % c.T
                x = codes[src, :, slot].float() * scale[src, :, slot, None]
                want[dst, :, slot] = x.to(out.dtype)
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,first,hkv,d,T", [
    ([1], [0], 1, 64, 64), ([130, 0, 64], [0, 0, 63], 2, 128, 64), ([300, 7], [129, 7], 3, 64, 128),
    ([128, 129, 127], [128, 128, 1], 1, 128, 128),
])
def test_values(lens, first, hkv, d, T, dtype, kind):
    c = Q8(lens, hkv, d, T, kind, seed=len(lens))
    k, v, table = destination(c, dtype)
    f = torch.tensor(first, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = santa.santa_q8_read(c.cache, c.table, c.seq_lens, k, v, table,
                            first=f if any(first) else None, device_status=status)
    assert r[0] is k and r[1] is v and int(status) == 0
    check(c, lens, first, k, v, table)


def test_every_code():
    """All 256 bytes under scales of every size."""
    for kind in (I8, E4M3):
        c = Q8([64], 4, 64, 64, kind)
        c.cache.k.view(torch.uint8)[:] = torch.arange(256, dtype=torch.uint8, device="cuda").view(4, 64)[:, None]
        s = torch.exp2(torch.linspace(-97, 120, 64)).cuda()
        c.cache.k_scale[:] = s * 1.2345
        for dtype in (F32, BF16):
            k, v, table = destination(c, dtype)
            santa.santa_q8_read(c.cache, c.table, c.seq_lens, k, v, table)
            p, o = int(c.table[0, 0]), int(table[0, 0])
            want = (c.cache.k[p].float() * c.cache.k_scale[p][..., None]).to(dtype)
            assert torch.equal(k[o].nan_to_num(nan=3.0), want.nan_to_num(nan=3.0))
            assert torch.equal(torch.isnan(k[o]), torch.isnan(want))


def test_bad_lengths_and_pages_are_skipped():
    lens, first = [70, 70, 70, 70, 70], [0, 0, 0, 0, 0]
    c = Q8(lens, 2, 64, 64, I8, seed=2)
    k, v, table = destination(c, F32)
    f = torch.tensor([0, 71, -1, 0, 0], dtype=torch.int32, device="cuda")
    c.seq_lens[3] = 129
    c.table[4, 1] = c.reps.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    santa.santa_q8_read(c.cache, c.table, c.seq_lens, k, v, table, first=f, device_status=status)
    assert int(status) == DEV_BAD_SEQLEN | DEV_BAD_PAGE
    check(c, [70, 0, 0, 0, 64], first, k, v, table)
    table[0, 0] = -1
    k[:], v[:] = 7.0, 7.0
    status.zero_()
    santa.santa_q8_read(c.cache, c.table, c.seq_lens, k, v, table, first=f, device_status=status)
    assert int(status) == DEV_BAD_SEQLEN | DEV_BAD_PAGE
    check(c, [70, 0, 0, 0, 64], [64, 0, 0, 0, 0], k, v, table)


def test_far_pages():
    """Codes and values behind element 2^31 of their pools."""
    P, hkv, T, d = 16500, 8, 128, 128
    cache = santa.Q8Cache.allocate(P, hkv, T, d, E4M3)
    assert cache.k.numel() > 2**31
    g = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randint(0, 120, (hkv, T, d), generator=g, device="cuda").to(torch.uint8)
    cache.k.view(torch.uint8)[P - 1], cache.v.view(torch.uint8)[P - 1] = last, last.flip(0)
    cache.k_scale[P - 1], cache.v_scale[P - 1] = 0.5, 2.0
    k = torch.zeros(P, hkv, T, d, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[P - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    santa.santa_q8_read(cache, table, lens, k, v, table)
    assert torch.equal(k[P - 1, :, :100].float(), cache.k[P - 1, :, :100].float() * 0.5)
    assert torch.equal(v[P - 1, :, :100].float(), cache.v[P - 1, :, :100].float() * 2.0)
    assert not k[P - 1, :, 100:].any() and not k[:P - 1].any()


@pytest.mark.parametrize("first", [[0] * 40, [70, 0, 511] + [1] * 37])
def test_wide_tables(first):
    """More (page, head) pairs in the tables than the launch has blocks."""
    lens = [900, 1, 512] + [65] * 37
    c = Q8(lens, 8, 64, 64, I8, seed=3)
    wide = torch.full((40, 300), 2**30, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    k, v, table = destination(c, BF16)
    f = torch.tensor(first, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    santa.santa_q8_read(c.cache, c.table, c.seq_lens, k, v, table, first=f, device_status=status)
    assert int(status) == 0
    check(c, lens, first, k, v, table)
