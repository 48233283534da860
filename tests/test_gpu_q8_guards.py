"""What the append and the sparse steps over 8-bit caches write stays inside their buffers: between guards, on
the first and last pages of a pool, and with bounds of chunks that are not in order."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DEV_BAD_SEQLEN, DecodeBuffers
from cache_cases import cu, rope_table
from q8_cases import E4M3, I8, Q8
from test_gpu_q8_streams import guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FILL = 0xab


class Guards:
    def __init__(self):
        self.raw = []

    def like(self, t, copy=True):
        g, raw = guarded(tuple(t.shape), t.dtype, FILL)
        if copy:
            g.view(torch.uint8).copy_(t.view(torch.uint8))
        self.raw.append(raw)
        return g

    def check(self):
        for raw in self.raw:
            assert bool((raw[:4096] == FILL).all()) and bool((raw[-4096:] == FILL).all())


def guard_cache(c, g):
    c.cache = santa.Q8Cache(*(g.like(t) for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale)))
    c.reps = g.like(c.reps)


def as_bytes(c):
    rows = [t.view(torch.uint8).view(*c.cache.k.shape[:3], -1).clone()
            for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale)]
    return rows + [c.reps.view(torch.uint8).clone()]


def changed_pages(before, after):
    return {p for a, b in zip(before, after) for p in range(a.shape[0]) if not torch.equal(a[p], b[p])}


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype,d,T", [(BF16, 128, 128), (BF16, 64, 64), (F32, 128, 64), (F32, 64, 128)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_between_guards(kind, dtype, d, T, norm):
    hkv, hq = 2, 6
    lens, new = [T - 1, 0], [2, T + 1]
    c = Q8(lens, hkv, d, T, kind, seed=1, spare=1, cap=2 * T)
    P = c.reps.shape[0]
    # tokens land on the pool's first and last pages
    c.table = torch.tensor([[1, P - 1], [0, 2]], dtype=torch.int32, device="cuda")
    g = Guards()
    guard_cache(c, g)
    gen = torch.Generator().manual_seed(3)
    n = sum(new)
    q, k, v = torch.randn(n, hq + 2 * hkv, d, generator=gen).to(dtype).cuda().split([hq, hkv, hkv], 1)
    q_out = g.like(torch.empty(n, hq, d, dtype=dtype, device="cuda"), copy=False)
    nxt = g.like(c.seq_lens, copy=False)
    w = torch.ones(d, device="cuda") if norm else None
    before = as_bytes(c)
    santa.santa_append_norm(q, k, v, cu(new), c.cache, c.reps, c.table, c.seq_lens, rope_table(512, d), q_norm=w,
                            k_norm=w, q_out=q_out, seq_lens_next=nxt)
    g.check()
    assert nxt.tolist() == [T + 1, T + 1]
    assert changed_pages(before, as_bytes(c)) == {1, P - 1, 0, 2}
    after = as_bytes(c)
    for a, b in zip(before[:4], after[:4]):              # one slot of a page at either end of a chunk
        assert torch.equal(a[1, :, :T - 1], b[1, :, :T - 1])
        assert torch.equal(a[P - 1, :, 1:], b[P - 1, :, 1:]) and torch.equal(a[2, :, 1:], b[2, :, 1:])
    for page in range(P):                                # no token: the other pages as they were
        if page not in (0, 1, 2, P - 1):
            assert all(torch.equal(a[page], b[page]) for a, b in zip(before, after))


BOUNDS = [
    [0, 9, 8, 12, 16], [-1, 4, 8, 12, 16], [5, 3, 8, 10, 16], [0, 4, 2**31 - 1, 8, 16], [16, 0, 8, 4, 16],
    [0, 0, -2**31, 3, 16], [3, 2, 1, 0, -1], [0, 17, 17, 17, 17], [2**31 - 1] * 5, [-2**31, 2**31 - 1, 0, 5, 9],
]


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("kind,dtype,d,T", [(E4M3, BF16, 128, 64), (I8, F32, 64, 128)])
def test_bounds_out_of_order(bounds, kind, dtype, d, T):
    """Only pages and query rows of sequences whose own bounds are valid may change."""
    hkv, hq, n = 2, 6, 16
    c = Q8([0, T - 3, 5, 0], hkv, d, T, kind, seed=2, cap=2 * T)
    g = Guards()
    guard_cache(c, g)
    gen = torch.Generator().manual_seed(3)
    q, k, v = torch.randn(n, hq + 2 * hkv, d, generator=gen).to(dtype).cuda().split([hq, hkv, hkv], 1)
    q_out = g.like(torch.empty(n, hq, d, dtype=dtype, device="cuda"), copy=False)
    fill = q_out.view(torch.uint8).clone()
    nxt = g.like(c.seq_lens, copy=False)
    untouched = nxt.clone()
    w = torch.ones(d, device="cuda")
    before, status = as_bytes(c), torch.zeros(1, dtype=torch.int32, device="cuda")
    santa.santa_append_norm(q, k, v, torch.tensor(bounds, dtype=torch.int32, device="cuda"), c.cache, c.reps,
                            c.table, c.seq_lens, rope_table(512, d), q_norm=w, k_norm=w, q_out=q_out,
                            seq_lens_next=nxt, device_status=status)
    assert int(status) & DEV_BAD_SEQLEN
    g.check()
    pages, rows = set(), set()
    for b, L in enumerate(c.lens):
        lo, hi = bounds[b], bounds[b + 1]
        if not 0 <= lo <= hi <= n:
            assert int(nxt[b]) == int(untouched[b])
            continue
        assert int(nxt[b]) in (int(untouched[b]), L + hi - lo)
        rows |= set(range(lo, hi))
        pages |= {int(c.table[b, i]) for i in range(L // T, -(-(L + hi - lo) // T)) if hi > lo}
    assert changed_pages(before, as_bytes(c)) <= pages
    got = q_out.view(torch.uint8)
    assert all(torch.equal(got[i], fill[i]) for i in range(n) if i not in rows)


@pytest.mark.parametrize("name", ["topk", "sampled"])
@pytest.mark.parametrize("dtype,d,M,lens", [(BF16, 128, 5, [900, 1, 300]), (F32, 64, 300, [700, 0, 64]),
                                            (BF16, 64, 1, [5000])])
def test_sparse_steps_between_guards(name, dtype, d, M, lens):
    hkv, hq, B = 2, 6, len(lens)
    c = Q8(lens, hkv, d, 64, I8, seed=3)
    gen = torch.Generator().manual_seed(1)
    c.reps += torch.randn(c.reps.shape, generator=gen).cuda()
    q = torch.randn(B, hq, d, generator=gen).to(dtype).cuda()
    g, i32 = Guards(), torch.int32
    shapes = [((B, hq, d), F32), ((B, hkv, M), i32), ((B, hkv, M), i32), ((B, hkv), i32), ((B, hkv, M), F32),
              ((B, hkv, c.table.shape[1]), F32),
              ((santa.santa_q8_workspace_bytes(B, hq, hkv, d, 64, c.table.shape[1]),), torch.uint8)]
    bufs = DecodeBuffers(*(g.like(torch.empty(s, dtype=t, device="cuda"), copy=False) for s, t in shapes),
                         device_status=g.like(torch.zeros(1, dtype=i32, device="cuda")))
    args = (q, c.cache, c.reps, c.table, c.seq_lens, M)
    if name == "topk":
        santa.santa_q8_topk_decode(*args, bufs=bufs)
        want = santa.santa_q8_topk_decode(*args)
    else:
        santa.santa_q8_decode(*args, seed=5, bufs=bufs)
        want = santa.santa_q8_decode(*args, seed=5)
    g.check()
    assert bufs.status() == want.status()
    for f in ("out", "sel_count"):
        assert torch.equal(getattr(bufs, f), getattr(want, f))
    for b in range(B):
        for h in range(hkv):
            m = int(bufs.sel_count[b, h])
            for f in ("sel_ids", "pi"):
                assert torch.equal(getattr(bufs, f)[b, h, :m], getattr(want, f)[b, h, :m])
