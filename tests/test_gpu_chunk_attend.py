"""santa_chunk_attend against a 64-bit reference: ragged chunks from one token to thousands,
groups of 1 to 8 heads, page borders, padding, unseen NaN and infinities, split tiles, bad
inputs seen on the device."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DEV_BAD_PAGE, DEV_BAD_SEQLEN
from cache_cases import Cache, attend64, cu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def run(c, q, cu_q, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    got = santa.santa_chunk_attend(q, c.k, c.v, c.table, c.seq_lens, cu_q, out=out,
                                   device_status=status, **kw)
    assert got is out
    return out, int(status)


def check_rows(c, q, out, b, first, n, rows=None):
    """Rows `rows` (default all) of sequence b's chunk against the reference."""
    rows = list(range(n)) if rows is None else rows
    L = c.lens[b]
    K, V = c.tokens(c.k, b, L), c.tokens(c.v, b, L)
    at = torch.tensor([first + i for i in rows], device="cuda")
    ref, mag, qk = attend64(q[at], K, V, [L - n + i + 1 for i in rows])
    # an fp32 score of d products and its scaling is off by (d + 2) 2^-24 of the sum of their
    # magnitudes, and a weight 2^(s - m) by that, by the rounding of the scaled difference and
    # by 2^-22 of the exponential; numerator and denominator each sum L weighted terms in fp32
    L_max = L
    rel = 2 * ((c.d + 8) * 2.0 ** -24 * qk + 2.0 ** -21) + 2 * L_max * 2.0 ** -24
    if q.dtype == BF16:
        half = torch.finfo(BF16).eps / 2
        tol = (half + rel) * mag + half * ref.abs()    # the weights' rounding, the output's
    else:
        tol = rel * mag + 2.0 ** -23 * ref.abs()
    err = (out[at].double() - ref).abs()
    assert (err <= tol).all(), f"sequence {b}: {(err / tol).max().item():.3g} of the tolerance"


CASES = [
    # ctx, new, hq, hkv, d, T, pad, lead
    ([0], [1], 1, 1, 64, 64, 0, 0),
    ([0], [1], 8, 1, 128, 128, 0, 0),
    ([100], [33], 28, 4, 128, 128, 0, 0),
    ([0, 1, 62, 64, 127], [1, 63, 2, 64, 129], 7, 1, 128, 64, 3, 0),
    ([500, 0, 9], [3, 0, 200], 6, 2, 64, 64, 0, 5),
    ([1000], [300], 5, 1, 128, 128, 0, 0),
    ([0], [257], 3, 3, 64, 128, 1, 0),
    ([37, 2000], [1, 1], 8, 2, 128, 128, 0, 0),
    ([3] * 50, [1 + i % 5 for i in range(50)], 4, 1, 64, 64, 0, 0),
    ([70, 0], [130, 515], 2, 1, 128, 64, 0, 0),
    ([0], [700], 4, 4, 128, 128, 0, 0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ctx,new,hq,hkv,d,T,pad,lead", CASES)
def test_matches_reference(ctx, new, hq, hkv, d, T, pad, lead, dtype):
    lens = [L + m for L, m in zip(ctx, new)]
    c = Cache(lens, hkv, d, T, dtype, seed=sum(new))
    g = torch.Generator().manual_seed(1)
    q = torch.randn(lead + sum(new) + pad, hq, d, generator=g).to(dtype).cuda()
    cu_q = cu(new, lead)
    out, status = run(c, q, cu_q)
    assert status == 0
    starts = cu_q.tolist()
    for b, m in enumerate(new):
        if m:
            check_rows(c, q, out, b, starts[b], m)
    assert (out[:lead] == 7).all() and (out[starts[-1]:] == 7).all(), "padding was written"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("L,n,hq,hkv,d", [(20000, 1, 8, 1, 128), (9001, 17, 7, 1, 128),
                                          (16384, 129, 4, 2, 64)])
def test_long_context_split_over_blocks(L, n, hq, hkv, d, dtype):
    """One short chunk over a long context: its keys are shared out over many blocks.  Peaked
    scores (queries four times larger) make the running maximum move."""
    c = Cache([L], hkv, d, 128, dtype, seed=L)
    q = (4 * torch.randn(n, hq, d, generator=torch.Generator().manual_seed(2))).to(dtype).cuda()
    out, status = run(c, q, cu([n]))
    assert status == 0
    check_rows(c, q, out, 0, 0, n, sorted({0, n // 2, n - 1}))
    again, _ = run(c, q, cu([n]))
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_rows_of_a_long_chunk(dtype):
    lens, new = [3000, 1500], [2900, 1500]
    c = Cache(lens, 2, 128, 128, dtype, seed=5)
    q = torch.randn(4400, 14, 128, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    out, status = run(c, q, cu(new))
    assert status == 0
    check_rows(c, q, out, 0, 0, 2900, [0, 1, 17, 18, 35, 36, 127, 128, 1000, 2048, 2898, 2899])
    check_rows(c, q, out, 1, 2900, 1500, [0, 63, 64, 700, 1499])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_has_no_influence(bad, dtype):
    """Later tokens of the chunk hold NaN or infinities in K and V: earlier rows are those of a
    clean cache (stale slots are NaN throughout)."""
    new, L = 90, 200
    c = Cache([L], 2, 64, 64, dtype, seed=8)
    q = torch.randn(new, 8, 64, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    clean, _ = run(c, q, cu([new]))
    for first in (199, 170, 120):
        page, slot = c.table[0, first // 64].long(), first % 64
        c.k[page, :, slot], c.v[page, :, slot] = bad, bad
        c.v[page, 0, slot] = 1.0                        # one head with a finite V
        out, status = run(c, q, cu([new]))
        assert status == 0
        rows = first - (L - new)
        assert torch.equal(out[:rows], clean[:rows])
        # rows that see it hold what the formula gives: NaN for NaN keys; +-inf * q has either
        # sign, so the softmax meets inf - inf in some head
        if bad != bad:
            assert out[rows:].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinite_value_reaches_the_rows_that_see_it(dtype):
    c = Cache([150], 1, 128, 128, dtype, seed=9)
    q = torch.randn(100, 2, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    clean, _ = run(c, q, cu([100]))
    page = c.table[0, 0].long()
    c.v[page, 0, 100, 5] = math.inf                     # token 100, one element
    out, _ = run(c, q, cu([100]))
    assert torch.equal(out[:50], clean[:50])
    assert (out[50:, :, 5] == math.inf).all()
    keep = [i for i in range(128) if i != 5]
    assert torch.equal(out[50:, :, keep], clean[50:, :, keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_whose_scores_are_all_minus_infinity(dtype):
    c = Cache([70], 1, 64, 64, dtype, seed=10)
    c.k[c.table[0, :2].long()] = -math.inf
    q = torch.ones(70, 2, 64, dtype=dtype, device="cuda")
    out, status = run(c, q, cu([70]))
    assert status == 0 and (out == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores_and_equal_scores(dtype):
    c = Cache([300], 1, 128, 128, dtype, seed=11)
    q = (50 * torch.randn(40, 4, 128, generator=torch.Generator().manual_seed(4))).to(dtype).cuda()
    out, _ = run(c, q, cu([40]))
    # scores of several hundred: the tolerance of check_rows grows with them
    check_rows(c, q, out, 0, 0, 40)
    q.zero_()
    out, _ = run(c, q, cu([40]))
    check_rows(c, q, out, 0, 0, 40)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_lengths_and_pages(dtype):
    lens, new = [40, 200, 65], [10, 30, 65]
    c = Cache(lens, 2, 64, 64, dtype, seed=12)
    q = torch.randn(105, 4, 64, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    cu_q = cu(new)
    clean, status = run(c, q, cu_q)
    assert status == 0
    for bad in (29, 64 * c.table.shape[1] + 1, -1):
        c.seq_lens[1] = bad
        out, status = run(c, q, cu_q)
        assert status == DEV_BAD_SEQLEN
        assert (out[10:40] == 7).all()
        assert torch.equal(out[:10], clean[:10]) and torch.equal(out[40:], clean[40:])
    c.seq_lens[1] = 200
    for bad in (-1, c.k.shape[0], 2**31 - 1):
        c.table[1, 2] = bad
        out, status = run(c, q, cu_q)
        assert status == DEV_BAD_PAGE
        assert torch.equal(out[:10], clean[:10]) and torch.equal(out[40:], clean[40:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bounds", [[0, 90, 40, 105], [-3, 10, 40, 105], [0, 10, 40, 106]])
def test_bad_cu_q(bounds, dtype):
    c = Cache([140, 200, 165], 2, 64, 64, dtype, seed=12)
    q = torch.randn(105, 4, 64, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    _, status = run(c, q, torch.tensor(bounds, dtype=torch.int32, device="cuda"))
    assert status & DEV_BAD_SEQLEN


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_streams_graphs_and_a_used_workspace(dtype):
    """The same bits from another stream, from a replayed graph and with a workspace full of
    NaN; two graphs with a workspace each replay side by side."""
    c = Cache([5000, 90], 2, 128, 128, dtype, seed=13)
    q = torch.randn(50, 8, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    cu_q = cu([40, 10])
    want, _ = run(c, q, cu_q)
    need = santa.santa_chunk_workspace_bytes(dtype, 2, 50, 8, 2, 128, 128, c.table.shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got, _ = run(c, q, cu_q, workspace=ws)
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = santa.santa_chunk_attend(q, c.k, c.v, c.table, c.seq_lens, cu_q, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    outs, graphs = [torch.zeros_like(q) for _ in range(2)], []
    for o in outs:
        h = santa.santa_chunk_attend_prepared(q, c.k, c.v, c.table, c.seq_lens, cu_q, out=o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            h.run()
        graphs.append((g, h))
    s2 = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_no_tokens():
    c = Cache([5], 1, 64, 64, BF16)
    out = santa.santa_chunk_attend(torch.empty(0, 2, 64, dtype=BF16, device="cuda"), c.k, c.v,
                                   c.table, c.seq_lens, cu([0]))
    assert out.shape == (0, 2, 64)


def test_single_token_agrees_with_dense_decode():
    """One new token per sequence is a dense decode step: both hold to the reference, so they
    agree within the sum of the tolerances (2e-3 for the dense step)."""
    lens = [1, 64, 777, 3000]
    c = Cache(lens, 2, 128, 128, BF16, seed=14, stale=0.0)
    q = torch.randn(4, 14, 128, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    out, _ = run(c, q, cu([1] * 4))
    table = torch.where(c.table == 2**30, torch.zeros_like(c.table), c.table)
    dense = santa.santa_dense_decode(q, c.k, c.v, table, c.seq_lens).out
    for b in range(4):
        check_rows(c, q, out, b, b, 1)
    half = torch.finfo(BF16).eps / 2
    vmax = c.v.abs().max().item()
    assert (out.double() - dense.double()).abs().max() <= 2e-3 + 2 * half * vmax


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_short_sequences(dtype):
    """300 sequences, a fifth of them without a new token, lengths from 0 to a few pages."""
    g = torch.Generator().manual_seed(31)
    new = [int(x) for x in torch.randint(0, 6, (300,), generator=g)]
    ctx = [int(x) for x in torch.randint(0, 200, (300,), generator=g)]
    new = [0 if i % 5 == 0 else m for i, m in enumerate(new)]
    lens = [L + m for L, m in zip(ctx, new)]
    c = Cache(lens, 2, 64, 64, dtype, seed=31)
    q = torch.randn(sum(new) + 2, 6, 64, generator=g).to(dtype).cuda()
    cu_q = cu(new)
    out, status = run(c, q, cu_q)
    assert status == 0
    starts = cu_q.tolist()
    for b in range(0, 300, 7):
        if new[b]:
            check_rows(c, q, out, b, starts[b], new[b])
    assert (out[starts[-1]:] == 7).all()
    # every row of every sequence was written
    assert not (out[:starts[-1]] == 7).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_output_at_any_16_byte_address(dtype):
    c = Cache([400], 2, 128, 64, dtype, seed=32)
    q = torch.randn(77, 8, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    want, _ = run(c, q, cu([77]))
    off = 16 // q.element_size()
    flat = torch.zeros(q.numel() + off, dtype=dtype, device="cuda")
    out = flat[off:].view_as(q)
    santa.santa_chunk_attend(q, c.k, c.v, c.table, c.seq_lens, cu([77]), out=out)
    assert torch.equal(out, want) and (flat[:off] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pool_larger_than_32_bit_offsets(dtype):
    """Pages behind element 2^31 of the pools."""
    hkv, T, d, L, new = 8, 128, 128, 300, 40
    pages = 2**31 // (hkv * T * d) + 8
    c = Cache([L], hkv, d, T, dtype, seed=33)
    q = torch.randn(new, 16, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    want, _ = run(c, q, cu([new]))
    k = torch.empty(pages, hkv, T, d, dtype=dtype, device="cuda")
    v = torch.empty(pages, hkv, T, d, dtype=dtype, device="cuda")
    n = c.k.shape[0]
    k[-n:], v[-n:] = c.k, c.v
    table = c.table + (pages - n)
    out = santa.santa_chunk_attend(q, k, v, table, c.seq_lens, cu([new]))
    assert torch.equal(out, want)
    # the single-token step and the append reach them too
    reps = torch.zeros(pages, hkv, d, device="cuda")
    reps[-n:] = santa.santa_build_reps(c.k, c.fill)
    a = santa.santa_topk_decode(q[:1], c.k, c.v, reps[-n:].contiguous(), c.table, c.seq_lens, 2)
    b = santa.santa_topk_decode(q[:1], k, v, reps, table, c.seq_lens, 2)
    assert torch.equal(a.out, b.out) and torch.equal(a.sel_ids, b.sel_ids)
    kn = torch.randn(50, hkv, d, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    for pool_k, pool_v, rep, tab in ((c.k, c.v, reps[-n:].clone(), c.table), (k, v, reps, table)):
        santa.santa_append_chunk(None, kn, kn, cu([50]), pool_k, pool_v, rep, tab, c.seq_lens)
        last = rep[-n:]
        it = torch.int16 if dtype == BF16 else torch.int32
        got = (pool_k[-n:].clone().view(it), pool_v[-n:].clone().view(it), last.clone())
        if pool_k is c.k:
            first = got
    assert all(torch.equal(x, y) for x, y in zip(first, got))


def test_keys_split_over_blocks_hold_nan_only_where_seen():
    """A long chunk whose items are split over blocks, with NaN in the last tokens: rows before
    them keep the bits of the clean cache, also in tiles that were joined."""
    c = Cache([6000], 1, 128, 128, BF16, seed=34)
    q = torch.randn(300, 4, 128, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    clean, _ = run(c, q, cu([300]))
    for first in (5999, 5900, 5760):
        page, slot = c.table[0, first // 128].long(), first % 128
        c.k[page, 0, slot], c.v[page, 0, slot] = math.nan, math.nan
        out, _ = run(c, q, cu([300]))
        rows = first - 5700
        assert torch.equal(out[:rows], clean[:rows])
        assert out[rows:].isnan().all()


def test_noted_values_outlast_the_items_behind_them():
    """One sequence in ten fills both tiles of an item and holds NaN behind its first tokens; the
    others have one token and use the first tile alone.  The second tile's rows are finished
    while later items are under way, and must still meet the NaN they see."""
    new = [20 if b % 10 == 0 else 1 for b in range(2000)]
    lens = [m + 3 for m in new]
    c = Cache(lens, 1, 64, 64, BF16, seed=35)
    q = torch.randn(sum(new), 8, 64, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    cu_q = cu(new)
    clean, _ = run(c, q, cu_q)
    pages = c.table[::10, 0].long()
    c.v[pages, :, 21] = math.nan                        # token 21 of 23: rows 18 and 19 see it
    starts = cu_q[:-1:10].long()
    for _ in range(5):
        out, status = run(c, q, cu_q)
        assert status == 0
        at = starts[:, None] + torch.arange(20, device="cuda")
        assert out[at[:, 18:]].isnan().all()
        rest = torch.ones(len(q), dtype=torch.bool, device="cuda")
        rest[at[:, 18:].flatten()] = False
        assert torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_replay_follows_lengths_and_bounds(dtype):
    """A captured call reads lengths, bounds and pages on the device: replays after they changed
    are calls with the new ones."""
    c = Cache([1500, 900, 300], 2, 64, 128, dtype, seed=36)
    q = torch.randn(200, 6, 64, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    cu_q, out = cu([200, 0, 0]), torch.zeros_like(q)
    h = santa.santa_chunk_attend_prepared(q, c.k, c.v, c.table, c.seq_lens, cu_q, out=out)
    h.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.run()
    for new in ([1, 198, 1], [0, 0, 200], [67, 66, 67], [200, 0, 0]):
        cu_q.copy_(cu(new))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want, _ = run(c, q, cu(new))
        assert torch.equal(out, want)
        first = 0
        for b, m in enumerate(new):
            if m:
                check_rows(c, q, out, b, first, m, sorted({0, m // 2, m - 1}))
            first += m


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_page_table_much_wider_than_the_lengths(dtype):
    c = Cache([130, 700], 2, 128, 64, dtype, seed=37)
    q = torch.randn(60, 4, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    wide = torch.full((2, 16384), -7, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    out, status = run(c, q, cu([20, 40]))
    assert status == 0
    check_rows(c, q, out, 0, 0, 20)
    check_rows(c, q, out, 1, 20, 40)
