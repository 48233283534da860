"""santa_select_topk and santa_topk_decode against 64-bit references: team counts around the
kernel's slices, ties, near ties below fp32, non-finite scores, bad inputs, and the whole run
from a prompt to sparse decode steps."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DEV_BAD_PAGE, DEV_BAD_SEQLEN
from cache_cases import Cache, attend64, best64, cu, rope_table, rotate64
from helpers import TOL_OUT

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAME = {F32: "f32", BF16: "bf16"}


def teams_only(n, hkv, d, T=64, B=1, seed=0, maxt=None):
    """q-independent inputs of a selection over n teams: reps, table, lengths (one-page pools
    would do for K and V; the selection does not read them)."""
    g = torch.Generator().manual_seed(seed)
    P = B * n + 1
    reps = torch.randn(P, hkv, d, generator=g).cuda()
    table = torch.full((B, maxt or n), 2**30, dtype=torch.int32)
    table[:, :n] = torch.randperm(P, generator=g)[:B * n].view(B, n).int()
    lens = torch.full((B,), n * T, dtype=torch.int32, device="cuda")
    pool = torch.zeros(P, hkv, T, d, dtype=BF16, device="cuda")
    return reps, table.cuda(), lens, pool


def select(q, pool, reps, table, lens, k):
    pool = pool if q.dtype == BF16 else pool.float()
    bufs = santa.santa_select_topk(q, pool, pool, reps, table, lens, k)
    return bufs, bufs.status()


def expect(q, reps, table, n, hkv, k, b=0):
    G = q.shape[1] // hkv
    pages = table[b, :n].long()
    return [best64(q[b, h * G:(h + 1) * G], reps[pages, h], k) for h in range(hkv)]


def check_sel(bufs, want, b, k):
    for h, w in enumerate(want):
        assert int(bufs.sel_count[b, h]) == len(w)
        assert bufs.sel_ids[b, h].tolist() == w + [-1] * (k - len(w))
        assert bufs.pi[b, h].tolist() == [1.0] * len(w) + [0.0] * (k - len(w))


@pytest.mark.parametrize("n,k,hq,hkv,d,dtype,maxt", [
    (1, 1, 1, 1, 64, BF16, None), (1, 5, 8, 1, 128, F32, 7), (2, 1, 4, 2, 64, F32, None),
    (31, 31, 7, 1, 128, BF16, None), (32, 31, 7, 1, 128, BF16, 100),
    (33, 8, 6, 2, 128, F32, None), (255, 64, 28, 4, 128, BF16, 256), (256, 31, 5, 1, 64, BF16, None),
    (257, 256, 3, 1, 128, F32, None), (1000, 100, 8, 1, 128, BF16, 1024),
    (5000, 4096, 2, 1, 64, F32, None), (16384, 700, 8, 1, 64, BF16, None),
])
def test_selection_matches_reference(n, k, hq, hkv, d, dtype, maxt):
    reps, table, lens, pool = teams_only(n, hkv, d, B=2, seed=n, maxt=maxt)
    q = torch.randn(2, hq, d, generator=torch.Generator().manual_seed(k)).to(dtype).cuda()
    bufs, status = select(q, pool, reps, table, lens, k)
    assert status == 0
    for b in range(2):
        check_sel(bufs, expect(q, reps, table, n, hkv, k, b), b, k)


@pytest.mark.parametrize("n", [40, 300, 2000])
def test_equal_scores_go_to_the_lowest_index(n):
    reps, table, lens, pool = teams_only(n, 1, 128, seed=3)
    q = torch.zeros(1, 4, 128, dtype=BF16, device="cuda")
    bufs, _ = select(q, pool, reps, table, lens, 17)
    check_sel(bufs, [list(range(17))], 0, 17)
    # groups of equal representatives across the border
    reps[:] = reps[torch.arange(reps.shape[0], device="cuda") % 7]
    q = torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    for k in (5, 17, 39):
        bufs, _ = select(q, pool, reps, table, lens, k)
        check_sel(bufs, expect(q, reps, table, n, 1, k), 0, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("step", [1, 3, 50])
def test_scores_closer_than_fp32_can_order(step, dtype):
    """Every representative is one vector with its last element some units in the last place
    higher or lower: fp32 sums of 128 products cannot order them, 64-bit ones can."""
    n, d = 500, 128
    reps, table, lens, pool = teams_only(n, 1, d, seed=4)
    g = torch.Generator().manual_seed(6)
    base = torch.randn(d, generator=g)
    base[-1] = 0.75
    ulps = torch.randint(-200, 200, (reps.shape[0],), generator=g) * step
    rows = base.repeat(reps.shape[0], 1)
    rows[:, -1] += ulps.float() * 2.0 ** -24
    reps[:, 0] = rows.cuda()
    q = torch.randn(1, 6, d, generator=g).to(dtype).cuda()
    for k in (1, 60, 499):
        bufs, _ = select(q, pool, reps, table, lens, k)
        check_sel(bufs, expect(q, reps, table, n, 1, k), 0, k)


@pytest.mark.parametrize("scale_q,scale_r", [(1e-25, 1e-18), (1e-30, 1e-30), (3e18, 3e18),
                                             (1e30, 1e30)])
def test_tiny_and_huge_scores(scale_q, scale_r):
    """Products in fp32's denormal range, below it and above its largest value."""
    reps, table, lens, pool = teams_only(300, 1, 64, seed=5)
    reps *= scale_r
    q = (torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(2)) * scale_q).cuda()
    bufs, _ = select(q, pool, reps, table, lens, 50)
    check_sel(bufs, expect(q, reps, table, 300, 1, 50), 0, 50)


def test_non_finite_representatives():
    reps, table, lens, pool = teams_only(100, 1, 64, seed=6)
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    reps[table[0, 10].long()] = math.nan
    reps[table[0, 20].long(), 0, 3] = math.inf
    reps[table[0, 30].long()] = -math.inf              # inf - inf: NaN in every head
    for k in (1, 50, 98, 99):
        bufs, status = select(q, pool, reps, table, lens, k)
        assert status == 0
        check_sel(bufs, expect(q, reps, table, 100, 1, k), 0, k)


def test_bad_lengths_and_pages():
    reps, table, lens, pool = teams_only(60, 1, 64, B=3, seed=7)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    clean, _ = select(q, pool, reps, table, lens, 20)
    for bad in (0, -4, 60 * 64 + 1):
        lens[1] = bad
        bufs, status = select(q, pool, reps, table, lens, 20)
        assert status == DEV_BAD_SEQLEN and int(bufs.sel_count[1, 0]) == 0
        for b in (0, 2):
            assert torch.equal(bufs.sel_ids[b], clean.sel_ids[b])
    lens[1] = 60 * 64
    best = int(clean.sel_ids[1, 0, 7])
    for bad in (-1, reps.shape[0]):
        table[1, best] = bad
        bufs, status = select(q, pool, reps, table, lens, 20)
        assert status == DEV_BAD_PAGE and best not in bufs.sel_ids[1, 0].tolist()


@pytest.mark.parametrize("lens,hq,hkv,d,T,dtype,k", [
    ([1], 1, 1, 64, 64, BF16, 1), ([700, 64, 65], 8, 2, 64, 64, F32, 4),
    ([5000, 129, 3], 28, 4, 128, 128, BF16, 9), ([2000] * 3, 6, 1, 128, 64, BF16, 31),
    ([4096, 100], 3, 3, 128, 128, F32, 64),
])
def test_topk_decode_matches_reference(lens, hq, hkv, d, T, dtype, k):
    c = Cache(lens, hkv, d, T, dtype, seed=len(lens) + k)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(len(lens), hq, d, generator=g).to(dtype).cuda()
    h = santa.santa_topk_decode_prepared(q, c.k, c.v, c.reps, c.table, c.seq_lens, k)
    bufs = h.run()
    assert bufs.status() == 0
    check_topk(c, q, bufs, k)
    other = santa.santa_topk_decode(q, c.k, c.v, c.reps, c.table, c.seq_lens, k)
    assert torch.equal(other.out, bufs.out) and torch.equal(other.sel_ids, bufs.sel_ids)


def check_topk(c, q, bufs, k):
    G = q.shape[1] // c.hkv
    for b, L in enumerate(c.lens):
        n = -(-L // c.T)
        want = expect(q, c.reps, c.table, n, c.hkv, k, b)
        check_sel(bufs, want, b, k)
        K, V = c.tokens(c.k, b, L), c.tokens(c.v, b, L)
        for h, w in enumerate(want):
            tok = torch.cat([torch.arange(i * c.T, min(L, (i + 1) * c.T)) for i in w]).cuda()
            ref, _, _ = attend64(q[b:b + 1, h * G:(h + 1) * G], K[h:h + 1, tok],
                                 V[h:h + 1, tok], [len(tok)])
            err = (bufs.out[b, h * G:(h + 1) * G].double() - ref[0]).abs().max()
            assert err <= TOL_OUT[NAME[c.dtype]]


def test_graph_replay_follows_new_queries():
    c = Cache([3000, 500], 2, 128, 128, BF16, seed=20)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    q = torch.randn(2, 8, 128).to(BF16).cuda()
    h = santa.santa_topk_decode_prepared(q, c.k, c.v, c.reps, c.table, c.seq_lens, 5)
    h.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.run()
    for seed in range(3):
        q.copy_(torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(seed)).to(BF16))
        g.replay()
        torch.cuda.synchronize()
        check_topk(c, q, h.run(), 5)
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_then_sparse_decode(dtype):
    """The operators together: two prompts appended in two chunks with attention after each,
    then decode steps (append one token, top-k attention), all against a cache kept in 64-bit
    from the stored values."""
    hq, hkv, d, T, k = 6, 2, 64, 64, 3
    c = Cache([0, 0], hkv, d, T, dtype, seed=21, cap=500)
    rope = rope_table(500, d)
    lens = c.seq_lens
    g = torch.Generator().manual_seed(9)
    half = torch.finfo(dtype).eps / 2
    for new in ([200, 37], [1, 150], [1, 1], [1, 1], [1, 1]):
        qkv = torch.randn(sum(new), hq + 2 * hkv, d, generator=g).to(dtype).cuda()
        q, kn, vn = qkv.split([hq, hkv, hkv], 1)
        nxt = torch.zeros_like(lens)
        qr = santa.santa_append_chunk(q, kn, vn, cu(new), c.k, c.v, c.reps, c.table, lens, rope,
                                      seq_lens_next=nxt)
        first = 0
        for b, m in enumerate(new):
            ref, mag = rotate64(q[first:first + m], rope[c.lens[b]:c.lens[b] + m], False)
            err = (qr[first:first + m].double() - ref).abs()
            assert (err <= half * ref.abs() + 2.01 * 2.0 ** -24 * mag * (1 + half)).all()
            c.lens[b] += m
            first += m
        lens = nxt
        assert lens.tolist() == c.lens
        c.seq_lens = lens
        if max(new) > 1:
            out = santa.santa_chunk_attend(qr, c.k, c.v, c.table, lens, cu(new))
            first = 0
            for b, m in enumerate(new):
                L = c.lens[b]
                K, V = c.tokens(c.k, b, L), c.tokens(c.v, b, L)
                ref, mag, qk = attend64(qr[first:first + m], K, V,
                                        [L - m + i + 1 for i in range(m)])
                rel = 2 * ((d + 8) * 2.0 ** -24 * qk + 2.0 ** -21) + 2 * L * 2.0 ** -24
                tol = (rel + (half if dtype == BF16 else 0)) * mag + max(half, 2.0 ** -23) * ref.abs()
                assert ((out[first:first + m].double() - ref).abs() <= tol).all()
                first += m
        else:
            check_topk(c, qr, santa.santa_topk_decode(qr, c.k, c.v, c.reps, c.table, lens, k), k)
            # the sampled step reads the same cache and representatives
            sampled = santa.santa_decode(qr, c.k, c.v, c.reps, c.table, lens, 4096, 1)
            assert sampled.status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chunk_tokens_as_rows_of_the_batch(dtype):
    """Several query tokens of one sequence, as rows with the same page-table row and growing
    lengths: each row is the step of its own length."""
    c = Cache([1000], 2, 64, 64, dtype, seed=40)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    rows = 6
    q = torch.randn(rows, 8, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    lens = torch.tensor([995 + i for i in range(rows)], dtype=torch.int32, device="cuda")
    table = c.table.expand(rows, -1).contiguous()
    got = santa.santa_topk_decode(q, c.k, c.v, c.reps, table, lens, 5)
    assert got.status() == 0
    for i in range(rows):
        c.lens = [995 + i]
        c.seq_lens = lens[i:i + 1].clone()
        one = santa.santa_topk_decode(q[i:i + 1], c.k, c.v, c.reps, c.table, c.seq_lens, 5)
        check_topk(c, q[i:i + 1], one, 5)
        assert torch.equal(got.sel_ids[i], one.sel_ids[0])
        assert (got.out[i] - one.out[0]).abs().max() <= TOL_OUT[NAME[dtype]]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_length_gives_zeros(dtype):
    c = Cache([300, 200], 1, 64, 64, dtype, seed=41, stale=0.0)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    c.seq_lens[0] = 64 * c.table.shape[1] + 1
    table = torch.where(c.table == 2**30, torch.zeros_like(c.table), c.table)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    bufs = santa.santa_topk_decode(q, c.k, c.v, c.reps, table, c.seq_lens, 3)
    assert bufs.status() == DEV_BAD_SEQLEN
    assert (bufs.out[0] == 0).all() and int(bufs.sel_count[0, 0]) == 0
    assert bufs.sel_count[1, 0] == 3 and not (bufs.out[1] == 0).all()


def test_side_stream_and_two_steps_at_once():
    """Two prepared steps on two streams, each with its own buffers."""
    c = Cache([2000, 300], 2, 128, 128, BF16, seed=42)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    qs = [torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(i)).to(BF16).cuda()
          for i in range(2)]
    hs = [santa.santa_topk_decode_prepared(q, c.k, c.v, c.reps, c.table, c.seq_lens, 4) for q in qs]
    want = []
    for h in hs:
        b = h.run()
        torch.cuda.synchronize()
        want.append((b.out.clone(), b.sel_ids.clone()))
    streams = [torch.cuda.Stream() for _ in hs]
    for _ in range(20):
        for h, s in zip(hs, streams):
            h.run(stream=s)
    torch.cuda.synchronize()
    for h, (out, ids) in zip(hs, want):
        assert torch.equal(h.run().out, out) and torch.equal(h.run().sel_ids, ids)
