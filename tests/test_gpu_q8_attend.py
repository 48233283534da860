"""Attention of one new token over 8-bit caches against 64-bit references: lengths around tiles, pages
and splits, groups of 1 to 8, windows, capped scores, listed teams with weights, what is not seen,
non-finite rows, bad inputs, far pages, graphs, and the run from a prompt to sparse steps."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DEV_BAD_PAGE, DEV_BAD_SEL, DEV_BAD_SEQLEN
from cache_cases import cu, rope_table
from q8_cases import E4M3, I8, Q8, attend64, close, values64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def queries(c, hq, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(len(c.lens), hq, c.d, generator=g)).to(dtype).cuda()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def check_dense(c, q, out, cap=0.0, window=0):
    for b, L in enumerate(c.lens):
        lo = max(0, L - window) if window else 0
        want, tol = attend64(q[b], c.tokens("k", b, L, lo), c.tokens("v", b, L, lo), cap=cap)
        close(out[b], want, tol)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,hq,hkv,d,T", [
    ([1], 1, 1, 64, 64), ([0, 1, 2, 31, 32, 33], 2, 2, 128, 64), ([63, 64, 65, 127, 128, 129], 8, 1, 128, 128),
    ([500, 0, 7], 6, 2, 64, 128), ([1000, 257, 3, 64], 28, 4, 128, 128), ([3001], 7, 1, 128, 64),
    ([90] * 40, 12, 4, 64, 64), ([20000, 5, 9000], 5, 1, 128, 128), ([4097, 8191], 15, 3, 64, 64),
])
def test_dense_matches_reference(lens, hq, hkv, d, T, dtype, kind):
    c = Q8(lens, hkv, d, T, kind, seed=hq)
    q, status = queries(c, hq, dtype), status_word()
    out = torch.full(q.shape, 9.0, device="cuda")
    r = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, out=out, device_status=status)
    assert r is out and int(status) == 0
    check_dense(c, q, out)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weights_and_queries_in_full(dtype, kind):
    """Two tokens of opposite values and nearly equal scores: an error of a weight shows whole, and
    the bound is far below what one 16-bit piece of a weight or of an fp32 query would give."""
    c = Q8([2] * 64, 1, 64, 64, kind, seed=3, size=0.5)
    for b in range(64):
        p = int(c.table[b, 0])
        c.cache.v.view(torch.uint8)[p, 0, 1] = c.cache.v.view(torch.uint8)[p, 0, 0]
        c.cache.v_scale[p, 0, 1] = -c.cache.v_scale[p, 0, 0]
    q = queries(c, 4, dtype, seed=1, size=0.5)
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    check_dense(c, q, out)
    want = torch.stack([attend64(q[b], c.tokens("k", b, 2), c.tokens("v", b, 2))[0] for b in range(64)])
    # root mean square: weights to 2^-21, scores to a few 2^-22
    assert float((out.double() - want).norm() / want.norm()) < 2.0**-18


@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("window", [1, 31, 32, 64, 100, 1000])
@pytest.mark.parametrize("dtype,d,T", [(BF16, 128, 128), (F32, 64, 64)])
def test_window_and_cap(dtype, d, T, window, cap):
    c = Q8([1, 30, 64, 65, 700, 1001, 2500], 2, d, T, I8, seed=window)
    # what lies before the window is stale
    for b, L in enumerate(c.lens):
        for t in range(max(0, L - window)):
            p = int(c.table[b, t // T])
            c.cache.k_scale[p, :, t % T] = math.nan
            c.cache.v_scale[p, :, t % T] = math.inf
    q = queries(c, 8, dtype, size=2.0)
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, softcap=cap, window=window)
    check_dense(c, q, out, cap, window)


def listed(c, M, seed, order="ascending"):
    """Random distinct teams of every unit with weights; ids padded with -1."""
    g = torch.Generator().manual_seed(seed)
    B = len(c.lens)
    ids = torch.full((B, c.hkv, M), -1, dtype=torch.int32)
    count, pi = torch.zeros(B, c.hkv, dtype=torch.int32), torch.zeros(B, c.hkv, M)
    for b, L in enumerate(c.lens):
        n = -(-L // c.T)
        for h in range(c.hkv):
            k = min(n, M) if h == 0 else int(torch.randint(0, min(n, M) + 1, (1,), generator=g))
            pick = torch.randperm(n, generator=g)[:k]
            ids[b, h, :k] = (pick.sort().values if order == "ascending" else pick).int()
            count[b, h], pi[b, h, :k] = k, 0.01 + 0.99 * torch.rand(k, generator=g)
    return ids.cuda(), count.cuda(), pi.cuda()


def check_listed(c, q, out, ids, count, pi, cap=0.0, window=0):
    G = q.shape[1] // c.hkv
    for b, L in enumerate(c.lens):
        K, V = c.tokens("k", b, L), c.tokens("v", b, L)
        for h in range(c.hkv):
            pos, bias = [], []
            for i in range(int(count[b, h])):
                t0 = int(ids[b, h, i]) * c.T
                see = [t for t in range(t0, min(L, t0 + c.T)) if not window or t >= L - window]
                pos += see
                bias += [-math.log(float(pi[b, h, i]))] * len(see)
            w = torch.tensor(bias, dtype=torch.float64, device="cuda")[None]
            want, tol = attend64(q[b, h * G:(h + 1) * G], K[h:h + 1, pos], V[h:h + 1, pos], w, cap)
            close(out[b, h * G:(h + 1) * G], want, tol)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,hq,hkv,d,T,M,cap,window", [
    ([1, 64, 0, 65], 3, 1, 64, 64, 1, 0.0, 0), ([1000, 130, 3], 8, 2, 128, 128, 5, 0.0, 0),
    ([5000, 4000], 28, 4, 128, 64, 40, 0.0, 0), ([700] * 5, 6, 3, 64, 128, 300, 3.0, 0),
    ([900, 100], 8, 1, 128, 64, 6, 0.0, 150), ([9000], 7, 1, 128, 128, 33, 20.0, 4000),
])
def test_listed_teams_match_reference(lens, hq, hkv, d, T, M, cap, window, dtype, kind):
    c = Q8(lens, hkv, d, T, kind, seed=M)
    q, status = queries(c, hq, dtype), status_word()
    ids, count, pi = listed(c, M, seed=hq, order="any")
    out = santa.santa_q8_attend(q, c.cache, c.table, c.seq_lens, ids, count, pi, softcap=cap,
                                window=window, device_status=status)
    assert int(status) == 0
    check_listed(c, q, out, ids, count, pi, cap, window)


def test_all_teams_with_weight_one_is_dense():
    c = Q8([1000, 77], 2, 128, 64, I8, seed=4)
    q = queries(c, 8, BF16)
    ids, count, pi = listed(c, 16, seed=1)
    for b, n in enumerate((16, 2)):
        ids[b, :, :n], count[b], pi[b, :, :n] = torch.arange(n, device="cuda").int(), n, 1.0
    out = santa.santa_q8_attend(q, c.cache, c.table, c.seq_lens, ids, count, pi)
    check_dense(c, q, out)


def many(B, seed, T=64):
    """Lengths of a large batch: empty runs, single tokens, a few long ones."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 3 * T, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.3] = 0
    lens[torch.rand(B, generator=g) < 0.2] = 1
    lens[B // 3:B // 2] = 0
    lens[B // 2], lens[-1] = 40 * T + 3, 7 * T
    return lens.tolist()


@pytest.mark.parametrize("B,hkv,hq,dtype,d,window", [
    (256, 2, 4, BF16, 128, 0), (257, 1, 8, BF16, 128, 0), (300, 3, 3, F32, 64, 100), (1500, 1, 2, BF16, 64, 0),
])
def test_large_batches(B, hkv, hq, dtype, d, window):
    """More sequences than a warp reads by itself, and than the grid has warps."""
    c = Q8(many(B, B), hkv, d, 64, I8, seed=1)
    q, status = queries(c, hq, dtype), status_word()
    out = torch.full(q.shape, 9.0, device="cuda")
    santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, window=window, out=out, device_status=status)
    assert int(status) == 0
    check_dense(c, q, out, window=window)
    c.seq_lens[5], c.seq_lens[B - 2] = -1, 10**6
    c.lens[5], c.lens[B - 2] = 0, 0
    santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, window=window, out=out, device_status=status)
    assert int(status) == DEV_BAD_SEQLEN
    check_dense(c, q, out, window=window)


@pytest.mark.parametrize("B,hkv", [(64, 4), (70, 4), (130, 3)])
def test_large_batches_of_lists(B, hkv):
    c = Q8(many(B, B), hkv, 128, 64, E4M3, seed=1)
    q, status = queries(c, 2 * hkv, BF16), status_word()
    ids, count, pi = listed(c, 6, seed=3)
    out = santa.santa_q8_attend(q, c.cache, c.table, c.seq_lens, ids, count, pi, device_status=status)
    assert int(status) == 0
    check_listed(c, q, out, ids, count, pi)


def test_one_long_sequence_behind_many_empty_ones():
    c = Q8([0] * 1000 + [9000] + [0] * 500, 2, 64, 64, I8, seed=1)
    q = queries(c, 4, BF16)
    check_dense(c, q, santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens))


def test_bad_lists_leave_teams_out():
    c = Q8([300, 300, 300, 300], 1, 64, 64, I8, seed=4)
    q = queries(c, 2, BF16)
    for bad in ("negative", "beyond", "pi_zero", "pi_nan", "pi_inf", "pi_negative"):
        ids, count, pi = listed(c, 3, seed=1)
        keep = ids.clone()
        if bad == "negative":
            ids[1, 0, 1] = -1
        elif bad == "beyond":
            ids[1, 0, 1] = 5
        else:
            pi[1, 0, 1] = {"pi_zero": 0.0, "pi_nan": math.nan, "pi_inf": math.inf, "pi_negative": -0.5}[bad]
        status = status_word()
        out = santa.santa_q8_attend(q, c.cache, c.table, c.seq_lens, ids, count, pi, device_status=status)
        assert int(status) == DEV_BAD_SEL
        ids2, count2, pi2 = keep.clone(), count.clone(), pi.clone()
        ids2[1, 0, 1], pi2[1, 0, 1], count2[1, 0] = keep[1, 0, 2], pi[1, 0, 2], 2
        check_listed(c, q, out, ids2, count2, pi2)
    ids, count, pi = listed(c, 3, seed=1)
    count[0, 0], count[2, 0], status = -1, 4, status_word()
    out = santa.santa_q8_attend(q, c.cache, c.table, c.seq_lens, ids, count, pi, device_status=status)
    assert int(status) == DEV_BAD_SEL
    count[0, 0], count[2, 0] = 0, 3
    check_listed(c, q, out, ids, count, pi)


def test_bad_lengths_and_pages():
    c = Q8([200, 200, 200, 130], 1, 128, 64, E4M3, seed=4)
    q, status = queries(c, 4, BF16), status_word()
    c.seq_lens[0], c.seq_lens[1] = -3, 4 * 64 + 1
    c.table[3, 1] = c.reps.shape[0]
    out = torch.full(q.shape, 9.0, device="cuda")
    santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, out=out, device_status=status)
    assert int(status) == DEV_BAD_SEQLEN | DEV_BAD_PAGE
    assert not out[:2].any()
    K, V = c.tokens("k", 2, 200), c.tokens("v", 2, 200)
    want, tol = attend64(q[2], K, V)
    close(out[2], want, tol)
    c.table[3, 1] = 0                          # any page: its tokens are cut out below
    see = list(range(64)) + [128, 129]
    want, tol = attend64(q[3], c.tokens("k", 3, 130)[:, see], c.tokens("v", 3, 130)[:, see])
    close(out[3], want, tol)


def test_rows_that_see_nothing_are_zero():
    c = Q8([0, 0, 50], 2, 64, 64, I8, seed=4)
    q = queries(c, 4, BF16)
    out = torch.full(q.shape, 9.0, device="cuda")
    santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, out=out)
    assert not out[:2].any() and out[2].any()
    # teams that the window leaves nothing of
    ids = torch.zeros(3, 2, 1, dtype=torch.int32, device="cuda")
    c = Q8([500, 400, 300], 2, 64, 64, I8, seed=4)
    count, pi = torch.ones(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, 2, 1, device="cuda")
    out = santa.santa_q8_attend(q, c.cache, c.table, c.seq_lens, ids, count, pi, window=100)
    assert not out.any()


@pytest.mark.parametrize("kind", [I8, E4M3])
def test_non_finite_rows_reach_only_what_sees_them(kind):
    c = Q8([300, 300, 300], 2, 128, 64, kind, seed=4)
    q = queries(c, 8, BF16)
    c.cache.k_scale[int(c.table[1, 2]), 1, 7] = math.nan
    c.cache.v_scale[int(c.table[2, 4]), 0, 43] = math.nan     # token 299
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    bad = torch.isnan(out).all(-1)
    assert not torch.isnan(out[~bad]).any()
    want = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    want[1, 4:], want[2, :4] = True, True
    assert torch.equal(bad, want)
    # a length or a window that ends before them does not see them
    lens = torch.tensor([300, 135, 299], dtype=torch.int32, device="cuda")
    assert bool(torch.isfinite(santa.santa_q8_dense_decode(q, c.cache, c.table, lens)).all())
    one = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, window=164)
    assert bool(torch.isfinite(one[1]).all())


def test_nan_codes_of_e4m3():
    c = Q8([100, 100], 1, 64, 64, E4M3, seed=4)
    c.cache.v.view(torch.uint8)[int(c.table[1, 1]), 0, 3, 5] = 0xff
    q = queries(c, 2, BF16)
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isnan(out[1, :, 5]).all())
    assert int(torch.isnan(out).sum()) == 2


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sizes_of_scales_and_queries(dtype):
    """Rows whose scales lie far apart, huge and tiny values, and queries of every size."""
    c = Q8([600] * 6, 1, 128, 128, I8, seed=4)
    c.cache.v_scale *= torch.exp2(torch.linspace(-60, 60, 128, device="cuda"))
    c.cache.k_scale[int(c.table[2, 0])] *= 1e-30
    q = queries(c, 4, dtype)
    q[3] *= 2.0**-40
    q[4] *= 0.0
    q[5, :, ::2] *= 2.0**-12
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    check_dense(c, q, out)
    # scores so far apart that most weights vanish, growing and falling along the sequence
    c = Q8([2000, 2000], 1, 128, 64, I8, seed=4)
    for b in range(2):
        for t in range(2000):
            f = 0.05 * (t if b else 2000 - t)
            c.cache.k_scale[int(c.table[b, t // 64]), 0, t % 64] = f / 127
        c.cache.k.view(torch.uint8)[c.table[b].long()] = 100
    q = queries(c, 3, dtype, size=0.3).abs()
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    check_dense(c, q, out)


def test_far_pages():
    """A long cache's last pages, behind element 2^31 of the codes."""
    P, hkv, T, d = 16500, 8, 128, 128
    cache = santa.Q8Cache.allocate(P, hkv, T, d, I8)
    c = Q8([700], hkv, d, T, I8, seed=2, spare=0)
    n = c.table.shape[1]
    far = torch.arange(P - n, P, device="cuda")
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(cache, name)[far] = getattr(c.cache, name)[c.table[0].long()]
    q = queries(c, 16, BF16)
    out = santa.santa_q8_dense_decode(q, cache, far.int()[None].contiguous(), c.seq_lens)
    check_dense(c, q, out)


def test_long_context_and_wide_table():
    c = Q8([100001], 1, 64, 128, I8, seed=2, cap=130000)
    q = queries(c, 8, BF16)
    check_dense(c, q, santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens))


def test_equal_calls_give_equal_bits():
    c = Q8([5000, 100, 9000, 0, 1], 4, 128, 128, E4M3, seed=2)
    q = queries(c, 16, BF16)
    h = santa.santa_q8_dense_decode_prepared(q, c.cache, c.table, c.seq_lens)
    first = h.run().clone()
    for _ in range(20):
        assert torch.equal(h.run(), first)
    # one workspace for calls of different shapes, one after the other
    ws = torch.full((santa.santa_q8_workspace_bytes(5, 16, 4, 128, 128, c.table.shape[1]),), 0xff,
                    dtype=torch.uint8, device="cuda")
    other = Q8([7000, 3000], 2, 64, 64, I8, seed=3)
    qo = queries(other, 6, F32)
    for _ in range(3):
        assert torch.equal(santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, workspace=ws), first)
        check_dense(other, qo, santa.santa_q8_dense_decode(qo, other.cache, other.table, other.seq_lens,
                                                           workspace=ws))


def test_replayed_for_other_lengths_on_another_stream():
    c = Q8([3000, 40, 500], 2, 128, 64, I8, seed=2)
    q = queries(c, 8, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        h = santa.santa_q8_dense_decode_prepared(q, c.cache, c.table, c.seq_lens, window=2000)
        h.run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = h.run()
    for lens in ([3000, 40, 500], [1, 0, 499], [2950, 13, 64]):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.lens = lens
        check_dense(c, q, out, window=2000)


def test_two_calls_at_once():
    c = Q8([8000, 8000], 4, 128, 128, I8, seed=2)
    q = [queries(c, 16, BF16, seed=s) for s in (1, 2)]
    want = [santa.santa_q8_dense_decode(x, c.cache, c.table, c.seq_lens) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    got = [[] for _ in q]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(santa.santa_q8_dense_decode(q[i], c.cache, c.table, c.seq_lens, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_from_a_prompt_to_sparse_steps(dtype, kind):
    """Prompts enter an 8-bit cache normed and turned, are read back for their own attention, and
    single tokens follow: dense, best teams and sampled teams, and a held set."""
    hq, hkv, d, T, M = 8, 2, 64, 64, 4
    lens = [700, 90, 333]
    c = Q8([0, 0, 0], hkv, d, T, kind, seed=1, cap=800)
    g = torch.Generator().manual_seed(5)
    w = (1 + 0.2 * torch.randn(2, d, generator=g)).cuda().unbind(0)
    w = [x.contiguous() for x in w]
    rope = santa.santa_rope_table(1024, d)

    def step(n, at, nxt):
        x = torch.randn(sum(n), hq + 2 * hkv, d, generator=g).to(dtype).cuda()
        q, k, v = x.split([hq, hkv, hkv], 1)
        return santa.santa_append_norm(q, k, v, cu(n), c.cache, c.reps, c.table, at, rope,
                                       q_norm=w[0], k_norm=w[1], seq_lens_next=nxt)

    now, nxt = c.seq_lens, torch.zeros_like(c.seq_lens)
    qr = step(lens, now, nxt)
    now, c.lens = nxt, lens
    P = c.reps.shape[0]
    k = torch.full((P, hkv, T, d), math.nan, dtype=dtype, device="cuda")
    v = k.clone()
    santa.santa_q8_read(c.cache, c.table, now, k, v, c.table)
    chunk = santa.santa_chunk_attend(qr, k, v, c.table, now, cu(lens))
    at = 0
    for b, L in enumerate(lens):
        K, V = c.tokens("k", b, L), c.tokens("v", b, L)
        for i in (0, 1, 63, L - 1):
            want, tol = attend64(qr[at + i], K[:, :i + 1], V[:, :i + 1])
            if dtype == BF16:           # weights, values read back and the output, to 2^-8 each
                tol = tol + 3 * 2.0**-8 * (V[:, :i + 1].abs().amax() + want.abs())
            close(chunk[at + i], want, tol)
        at += L
    for _ in range(3):
        nxt = torch.zeros_like(now)
        q1 = step([1, 1, 1], now, nxt)
        now, c.lens = nxt, [L + 1 for L in c.lens]
        out = santa.santa_q8_dense_decode(q1, c.cache, c.table, now)
        check_dense(c, q1, out)
        top = santa.santa_q8_topk_decode(q1, c.cache, c.reps, c.table, now, M)
        assert top.status() == 0
        plain = santa.santa_select_topk(q1, k, v, c.reps, c.table, now, M)
        assert torch.equal(top.sel_ids, plain.sel_ids) and torch.equal(top.pi, plain.pi)
        check_listed(c, q1, top.out, top.sel_ids, top.sel_count, top.pi)
        bufs = santa.santa_q8_decode(q1, c.cache, c.reps, c.table, now, M, seed=11)
        drawn = santa.santa_sample(q1, k, v, c.reps, c.table, now, M, 11)
        assert bufs.status() == 0
        for f in ("draw_ids", "sel_ids", "sel_count", "pi"):
            assert torch.equal(getattr(bufs, f), getattr(drawn, f))
        check_listed(c, q1, bufs.out, bufs.sel_ids, bufs.sel_count, bufs.pi)
        held = santa.santa_q8_attend(q1, c.cache, c.table, now, bufs.sel_ids, bufs.sel_count, bufs.pi)
        assert torch.equal(held, bufs.out)
        again = santa.santa_q8_topk_decode_prepared(q1, c.cache, c.reps, c.table, now, M, bufs=top)
        first = top.out.clone()
        assert torch.equal(again.run().out, first)


def test_values_helper_is_the_definition():
    x = torch.tensor([[1, -2, 127]], dtype=torch.int8)
    assert values64(x, torch.tensor([0.5])).tolist() == [[0.5, -1.0, 63.5]]
