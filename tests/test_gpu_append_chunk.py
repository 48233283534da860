"""santa_append_chunk and santa_rope_table against 64-bit references: ragged chunks, both pair
orders, partial rotation, strided inputs, padding, page borders, refusals seen on the device."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import Cache, cu, rope_table, rotate64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(ctx, new, hq, hkv, d, T, dtype, seed=0, pad=0, lead=0, cap=None):
    c = Cache(ctx, hkv, d, T, dtype, seed, cap=cap or max(L + m for L, m in zip(ctx, new)))
    g = torch.Generator().manual_seed(seed + 1)
    tok = lead + sum(new) + pad
    qkv = torch.randn(tok, hq + 2 * hkv, d, generator=g).to(dtype).cuda()
    return c, qkv.split([hq, hkv, hkv], 1), cu(new, lead)


def check(c, qkv, cu_q, new, rope, interleaved, q_out, before, lens_next, skip=()):
    """The cache, queries, lengths and representatives after an append of `new` tokens."""
    q, k, v = qkv
    k0, v0 = before
    starts = cu_q.tolist()
    want_v, touched = v0.clone(), torch.zeros(k0.shape[0], k0.shape[2], dtype=torch.bool)
    half_step = torch.finfo(c.dtype).eps / 2 if c.dtype == BF16 else 0.0
    wrote = torch.zeros(q.shape[0], dtype=torch.bool)
    for b, m in enumerate(new):
        L = c.lens[b]
        if b in skip:
            continue
        assert lens_next is None or int(lens_next[b]) == L + m
        if m == 0:
            continue
        sl = slice(starts[b], starts[b] + m)
        wrote[sl] = True
        pos = torch.arange(L, L + m)
        page, slot = c.table_cpu[b].long()[pos // c.T], pos % c.T
        touched[page, slot] = True
        want_v[page.cuda(), :, slot.cuda()] = v[sl]
        rows = rope[L:L + m] if rope is not None else torch.zeros(m, 0, device="cuda")
        for x, got in ((q[sl], q_out[sl]), (k[sl], c.k[page.cuda(), :, slot.cuda()])):
            ref, mag = rotate64(x, rows, interleaved)
            # two products and a sum in fp32 (a rounding of 2^-24 each, the sum's of at most
            # the products' magnitude), then one rounding to the cache's type
            err = (got.double() - ref).abs()
            assert (err <= half_step * ref.abs() + 2.01 * 2.0 ** -24 * mag * (1 + half_step)).all()
    old = ~touched.cuda()[:, None, :, None].expand_as(k0)
    same = torch.equal(c.k[old].view(torch.int16 if c.dtype == BF16 else torch.int32),
                       k0[old].view(torch.int16 if c.dtype == BF16 else torch.int32))
    assert same, "a slot outside the chunk changed"
    it = torch.int16 if c.dtype == BF16 else torch.int32
    assert torch.equal(c.v.view(it), want_v.view(it))
    assert (q_out[(~wrote).cuda()] == 7).all(), "a padding row was written"
    # the representatives are those of a rebuild, bit for bit
    fill = torch.zeros_like(c.fill)
    for b, m in enumerate(new):
        L = c.lens[b] + (0 if b in skip else m)
        for i in range(-(-L // c.T)):
            fill[c.table_cpu[b, i]] = min(c.T, L - i * c.T)
    assert torch.equal(c.reps, santa.santa_build_reps(c.k, fill))


@pytest.mark.parametrize("ctx,new,hq,hkv,d,T,dtype,R,inter,pad,lead", [
    ([0], [1], 1, 1, 64, 64, BF16, 64, False, 0, 0),
    ([63], [2], 7, 1, 128, 64, BF16, 128, False, 0, 0),          # over a page border
    ([128, 0, 127], [1, 128, 129], 28, 4, 128, 128, BF16, 128, False, 5, 0),
    ([5, 300, 0, 64], [0, 77, 0, 200], 6, 2, 64, 64, BF16, 32, True, 0, 3),
    ([100, 1], [33, 500], 5, 1, 128, 128, F32, 128, True, 1, 0),
    ([0, 0, 64], [63, 64, 65], 4, 2, 64, 64, F32, 16, False, 0, 0),
    ([17], [1000], 16, 2, 128, 64, F32, 64, False, 0, 1),
    ([10, 20], [40, 3], 3, 3, 128, 128, BF16, 0, False, 0, 0),   # no rotation
    ([0] * 40, list(range(40)), 2, 1, 64, 64, BF16, 64, True, 9, 0),
    ([3] * 70, [1] * 70, 4, 2, 128, 128, BF16, 112, False, 0, 0),
])
def test_append_matches_reference(ctx, new, hq, hkv, d, T, dtype, R, inter, pad, lead):
    c, qkv, cu_q = make(ctx, new, hq, hkv, d, T, dtype, seed=len(ctx) + d, pad=pad, lead=lead)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    rope = rope_table(max(L + m for L, m in zip(ctx, new)), R) if R else None
    before = c.k.clone(), c.v.clone()
    q_out = torch.full(qkv[0].shape, 7.0, dtype=dtype, device="cuda")
    nxt = torch.full((len(ctx),), -5, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = santa.santa_append_chunk(*qkv, cu_q, c.k, c.v, c.reps, c.table, c.seq_lens, rope,
                                   seq_lens_next=nxt, q_out=q_out, interleaved=inter,
                                   device_status=status)
    assert got is q_out and int(status) == 0
    check(c, qkv, cu_q, new, rope, inter, q_out, before, nxt)


def test_single_tokens_equal_append_kv():
    """Without rotation, one token per sequence gives what santa_append_kv gives, bit for bit."""
    ctx = [0, 1, 63, 64, 127, 128, 200]
    c, (q, k, v), cu_q = make(ctx, [1] * 7, 4, 2, 128, 128, BF16)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    k2, v2, r2 = c.k.clone(), c.v.clone(), c.reps.clone()
    n1, n2 = torch.zeros_like(c.seq_lens), torch.zeros_like(c.seq_lens)
    assert santa.santa_append_chunk(None, k, v, cu_q, c.k, c.v, c.reps, c.table, c.seq_lens,
                                    seq_lens_next=n1) is None
    santa.santa_append_kv(k.contiguous(), v.contiguous(), k2, v2, r2, c.table, c.seq_lens, n2)
    assert torch.equal(c.k.view(torch.int16), k2.view(torch.int16))
    assert torch.equal(c.v.view(torch.int16), v2.view(torch.int16))
    assert torch.equal(c.reps, r2) and torch.equal(n1, n2)


def test_split_chunk_equals_whole():
    """A prompt appended in three pieces leaves the cache of one append, bit for bit."""
    whole = [0, 130, 77]
    a, qkv, cu_q = make([0, 5, 64], [300, 130, 1], 4, 2, 64, 64, BF16)
    rope = rope_table(400, 64)
    b_k, b_v, b_r = a.k.clone(), a.v.clone(), a.reps.clone()
    out = santa.santa_append_chunk(*qkv, cu_q, a.k, a.v, a.reps, a.table, a.seq_lens, rope)
    lens, done = a.seq_lens.clone(), [0, 0, 0]
    starts, parts = cu_q.tolist(), []
    for piece in ([100, 130, 0], [29, 0, 1], [171, 0, 0]):
        rows = torch.cat([torch.arange(starts[i] + done[i], starts[i] + done[i] + piece[i])
                          for i in range(3)]).cuda()
        nxt = torch.empty_like(lens)
        sub = [x[rows] for x in qkv]
        parts.append((rows, santa.santa_append_chunk(*sub, cu(piece), b_k, b_v, b_r, a.table,
                                                     lens, rope, seq_lens_next=nxt)))
        lens = nxt
        done = [x + y for x, y in zip(done, piece)]
    assert torch.equal(a.k.view(torch.int16), b_k.view(torch.int16))
    assert torch.equal(a.v.view(torch.int16), b_v.view(torch.int16))
    assert torch.equal(a.reps, b_r) and lens.tolist() == [300, 135, 65]
    for rows, o in parts:
        assert torch.equal(out[rows], o)
    assert whole


def test_in_place_queries_and_graph_replay():
    c, (q, k, v), cu_q = make([9, 70], [20, 60], 6, 2, 128, 64, BF16)
    rope = rope_table(200, 128)
    q = q.contiguous()
    want = santa.santa_append_chunk(q, k, v, cu_q, c.k, c.v, c.reps, c.table, c.seq_lens, rope)
    handle = santa.santa_append_chunk_prepared(q, k, v, cu_q, c.k, c.v, c.reps, c.table,
                                               c.seq_lens, rope, q_out=q)
    first = q.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        handle.run()
    for _ in range(2):
        q.copy_(first)
        c.k.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, want)
        assert c.k.abs().sum() > 0


def test_empty_chunk_copies_lengths():
    c, (q, k, v), cu_q = make([5, 6], [0, 0], 2, 1, 64, 64, F32, cap=64)
    before = c.k.clone()
    nxt = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = santa.santa_append_chunk(q, k, v, cu_q, c.k, c.v, c.reps, c.table, c.seq_lens,
                                   rope_table(64, 64), seq_lens_next=nxt)
    assert out.shape == (0, 2, 64) and nxt.tolist() == [5, 6]
    assert torch.equal(c.k.view(torch.int32), before.view(torch.int32))


@pytest.mark.parametrize("what", ["negative", "past_the_table", "past_the_rope", "page"])
def test_bad_sequences_are_reported_and_skipped(what):
    """Sequence 1 of 3 is out of range: the others are appended, it is left alone."""
    ctx, new = [3, 60, 100], [5, 70, 9]
    c, qkv, cu_q = make(ctx, new, 4, 2, 64, 64, BF16, cap=200)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    before = c.k.clone(), c.v.clone()
    rope = rope_table(129 if what == "past_the_rope" else 300, 64)
    lens, table = c.seq_lens.clone(), c.table
    if what == "negative":
        lens[1] = -1
    elif what == "past_the_table":
        lens[1] = 4 * 64 - 69
    elif what == "page":
        table = table.clone()
        table[1, 0], table[1, 1], table[1, 2] = -1, c.k.shape[0], 2**31 - 1
    q_out = torch.full(qkv[0].shape, 7.0, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nxt = torch.full((3,), -5, dtype=torch.int32, device="cuda")
    santa.santa_append_chunk(*qkv, cu_q, c.k, c.v, c.reps, table, lens, rope, seq_lens_next=nxt,
                             q_out=q_out, device_status=status)
    from sampled_sparse_decode_gb300.binding import DEV_BAD_PAGE, DEV_BAD_SEQLEN
    assert int(status) == (DEV_BAD_PAGE if what == "page" else DEV_BAD_SEQLEN)
    if what == "page":               # the queries and the length are not the page's
        assert int(nxt[1]) == 130
        q_out[5:75] = 7
    else:
        assert int(nxt[1]) == -5
    check(c, qkv, cu_q, new, rope, False, q_out, before, nxt, skip=(1,))


@pytest.mark.parametrize("bounds", [[0, 9, 5, 12], [-3, 4, 8, 12], [0, 4, 8, 13]])
def test_bad_cu_q_is_reported(bounds):
    c, qkv, _ = make([3, 60, 100], [4, 4, 4], 4, 2, 64, 64, BF16, cap=200)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    santa.santa_append_chunk(*qkv, torch.tensor(bounds, dtype=torch.int32, device="cuda"), c.k,
                             c.v, c.reps, c.table, c.seq_lens, rope_table(300, 64),
                             device_status=status)
    assert int(status) & santa.DEV_BAD_SEQLEN


@pytest.mark.parametrize("positions,R,theta", [(1, 16, 10000.0), (131073, 128, 10000.0),
                                               (5000, 64, 5e5)])
def test_rope_table(positions, R, theta):
    got = santa.santa_rope_table(positions, R, theta).double()
    half = R // 2
    f = theta ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    # one rounding to fp32 (2^-24 of at most 1), and the angles' 64-bit error of a few 2^-52
    # of the angle (the power, the product)
    tol = 2.0 ** -24 + 2.0 ** -49 * positions
    assert (got[:, :half] - a.cos()).abs().max() <= tol
    assert (got[:, half:] - a.sin()).abs().max() <= tol
