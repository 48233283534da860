"""The calls over 8-bit caches on streams other than the current one, from graphs that share a workspace,
with handles dropped while runs are in flight, and between guards that no call may touch."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import cu, rope_table
from q8_cases import E4M3, I8, Q8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def case(kind=I8, dtype=BF16, d=64):
    c = Q8([700, 90, 0], 2, d, 64, kind, seed=3, cap=800)
    g = torch.Generator().manual_seed(1)
    c.q = torch.randn(3, 8, d, generator=g).to(dtype).cuda()
    c.new = torch.randn(3, 2, d, generator=g).to(dtype).cuda()
    c.cu = cu([1, 1, 1])
    c.k_out = torch.zeros(c.reps.shape[0], 2, 64, d, dtype=dtype, device="cuda")
    c.v_out = torch.zeros_like(c.k_out)
    c.reps += torch.randn(c.reps.shape, generator=g).cuda()
    return c


def handle(name, c, **kw):
    if name == "append":
        return santa.santa_append_norm_prepared(c.q, c.new, c.new, c.cu, c.cache, c.reps, c.table,
                                                c.seq_lens, **kw)
    if name == "read":
        return santa.santa_q8_read_prepared(c.cache, c.table, c.seq_lens, c.k_out, c.v_out, c.table)
    if name == "topk":
        return santa.santa_q8_topk_decode_prepared(c.q[:2], c.cache, c.reps, c.table[:2], c.seq_lens[:2], 3)
    return santa.santa_q8_dense_decode_prepared(c.q, c.cache, c.table, c.seq_lens, **kw)


def result(name, c, r):
    if name == "append":
        return [r, c.cache.k.view(torch.uint8), c.cache.v.view(torch.uint8), c.cache.k_scale.nan_to_num(),
                c.cache.v_scale.nan_to_num(), c.reps]
    if name == "topk":
        return [r.out, r.sel_ids, r.sel_count, r.pi]
    return list(r) if name == "read" else [r]


def expected(name):
    c = case()
    return [t.clone() for t in result(name, c, handle(name, c).run())]


NAMES = ["append", "read", "topk", "dense"]


@pytest.mark.parametrize("how", ["given", "raw", "current"])
@pytest.mark.parametrize("name", NAMES)
def test_dropped_handles_on_another_stream(name, how):
    want = expected(name)
    side = torch.cuda.Stream()
    c = case()
    h = handle(name, c)
    torch.cuda.synchronize()
    stream = {"given": side, "raw": side.cuda_stream, "current": None}[how]
    with torch.cuda.stream(side if how == "current" else torch.cuda.current_stream()):
        with torch.cuda.stream(side):
            torch.cuda._sleep(10**7)               # the run waits behind this
        r = h.run(stream)
    del h
    # what the handle had made is not given out to another stream before the run is over
    noise = [torch.full((1 << 16,), 5.0, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del noise
    for a, b in zip(want, result(name, c, r)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["dense", "append"])
def test_direct_calls_on_a_given_stream(name):
    want = expected(name)
    c, side = case(), torch.cuda.Stream()
    torch.cuda.synchronize()
    if name == "dense":
        r = santa.santa_q8_dense_decode(c.q, c.cache, c.table, c.seq_lens, stream=side)
    else:
        r = santa.santa_append_norm(c.q, c.new, c.new, c.cu, c.cache, c.reps, c.table, c.seq_lens,
                                    stream=side)
    side.synchronize()
    for a, b in zip(want, result(name, c, r)):
        assert torch.equal(a, b)


def capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        fn()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            fn()
    torch.cuda.synchronize()
    return graph


def test_two_graphs_share_a_workspace():
    """Of two shapes, replayed in turn, eager calls between them."""
    a, b = Q8([9000, 40], 4, 128, 128, I8, seed=1), Q8([300, 7000, 5], 2, 64, 64, E4M3, seed=2)
    g = torch.Generator().manual_seed(1)
    qa = torch.randn(2, 28, 128, generator=g).to(BF16).cuda()
    qb = torch.randn(3, 4, 64, generator=g).cuda()
    ws = torch.empty(max(santa.santa_q8_workspace_bytes(2, 28, 4, 128, 128, a.table.shape[1]),
                         santa.santa_q8_workspace_bytes(3, 4, 2, 64, 64, b.table.shape[1])),
                     dtype=torch.uint8, device="cuda")
    want = [santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens) for q, c in ((qa, a), (qb, b))]
    hs = [santa.santa_q8_dense_decode_prepared(q, c.cache, c.table, c.seq_lens, workspace=ws)
          for q, c in ((qa, a), (qb, b))]
    graphs = [capture(h.run) for h in hs]
    outs = [h.run() for h in hs]
    for _ in range(5):
        for i in (0, 1, 1, 0):
            outs[i].fill_(7.0)
            graphs[i].replay()
            assert torch.equal(outs[i], want[i])
            hs[1 - i].run()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_a_step_as_one_graph():
    """Append, dense attention and best teams of a step captured together and replayed over a growing
    cache equal the eager calls."""
    def build():
        c = case(E4M3)
        c.next = torch.zeros_like(c.seq_lens)
        c.rope, c.w = rope_table(1024, 64), torch.linspace(0.5, 1.5, 64).cuda()
        c.h = [santa.santa_append_norm_prepared(c.q, c.new, c.new, c.cu, c.cache, c.reps, c.table, c.seq_lens,
                                                c.rope, q_norm=c.w, k_norm=c.w, seq_lens_next=c.next)]
        qr = c.h[0]._result
        c.h += [santa.santa_q8_dense_decode_prepared(qr, c.cache, c.table, c.next),
                santa.santa_q8_topk_decode_prepared(qr, c.cache, c.reps, c.table, c.next, 3)]
        return c

    def step(c):
        r = [h.run() for h in c.h]
        return [r[0], r[1], r[2].out, r[2].sel_ids]

    eager, replayed = build(), build()
    saved = [t.clone() for t in (replayed.cache.k.view(torch.uint8), replayed.cache.v.view(torch.uint8),
                                 replayed.cache.k_scale, replayed.cache.v_scale, replayed.reps)]
    graph = capture(lambda: step(replayed))
    for t, s in zip((replayed.cache.k.view(torch.uint8), replayed.cache.v.view(torch.uint8),
                     replayed.cache.k_scale, replayed.cache.v_scale, replayed.reps), saved):
        t.copy_(s)
    for i in range(70):
        want = [t.clone() for t in step(eager)]
        graph.replay()
        got = [replayed.h[0]._result, replayed.h[1]._result, replayed.h[2]._result.out,
               replayed.h[2]._result.sel_ids]
        for a, b in zip(want, got):
            assert torch.equal(a, b), i
        eager.seq_lens.copy_(eager.next)
        replayed.seq_lens.copy_(replayed.next)
        eager.q.add_(0.01)
        replayed.q.add_(0.01)


def guarded(shape, dtype, fill):
    """A tensor between two guards of 4 KiB in one storage, and the storage as bytes."""
    n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n + 8192,), fill, dtype=torch.uint8, device="cuda")
    return raw[4096:4096 + n].view(dtype).view(shape), raw


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_guards_around_outputs(dtype, d):
    c = case(I8, dtype, d)
    out, raw_out = guarded((3, 8, d), F32, 0xab)
    ws, raw_ws = guarded((santa.santa_q8_workspace_bytes(3, 8, 2, d, 64, c.table.shape[1]),), torch.uint8, 0xab)
    santa.santa_q8_dense_decode(c.q, c.cache, c.table, c.seq_lens, out=out, workspace=ws)
    q_out, raw_q = guarded((3, 8, d), dtype, 0xab)
    nxt, raw_n = guarded((3,), torch.int32, 0xab)
    reps, raw_r = guarded(tuple(c.reps.shape), F32, 0xab)
    reps.copy_(c.reps)
    santa.santa_append_norm(c.q, c.new, c.new, c.cu, c.cache, reps, c.table, c.seq_lens,
                            k_norm=torch.ones(d, device="cuda"), q_out=q_out, seq_lens_next=nxt)
    k, raw_k = guarded(tuple(c.k_out.shape), dtype, 0xab)
    v, raw_v = guarded(tuple(c.k_out.shape), dtype, 0xab)
    santa.santa_q8_read(c.cache, c.table, nxt, k, v, c.table)
    for raw in (raw_out, raw_ws, raw_q, raw_n, raw_r, raw_k, raw_v):
        assert bool((raw[:4096] == 0xab).all()) and bool((raw[-4096:] == 0xab).all())
