"""Buffers that a prepared call makes: their memory is not handed out again while another stream
that ran the call has work of it in flight."""
import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import Cache, cu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def inputs():
    """A cache, its representatives and the other tensors of a call of one token per sequence."""
    c = Cache([700, 90], 2, 64, 64, BF16, seed=3, cap=800)
    c.reps = santa.santa_build_reps(c.k, c.fill)
    g = torch.Generator().manual_seed(1)
    c.q = torch.randn(2, 8, 64, generator=g).to(BF16).cuda()
    c.new = torch.randn(2, 2, 64, generator=g).to(BF16).cuda()
    c.cu = cu([1, 1])
    return c


def handle(name, c, **given):
    if name == "chunk":
        return santa.santa_chunk_attend_prepared(c.q, c.k, c.v, c.table, c.seq_lens, c.cu, **given)
    if name == "topk":
        return santa.santa_topk_decode_prepared(c.q, c.k, c.v, c.reps, c.table, c.seq_lens, 3, **given)
    return santa.santa_append_chunk_prepared(c.q, c.new, c.new, c.cu, c.k, c.v, c.reps, c.table,
                                             c.seq_lens, **given)


def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    if isinstance(x, (tuple, list)):
        return [t for y in x for t in tensors(y)]
    if isinstance(x, santa.DecodeBuffers):
        return tensors(list(vars(x).values()))
    return []


def held(h):
    """Address and size of every storage that the handle holds."""
    stores = [t.untyped_storage() for t in tensors((h._keep, h._result))]
    return {s.data_ptr(): s.nbytes() for s in stores}


@pytest.mark.parametrize("how", ["given", "given_raw", "current"])
@pytest.mark.parametrize("name", ["chunk", "topk", "append"])
def test_dropped_handle_keeps_its_memory_from_other_streams(name, how):
    c = inputs()
    h = handle(name, c)
    given = {t.untyped_storage().data_ptr() for t in tensors(list(vars(c).values()))}
    sizes = {at: n for at, n in held(h).items() if at not in given}
    assert sizes
    h.run()                                    # loads the kernels, which may wait for the device
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)         # a fifth of a second: the work behind it is pending
        if how == "current":
            h.run()
    if how != "current":
        h.run(stream=side if how == "given" else side.cuda_stream)
    del h
    pending, fresh, reused = not side.query(), [], []
    for n in sizes.values():
        fresh.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
        # memory that came back although the side stream is still at work after that
        reused.append(fresh[-1].untyped_storage().data_ptr() in sizes and not side.query())
    side.synchronize()
    assert pending, "the side stream finished too early for the test"
    assert not any(reused)


def test_replaced_fields_of_the_buffers_do_not_move_the_call():
    """bufs.out set to another tensor after the preparation: the call still owns the one it was
    prepared on."""
    h = handle("topk", inputs())
    bufs = h.run()
    at = bufs.out.data_ptr()
    bufs.out = torch.zeros_like(bufs.out)
    assert at in {t.data_ptr() for t in tensors(h._keep)}


def test_tensors_of_the_caller_are_left_to_the_caller():
    """Results that the caller gave are not named to the allocator: once the caller has waited and
    dropped them, their memory is free at once."""
    c = inputs()
    out, ws = torch.zeros_like(c.q), torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    h = handle("chunk", c, out=out, workspace=ws)
    assert h._made == ()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = h.run().clone()
    torch.cuda.synchronize()
    got = h.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    at = ws.data_ptr()
    del h, ws
    assert torch.empty(1 << 26, dtype=torch.uint8, device="cuda").data_ptr() == at
