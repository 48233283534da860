"""Arguments of the chunk and top-k calls that are refused on the host (CPU): buffers that overlap
what a call still reads, and buffers on another device."""
import ctypes

import pytest
import torch

from sampled_sparse_decode_gb300 import binding, build
from sampled_sparse_decode_gb300.binding import DecodeBuffers, SantaError


class _OnDevice(torch.Tensor):
    """A CPU tensor that claims to live on a CUDA device: what the checks look at."""
    index = 0
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index)


def on(t, index=0):
    t = t.as_subclass(_OnDevice)
    t.index = index
    return t


TOPK_FIELDS = ["out", "sel_ids", "sel_count", "pi", "workspace", "device_status"]


@pytest.mark.parametrize("field", TOPK_FIELDS)
def test_topk_buffers_of_another_device_are_refused(field, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    B, hq, hkv, d, T, k, P = 1, 4, 2, 64, 64, 3, 8
    i32 = torch.int32
    bufs = DecodeBuffers(
        out=on(torch.zeros(B, hq, d)), draw_ids=on(torch.zeros(B, hkv, k, dtype=i32)),
        sel_ids=on(torch.zeros(B, hkv, k, dtype=i32)), sel_count=on(torch.zeros(B, hkv, dtype=i32)),
        pi=on(torch.zeros(B, hkv, k)), team_probs=None,
        workspace=on(torch.zeros(256, dtype=torch.uint8)), device_status=on(torch.zeros(1, dtype=i32)))
    pool = on(torch.zeros(P, hkv, T, d))
    args = [on(torch.zeros(B, hq, d)), pool, pool, on(torch.zeros(P, hkv, d)),
            on(torch.zeros(B, P, dtype=i32)), on(torch.ones(B, dtype=i32)), k, bufs, None]
    setattr(bufs, field, on(getattr(bufs, field), 1))
    with pytest.raises(SantaError, match=field):
        binding._topk("santa_topk_decode", *args)


# ---------------------------------------------------------------- overlapping buffers

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(build.build())
    for f in ("santa_append_chunk", "santa_chunk_attend"):
        getattr(L, f).restype = ctypes.c_int
        getattr(L, f).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    return L


def fake(cls, **values):
    """Arguments with pointers a gigabyte apart that are never dereferenced: every call here fails
    a check (calls that pass them are made on the GPU, with memory behind the pointers)."""
    a, at = cls(), 1 << 32
    for name, t in cls._fields_:
        if t is ctypes.c_void_p:
            setattr(a, name, at)
            at += 1 << 30
    for name, v in values.items():
        setattr(a, name, v)
    return a


def append(**kw):
    """Ten tokens of a fused projection: rows of 6 + 2 + 2 heads of 64 bf16 values at 1 << 32."""
    base, row = 1 << 32, 10 * 64
    v = dict(q=base, k_new=base + 6 * 128, v_new=base + 8 * 128, q_stride=row, k_stride=row,
             v_stride=row, rope=None, rope_dim=0, rope_positions=0, num_tokens=10, num_pages=64,
             dtype=1, batch=3, num_q_heads=6, num_kv_heads=2, head_dim=64, team_size=64,
             max_teams=16)
    return fake(binding._AppendChunkArgs, **dict(v, **kw))


Q = 1 << 32
TOTAL = 10 * 6 * 128                     # bytes of the ten tokens' queries


@pytest.mark.parametrize("kw", [
    dict(q_out=Q + 16), dict(q_out=Q + 6 * 128), dict(q_out=Q + 9 * 1280),
    dict(q_out=Q - TOTAL + 16),                                     # ends inside the first row
    dict(q_stride=6 * 64, q_out=Q + 128),                           # packed, a head further on
    dict(q=Q - (1 << 28), q_out=Q + 6 * 128 + 16),                  # over the keys
    dict(q=Q - (1 << 28), q_out=Q + 9 * 1280 + 10 * 128 - 16),      # over the last value row's end
], ids=str)
def test_rotated_queries_over_rows_that_are_read(lib, kw):
    assert lib.santa_append_chunk(ctypes.addressof(append(**kw)), None) == INVALID


@pytest.mark.parametrize("field", ["seq_lens", "cu_q"])
@pytest.mark.parametrize("shift", [-8, 0, 8])
def test_new_lengths_over_arrays_that_are_read(lib, field, shift):
    a = append()
    a.seq_lens_next = getattr(a, field) + shift
    assert lib.santa_append_chunk(ctypes.addressof(a), None) == INVALID


@pytest.mark.parametrize("shift", [0, 16, -16, 10 * 6 * 64 * 2 - 16])
def test_chunk_output_over_its_queries(lib, shift):
    a = fake(binding._ChunkArgs, num_tokens=10, num_pages=64, dtype=1, batch=2, num_q_heads=6,
             num_kv_heads=2, head_dim=64, team_size=64, max_teams=16, workspace_bytes=1 << 29)
    a.out = a.q + shift
    assert lib.santa_chunk_attend(ctypes.addressof(a), None) == INVALID
