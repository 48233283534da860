"""Refusals of the chunk append, the chunk attention and the top-k step on the host (CPU): bad
arguments are turned down by the C entry points before any CUDA call, and by the binding before
the library is entered."""
import ctypes

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300 import binding
from sampled_sparse_decode_gb300 import build as B
from sampled_sparse_decode_gb300.binding import (SantaError, _AppendChunkArgs, _ChunkArgs,
                                                 _DecodeArgs)

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(B.build())
    for f in ("santa_append_chunk", "santa_chunk_attend", "santa_select_topk",
              "santa_topk_decode"):
        getattr(L, f).restype = ctypes.c_int
        getattr(L, f).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    return L


def fake(cls, **values):
    """Arguments whose pointers are aligned addresses that are never dereferenced: every call
    fails a check first."""
    a, at = cls(), 0x10000
    for name, t in cls._fields_:
        if t is ctypes.c_void_p:
            setattr(a, name, at)
            at += 0x10000
    for name, v in values.items():
        setattr(a, name, v)
    return a


def append_args(**kw):
    base = dict(q_stride=28 * 128, k_stride=512, v_stride=512, rope_positions=4096,
                num_tokens=10, num_pages=64, dtype=1, batch=2, num_q_heads=28, num_kv_heads=4,
                head_dim=128, team_size=128, max_teams=16, rope_dim=128)
    return fake(_AppendChunkArgs, **dict(base, **kw))


@pytest.mark.parametrize("field,value,expect", [
    ("dtype", 2, UNSUPPORTED), ("batch", 0, INVALID), ("num_kv_heads", 0, INVALID),
    ("head_dim", 96, UNSUPPORTED), ("team_size", 32, UNSUPPORTED), ("max_teams", 0, INVALID),
    ("max_teams", 16385, UNSUPPORTED), ("batch", 65536, UNSUPPORTED), ("num_tokens", -1, INVALID),
    ("num_tokens", (1 << 24) + 1, UNSUPPORTED), ("num_pages", 0, INVALID), ("q", 0, INVALID),
    ("q_out", 0, INVALID), ("num_q_heads", 0, INVALID), ("rope_dim", 24, UNSUPPORTED),
    ("rope_dim", 144, UNSUPPORTED), ("rope_dim", -16, UNSUPPORTED), ("rope", 0, INVALID),
    ("rope_positions", 0, INVALID), ("k_new", 0, INVALID), ("v_new", 0, INVALID),
    ("k_stride", 504, INVALID), ("v_stride", 516, INVALID), ("q_stride", 128, INVALID),
    ("q_stride", 28 * 128 + 4, INVALID), ("cu_q", 0, INVALID), ("page_table", 0, INVALID),
    ("seq_lens", 0, INVALID), ("k_pool", 0, INVALID), ("v_pool", 0, INVALID), ("reps", 0, INVALID),
    ("k_pool", 0x10008, INVALID), ("cu_q", 0x10002, INVALID), ("device_status", 0x10001, INVALID),
])
def test_append_chunk_refusals(lib, field, value, expect):
    assert lib.santa_append_chunk(ctypes.addressof(append_args(**{field: value})), None) == expect


def test_append_chunk_refuses_aliased_buffers(lib):
    a = append_args()
    a.seq_lens_next = a.seq_lens
    assert lib.santa_append_chunk(ctypes.addressof(a), None) == INVALID
    a = append_args(q_stride=36 * 128)          # in place, but q is a strided view
    a.q_out = a.q
    assert lib.santa_append_chunk(ctypes.addressof(a), None) == INVALID
    # more blocks than a launch holds
    a = append_args(batch=65535, num_kv_heads=65535, k_stride=65535 * 128, v_stride=65535 * 128)
    assert lib.santa_append_chunk(ctypes.addressof(a), None) == UNSUPPORTED


@pytest.mark.parametrize("kw,expect", [
    (dict(table=0), INVALID), (dict(table=0x10004), INVALID), (dict(positions=0), INVALID),
    (dict(rope_dim=8), UNSUPPORTED), (dict(rope_dim=130), UNSUPPORTED),
    (dict(rope_dim=256), UNSUPPORTED), (dict(theta=1.0), INVALID),
    (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(positions=1 << 31), UNSUPPORTED),
])
def test_rope_table_refusals(lib, kw, expect):
    f = lib.santa_rope_table
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p]
    a = dict(dict(table=0x10000, positions=64, rope_dim=64, theta=10000.0), **kw)
    assert f(a["table"], a["positions"], a["rope_dim"], a["theta"], None) == expect


def chunk_args(**kw):
    base = dict(num_tokens=10, num_pages=64, dtype=1, batch=2, num_q_heads=28, num_kv_heads=4,
                head_dim=128, team_size=128, max_teams=16, workspace_bytes=0)
    return fake(_ChunkArgs, **dict(base, **kw))


@pytest.mark.parametrize("field,value,expect", [
    ("dtype", -1, UNSUPPORTED), ("batch", 0, INVALID), ("num_q_heads", 30, INVALID),
    ("num_q_heads", 36, UNSUPPORTED), ("num_q_heads", 0, INVALID), ("head_dim", 256, UNSUPPORTED),
    ("team_size", 256, UNSUPPORTED), ("max_teams", 20000, UNSUPPORTED), ("num_tokens", -5, INVALID),
    ("num_tokens", 1 << 25, UNSUPPORTED), ("num_pages", 0, INVALID), ("q", 0, INVALID),
    ("out", 0, INVALID), ("k_pool", 0, INVALID), ("v_pool", 0x10004, INVALID), ("cu_q", 0, INVALID),
    ("seq_lens", 0, INVALID), ("page_table", 0x10002, INVALID), ("out", 0x10008, INVALID),
])
def test_chunk_attend_refusals(lib, field, value, expect):
    assert lib.santa_chunk_attend(ctypes.addressof(chunk_args(**{field: value})), None) == expect


def test_chunk_attend_without_tokens_does_nothing(lib):
    a = chunk_args(num_tokens=0)
    a.q = a.out = a.workspace = None
    assert lib.santa_chunk_attend(ctypes.addressof(a), None) == OK


def topk_args(**kw):
    base = dict(num_pages=64, dtype=1, batch=2, num_q_heads=28, num_kv_heads=4, head_dim=128,
                team_size=128, max_teams=16, num_draws=4)
    return fake(_DecodeArgs, **dict(base, **kw))


@pytest.mark.parametrize("field,value,expect", [
    ("dtype", 5, UNSUPPORTED), ("num_draws", 0, UNSUPPORTED), ("num_draws", 4097, UNSUPPORTED),
    ("num_q_heads", 36, UNSUPPORTED), ("head_dim", 32, UNSUPPORTED), ("reps", 0, INVALID),
    ("reps", 0x10004, INVALID), ("q", 0, INVALID), ("sel_ids", 0, INVALID), ("pi", 0, INVALID),
    ("sel_count", 0x10001, INVALID), ("seq_lens", 0, INVALID), ("page_table", 0, INVALID),
])
def test_select_topk_refusals(lib, field, value, expect):
    assert lib.santa_select_topk(ctypes.addressof(topk_args(**{field: value})), None) == expect


@pytest.mark.parametrize("field,value,expect", [
    ("out", 0, INVALID), ("k_pool", 0, INVALID), ("v_pool", 0x10004, INVALID), ("batch", 0, INVALID),
    ("num_draws", 0, UNSUPPORTED),
])
def test_topk_decode_refuses_before_the_selection(lib, field, value, expect):
    assert lib.santa_topk_decode(ctypes.addressof(topk_args(**{field: value})), None) == expect


def test_null_arguments(lib):
    for f in ("santa_append_chunk", "santa_chunk_attend", "santa_select_topk",
              "santa_topk_decode"):
        assert getattr(lib, f)(None, None) == INVALID


# ---------------------------------------------------------------- the binding

def _cpu():
    z = torch.zeros
    bf = torch.bfloat16
    return dict(q=z(3, 4, 64, dtype=bf), k=z(3, 2, 64, dtype=bf), pool=z(8, 2, 64, 64, dtype=bf),
                reps=z(8, 2, 64), table=z(1, 8, dtype=torch.int32),
                lens=z(1, dtype=torch.int32), cu=torch.tensor([0, 3], dtype=torch.int32))


CALLS = {
    "append": lambda t: santa.santa_append_chunk(t["q"], t["k"], t["k"], t["cu"], t["pool"],
                                                 t["pool"], t["reps"], t["table"], t["lens"]),
    "append_prepared": lambda t: santa.santa_append_chunk_prepared(
        t["q"], t["k"], t["k"], t["cu"], t["pool"], t["pool"], t["reps"], t["table"], t["lens"]),
    "chunk": lambda t: santa.santa_chunk_attend(t["q"], t["pool"], t["pool"], t["table"],
                                                t["lens"], t["cu"]),
    "chunk_prepared": lambda t: santa.santa_chunk_attend_prepared(
        t["q"], t["pool"], t["pool"], t["table"], t["lens"], t["cu"]),
    "select": lambda t: santa.santa_select_topk(t["q"][:1], t["pool"], t["pool"], t["reps"],
                                                t["table"], t["lens"], 2),
    "topk": lambda t: santa.santa_topk_decode(t["q"][:1], t["pool"], t["pool"], t["reps"],
                                              t["table"], t["lens"], 2),
    "topk_prepared": lambda t: santa.santa_topk_decode_prepared(
        t["q"][:1], t["pool"], t["pool"], t["reps"], t["table"], t["lens"], 2),
    "rope": lambda t: santa.santa_rope_table(16, 64, device="cpu"),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_cpu_tensors_are_refused(name):
    with pytest.raises(SantaError):
        CALLS[name](_cpu())


class _Cuda:
    """A stand-in for a CUDA tensor on `index`: what the device check looks at."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    binding._same_device(q=_Cuda(0), out=None)
    with pytest.raises(SantaError, match="v_pool"):
        binding._same_device(q=_Cuda(0), v_pool=_Cuda(1))


def test_a_prepared_call_stays_on_its_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    h = binding._Prepared("santa_chunk_attend", chunk_args(batch=0), (), None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(SantaError, match="cuda:0"):
        h.run(0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(SantaError, match="santa_chunk_attend"):
        h.run(0)


class _Rows(torch.Tensor):
    is_cuda = True


def test_token_rows_must_hold_whole_heads():
    def rows(*shape, strides=None):
        t = torch.zeros(4000)
        return t.as_strided(shape, strides or torch.zeros(shape).stride()).as_subclass(_Rows)

    assert binding._token_rows(rows(3, 2, 64), "q", torch.float32, 2, 64) == 128
    assert binding._token_rows(rows(3, 2, 64, strides=(400, 64, 1)), "q", torch.float32, 2, 64) == 400
    assert binding._token_rows(rows(1, 2, 64, strides=(1, 64, 1)), "q", torch.float32, 2, 64) == 128
    assert binding._token_rows(rows(0, 2, 64), "q", torch.float32, 2, 64) == 128
    for bad in ((400, 128, 1), (400, 64, 2), (400, 1, 2)):
        with pytest.raises(SantaError):
            binding._token_rows(rows(3, 2, 64, strides=bad), "q", torch.float32, 2, 64)
    for shape in ((3, 3, 64), (3, 2, 32)):
        with pytest.raises(SantaError):
            binding._token_rows(rows(*shape), "q", torch.float32, 2, 64)
