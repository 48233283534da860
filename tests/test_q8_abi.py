"""Refusals of the calls over 8-bit caches on the host (CPU): bad arguments are turned down by the C
entry points before any CUDA call, and by the binding before the library is entered."""
import ctypes
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300 import binding
from sampled_sparse_decode_gb300 import build as B
from sampled_sparse_decode_gb300.binding import (SantaError, _AppendNormArgs, _DecodeArgs, _Q8Args,
                                                 _Q8ReadArgs)
from test_cache_abi import append_args, fake
from test_cache_args import on

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(B.build())
    for f in ("santa_append_norm", "santa_q8_read"):
        getattr(L, f).restype = ctypes.c_int
        getattr(L, f).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    for f in ("santa_q8_dense_decode", "santa_q8_attend", "santa_q8_topk_decode", "santa_q8_decode"):
        getattr(L, f).restype = ctypes.c_int
        getattr(L, f).argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    return L


def norm_args(chunk=(), **kw):
    a = fake(_AppendNormArgs, **dict(dict(cache_type=2, eps=1e-6, q_norm=0x900000, k_norm=0x910000,
                                          k_scale=0x920000, v_scale=0x930000), **kw))
    a.chunk = append_args(**dict(chunk))
    return a


@pytest.mark.parametrize("kw,expect", [
    (dict(cache_type=0), UNSUPPORTED), (dict(cache_type=4), UNSUPPORTED), (dict(cache_type=-1), UNSUPPORTED),
    (dict(cache_type=1), INVALID), (dict(k_scale=0), INVALID), (dict(v_scale=0), INVALID),
    (dict(k_scale=0x920004), INVALID), (dict(v_scale=0x930008), INVALID),
    (dict(q_norm=0x900004), INVALID), (dict(k_norm=0x910008), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(chunk=dict(dtype=2)), UNSUPPORTED), (dict(chunk=dict(dtype=3)), UNSUPPORTED),
    (dict(chunk=dict(head_dim=96)), UNSUPPORTED), (dict(chunk=dict(k_stride=504)), INVALID),
    (dict(chunk=dict(rope_dim=24)), UNSUPPORTED), (dict(chunk=dict(k_pool=0)), INVALID),
    (dict(chunk=dict(num_pages=0)), INVALID), (dict(chunk=dict(q_out=0)), INVALID),
])
def test_append_norm_refusals(lib, kw, expect):
    assert lib.santa_append_norm(ctypes.addressof(norm_args(**kw)), None) == expect


def test_append_norm_refuses_overlaps(lib):
    a = norm_args()
    a.chunk.seq_lens_next = a.chunk.cu_q
    assert lib.santa_append_norm(ctypes.addressof(a), None) == INVALID
    a = norm_args()
    a.chunk.q_out = a.chunk.k_new
    assert lib.santa_append_norm(ctypes.addressof(a), None) == INVALID
    assert lib.santa_append_norm(None, None) == INVALID


def step_args(**kw):
    base = dict(num_pages=64, dtype=1, batch=2, num_q_heads=28, num_kv_heads=4, head_dim=128,
                team_size=128, max_teams=16, num_draws=4, workspace_bytes=0)
    return fake(_DecodeArgs, **dict(base, **kw))


def cache_args(**kw):
    return fake(_Q8Args, **dict(dict(k=0x1000000, v=0x2000000, k_scale=0x3000000, v_scale=0x3100000,
                                     type=2), **kw))


ATTEND = ["santa_q8_dense_decode", "santa_q8_attend", "santa_q8_topk_decode", "santa_q8_decode"]


@pytest.mark.parametrize("f", ATTEND)
@pytest.mark.parametrize("kw,cw,expect", [
    (dict(dtype=2), {}, UNSUPPORTED), (dict(batch=0), {}, INVALID), (dict(num_q_heads=30), {}, INVALID),
    (dict(num_q_heads=36), {}, UNSUPPORTED), (dict(head_dim=256), {}, UNSUPPORTED),
    (dict(team_size=32), {}, UNSUPPORTED), (dict(max_teams=16385), {}, UNSUPPORTED),
    (dict(batch=65536), {}, UNSUPPORTED), (dict(num_pages=0), {}, INVALID),
    (dict(num_pages=1 << 31), {}, UNSUPPORTED), (dict(q=0), {}, INVALID), (dict(out=0), {}, INVALID),
    (dict(page_table=0), {}, INVALID), (dict(seq_lens=0), {}, INVALID), (dict(q=0x10008), {}, INVALID),
    (dict(out=0x70008), {}, INVALID), (dict(device_status=0x10001), {}, INVALID),
    ({}, dict(type=1), UNSUPPORTED), ({}, dict(type=4), UNSUPPORTED), ({}, dict(k=0), INVALID),
    ({}, dict(v=0x2000008), INVALID), ({}, dict(k_scale=0), INVALID), ({}, dict(v_scale=0x3100004), INVALID),
    ({}, dict(softcap=-1.0), INVALID), ({}, dict(softcap=math.nan), INVALID),
    ({}, dict(softcap=math.inf), INVALID), ({}, dict(window=-1), INVALID),
    ({}, dict(softcap=9e-7), INVALID), ({}, dict(softcap=1.1e6), INVALID),
])
def test_attend_refusals(lib, f, kw, cw, expect):
    a, c = step_args(**kw), cache_args(**cw)
    assert getattr(lib, f)(ctypes.addressof(a), ctypes.addressof(c), None) == expect


def test_more_tiles_than_32_bits_count(lib):
    a, c = step_args(batch=65535, num_kv_heads=8, num_q_heads=8, max_teams=16384), cache_args()
    assert lib.santa_q8_dense_decode(ctypes.addressof(a), ctypes.addressof(c), None) == UNSUPPORTED
    a = step_args(batch=65535, num_kv_heads=64, num_q_heads=64, num_draws=4096)
    assert lib.santa_q8_attend(ctypes.addressof(a), ctypes.addressof(c), None) == UNSUPPORTED


@pytest.mark.parametrize("f", ATTEND[1:])
@pytest.mark.parametrize("kw,expect", [
    (dict(num_draws=0), UNSUPPORTED), (dict(num_draws=4097), UNSUPPORTED), (dict(sel_ids=0), INVALID),
    (dict(sel_count=0), INVALID), (dict(pi=0), INVALID), (dict(pi=0x50002), INVALID),
])
def test_listed_refusals(lib, f, kw, expect):
    a, c = step_args(**kw), cache_args()
    assert getattr(lib, f)(ctypes.addressof(a), ctypes.addressof(c), None) == expect


def test_null_structures(lib):
    a, c = step_args(), cache_args()
    for f in ATTEND:
        assert getattr(lib, f)(None, ctypes.addressof(c), None) == INVALID
        assert getattr(lib, f)(ctypes.addressof(a), None, None) == INVALID
    assert lib.santa_q8_read(None, None) == INVALID


def read_args(**kw):
    base = dict(k=0x1000000, v=0x2000000, k_scale=0x3000000, v_scale=0x3100000, k_out=0x10000000,
                v_out=0x20000000, num_pages=64, dst_pages=64, type=3, out_dtype=1, batch=2,
                num_kv_heads=4, head_dim=128, team_size=128, max_teams=16)
    return fake(_Q8ReadArgs, **dict(base, **kw))


@pytest.mark.parametrize("kw,expect", [
    (dict(type=0), UNSUPPORTED), (dict(out_dtype=2), UNSUPPORTED), (dict(batch=0), INVALID),
    (dict(head_dim=80), UNSUPPORTED), (dict(team_size=16), UNSUPPORTED), (dict(max_teams=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(dst_pages=0), INVALID), (dict(dst_pages=1 << 31), UNSUPPORTED),
    (dict(k=0), INVALID), (dict(k_scale=0), INVALID), (dict(k_out=0), INVALID), (dict(v_out=0), INVALID),
    (dict(dst_table=0), INVALID), (dict(page_table=0), INVALID), (dict(seq_lens=0), INVALID),
    (dict(k_out=0x10000008), INVALID), (dict(first=0x10002), INVALID), (dict(v=0x2000008), INVALID),
    (dict(k_out=0x1000000), INVALID), (dict(v_out=0x10000010), INVALID), (dict(v_out=0x30ffff0), INVALID),
])
def test_read_refusals(lib, kw, expect):
    assert lib.santa_q8_read(ctypes.addressof(read_args(**kw)), None) == expect


# ---------------------------------------------------------------- the binding

def cpu_cache(dtype=torch.int8, P=4, hkv=2, T=64, d=64):
    c = santa.Q8Cache.allocate(P, hkv, T, d, dtype, device="cpu")
    return santa.Q8Cache(*(on(t) for t in (c.k, c.v, c.k_scale, c.v_scale)))


def call(**kw):
    base = dict(q=on(torch.zeros(2, 4, 64, dtype=torch.bfloat16)), cache=cpu_cache(),
                page_table=on(torch.zeros(2, 2, dtype=torch.int32)),
                seq_lens=on(torch.zeros(2, dtype=torch.int32)), sel=None, softcap=0.0, window=0,
                out=None, workspace=None, device_status=None, stream=None)
    base.update(kw)
    return binding._q8_attend(**base)


def part(**kw):
    c = cpu_cache()
    for name, t in kw.items():
        setattr(c, name, t)
    return c


@pytest.mark.parametrize("kw,match", [
    (dict(cache=(1, 2)), "Q8Cache"), (dict(cache=part(k=on(torch.zeros(4, 2, 64, 64)))), "int8 or float8"),
    (dict(cache=part(v=cpu_cache(torch.float8_e4m3fn).v)), "cache.v"),
    (dict(cache=part(k_scale=on(torch.zeros(4, 2, 63)))), "scales"),
    (dict(cache=part(v_scale=on(torch.zeros(4, 2, 64, dtype=torch.float64)))), "v_scale"),
    (dict(q=on(torch.zeros(2, 4, 64, dtype=torch.float16))), "float32 or bfloat16"),
    (dict(q=on(torch.zeros(2, 4, 128))), "mismatch"), (dict(q=torch.zeros(2, 4, 64)), "CUDA"),
    (dict(seq_lens=on(torch.zeros(3, dtype=torch.int32))), "mismatch"),
    (dict(page_table=on(torch.zeros(2, 2, dtype=torch.int64))), "page_table"),
    (dict(out=on(torch.zeros(2, 4, 64, dtype=torch.bfloat16))), "out"),
    (dict(out=on(torch.zeros(2, 5, 64))), "out"),
    (dict(workspace=on(torch.zeros(8))), "workspace"),
    (dict(device_status=on(torch.zeros(1))), "device_status"),
    (dict(sel=(on(torch.zeros(2, 2, 3, dtype=torch.int32)), on(torch.zeros(2, 2, dtype=torch.int32)),
               on(torch.zeros(2, 2, 4)))), "pi must"),
])
def test_binding_refuses(kw, match):
    with pytest.raises(SantaError, match=match):
        call(**kw)


@pytest.mark.parametrize("name", ["q", "page_table", "seq_lens", "cache_k", "cache_v", "cache_k_scale",
                                  "cache_v_scale", "out", "workspace", "device_status", "sel_ids"])
def test_binding_refuses_another_device(name, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i32 = torch.int32
    given = dict(q=on(torch.zeros(2, 4, 64)), page_table=on(torch.zeros(2, 2, dtype=i32)),
                 seq_lens=on(torch.zeros(2, dtype=i32)), out=on(torch.zeros(2, 4, 64)),
                 workspace=on(torch.zeros(8, dtype=torch.uint8)), device_status=on(torch.zeros(1, dtype=i32)))
    cache, ids = cpu_cache(), on(torch.zeros(2, 2, 3, dtype=i32))
    if name in given:
        given[name] = on(given[name], 1)
    elif name == "sel_ids":
        ids = on(ids, 1)
    else:
        setattr(cache, name[6:], on(getattr(cache, name[6:]), 1))
    sel = (ids, on(torch.zeros(2, 2, dtype=i32)), on(torch.zeros(2, 2, 3)))
    with pytest.raises(SantaError, match=name):
        call(cache=cache, sel=sel, **given)


def test_append_binding_refuses():
    d, x = 64, on(torch.zeros(3, 2, 64))
    i32 = torch.int32
    args = dict(q=x, k_new=x, v_new=x, cu_q=on(torch.zeros(2, dtype=i32)), cache=cpu_cache(),
                reps=on(torch.zeros(4, 2, d)), page_table=on(torch.zeros(1, 2, dtype=i32)),
                seq_lens=on(torch.zeros(1, dtype=i32)), rope=None, q_norm=None, k_norm=None, eps=1e-6,
                seq_lens_next=None, q_out=None, interleaved=False, device_status=None, stream=None)
    for kw, match in [
            (dict(cache=5), "Q8Cache or"), (dict(cache=(x,)), "Q8Cache or"),
            (dict(cache=(cpu_cache().k, cpu_cache().v)), "k_pool"),
            (dict(k_norm=on(torch.zeros(32))), "k_norm"),
            (dict(q_norm=on(torch.zeros(d, dtype=torch.bfloat16))), "q_norm"),
            (dict(q=None, q_norm=on(torch.zeros(d))), "q_norm without q"),
            (dict(k_new=on(torch.zeros(3, 2, d, dtype=torch.float16))), "k_new"),
            (dict(v_new=on(torch.zeros(3, 2, d, dtype=torch.bfloat16))), "v_new"),
            (dict(reps=on(torch.zeros(4, 1, d))), "reps")]:
        with pytest.raises(SantaError, match=match):
            binding._append_norm(**dict(args, **kw))


def test_read_binding_refuses():
    i32 = torch.int32
    pool = on(torch.zeros(3, 2, 64, 64))
    args = dict(cache=cpu_cache(), page_table=on(torch.zeros(1, 2, dtype=i32)),
                seq_lens=on(torch.zeros(1, dtype=i32)), k_out=pool, v_out=pool.clone(),
                dst_table=on(torch.zeros(1, 2, dtype=i32)), first=None, device_status=None, stream=None)
    for kw, match in [
            (dict(cache=None), "Q8Cache"), (dict(k_out=on(torch.zeros(3, 2, 64, 64, dtype=torch.float16))), "k_out"),
            (dict(v_out=on(torch.zeros(3, 2, 64, 64, dtype=torch.bfloat16))), "v_out"),
            (dict(k_out=on(torch.zeros(3, 2, 64, 128))), "k_out and v_out"),
            (dict(dst_table=on(torch.zeros(1, 3, dtype=i32))), "dst_table"),
            (dict(first=on(torch.zeros(2, dtype=i32))), "first")]:
        with pytest.raises(SantaError, match=match):
            binding._q8_read(**dict(args, **kw))


@pytest.mark.parametrize("call,name", [
    (c, n) for c, names in (("append", ["q", "k_new", "v_new", "cu_q", "reps", "page_table", "seq_lens", "rope",
                                        "q_norm", "k_norm", "seq_lens_next", "q_out", "device_status",
                                        "k_pool", "v_pool", "k_scale", "v_scale"]),
                            ("read", ["page_table", "dst_table", "seq_lens", "first", "k_out", "v_out",
                                      "device_status", "cache_k", "cache_v", "cache_k_scale",
                                      "cache_v_scale"])) for n in names])
def test_other_calls_refuse_another_device(call, name, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i32, d = torch.int32, 64
    cache = cpu_cache()
    parts = dict(k_pool="k", v_pool="v", k_scale="k_scale", v_scale="v_scale", cache_k="k", cache_v="v",
                 cache_k_scale="k_scale", cache_v_scale="v_scale")
    if name in parts:
        setattr(cache, parts[name], on(getattr(cache, parts[name]), 1))
    if call == "append":
        given = dict(q=on(torch.zeros(3, 2, d)), k_new=on(torch.zeros(3, 2, d)), v_new=on(torch.zeros(3, 2, d)),
                     cu_q=on(torch.zeros(2, dtype=i32)), reps=on(torch.zeros(4, 2, d)),
                     page_table=on(torch.zeros(1, 2, dtype=i32)), seq_lens=on(torch.zeros(1, dtype=i32)),
                     rope=on(torch.zeros(9, 64)), q_norm=on(torch.zeros(d)), k_norm=on(torch.zeros(d)),
                     seq_lens_next=on(torch.zeros(1, dtype=i32)), q_out=on(torch.zeros(3, 2, d)),
                     device_status=on(torch.zeros(1, dtype=i32)))
        rest = dict(cache=cache, eps=1e-6, interleaved=False, stream=None)
        f = binding._append_norm
    else:
        pool = torch.zeros(3, 2, 64, d)
        given = dict(page_table=on(torch.zeros(1, 2, dtype=i32)), dst_table=on(torch.zeros(1, 2, dtype=i32)),
                     seq_lens=on(torch.zeros(1, dtype=i32)), first=on(torch.zeros(1, dtype=i32)),
                     k_out=on(pool), v_out=on(pool.clone()), device_status=on(torch.zeros(1, dtype=i32)))
        rest = dict(cache=cache, stream=None)
        f = binding._q8_read
    if name in given:
        given[name] = on(given[name], 1)
    with pytest.raises(SantaError, match=f"^{name} is on"):
        f(**given, **rest)


@pytest.mark.parametrize("name", ["q", "reps", "page_table", "cache_k", "out", "sel_ids", "sel_count", "pi",
                                  "draw_ids", "workspace", "device_status"])
def test_sparse_steps_refuse_another_device(name, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i32 = torch.int32
    bufs = binding.DecodeBuffers(
        out=on(torch.zeros(2, 4, 64)), draw_ids=on(torch.zeros(2, 2, 3, dtype=i32)),
        sel_ids=on(torch.zeros(2, 2, 3, dtype=i32)), sel_count=on(torch.zeros(2, 2, dtype=i32)),
        pi=on(torch.zeros(2, 2, 3)), team_probs=None, workspace=on(torch.zeros(256, dtype=torch.uint8)),
        device_status=on(torch.zeros(1, dtype=i32)))
    cache = cpu_cache()
    given = dict(q=on(torch.zeros(2, 4, 64)), reps=on(torch.zeros(4, 2, 64)),
                 page_table=on(torch.zeros(2, 2, dtype=i32)), seq_lens=on(torch.zeros(2, dtype=i32)))
    if name in given:
        given[name] = on(given[name], 1)
    elif name == "cache_k":
        cache.k = on(cache.k, 1)
    else:
        setattr(bufs, name, on(getattr(bufs, name), 1))
    with pytest.raises(SantaError, match=f"^{name} is on"):
        binding._q8_sparse("santa_q8_decode", cache=cache, num_teams=3, softcap=0.0, window=0, bufs=bufs,
                           stream=None, **given)


def test_allocate_refuses_other_types():
    with pytest.raises(SantaError, match="int8 or float8"):
        santa.Q8Cache.allocate(1, 1, 64, 64, torch.uint8, device="cpu")
