"""santa_append_norm refuses outputs that overlap each other or what the call reads (CPU: no address here is
ever read, every call is turned down by a check)."""
import ctypes

import pytest

from sampled_sparse_decode_gb300 import build as B
from sampled_sparse_decode_gb300.binding import _AppendChunkArgs, _AppendNormArgs

INVALID = 1
TOKENS, BATCH, HQ, HKV, D, T, TEAMS, PAGES, ROPE = 10, 2, 28, 4, 128, 128, 16, 64, 128
ROWS = PAGES * HKV * T


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(B.build())
    L.santa_append_norm.restype = ctypes.c_int
    L.santa_append_norm.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    return L


def sizes(bits):
    """Bytes of every buffer: bf16 tokens into an 8-bit cache or (16) a bf16 one."""
    pool = ROWS * D * bits // 8
    sz = dict(q_out=TOKENS * HQ * D * 2, k_pool=pool, v_pool=pool, k_scale=ROWS * 4, v_scale=ROWS * 4,
              reps=PAGES * HKV * D * 4, seq_lens_next=BATCH * 4, q=TOKENS * HQ * D * 2,
              k_new=TOKENS * HKV * D * 2, v_new=TOKENS * HKV * D * 2, cu_q=(BATCH + 1) * 4,
              page_table=BATCH * TEAMS * 4, seq_lens=BATCH * 4, rope=TEAMS * T * ROPE * 4, q_norm=D * 4,
              k_norm=D * 4)
    return sz if bits == 8 else {k: v for k, v in sz.items() if k not in ("k_scale", "v_scale")}


OUT = ["q_out", "k_pool", "v_pool", "k_scale", "v_scale", "reps", "seq_lens_next"]


def args(bits, **moved):
    """Buffers far from each other, but for those in `moved`."""
    chunk = dict(q_stride=HQ * D, k_stride=HKV * D, v_stride=HKV * D, rope_positions=1 << 20,
                 num_tokens=TOKENS, num_pages=PAGES, dtype=1, batch=BATCH, num_q_heads=HQ, num_kv_heads=HKV,
                 head_dim=D, team_size=T, max_teams=TEAMS, rope_dim=ROPE)
    a = _AppendNormArgs(chunk=_AppendChunkArgs(**chunk), cache_type=2 if bits == 8 else 1, eps=1e-6)
    for i, name in enumerate(sizes(bits)):
        at = moved.get(name, (i + 1) << 32)
        setattr(a.chunk if hasattr(a.chunk, name) else a, name, at)
    return a


def pairs():
    for bits in (8, 16):
        names = list(sizes(bits))
        for o in OUT:
            for other in names:
                if o in names and o != other and not (other in OUT and names.index(other) < names.index(o)):
                    yield bits, o, other


@pytest.mark.parametrize("bits,out,other", list(pairs()))
def test_overlaps_are_refused(lib, bits, out, other):
    sz = sizes(bits)
    base = 1 << 50
    for at in {base + (sz[out] - 1) // 16 * 16, base - (sz[other] - 1) // 16 * 16}:
        a = args(bits, **{out: base, other: at})
        assert lib.santa_append_norm(ctypes.addressof(a), None) == INVALID, at - base


def test_queries_in_place_only_row_for_row(lib):
    a = args(8, q=1 << 50, q_out=1 << 50)
    a.chunk.q_stride = HQ * D + 64
    assert lib.santa_append_norm(ctypes.addressof(a), None) == INVALID
    # queries in place do not allow the rest to overlap them
    a = args(8, q=1 << 50, q_out=1 << 50, k_scale=(1 << 50) + 16)
    assert lib.santa_append_norm(ctypes.addressof(a), None) == INVALID
    a = args(8, q=1 << 50, q_out=1 << 50, v_pool=(1 << 50) - 16)
    assert lib.santa_append_norm(ctypes.addressof(a), None) == INVALID


def test_rows_of_a_strided_product(lib):
    """Outputs between the rows that are read would pass; one that meets the last row does not."""
    a = args(8, k_new=1 << 50)
    a.chunk.k_stride = HKV * D + 512
    last = (1 << 50) + (TOKENS - 1) * a.chunk.k_stride * 2
    a.chunk.seq_lens_next = last + HKV * D * 2 - 4
    assert lib.santa_append_norm(ctypes.addressof(a), None) == INVALID
