"""santa_append_norm against 64-bit references: norms, rotations and 8-bit rows at page borders, ragged
and padded chunks, strided inputs, non-finite and tiny rows, equality with santa_append_chunk where
both can do it, bad lengths and pages, and independence of how tokens are divided among calls."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from sampled_sparse_decode_gb300.binding import DEV_BAD_PAGE, DEV_BAD_SEQLEN
from cache_cases import Cache, cu, rope_table, rotate64
from q8_cases import E4M3, I8, Q8, TOP, quantise, values64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = {F32: 2.0**-24, BF16: 2.0**-8}   # half a step, relative
# A norm: 16 squares in a chain and 4 shuffle sums, the mean and eps (at most 22 roundings of a sum of
# positive terms, half of them under the root), the root, two products; a rotation: products and sum.
NORM = (11 + 1 + 2 + 2) * 2.0**-24


def norm64(x, w, eps):
    x = x.double()
    return x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def make(seed, n, hq, hkv, d, dtype, strided=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, hq + 2 * hkv, d, generator=g) * torch.exp2(torch.randn(n, hq + 2 * hkv, 1, generator=g))
    q, k, v = x.to(dtype).cuda().split([hq, hkv, hkv], 1)
    return (q, k, v) if strided else (q.contiguous(), k.contiguous(), v.contiguous())


def target(lens, new, hkv, d, T, dtype, kind, seed, cap=None):
    """A cache holding `lens` tokens with room for `new` more: (object, what the call takes)."""
    cap = cap or max(L + m for L, m in zip(lens, new))
    if kind is None:
        c = Cache(lens, hkv, d, T, dtype, seed=seed, cap=cap)
        return c, (c.k, c.v)
    c = Q8(lens, hkv, d, T, kind, seed=seed, cap=cap)
    return c, c.cache


def snapshot(c):
    ts = (c.k, c.v) if isinstance(c, Cache) else (c.cache.k.view(torch.uint8), c.cache.v.view(torch.uint8),
                                                  c.cache.k_scale, c.cache.v_scale)
    return [t.clone() for t in ts]


def stored(c, which, page, slots):
    """Rows of a page in 64 bits, [hkv][slots][d]."""
    if isinstance(c, Cache):
        return getattr(c, which)[page, :, slots].double()
    codes = getattr(c.cache, which).view(torch.uint8)[page, :, slots].view(c.dtype)
    return values64(codes, getattr(c.cache, which + "_scale")[page, :, slots])


def check(c, lens, new, q, k, v, rope, qn, kn, eps, inter, q_out, T, before, lead=0):
    dtype, kind = q.dtype, None if isinstance(c, Cache) else c.dtype
    touched = torch.zeros(c.reps.shape[0], T, dtype=torch.bool, device="cuda")
    at = lead
    for b, (L, m) in enumerate(zip(lens, new)):
        rows = rope[L:L + m] if rope is not None else torch.zeros(m, 0, device="cuda")
        sl = slice(at, at + m)
        at += m
        yq, mq = rotate64(norm64(q[sl], qn, eps), rows, inter)
        tol = NORM * mq + EPS[dtype] * yq.abs() * (1 + 2.0**-7)
        assert bool(((q_out[sl].double() - yq).abs() <= tol).all())
        yk, mk = rotate64(norm64(k[sl], kn, eps), rows, inter)
        for i in range(m):
            p, slot = int(c.table[b, (L + i) // T]), (L + i) % T
            touched[p, slot] = True
            for which, y, mag in (("k", yk[i], NORM * mk[i]), ("v", v[sl][i].double(), 0 * mk[i])):
                got = stored(c, which, p, slice(slot, slot + 1))[:, 0]
                if kind is None:
                    tol = mag + EPS[dtype] * y.abs() * (1 + 2.0**-7)
                else:
                    s = getattr(c.cache, which + "_scale")[p, :, slot].double()
                    amax = y.abs().amax(-1)
                    # the largest element's error, and the quotient's rounding
                    ds = mag.amax(-1) / TOP[kind] + s * 2.0**-23
                    assert bool(((s - amax / TOP[kind]).abs() <= ds).all())
                    # half a step of the code, an element's own error, the quotient's rounding
                    half = (s[:, None] / 2 if kind == I8 else
                            torch.maximum(y.abs() * 2.0**-4, s[:, None] * 2.0**-10))
                    tol = half * (1 + 2.0**-14) + mag * 1.1 + y.abs() * 2.0**-22
                assert bool(((got - y).abs() <= tol).all()), (which, b, i)
    # nothing else was written
    now = snapshot(c)
    for old, new_ in zip(before, now):
        keep = ~touched[:, None].expand(-1, old.shape[1], -1)
        a, b_ = old[keep], new_[keep]
        assert torch.equal(a.view(torch.uint8) if a.dtype != torch.float32 else a.view(torch.int32),
                           b_.view(torch.uint8) if b_.dtype != torch.float32 else b_.view(torch.int32))
    # representatives: c s rounded, at most 16 + 16 additions, a division
    for b, (L, m) in enumerate(zip(lens, new)):
        for team in range(L // T, -(-(L + m) // T)) if m else ():
            p, fill = int(c.table[b, team]), min(T, L + m - team * T)
            rows = stored(c, "k", p, slice(0, fill))
            tol = 36 * 2.0**-24 * rows.abs().mean(1)
            assert bool(((c.reps[p].double() - rows.mean(1)).abs() <= tol).all())


SHAPES = [
    # lens, new, hq, hkv, d, T, rope, interleaved, pad
    ([0], [1], 1, 1, 64, 64, 64, False, 0),
    ([63, 64, 0, 127], [1, 1, 1, 1], 7, 1, 128, 64, 128, False, 0),
    ([5, 0, 200], [130, 0, 57], 8, 2, 128, 128, 64, True, 3),
    ([0, 1, 127, 128], [128, 127, 2, 129], 5, 5, 64, 128, 16, True, 0),
    ([17, 3], [300, 64], 6, 3, 64, 64, 32, False, 9),
    ([100], [33], 9, 1, 128, 64, 0, False, 0),
    ([0] * 70, [(7 * i) % 13 for i in range(70)], 2, 2, 64, 64, 64, True, 1),
]


@pytest.mark.parametrize("kind", [None, I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_append_matches_reference(case, dtype, kind):
    lens, new, hq, hkv, d, T, R, inter, pad = SHAPES[case]
    c, cache = target(lens, new, hkv, d, T, dtype, kind, seed=case)
    n = sum(new) + pad
    q, k, v = make(case + 50, n, hq, hkv, d, dtype)
    g = torch.Generator().manual_seed(case)
    qn, kn = (1 + 0.3 * torch.randn(2, d, generator=g)).cuda().unbind(0)
    qn, kn = qn.contiguous(), kn.contiguous()
    if case == 1:
        qn = None
    if case == 2:
        kn = None
    rope = rope_table(512, R) if R else None
    nxt = torch.zeros_like(c.seq_lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((n, hq, d), 7.0, dtype=dtype, device="cuda")
    before = snapshot(c)
    santa.santa_append_norm(q, k, v, cu(new), cache, c.reps, c.table, c.seq_lens, rope, q_norm=qn,
                            k_norm=kn, eps=1e-5, seq_lens_next=nxt, q_out=q_out,
                            interleaved=inter, device_status=status)
    assert int(status) == 0
    assert nxt.tolist() == [L + m for L, m in zip(lens, new)]
    assert bool((q_out[sum(new):] == 7.0).all())
    check(c, lens, new, q, k, v, rope, qn, kn, 1e-5, inter, q_out, T, before)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_without_norms_it_is_append_chunk(dtype):
    lens, new = [100, 0, 64], [77, 129, 1]
    q, k, v = make(1, sum(new), 6, 2, 128, dtype)
    rope = rope_table(256, 128)
    outs = []
    for f in ("chunk", "norm"):
        c, cache = target(lens, new, 2, 128, 64, dtype, None, seed=4)
        args = (c.reps, c.table, c.seq_lens, rope)
        qo = (santa.santa_append_chunk(q, k, v, cu(new), *cache, *args) if f == "chunk" else
              santa.santa_append_norm(q, k, v, cu(new), cache, *args))
        outs.append((qo, c.k, c.v, c.reps))
    for a, b in zip(*outs):
        assert torch.equal(a.nan_to_num(nan=9.0), b.nan_to_num(nan=9.0))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,T", [(64, 64), (128, 128)])
def test_representatives_are_build_reps_of_the_cache(d, T, dtype):
    lens, new = [30, 0], [2 * T, T + 5]
    c, cache = target(lens, new, 2, d, T, dtype, None, seed=2)
    q, k, v = make(3, sum(new), 4, 2, d, dtype)
    w = torch.linspace(0.5, 1.5, d).cuda()
    santa.santa_append_norm(q, k, v, cu(new), cache, c.reps, c.table, c.seq_lens, rope_table(512, d),
                            q_norm=w, k_norm=w)
    fill = torch.zeros(c.k.shape[0], dtype=torch.int32, device="cuda")
    for b in range(2):
        for i in range(-(-(lens[b] + new[b]) // T)):
            fill[c.table[b, i]] = min(T, lens[b] + new[b] - i * T)
    assert torch.equal(c.reps, santa.santa_build_reps(c.k, fill))


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_codes_are_those_of_any_fp32_program(kind, dtype):
    """Without norms every operation is one that torch rounds alike: equal codes and scales, with
    ties, rows of zeros, tiny and huge rows among them."""
    T, hkv, d, n = 64, 2, 64, 150
    c, cache = target([10], [n], hkv, d, T, dtype, kind, seed=1)
    _, k, v = make(9, n, 2, hkv, d, dtype, strided=False)
    k[3], v[5] = 0.0, 0.0
    k[7] *= 2.0**-100
    v[8] *= 2.0**-110
    k[9] *= 2.0**60
    v[10] = torch.where(v[10] > 0, 3e38, -2e38)
    v[11] = torch.arange(64, device="cuda") * 2.0 - 63.5        # quotients at half codes
    v[11, :, 0] = 127.0 if kind == I8 else 448.0
    santa.santa_append_norm(None, k, v, cu([n]), cache, c.reps, c.table, c.seq_lens)
    pos = torch.arange(10, 10 + n, device="cuda")
    page, slot = c.table[0].long()[pos // T], pos % T
    for x, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        want, s = quantise(x.float(), kind)
        assert torch.equal(scale[page, :, slot], s)
        assert torch.equal(codes.view(torch.uint8)[page, :, slot], want.view(torch.uint8))


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_non_finite_rows_stay_by_themselves(kind, bad):
    T, n = 64, 40
    c, cache = target([0], [n], 1, 128, T, BF16, kind, seed=1)
    q, k, v = make(4, n, 2, 1, 128, BF16, strided=False)
    k[5, 0, 17], v[9, 0, 127], q[3, 1, 0] = bad, bad, bad
    w = torch.ones(128, device="cuda")
    qo = santa.santa_append_norm(q, k, v, cu([n]), cache, c.reps, c.table, c.seq_lens,
                                 rope_table(64, 128), q_norm=w, k_norm=w)
    p = int(c.table[0, 0])
    for scale, codes, row in ((cache.k_scale, cache.k, 5), (cache.v_scale, cache.v, 9)):
        s = scale[p, 0, :n]
        assert bool(torch.isnan(s[row])) and bool(torch.isfinite(s[torch.arange(n) != row]).all())
        assert not codes.view(torch.uint8)[p, 0, row].any()
    fin = torch.isfinite(qo)
    fin[3, 1] = True
    assert bool(fin.all())


@pytest.mark.parametrize("kind", [None, I8, E4M3])
def test_one_call_or_many(kind):
    T, total = 64, 150
    q, k, v = make(6, total, 4, 2, 128, BF16)
    rope, w = rope_table(512, 128), torch.linspace(0.5, 2, 128).cuda()
    got = []
    for sizes in ([150], [1] * 150, [63, 1, 1, 64, 21]):
        c, cache = target([37], [total], 2, 128, T, BF16, kind, seed=8)
        at, lens, outs = 0, c.seq_lens, []
        # the earlier tokens' representatives are those of the cache
        for m in sizes:
            nxt = torch.empty_like(lens)
            sl = slice(at, at + m)
            outs.append(santa.santa_append_norm(q[sl], k[sl], v[sl], cu([m]), cache, c.reps,
                                                c.table, lens, rope, q_norm=w, k_norm=w,
                                                seq_lens_next=nxt))
            at, lens = at + m, nxt
        got.append([torch.cat(outs), *snapshot(c), c.reps])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a.nan_to_num(nan=5.0), b.nan_to_num(nan=5.0))


def test_queries_in_place_and_default_output():
    c, cache = target([0, 3], [5, 60], 2, 64, 64, BF16, I8, seed=8)
    q, k, v = make(6, 70, 4, 2, 64, BF16, strided=False)
    w, rope = torch.linspace(0.5, 2, 64).cuda(), rope_table(128, 64)
    args = (k, v, cu([5, 60]), cache, c.reps, c.table, c.seq_lens, rope)
    out = santa.santa_append_norm(q, *args, q_norm=w)
    assert not out[65:].any()
    tail = q[65:].clone()
    same = santa.santa_append_norm(q, *args, q_norm=w, q_out=q)
    assert same is q and torch.equal(q[:65], out[:65]) and torch.equal(q[65:], tail)


@pytest.mark.parametrize("kind", [None, I8])
def test_bad_lengths_and_pages_are_skipped(kind):
    T, new = 64, [10, 10, 10, 10]
    c, cache = target([5, 5, 5, 60], new, 1, 64, T, F32, kind, seed=3, cap=128)
    q, k, v = make(2, 40, 1, 1, 64, F32)
    c.seq_lens[0], c.seq_lens[1] = -1, 2 * T - 9
    c.table[3, 1] = c.reps.shape[0]
    before, status = snapshot(c), torch.zeros(1, dtype=torch.int32, device="cuda")
    reps = c.reps.clone()
    q_out = torch.full((40, 1, 64), 7.0, device="cuda")
    nxt = torch.full((4,), -5, dtype=torch.int32, device="cuda")
    santa.santa_append_norm(q, k, v, cu(new), cache, c.reps, c.table, c.seq_lens, q_norm=None,
                            q_out=q_out, seq_lens_next=nxt, device_status=status)
    assert int(status) == DEV_BAD_SEQLEN | DEV_BAD_PAGE
    assert nxt.tolist() == [-5, -5, 15, 70]
    assert bool((q_out[:20] == 7.0).all()) and not bool((q_out[20:] == 7.0).any())
    changed = {int(c.table[2, 0]), int(c.table[3, 0])}
    for p in range(c.reps.shape[0]):
        for a, b in zip(before, snapshot(c)):
            same = torch.equal(a[p].nan_to_num(nan=5.0), b[p].nan_to_num(nan=5.0))
            assert same == (p not in changed)
        assert torch.equal(reps[p], c.reps[p]) == (p not in changed)


def test_bad_bounds_touch_nothing_outside():
    c, cache = target([0, 0], [4, 4], 1, 64, 64, BF16, E4M3, seed=3)
    q, k, v = make(2, 8, 2, 1, 64, BF16)
    for bounds in ([0, 9, 8], [-1, 4, 8], [5, 3, 8], [0, 4, 2**31 - 1]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        santa.santa_append_norm(q, k, v, torch.tensor(bounds, dtype=torch.int32, device="cuda"),
                                cache, c.reps, c.table, c.seq_lens, device_status=status)
        assert int(status) & DEV_BAD_SEQLEN


def test_empty_chunk_copies_lengths():
    c, cache = target([3, 70], [0, 0], 1, 64, 64, BF16, I8, seed=3)
    nxt, before = torch.zeros_like(c.seq_lens), snapshot(c)
    x = torch.zeros(0, 1, 64, dtype=BF16, device="cuda")
    santa.santa_append_norm(x, x, x, cu([0, 0]), cache, c.reps, c.table, c.seq_lens,
                            seq_lens_next=nxt)
    assert nxt.tolist() == [3, 70]
    for a, b in zip(before, snapshot(c)):
        assert torch.equal(a.nan_to_num(nan=5.0), b.nan_to_num(nan=5.0))


def test_replayed_for_other_lengths():
    c, cache = target([10, 90], [30, 30], 2, 128, 64, BF16, E4M3, seed=5)
    q, k, v = make(7, 8, 4, 2, 128, BF16, strided=False)
    w, rope = torch.linspace(0.5, 2, 128).cuda(), rope_table(256, 128)
    nxt, bounds = torch.zeros_like(c.seq_lens), cu([3, 5])
    h = santa.santa_append_norm_prepared(q, k, v, bounds, cache, c.reps, c.table, c.seq_lens, rope,
                                         q_norm=w, k_norm=w, seq_lens_next=nxt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        h.run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = h.run()
    torch.cuda.synchronize()
    other, other_cache = target([10, 90], [30, 30], 2, 128, 64, BF16, E4M3, seed=5)
    for lens, new in (([13, 90], [0, 8]), ([20, 63], [7, 1])):
        other.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.seq_lens.copy_(other.seq_lens)
        bounds.copy_(cu(new))
        graph.replay()
        torch.cuda.synchronize()
        want = santa.santa_append_norm(q, k, v, cu(new), other_cache, other.reps, other.table,
                                       other.seq_lens, rope, q_norm=w, k_norm=w)
        assert torch.equal(out, want)
        assert nxt.tolist() == [L + m for L, m in zip(lens, new)]
        for b, (L, m) in enumerate(zip(lens, new)):
            for i in range(m):
                p, slot = int(c.table[b, (L + i) // 64]), (L + i) % 64
                for t, o in zip(snapshot(c), snapshot(other)):
                    assert torch.equal(t[p, :, slot], o[p, :, slot])
