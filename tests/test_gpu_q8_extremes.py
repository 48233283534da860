"""The ends of the ranges of the calls over 8-bit caches: many heads, the longest cache, the widest batch, codes of
any byte, queries of every size and non-finite ones."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from cache_cases import cu, rope_table
from q8_cases import E4M3, I8, Q8, attend64, close, values64
from test_gpu_append_norm import check, make, snapshot, target
from test_gpu_q8_attend import check_dense, check_listed, listed, queries, status_word

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype,d,hkv,hq", [(BF16, 64, 71, 71), (F32, 128, 40, 80)])
def test_many_heads(dtype, d, hkv, hq):
    c = Q8([300, 0, 65, 1], hkv, d, 64, I8, seed=1)
    q = queries(c, hq, dtype)
    check_dense(c, q, santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens))
    ids, count, pi = listed(c, 3, seed=1, order="any")
    out = santa.santa_q8_attend(q, c.cache, c.table, c.seq_lens, ids, count, pi)
    check_listed(c, q, out, ids, count, pi)


@pytest.mark.parametrize("kind", [None, I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_append_of_many_heads(dtype, kind):
    lens, new, hq, hkv, d, T = [60, 0], [9, 70], 71, 71, 64, 64
    c, cache = target(lens, new, hkv, d, T, dtype, kind, seed=1)
    q, k, v = make(4, sum(new), hq, hkv, d, dtype)
    w, rope, before = torch.linspace(0.5, 1.5, d).cuda(), rope_table(256, d), snapshot(c)
    q_out = torch.zeros(sum(new), hq, d, dtype=dtype, device="cuda")
    santa.santa_append_norm(q, k, v, cu(new), cache, c.reps, c.table, c.seq_lens, rope, q_norm=w, k_norm=w, eps=1e-5,
                            q_out=q_out)
    check(c, lens, new, q, k, v, rope, w, w, 1e-5, False, q_out, T, before)


@pytest.mark.parametrize("kind", [I8, E4M3])
def test_the_longest_cache(kind):
    """16384 pages of 128 tokens, from a pool of 90 (a page may stand in a table many times)."""
    P, T, d, teams = 90, 128, 64, 16384
    c = Q8([P * T], 1, d, T, kind, seed=1, spare=0)
    g = torch.Generator().manual_seed(1)
    table = torch.randint(0, P, (2, teams), generator=g).int().cuda()
    lens = torch.tensor([teams * T, teams * T - 77], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, d, generator=g).cuda()
    status = status_word()
    for window in (0, 1000000):
        out = santa.santa_q8_dense_decode(q, c.cache, table, lens, window=window, device_status=status)
        assert int(status) == 0
        for b in range(2):
            L = int(lens[b])
            K, V = (values64(x.view(torch.uint8)[table[b].long()].view(kind), s[table[b].long()]).reshape(1, -1, d)
                    for x, s in ((c.cache.k, c.cache.k_scale), (c.cache.v, c.cache.v_scale)))
            lo = max(0, L - window) if window else 0
            want, tol = attend64(q[b], K[:, lo:L], V[:, lo:L])
            # a warp adds up to 2^21 / 32 / 1216 tiles, pieces and parts after them: 2^7 roundings of 2^-24, in
            # the 2^-18 of the bound
            close(out[b], want, tol)


def test_the_widest_batch():
    """65535 sequences, most of them empty or of one token."""
    P, B, T, d = 40, 65535, 64, 64
    c = Q8([P * T], 1, d, T, I8, seed=1, spare=0)
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 4, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.5] = 0
    lens[0], lens[70], lens[40000], lens[-1] = 2 * T, 65, 2 * T - 1, 3
    table = torch.randint(0, P, (B, 2), generator=g).int().cuda()
    q = torch.randn(B, 2, d, generator=g).to(BF16).cuda()
    out = torch.full((B, 2, d), 9.0, device="cuda")
    status = status_word()
    santa.santa_q8_dense_decode(q, c.cache, table, lens.int().cuda(), out=out, device_status=status)
    assert int(status) == 0
    assert not out[(lens == 0).cuda()].any()
    K, V = (values64(x.view(torch.uint8).view(I8), s)[:, 0] for x, s in ((c.cache.k, c.cache.k_scale),
                                                                         (c.cache.v, c.cache.v_scale)))
    for n in (1, 2, 3):                        # all sequences of a length at once
        at = (lens == n).nonzero().flatten().cuda()
        k, v = K[table[at, 0].long(), :n], V[table[at, 0].long(), :n]
        s = torch.einsum("bhd,bnd->bhn", q[at].double(), k) / math.sqrt(d)
        w = torch.softmax(s, -1)
        want, mag = torch.einsum("bhn,bnd->bhd", w, v), torch.einsum("bhn,bnd->bhd", w, v.abs())
        qk = torch.einsum("bhd,bnd->bhn", q[at].double().abs(), k.abs()).amax(-1) / math.sqrt(d)
        ds = (17 * (d / 16 + 1) + 8) * 2.0**-24 * qk
        tol = (2 * (ds + 2.0**-21) + 2.0**-18)[..., None] * mag + 2.0**-21 * mag.amax(-1, keepdim=True)
        assert bool(((out[at].double() - want).abs() <= tol).all())
    for b in (0, 70, 40000):
        L = int(lens[b])
        k, v = (x[table[b].long()].reshape(1, -1, d)[:, :L] for x in (K, V))
        want, tol = attend64(q[b], k, v)
        close(out[b], want, tol)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_codes_of_any_byte(kind, dtype, d):
    """int8's -128 and e4m3's smallest and largest numbers, scales of either sign and of zero."""
    lens = [500, 33, 1]
    c = Q8(lens, 2, d, 64, kind, seed=1)
    g = torch.Generator().manual_seed(3)
    for x in (c.cache.k, c.cache.v):
        b = torch.randint(0, 256, tuple(x.shape), generator=g).to(torch.uint8)
        if kind == E4M3:
            b[(b & 0x7f) == 0x7f] = 0x01
        x.view(torch.uint8).copy_(b.cuda())
    for s, size in ((c.cache.k_scale, 2.0**-5 if kind == I8 else 2.0**-7), (c.cache.v_scale, 1.0)):
        y = size * torch.randn(s.shape, generator=g)
        y[torch.rand(y.shape, generator=g) < 0.1] = 0.0
        s.copy_(y.cuda())
    q = queries(c, 6, dtype, size=0.3)
    check_dense(c, q, santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens))
    out = [torch.zeros(tuple(c.cache.k.shape), dtype=F32, device="cuda") for _ in "kv"]
    santa.santa_q8_read(c.cache, c.table, c.seq_lens, *out, c.table)
    for b, L in enumerate(lens):
        for i in range(-(-L // 64)):
            p, m = int(c.table[b, i]), min(64, L - i * 64)
            for o, x, s in ((out[0], c.cache.k, c.cache.k_scale), (out[1], c.cache.v, c.cache.v_scale)):
                codes = x.view(torch.uint8)[p].view(kind).float()
                assert torch.equal(o[p, :, :m], (codes * s[p][..., None])[:, :m])


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype,d,hq,hkv", [(BF16, 128, 8, 2), (F32, 64, 3, 1)])
def test_queries_of_every_size(kind, dtype, d, hq, hkv):
    """Heads from 2^-120 to 2^107 over keys whose scales bring the scores back, the last to about 2^21."""
    e = [-120, -100, -60, -20, 20, 60, 100, 105]
    c = Q8([200] * len(e), hkv, d, 64, kind, seed=2)
    q = queries(c, hq, F32, seed=1).clamp(-3.9, 3.9)
    for b, x in enumerate(e):
        q[b] *= 2.0**x
        c.cache.k_scale[c.table[b, :4].long()] *= 2.0**max(-x, -90)
    if dtype == BF16:
        q = q.to(BF16)
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens, softcap=0.0)
    check_dense(c, q, out)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype,d,hq,hkv", [(BF16, 128, 8, 2), (F32, 64, 3, 1)])
@pytest.mark.parametrize("top", [2.0**15, 2.0**20, 2.0**25])
def test_scores_of_the_largest_size(kind, dtype, d, hq, hkv, top):
    """Largest scores up to the stated 2^25: the value of the largest where it stands out.  A score's exponent
    is formed from the exact product less the rounded reference, and may lie half a step of the reference above
    it, which is 2 for one of 2^25 log2(e): weights stay below 2^8 2^2, and fp16 ends at 65504."""
    lens = [200, 3000]
    c = Q8(lens, hkv, d, 64, kind, seed=2)
    q = queries(c, hq, dtype, seed=1)
    for b, L in enumerate(lens):
        qk = (q[b].double().view(hkv, -1, d) @ c.tokens("k", b, L).transpose(1, 2)).abs().amax() / math.sqrt(d)
        c.cache.k_scale[c.table[b, :-(-L // 64)].long()] *= float(0.99 * top / qk)
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    assert bool(torch.isfinite(out).all())
    for b, L in enumerate(lens):
        K, V = c.tokens("k", b, L), c.tokens("v", b, L)
        want, _ = attend64(q[b], K, V)
        # heads whose largest score stands out by more than the sum's rounding (17 (d / 16 + 1) + 8 steps)
        qi = q[b].double().view(hkv, -1, d)
        s = (qi @ K.transpose(1, 2) / math.sqrt(d)).reshape(hq, L).topk(2, -1).values
        slack = 2 * (17 * (d / 16 + 1) + 8) * 2.0**-24 * (qi.abs() @ K.abs().transpose(1, 2)).amax(-1) / math.sqrt(d)
        clear = s[:, 0] - s[:, 1] > slack.reshape(hq) + 40
        assert bool(clear.any())
        err = (out[b].double() - want).abs() / want.abs().amax(-1, keepdim=True)
        assert float(err[clear].amax()) <= 2.0**-18


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_non_finite_queries_stay_with_their_head(bad, dtype, d):
    c = Q8([700, 40], 2, d, 64, I8, seed=2)
    q = queries(c, 8, dtype)
    want = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    hurt = q.clone()
    hurt[0, 5, 3] = bad
    out = santa.santa_q8_dense_decode(hurt, c.cache, c.table, c.seq_lens)
    assert bool(torch.isnan(out[0, 5]).all())
    keep = torch.ones(2, 8, dtype=torch.bool, device="cuda")
    keep[0, 5] = False
    # a tile's references are raised for all heads at once: equal up to rounding
    assert bool(torch.isfinite(out[keep]).all())
    assert bool(((out - want)[keep].abs() <= 2.0**-17 * want.abs().amax()).all())
