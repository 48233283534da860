"""How many bits of small weights and of small elements of a query reach the result over 8-bit caches:
what lies beside them in the same row or tile may be far larger."""
import math

import pytest
import torch

import sampled_sparse_decode_gb300 as santa
from q8_cases import E4M3, I8, Q8, attend64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 1), (128, 12, 2)])
@pytest.mark.parametrize("down,tol", [(10, 2.0**-18), (18, 2.0**-18), (24, 2.0**-17)])
@pytest.mark.parametrize("first", [True, False])
def test_small_weights_beside_a_large_one(kind, d, hq, hkv, down, tol, first):
    """Queries of zeros, so that every weight is its value's scale.  One token's scale is 2^down times the
    others', with a value in dimension 0 alone; the other dimensions hold the small weights' sums only, of
    one sign.

    Weights whose largest is scaled to 2^7 .. 2^8 are 2^(7 - down) here.  As two fp16 pieces, the second 2^11
    up, they carry 2^-22 of themselves down to 2^-14, and 2^-36 below (down = 24: 2^-19 of 2^-17).  Two
    products of 16 tokens cut 17 terms each at 2^-24 (2^-18.9); sums of tiles and pieces, a division and the
    64-bit result's fp32 take 2^-21."""
    lens = [32, 33, 96, 64, 500, 2, 31, 128] * 3
    c = Q8(lens, hkv, d, 64, kind, seed=down)
    g = torch.Generator().manual_seed(down)
    for b, L in enumerate(lens):
        pages = c.table[b, :-(-L // 64)].long()
        v = c.cache.v.view(torch.uint8)
        v[pages] = v[pages] & 0x7f                  # no signs; an e4m3 0x7f is a NaN and cut below
        if kind == E4M3:
            v[pages] = v[pages].clamp(max=0x7e)
        v[pages, :, :, 0] = 0
        c.cache.v_scale[pages] = (1 + torch.rand(len(pages), hkv, 64, generator=g)).cuda()
        at = 0 if first else L - 1
        strong = torch.zeros(d, dtype=torch.uint8, device="cuda")
        strong[0] = 127 if kind == I8 else 0x7e
        v[pages[at // 64], :, at % 64] = strong
        c.cache.v_scale[pages[at // 64], :, at % 64] *= 2.0**down
    q = torch.zeros(len(lens), hq, d, device="cuda")
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    for b, L in enumerate(lens):
        want = c.tokens("v", b, L).mean(1).repeat_interleave(hq // hkv, 0)
        over = float(((out[b].double() - want).abs() - tol * want).max())
        assert over <= 0, (b, L)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("up", [2.0**12, -2.0**20])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 1), (128, 12, 2)])
def test_small_elements_beside_a_large_one(kind, dtype, up, d, hq, hkv):
    """A query with one element far above the others, in a dimension where the keys are zeros.

    bf16 elements are fp16 numbers down to 2^-17 with the largest at 2^14 .. 2^15; of fp32 ones two pieces,
    the second 2^11 up, carry 2^-22 down to 2^-14: both hold at 2^-20 of the largest.  A score then has the
    cuts of d / 16 chained products (17 terms at 2^-24 each; one more for the sum of two chains) and 2^-22 of
    its products' magnitudes, and the rest is as in q8_cases.bound."""
    lens = [33, 100, 500, 2]
    c = Q8(lens, hkv, d, 64, kind, seed=3)
    c.cache.k.view(torch.uint8)[..., 5] = 0
    g = torch.Generator().manual_seed(1)
    q = torch.randn(len(lens), hq, d, generator=g).to(dtype).cuda()
    q[..., 5] = up
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    for b, L in enumerate(lens):
        K, V = c.tokens("k", b, L), c.tokens("v", b, L)
        want, _ = attend64(q[b], K, V)
        qi = q[b].double().view(hkv, hq // hkv, d)
        qk = (qi.abs() @ K.abs().transpose(1, 2)).amax(-1) / math.sqrt(d)
        ds = (17 * (d / 16 + 1) * 2.0**-24 + 2.0**-22 + 8 * 2.0**-24) * qk
        rel = (2 * (ds + 2.0**-21) + 2.0**-18).reshape(-1, 1)
        mag, _ = attend64(q[b], K, V.abs())
        tol = rel * mag + 2.0**-21 * mag.amax(-1, keepdim=True)
        worst = float(((out[b].double() - want).abs() / tol).max())
        assert worst <= 1, (b, L)


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 1), (128, 8, 2)])
def test_no_further_from_64_bits_than_fp32(kind, d, hq, hkv):
    """fp32 queries, scores of all sizes: a plain fp32 evaluation sums its d products in some order and
    rounds each sum; the kernel's distance from the 64-bit result (root mean square) is not more."""
    lens = [4000, 900, 77]
    c = Q8(lens, hkv, d, 64, kind, seed=4)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(len(lens), hq, d, generator=g).cuda()
    out = santa.santa_q8_dense_decode(q, c.cache, c.table, c.seq_lens)
    here, plain = [], []
    for b, L in enumerate(lens):
        K, V = c.tokens("k", b, L), c.tokens("v", b, L)
        want, _ = attend64(q[b], K, V)
        s = (q[b].view(hkv, -1, 1, d) * K.float()[:, None]).cumsum(-1)[..., -1] / math.sqrt(d)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        flat = (p[..., None] * V.float()[:, None]).cumsum(-2)[..., -1, :] / p.sum(-1, keepdim=True)
        here.append((out[b].double() - want).flatten())
        plain.append((flat.reshape(hq, d).double() - want).flatten())
    assert float(torch.cat(here).norm()) <= float(torch.cat(plain).norm())
