"""8-bit paged caches of random rows, and 64-bit references of what is computed over them, written
from the definitions (torch, no code of the package)."""
import math

import torch

import sampled_sparse_decode_gb300 as santa

I8, E4M3 = torch.int8, torch.float8_e4m3fn
TOP = {I8: 127.0, E4M3: 448.0}
TINY = 2.0 ** -90


def quantise(x, dtype):
    """Codes and scales of fp32 rows x, each operation rounded to fp32."""
    s = x.abs().amax(-1).clamp(min=TINY)
    s = s / torch.full_like(s, TOP[dtype])      # torch multiplies by a number's rounded reciprocal
    y = x / s[..., None]
    return (y.round().to(I8) if dtype == I8 else y.to(E4M3)), s


def values64(codes, scale):
    """What rows of codes stand for, in 64 bits."""
    return codes.float().double() * scale.double()[..., None]


class Q8:
    """A Q8Cache with random rows for sequences of the given lengths on randomly placed pages.  Slots
    of no token hold bytes 0x7f (an e4m3 NaN, int8's largest) and NaN scales; table entries that no
    token reaches are out of range."""

    def __init__(self, lens, hkv, d, T, dtype, seed=0, spare=2, cap=None, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.T, self.hkv, self.d, self.dtype = list(lens), T, hkv, d, dtype
        caps = [max(1, -(-(L if cap is None else cap) // T)) for L in lens]
        P = sum(caps) + spare
        perm = torch.randperm(P, generator=g).int()
        self.table = torch.full((len(lens), max(caps)), 2**30, dtype=torch.int32)
        at = 0
        for b, c in enumerate(caps):
            self.table[b, :c] = perm[at:at + c]
            at += c
        shape = (P, hkv, T, d)
        parts = []
        for _ in range(2):
            codes = torch.full(shape, 0x7f, dtype=torch.uint8)
            scale = torch.full(shape[:3], math.nan)
            for b, L in enumerate(lens):
                for i in range(-(-L // T)):
                    m = min(T, L - i * T)
                    x = size * torch.randn(hkv, m, d, generator=g)
                    x *= torch.exp2(torch.randn(hkv, m, 1, generator=g))
                    c, s = quantise(x, dtype)
                    codes[self.table[b, i], :, :m] = c.view(torch.uint8)
                    scale[self.table[b, i], :, :m] = s
            parts += [codes.cuda().view(dtype), scale.cuda()]
        self.cache = santa.Q8Cache(parts[0], parts[2], parts[1], parts[3])
        self.table = self.table.cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.reps = torch.zeros(P, hkv, d, device="cuda")

    def tokens(self, which, b, n, start=0):
        """Tokens start .. n - 1 of sequence b as [hkv][n - start][d] float64."""
        pages = self.table[b, :-(-n // self.T)].long()
        codes, scale = getattr(self.cache, which), getattr(self.cache, which + "_scale")
        x = values64(codes.view(torch.uint8)[pages].view(self.dtype), scale[pages]).transpose(0, 1)
        return x.reshape(self.hkv, -1, self.d)[:, start:n]


def attend64(q, K, V, bias=None, cap=0.0):
    """q [Hq][d] over K, V [hkv][L][d] with bias [hkv][L] added to the scores.  Returns the output
    and its bound: the largest error that the arithmetic of the kernels allows (see `bound`)."""
    hq, d = q.shape
    hkv, L = K.shape[:2]
    if L == 0:
        return torch.zeros(hq, d, dtype=torch.float64, device=q.device), 0.0
    qi = q.double().view(hkv, hq // hkv, d)
    s = qi @ K.transpose(1, 2) / math.sqrt(d)
    if cap:
        s = cap * torch.tanh(s / cap)
    if bias is not None:
        s = s + bias[:, None]
    m = s.amax(-1, keepdim=True)
    p = torch.where(m == -math.inf, torch.zeros_like(s), torch.exp(s - m))
    z = p.sum(-1, keepdim=True)
    w = torch.where(z == 0, torch.zeros_like(p), p / z)
    out, mag = (w @ V).reshape(hq, d), (w @ V.abs()).reshape(hq, d)
    return out, bound(qi, K, s, mag, d, cap)


def bound(qi, K, s, mag, d, cap):
    """A score is a sum of d products in fp32 on the matrix units: at most d / 16 + 1 steps, each of
    which may cut 17 terms at 2^-24 of the largest (17 (d / 16 + 1) 2^-24 of the sum of magnitudes),
    of queries carried to 2^-22 of their largest element.  Its exponent is formed by a few operations
    that round to 2^-24 of it (8 taken), a tanh adds 2^-20 of the cap, and the exponential 2^-21.  A
    weight's error enters numerator and denominator; the sums of weights and of weighted values are
    fp32 again, over at most 2^5 tokens of a step at a time and then across steps (2^-18 taken), and a
    weight is carried to 2^-21 of the largest."""
    qk = (qi.abs() @ K.abs().transpose(1, 2)).amax(-1) / math.sqrt(d)
    qmax = (qi.abs().amax(-1, keepdim=True) * K.abs().sum(-1)[:, None]).amax(-1) / math.sqrt(d)
    fin = torch.where(torch.isfinite(s), s.abs(), torch.zeros_like(s)).amax(-1)
    ds = 17 * (d / 16 + 1) * 2.0**-24 * qk + 2.0**-22 * qmax + 8 * 2.0**-24 * fin + 2.0**-20 * cap
    rel = 2 * (ds + 2.0**-21) + 2.0**-18
    return rel.reshape(-1, 1) * mag + 2.0**-21 * mag.amax(-1, keepdim=True)


def close(got, want, tol):
    """Finite and within tol element by element; returns the worst excess ratio for the message."""
    err = (got.double() - want).abs()
    ok = bool(torch.isfinite(got).all()) and bool((err <= tol + 1e-300).all())
    assert ok, f"largest error {float(err.max()):.3g}, {float((err / (tol + 1e-300)).max()):.3g} of the bound"
