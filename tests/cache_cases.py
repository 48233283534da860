"""Ragged paged-cache cases and 64-bit references of the chunk append, the chunk attention and
the top-k selection, written from their definitions (torch float64, no code of the package)."""
import math

import torch


class Cache:
    """A paged cache of random tokens: k_pool, v_pool, page table and lengths on the GPU.  Slots
    that hold no token of a sequence carry `stale`."""

    def __init__(self, lens, hkv, d, T, dtype, seed=0, spare=2, cap=None, stale=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.T, self.hkv, self.d, self.dtype = list(lens), T, hkv, d, dtype
        caps = [max(1, -(-(L if cap is None else cap) // T)) for L in lens]
        P = sum(caps) + spare
        perm = torch.randperm(P, generator=g).int()
        # table entries that no token reaches are out of range on purpose
        self.table = torch.full((len(lens), max(caps)), 2**30, dtype=torch.int32)
        at = 0
        for b, c in enumerate(caps):
            self.table[b, :c] = perm[at:at + c]
            at += c
        k = torch.full((P, hkv, T, d), stale).to(dtype)
        v = torch.full((P, hkv, T, d), stale).to(dtype)
        for b, L in enumerate(lens):
            for i in range(-(-L // T)):
                m = min(T, L - i * T)
                k[self.table[b, i], :, :m] = torch.randn(hkv, m, d, generator=g).to(dtype)
                v[self.table[b, i], :, :m] = torch.randn(hkv, m, d, generator=g).to(dtype)
        self.k, self.v = k.cuda(), v.cuda()
        self.table_cpu, self.table = self.table, self.table.cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.reps = torch.zeros(P, hkv, d, device="cuda")
        self.fill = torch.zeros(P, dtype=torch.int32)
        for b, L in enumerate(lens):
            for i in range(-(-L // T)):
                self.fill[self.table_cpu[b, i]] = min(T, L - i * T)
        self.fill = self.fill.cuda()

    def tokens(self, pool, b, n):
        """The first n tokens of sequence b, [hkv][n][d] float64."""
        pages = self.table[b, :-(-n // self.T)].long()
        x = pool[pages].double().transpose(0, 1)
        return x.reshape(self.hkv, -1, self.d)[:, :n]


def cu(new, lead=0):
    out = [lead]
    for m in new:
        out.append(out[-1] + m)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def rope_table(positions, rope_dim, theta=10000.0):
    half = rope_dim // 2
    f = theta ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def rotate64(x, rows, interleaved):
    """x [n][H][d] rotated by table rows [n][R] in float64, and the sum of the magnitudes of the
    two products behind every element (for the rounding bound)."""
    x = x.double()
    half = rows.shape[1] // 2
    c, s = rows[:, None, :half].double(), rows[:, None, half:].double()
    ia = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else half)
    a, b = x[..., ia], x[..., ib]
    y, mag = x.clone(), x.abs()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return y, mag


def attend64(q, K, V, see):
    """q [n][Hq][d] over K, V [hkv][L][d]; row i sees the first see[i] tokens.  Returns the
    output, the same attention over |V|, and the largest sum |q||k| / sqrt(d) of each row."""
    n, hq, d = q.shape
    hkv = K.shape[0]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    mag, qk = torch.zeros_like(out), torch.zeros(n, hq, 1, dtype=torch.float64, device=q.device)
    for i in range(n):
        L = int(see[i])
        qi = q[i].double().view(hkv, hq // hkv, d)
        k, v = K[:, :L], V[:, :L]
        s = qi @ k.transpose(1, 2) / math.sqrt(d)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        w = torch.where(z == 0, torch.zeros_like(p), p / z)
        out[i] = (w @ v).reshape(hq, d)
        mag[i] = (w @ v.abs()).reshape(hq, d)
        qk[i] = (qi.abs() @ k.abs().transpose(1, 2) / math.sqrt(d)).amax(-1).reshape(hq, 1)
    return out, mag, qk


def best64(q, reps, k):
    """Team indices [min(k, n)] ascending: largest max_g q_g . rep_i, ties to the lower index."""
    s = (q.double() @ reps.double().T).amax(0).tolist()
    s = [-math.inf if x != x else x for x in s]
    return sorted(sorted(range(len(s)), key=lambda i: (-s[i], i))[:k])
