"""Cases of the paged-cache operators: chunk append with rotation, chunk attention, top-k decode.

``own`` false computes each operator in plain torch operations; ``own`` true calls the
package's entry points.  Both take the state that ``prepare`` makes and write the same
buffers (the cache is updated in place, as a serving loop does).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _ints(text):
    """"4,7x3" -> [4, 7, 7, 7]"""
    out = []
    for part in str(text).split(","):
        if "x" in part:
            v, n = part.split("x")
            out += [int(v)] * int(n)
        else:
            out.append(int(part))
    return out


def _text(values):
    return ",".join(str(v) for v in values)


def listed():
    return [
        # one generated token for each of 8 sequences deep in a 32K context: the append of a
        # decode step, all latency
        dict(name="append_step_b8", op="append", dtype="bf16", hq=28, hkv=4, d=128, T=128,
             ctx="32000,32383,31744,32767,29000,32640,30001,32255", new="1x8", rope=128,
             style="half", pad=0),
        # prompts of different lengths arriving together on top of earlier turns, fp32 cache,
        # interleaved pairs on half of the head, padded to a multiple of 64 tokens
        dict(name="append_ragged_f32", op="append", dtype="f32", hq=16, hkv=2, d=64, T=64,
             ctx="0,777,64,5,1023,0,4096,310", new="1,300,64,63,129,700,2,45", rope=32,
             style="interleaved", pad=40),
        # a full prefill batch: 8 prompts of 4096 tokens from an empty cache
        dict(name="append_prefill_b8_4k", op="append", dtype="bf16", hq=32, hkv=8, d=128, T=128,
             ctx="0x8", new="4096x8", rope=128, style="half", pad=0),
        # the first chunk of a short question: one sequence, 33 tokens after 100 cached ones
        dict(name="chunk_short_b1", op="chunk", dtype="bf16", hq=28, hkv=4, d=128, T=128,
             ctx="100", new="33", pad=0),
        # checking 4 drafted tokens of 16 sequences against 32K of context: cache-bound
        dict(name="chunk_verify_b16_32k", op="chunk", dtype="bf16", hq=32, hkv=8, d=128, T=128,
             ctx="32764x16", new="4x16", pad=0),
        # one 2048-token chunk of a long prompt, 32K already cached
        dict(name="chunk_2k_on_32k", op="chunk", dtype="bf16", hq=28, hkv=4, d=128, T=128,
             ctx="32768", new="2048", pad=0),
        # prefill of a batch of ragged prompts from an empty cache, padded
        dict(name="chunk_prefill_ragged", op="chunk", dtype="bf16", hq=32, hkv=8, d=128, T=128,
             ctx="0x6", new="8192,4097,1,2500,777,6001", pad=16),
        # fp32 cache, small heads, mixed prompts and single tokens in one batch
        dict(name="chunk_mixed_f32", op="chunk", dtype="f32", hq=8, hkv=2, d=64, T=64,
             ctx="2000,0,511,4095", new="1,513,64,1", pad=0),
        # the sparse decode step of one sequence at 32K, 31 of 256 teams
        dict(name="topk_32k_b1_k31", op="topk", dtype="bf16", hq=28, hkv=4, d=128, T=128,
             ctx="32768", k=31),
        # 16 sequences at 32K over a shared pool
        dict(name="topk_32k_b16_k32", op="topk", dtype="bf16", hq=32, hkv=8, d=128, T=128,
             ctx="32768x8,20000,31000,32000,1000,32700,12345,127,30001", k=32),
        # long context: 4 sequences of 128K tokens, 64 of 1024 teams
        dict(name="topk_128k_b4_k64", op="topk", dtype="bf16", hq=28, hkv=4, d=128, T=128,
             ctx="131072x3,100001", k=64),
        # small fp32 cache, 64-token teams
        dict(name="topk_2k_f32_k8", op="topk", dtype="f32", hq=2, hkv=1, d=64, T=64,
             ctx="2048,1999,3", k=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "chunk", "topk"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    T = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    c = dict(op=op, dtype=dtype, hq=hkv * group, hkv=hkv, d=d, T=T)
    if op == "topk":
        batch = _log(rng, 1, 16)
        top = min(131072, 524288 // batch)
        c["ctx"] = _text(_log(rng, 1, top) for _ in range(batch))
        c["k"] = _log(rng, 1, 128)
        return c
    batch = _log(rng, 1, 16)
    if op == "append":
        c["new"] = _text(_log(rng, 1, 16384 // batch) for _ in range(batch))
        c["ctx"] = _text(rng.choice([0, _log(rng, 1, 131072 // batch)]) for _ in range(batch))
        c["rope"] = rng.choice([d, d, d // 2, 16])
        c["style"] = rng.choice(["half", "interleaved"])
    else:
        # the largest listed chunk has about 2e9 visible (head, query, key) triples at d = 128
        new = [_log(rng, 1, (8192 if dtype == "bf16" else 1024) // batch) for _ in range(batch)]
        room = (1.0e9 if dtype == "bf16" else 6.0e7) / (c["hq"] * sum(new))
        ctx = [rng.choice([0, _log(rng, 1, max(1, min(65536, int(room))))]) for _ in range(batch)]
        c["new"], c["ctx"] = _text(new), _text(ctx)
    c["pad"] = rng.choice([0, 0, rng.randint(1, 64)])
    return c


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d, T = case["hq"], case["hkv"], case["d"], case["T"]
    ctx = _ints(case["ctx"])
    if case["op"] == "topk":
        # representatives, page ids, the chosen teams' K and V, q and the results
        n = [-(-L // T) for L in ctx]
        toks = sum(min(L, min(case["k"], -(-L // T)) * T) for L in ctx)
        b = sum(n) * (hkv * d * 4 + 4) + toks * hkv * 2 * d * es
        b += len(ctx) * (hq * d * (es + 4) + 4 + hkv * (case["k"] + 1) * 4)
        return {"bytes": b, "flops": 2 * d * hq * sum(n) + 4 * d * hq * toks}
    new = _ints(case["new"])
    tok, batch = sum(new), len(new)
    if case["op"] == "append":
        # the new rows in and out, the table rows, the earlier rows of a page that is already
        # begun (its mean is needed), the touched representatives, page ids and lengths
        old = sum(L % T for L, m in zip(ctx, new) if m)
        pages = sum(-(-(L % T + m) // T) for L, m in zip(ctx, new))
        b = 2 * tok * (hq + 2 * hkv) * d * es + tok * case["rope"] * 4 + old * hkv * d * es
        b += pages * (hkv * d * 4 + 4) + batch * 12
        f = tok * (hq + hkv) * case["rope"] * 3 + (old + tok) * hkv * d
        return {"bytes": b, "flops": f}
    total = [L + m for L, m in zip(ctx, new)]
    seen = sum(m * L + m * (m + 1) // 2 for L, m in zip(ctx, new))
    b = 2 * tok * hq * d * es + sum(total) * hkv * 2 * d * es
    b += sum(-(-L // T) for L in total) * 4 + batch * 8
    return {"bytes": b, "flops": 4 * d * hq * seen}


# ---------------------------------------------------------------- inputs

def _mixture_keys(gen, lens, hkv, d):
    """Keys in runs that share one of 64 component means, as contexts that stay on a topic for
    a while give: one [hkv][L][d] tensor for each sequence, and the means [B][hkv][64][d]."""
    means = torch.randn(len(lens), hkv, 64, d, generator=gen, device="cuda")
    keys = []
    for b, L in enumerate(lens):
        runs = torch.randint(32, 513, (L // 32 + 1,), generator=gen, device="cuda")
        at = torch.searchsorted(torch.cumsum(runs, 0), torch.arange(L, device="cuda"), right=True)
        comp = torch.randint(0, 64, (hkv, L // 32 + 1), generator=gen, device="cuda")[:, at]
        mu = means[b].gather(1, comp[:, :, None].expand(-1, -1, d))
        keys.append(mu + 0.5 * torch.randn(hkv, L, d, generator=gen, device="cuda"))
    return keys, means


def _queries(gen, means, counts, group):
    """Each head's query leans on three components of its KV head's keys."""
    out = []
    for b, m in enumerate(counts):
        hkv, _, d = means[b].shape
        pick = torch.rand(m, hkv, group, 64, generator=gen, device="cuda").topk(3, -1).indices
        mu = means[b][torch.arange(hkv, device="cuda")[None, :, None, None], pick]
        q = 0.7 * mu.mean(3) + 0.3 * torch.randn(m, hkv, group, d, generator=gen, device="cuda")
        out.append(q.reshape(m, hkv * group, d))
    return torch.cat(out)


def _paged(gen, lens, hkv, T, d, dtype, keys):
    """Pools with the sequences' tokens on randomly placed pages (stale values elsewhere)."""
    n = [-(-L // T) for L in lens]
    pages = sum(n) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(n), dtype=torch.int32, device="cuda")
    k_pool = torch.randn(pages, hkv, T, d, generator=gen, device="cuda").to(dtype)
    v_pool = torch.randn(pages, hkv, T, d, generator=gen, device="cuda").to(dtype)
    at = 0
    for b, L in enumerate(lens):
        ids = perm[at:at + n[b]]
        at += n[b]
        table[b, :n[b]] = ids
        if keys is not None and L:
            slot = torch.arange(L, device="cuda")
            k_pool[ids.long()[slot // T], :, slot % T] = keys[b].transpose(0, 1).to(dtype)
    return k_pool, v_pool, table


def _means(k_pool, table, lens, T):
    """fp32 mean of every page's valid keys."""
    reps = torch.zeros(k_pool.shape[0], k_pool.shape[1], k_pool.shape[3], device="cuda")
    for b, L in enumerate(lens):
        n = -(-L // T)
        if n == 0:
            continue
        ids = table[b, :n].long()
        reps[ids] = k_pool[ids].float().mean(2)
        last = L - (n - 1) * T
        reps[ids[-1]] = k_pool[ids[-1], :, :last].float().mean(1)
    return reps


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    hq, hkv, d, T = case["hq"], case["hkv"], case["d"], case["T"]
    ctx = _ints(case["ctx"])
    st = dict(case=case, op=case["op"], ctx=ctx)
    if case["op"] == "topk":
        keys, means = _mixture_keys(gen, ctx, hkv, d)
        st["q"] = _queries(gen, means, [1] * len(ctx), hq // hkv).to(dtype)
        st["k_pool"], st["v_pool"], st["table"] = _paged(gen, ctx, hkv, T, d, dtype, keys)
        st["reps"] = _means(st["k_pool"], st["table"], ctx, T)
        st["lens"] = _i32(ctx)
        if own:
            import sampled_sparse_decode_gb300 as santa
            st["handle"] = santa.santa_topk_decode_prepared(
                st["q"], st["k_pool"], st["v_pool"], st["reps"], st["table"], st["lens"],
                case["k"])
        return st
    new = _ints(case["new"])
    total = [L + m for L, m in zip(ctx, new)]
    tok = sum(new) + case["pad"]
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    st.update(new=new, starts=starts, cu_q=_i32(starts))
    if case["op"] == "chunk":
        keys, means = _mixture_keys(gen, total, hkv, d)
        q = _queries(gen, means, new, hq // hkv)
        pad = torch.randn(case["pad"], hq, d, generator=gen, device="cuda")
        st["q"] = torch.cat([q, pad]).to(dtype)
        st["k_pool"], st["v_pool"], st["table"] = _paged(gen, total, hkv, T, d, dtype, keys)
        st["lens"] = _i32(total)
        st["out"] = torch.zeros(tok, hq, d, dtype=dtype, device="cuda")
        if own:
            import sampled_sparse_decode_gb300 as santa
            st["handle"] = santa.santa_chunk_attend_prepared(
                st["q"], st["k_pool"], st["v_pool"], st["table"], st["lens"], st["cu_q"],
                out=st["out"])
        return st
    # append: the three projections of one fused product, so q, k and v are strided views
    qkv = torch.randn(tok, hq + 2 * hkv, d, generator=gen, device="cuda").to(dtype)
    st["q"], st["k"], st["v"] = qkv.split([hq, hkv, hkv], 1)
    st["k_pool"], st["v_pool"], st["table"] = _paged(gen, total, hkv, T, d, dtype, None)
    st["reps"] = _means(st["k_pool"], st["table"], ctx, T)
    st["lens"] = _i32(ctx)
    half = case["rope"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = torch.arange(max(total), dtype=torch.float64, device="cuda")[:, None] * freq
    st["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    st["q_out"] = torch.zeros(tok, hq, d, dtype=dtype, device="cuda")
    st["lens_next"] = torch.zeros_like(st["lens"])
    if own:
        import sampled_sparse_decode_gb300 as santa
        st["handle"] = santa.santa_append_chunk_prepared(
            st["q"], st["k"], st["v"], st["cu_q"], st["k_pool"], st["v_pool"], st["reps"],
            st["table"], st["lens"], st["rope"], seq_lens_next=st["lens_next"],
            q_out=st["q_out"], interleaved=case["style"] == "interleaved")
    return st


# ---------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, style, wide):
    """x [n][H][d] with its first 2 * cos.shape[1] elements rotated pair by pair, in `wide`."""
    x = x.to(wide)
    half = cos.shape[1]
    c, s = cos.to(wide)[:, None], sin.to(wide)[:, None]
    y = x.clone()
    if style == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    return y


def _append_plain(st):
    case, T, half = st["case"], st["case"]["T"], st["case"]["rope"] // 2
    dtype = st["q"].dtype
    for b, (L, m) in enumerate(zip(st["ctx"], st["new"])):
        if m == 0:
            continue
        lo, hi = st["starts"][b], st["starts"][b + 1]
        rows = st["rope"][L:L + m]
        cos, sin = rows[:, :half], rows[:, half:]
        pos = torch.arange(L, L + m, device="cuda")
        ids = st["table"][b].long()
        st["q_out"][lo:hi] = _rotate(st["q"][lo:hi], cos, sin, case["style"],
                                     torch.float32).to(dtype)
        st["k_pool"][ids[pos // T], :, pos % T] = _rotate(
            st["k"][lo:hi], cos, sin, case["style"], torch.float32).to(dtype)
        st["v_pool"][ids[pos // T], :, pos % T] = st["v"][lo:hi]
        first, last = L // T, (L + m - 1) // T
        st["reps"][ids[first:last]] = st["k_pool"][ids[first:last]].float().mean(2)
        fill = L + m - last * T
        st["reps"][ids[last]] = st["k_pool"][ids[last], :, :fill].float().mean(1)
    torch.add(st["lens"], st["cu_q"][1:] - st["cu_q"][:-1], out=st["lens_next"])
    return [st["q_out"], st["k_pool"], st["v_pool"], st["reps"], st["lens_next"]]


def _tokens(pool, ids, L, wide):
    """The first L tokens on pages `ids` as [hkv][L][d]."""
    x = pool[ids].to(wide)
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :L]


def _chunk_plain(st):
    case, T, d = st["case"], st["case"]["T"], st["case"]["d"]
    group = case["hq"] // case["hkv"]
    for b, (L, m) in enumerate(zip(st["ctx"], st["new"])):
        ids = st["table"][b, :-(-(L + m) // T)].long()
        K = _tokens(st["k_pool"], ids, L + m, torch.float32)
        V = _tokens(st["v_pool"], ids, L + m, torch.float32)
        for i in range(0, m, 1024):
            e = min(m, i + 1024)
            see = L + e
            lo = st["starts"][b] + i
            q = st["q"][lo:lo + e - i].float().view(e - i, case["hkv"], group, d)
            q = q.permute(1, 2, 0, 3).reshape(case["hkv"], -1, d)
            s = (q @ K[:, :see].transpose(1, 2) / math.sqrt(d)).view(case["hkv"], group, e - i, see)
            late = torch.arange(see, device="cuda")[None] > L + torch.arange(i, e, device="cuda")[:, None]
            s.masked_fill_(late, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = (p.view(case["hkv"], -1, see) @ V[:, :see]).view(case["hkv"], group, e - i, d)
            o /= p.sum(-1, keepdim=True)
            st["out"][lo:lo + e - i] = o.permute(2, 0, 1, 3).reshape(e - i, -1, d).to(st["out"].dtype)
    return st["out"]


def _best(q, reps, k):
    """The k best teams of [hkv][n] scores, ascending; a score is the group's largest product
    of query and representative (64 bits: the choice stands next to a border)."""
    s = torch.einsum("hgd,nhd->hgn", q.double(), reps.double()).amax(1)
    order = torch.sort(s, dim=1, descending=True, stable=True).indices
    return order[:, :min(k, s.shape[1])].sort(1).values


def _topk_plain(st):
    case, T, d, k = st["case"], st["case"]["T"], st["case"]["d"], st["case"]["k"]
    hkv, group = case["hkv"], case["hq"] // case["hkv"]
    out = torch.empty(len(st["ctx"]), case["hq"], d, device="cuda")
    sel = torch.full((len(st["ctx"]), hkv, k), -1, dtype=torch.int32, device="cuda")
    count = torch.empty(len(st["ctx"]), hkv, dtype=torch.int32, device="cuda")
    heads = torch.arange(hkv, device="cuda")[:, None]
    for b, L in enumerate(st["ctx"]):
        n = -(-L // T)
        ids = st["table"][b, :n].long()
        q = st["q"][b].view(hkv, group, d)
        best = _best(q, st["reps"][ids], k)
        sel[b, :, :best.shape[1]] = best.int()
        count[b] = best.shape[1]
        K = st["k_pool"][ids[best], heads].float().view(hkv, -1, d)
        V = st["v_pool"][ids[best], heads].float().view(hkv, -1, d)
        tok = best[:, :, None] * T + torch.arange(T, device="cuda")
        s = q.float() @ K.transpose(1, 2) / math.sqrt(d)
        s.masked_fill_((tok >= L).view(hkv, 1, -1), -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        # slots behind the sequence's end hold anything: they do not enter the sum
        V.masked_fill_((tok >= L).view(hkv, -1, 1), 0.0)
        out[b] = ((p @ V) / p.sum(-1, keepdim=True)).view(-1, d)
    return [out, sel, count]


def run(st):
    if own:
        r = st["handle"].run()
        if st["op"] == "append":
            return [st["q_out"], st["k_pool"], st["v_pool"], st["reps"], st["lens_next"]]
        return r if st["op"] == "chunk" else [r.out, r.sel_ids, r.sel_count]
    return {"append": _append_plain, "chunk": _chunk_plain, "topk": _topk_plain}[st["op"]](st)


# ---------------------------------------------------------------- 64-bit definition

def _exact_append(case, st):
    """Token by token position: a complex product for each pair."""
    T, half = case["T"], case["rope"] // 2
    q_out = torch.zeros(st["q_out"].shape, dtype=torch.float64, device="cuda")
    k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
    reps = st["reps"].double()
    for b, (L, m) in enumerate(zip(st["ctx"], st["new"])):
        sl = slice(st["starts"][b], st["starts"][b] + m)
        row = st["rope"][L:L + m].double()
        turn = torch.complex(row[:, :half].contiguous(), row[:, half:].contiguous())[:, None]
        done = []
        for x in (st["q"][sl].double(), st["k"][sl].double()):
            head, rest = x[..., :2 * half], x[..., 2 * half:]
            if case["style"] == "half":
                z = torch.complex(*[t.contiguous() for t in head.chunk(2, -1)]) * turn
                head = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.view_as_complex(head.reshape(*head.shape[:2], half, 2)) * turn
                head = torch.view_as_real(z).flatten(2)
            done.append(torch.cat([head, rest], -1))
        q_out[sl] = done[0]
        for page in range(L // T, -(-(L + m) // T)):
            p = int(st["table"][b, page])
            lo, hi = max(L, page * T), min(L + m, (page + 1) * T)
            k_pool[p, :, lo - page * T:hi - page * T] = done[1][lo - L:hi - L].transpose(0, 1)
            v_pool[p, :, lo - page * T:hi - page * T] = st["v"][sl][lo - L:hi - L].transpose(0, 1).double()
            reps[p] = k_pool[p, :, :hi - page * T].sum(1) / (hi - page * T)
    lens = torch.tensor([L + m for L, m in zip(st["ctx"], st["new"])], dtype=torch.int32,
                        device="cuda")
    # a mean of keys that were rounded to 16 bits has no exact value: it jumps with every key
    # that stands next to a rounding border
    return [q_out, k_pool, v_pool, reps if case["dtype"] == "f32" else None, lens]


def _exact_chunk(case, st):
    """Head by head, with the softmax as weights that sum to one."""
    T, d, group = case["T"], case["d"], case["hq"] // case["hkv"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b, (L, m) in enumerate(zip(st["ctx"], st["new"])):
        pos = torch.arange(L + m, device="cuda")
        page = st["table"][b].long()[pos // T]
        for h in range(case["hkv"]):
            K = st["k_pool"][page, h, pos % T].double()
            V = st["v_pool"][page, h, pos % T].double()
            for hq in range(h * group, (h + 1) * group):
                for i in range(0, m, 2048):
                    rows = torch.arange(i, min(m, i + 2048), device="cuda")
                    at = st["starts"][b] + rows
                    s = torch.mm(st["q"][at, hq].double(), K.T) * d ** -0.5
                    s = torch.where(pos[None] <= L + rows[:, None], s, -math.inf)
                    out[at, hq] = torch.mm(torch.softmax(s, 1), V)
    return out


def _exact_topk(case, st):
    T, d, k, group = case["T"], case["d"], case["k"], case["hq"] // case["hkv"]
    out = torch.zeros(len(st["ctx"]), case["hq"], d, dtype=torch.float64, device="cuda")
    sel = torch.full((len(st["ctx"]), case["hkv"], k), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(len(st["ctx"]), case["hkv"], dtype=torch.int32, device="cuda")
    for b, L in enumerate(st["ctx"]):
        page = st["table"][b, :-(-L // T)].long()
        for h in range(case["hkv"]):
            q = st["q"][b, h * group:(h + 1) * group].double()
            score = (st["reps"][page, h].double() @ q.T).max(1).values.tolist()
            best = sorted(sorted(range(len(score)), key=lambda i: (-score[i], i))[:k])
            sel[b, h, :len(best)] = torch.tensor(best, dtype=torch.int32)
            count[b, h] = len(best)
            pos = torch.cat([torch.arange(i * T, min(L, (i + 1) * T)) for i in best]).cuda()
            K = st["k_pool"][page[pos // T], h, pos % T].double()
            V = st["v_pool"][page[pos // T], h, pos % T].double()
            out[b, h * group:(h + 1) * group] = torch.softmax(q @ K.T * d ** -0.5, 1) @ V
    return [out, sel, count]


def exact(case, seed):
    if case["op"] == "chunk" and work(case)["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    st.pop("handle", None)
    return {"append": _exact_append, "chunk": _exact_chunk, "topk": _exact_topk}[case["op"]](case, st)
