"""Cases of the 8-bit paged cache: append with the heads' norms, rotation and quantisation in one
pass, attention of one new token over the quantised cache, and reading the cache back.

``own`` false computes each operator in plain torch operations; ``own`` true calls the package's
entry points.  Both take the state that ``prepare`` makes and write the same buffers (the cache is
updated in place, as a serving loop does).

A row of d elements x is held as 8-bit codes c and one fp32 scale s, standing for c s:
s = max(max |x|, 2^-90) / top and c = x / s rounded to the nearest code (ties to even), top = 127
for int8 and 448 for e4m3.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8,
          "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -90
EPS = 1e-6


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
        # one generated token for each of 8 sequences deep in a 32K context, int8 cache: the
        # append of a decode step, all latency
        dict(name="append_step_b8_i8", op="append", dtype="bf16", cache="i8", hq=28, hkv=4, d=128,
             T=128, ctx="32000,32383,31744,32767,29000,32640,30001,32255", new="1x8", rope=128,
             style="half", norm=False, pad=0),
        # prompts of different lengths on top of earlier turns into an fp32 cache, with norms of
        # queries and keys, interleaved pairs on half of the head, padded
        dict(name="append_ragged_f32_norm", op="append", dtype="f32", cache="same", hq=16, hkv=2,
             d=64, T=64, ctx="0,777,64,5,1023,0,4096,310", new="1,300,64,63,129,700,2,45", rope=32,
             style="interleaved", norm=True, pad=40),
        # a few bf16 prompts with norms into a bf16 cache
        dict(name="append_bf16_norm", op="append", dtype="bf16", cache="same", hq=32, hkv=8, d=128,
             T=128, ctx="0,100,4000", new="1500,37,611", rope=128, style="half", norm=True, pad=4),
        # a full prefill batch with norms into an e4m3 cache: 8 prompts of 4096 tokens
        dict(name="append_prefill_b8_4k_e4m3", op="append", dtype="bf16", cache="e4m3", hq=32,
             hkv=8, d=128, T=128, ctx="0x8", new="4096x8", rope=128, style="half", norm=True, pad=0),
        # the first generated tokens of one short question: latency
        dict(name="attend_short_b1_i8", op="attend", dtype="bf16", cache="i8", hq=28, hkv=4, d=128,
             T=128, ctx="523", teams=0, cap=0.0, window=0),
        # a decode step of one sequence at 32K
        dict(name="attend_32k_b1_i8", op="attend", dtype="bf16", cache="i8", hq=28, hkv=4, d=128,
             T=128, ctx="32768", teams=0, cap=0.0, window=0),
        # a batch at 32K and below, some sequences short: bound by the cache's bytes
        dict(name="attend_32k_b16_i8", op="attend", dtype="bf16", cache="i8", hq=32, hkv=8, d=128,
             T=128, ctx="32768x8,20000,31000,32000,1000,32700,12345,127,30001", teams=0, cap=0.0,
             window=0),
        # long contexts with scores capped by a tanh, e4m3 cache
        dict(name="attend_128k_b4_e4m3_cap", op="attend", dtype="bf16", cache="e4m3", hq=28, hkv=4,
             d=128, T=128, ctx="131072x3,100001", teams=0, cap=30.0, window=0),
        # fp32 queries, small heads, a layer that sees the last 1000 tokens only
        dict(name="attend_window_f32_i8", op="attend", dtype="f32", cache="i8", hq=8, hkv=2, d=64,
             T=64, ctx="4096,999,1,2500,64,7001", teams=0, cap=0.0, window=1000),
        # the sparse step over sampled teams with their weights, 32 of 256 teams of 16 sequences
        dict(name="attend_teams_b16_i8", op="attend", dtype="bf16", cache="i8", hq=32, hkv=8, d=128,
             T=128, ctx="32768x8,20000,31000,32000,1000,32700,12345,127,30001", teams=32, cap=0.0,
             window=0),
        # the last chunk of one prompt out of an int8 cache, behind what was read back before
        dict(name="read_chunk_i8_f32", op="read", dtype="f32", cache="i8", hkv=4, d=128, T=128,
             ctx="1800", first="1536"),
        # a batch of prompts read back as bf16 pages for the attention of their next chunk
        dict(name="read_b8_8k_e4m3_bf16", op="read", dtype="bf16", cache="e4m3", hkv=8, d=128, T=128,
             ctx="8192,8000,4097,8192,1,2500,777,6001", first="0x8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "read"])
    d = rng.choice([64, 128, 128])
    T = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), cache=rng.choice(["i8", "e4m3"]),
             hkv=hkv, d=d, T=T)
    batch = _log(rng, 1, 16)
    if op == "attend":
        c["hq"] = hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        top = min(131072, 400000 // batch)
        c["ctx"] = _text(_log(rng, 1, top) for _ in range(batch))
        c["teams"] = rng.choice([0, 0, _log(rng, 1, 128)])
        c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 8000)]) if c["teams"] == 0 else 0
        return c
    if op == "append":
        c["hq"] = hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        c["new"] = _text(_log(rng, 1, 16384 // batch) for _ in range(batch))
        c["ctx"] = _text(rng.choice([0, _log(rng, 1, 131072 // batch)]) for _ in range(batch))
        c["rope"] = rng.choice([d, d, d // 2, 16, 0])
        c["style"] = rng.choice(["half", "interleaved"])
        c["norm"] = rng.choice([False, True])
        # whole numbers are compared bit for bit, which a norm's last rounding would upset
        c["cache"] = rng.choice(["same", "e4m3"]) if c["norm"] else rng.choice(["i8", "e4m3"])
        c["pad"] = rng.choice([0, 0, rng.randint(1, 64)])
        return c
    ctx = [_log(rng, 1, 32768 // batch) for _ in range(batch)]
    c["ctx"] = _text(ctx)
    c["first"] = _text(rng.choice([0, rng.randint(0, L)]) for L in ctx)
    if c["first"] == c["ctx"]:
        c["first"] = _text(0 for _ in ctx)
    return c


def _size(case):
    """Bytes of an element of the activations, and of a cached row of d elements."""
    es = 2 if case["dtype"] == "bf16" else 4
    return es, case["d"] * es if case["cache"] == "same" else case["d"] + 4


def _seen(case):
    """Visible tokens of each sequence (of a head that takes `teams` teams, if not 0)."""
    ctx, T = _ints(case["ctx"]), case["T"]
    if case["teams"]:
        return [min(L, case["teams"] * T) for L in ctx]
    return [min(L, case["window"]) if case["window"] else L for L in ctx]


def work(case):
    hkv, d, T = case["hkv"], case["d"], case["T"]
    es, row = _size(case)
    ctx = _ints(case["ctx"])
    if case["op"] == "attend":
        seen = sum(_seen(case))
        b = seen * hkv * 2 * row + len(ctx) * (case["hq"] * d * (es + 4) + 4)
        b += -(-seen // T) * 4 + len(ctx) * hkv * case["teams"] * 8
        return {"bytes": b, "flops": 4 * d * case["hq"] * seen}
    if case["op"] == "read":
        tok = sum(L - f for L, f in zip(ctx, _ints(case["first"])))
        return {"bytes": tok * hkv * 2 * (row + d * es) + len(ctx) * 8, "flops": 2 * tok * hkv * d}
    new = _ints(case["new"])
    tok, batch, hq = sum(new), len(new), case["hq"]
    # the new rows in, the queries and the cached rows out, the table's rows, the earlier rows of
    # a page that is already begun (its mean is needed), representatives, page ids and lengths
    old = sum(L % T for L, m in zip(ctx, new) if m)
    pages = sum(-(-(L % T + m) // T) for L, m in zip(ctx, new))
    b = tok * (2 * hq + 2 * hkv) * d * es + tok * 2 * hkv * row + tok * case["rope"] * 4
    b += old * hkv * row + pages * (hkv * d * 4 + 4) + batch * 12
    f = tok * (hq + hkv) * (case["rope"] * 3 + (4 * d if case["norm"] else 0))
    return {"bytes": b, "flops": f + (old + tok) * hkv * d}


# ---------------------------------------------------------------- inputs

def _scale(x, top):
    # divided by a tensor: torch multiplies by a plain number's rounded reciprocal instead
    a = x.abs().amax(-1).clamp(min=TINY)
    return a / torch.full_like(a, top)


def _codes(x, scale, kind):
    """The nearest codes of fp32 rows x."""
    y = x / scale[..., None]
    return y.round().to(torch.int8) if kind == "i8" else y.to(torch.float8_e4m3fn)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(gen, lens, T):
    """Randomly placed pages for sequences of these lengths: the table and the page count."""
    n = [-(-L // T) for L in lens]
    perm = torch.randperm(sum(n) + 3, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(max(n), 1), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(n):
        table[b, :c] = perm[at:at + c]
        at += c
    return table, sum(n) + 3


def _fill(gen, pages, case, means=None):
    """K, V and their scales of `pages` pages in the case's cache type: values of both signs whose
    rows differ in size, as projections give them; keys lean on one of 64 directions per page."""
    shape = (pages, case["hkv"], case["T"], case["d"])
    kind = case["cache"]
    same = kind == "same"
    dt = DTYPES[case["dtype"] if same else kind]
    codes = [torch.empty(shape, dtype=dt, device="cuda") for _ in range(2)]
    scales = [None if same else torch.empty(shape[:3], device="cuda") for _ in range(2)]
    for p in range(0, pages, 512):
        n = min(512, pages - p)
        for i in range(2):
            x = torch.randn((n,) + shape[1:], generator=gen, device="cuda")
            if i == 0 and means is not None:
                at = torch.randint(0, 64, (n,), generator=gen, device="cuda")
                x = means[:, at].transpose(0, 1)[:, :, None] + 0.5 * x
            x = x * torch.exp2(0.5 * torch.randn(n, *shape[1:3], 1, generator=gen, device="cuda"))
            if not same:
                scales[i][p:p + n] = _scale(x, TOP[kind])
                x = _codes(x, scales[i][p:p + n], kind)
            codes[i][p:p + n] = x.to(dt)
    return codes, scales


def _cache(st):
    """The package's handle of a cache: the two pools, or codes with their scales."""
    if st["case"]["cache"] == "same":
        return st["k_pool"], st["v_pool"]
    import sampled_sparse_decode_gb300 as santa
    return santa.Q8Cache(st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"])


def _stored(st, ids):
    """The keys on pages `ids` as the fp32 values they stand for."""
    k = st["k_pool"][ids].float()
    return k if st["k_scale"] is None else k * st["k_scale"][ids][..., None]


def _prepare_attend(case, gen, st):
    dtype, hq, hkv, d, T = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"], case["T"]
    ctx = st["ctx"]
    st["table"], pages = _table(gen, ctx, T)
    means = torch.randn(hkv, 64, d, generator=gen, device="cuda")
    (st["k_pool"], st["v_pool"]), (st["k_scale"], st["v_scale"]) = _fill(gen, pages, case, means)
    pick = torch.rand(len(ctx), hkv, hq // hkv, 64, generator=gen, device="cuda").topk(3, -1).indices
    mu = means[torch.arange(hkv, device="cuda")[None, :, None, None], pick].mean(3)
    q = 0.7 * mu + 0.3 * torch.randn(mu.shape, generator=gen, device="cuda")
    st["q"] = q.reshape(len(ctx), hq, d).to(dtype)
    st["lens"] = _i32(ctx)
    st["out"] = torch.zeros(len(ctx), hq, d, device="cuda")
    sel = None
    if case["teams"]:
        # distinct teams in ascending order and the chance that each was drawn
        m = case["teams"]
        ids = torch.full((len(ctx), hkv, m), -1, dtype=torch.int32, device="cuda")
        pi = torch.zeros(len(ctx), hkv, m, device="cuda")
        for b, L in enumerate(ctx):
            n = -(-L // T)
            keep = min(n, m)
            order = torch.rand(hkv, n, generator=gen, device="cuda").argsort(1)[:, :keep]
            ids[b, :, :keep] = order.sort(1).values.int()
            pi[b, :, :keep] = 0.05 + 0.95 * torch.rand(hkv, keep, generator=gen, device="cuda")
        count = _i32([min(-(-L // T), m) for L in ctx])[:, None].repeat(1, hkv).contiguous()
        st["sel"] = sel = (ids, count, pi)
    if own:
        import sampled_sparse_decode_gb300 as santa
        args = (st["q"], _cache(st), st["table"], st["lens"])
        opts = dict(softcap=case["cap"], window=case["window"], out=st["out"])
        st["handle"] = (santa.santa_q8_attend_prepared(*args, *sel, **opts) if sel else
                        santa.santa_q8_dense_decode_prepared(*args, **opts))
    return st


def _prepare_read(case, gen, st):
    st["first"] = _ints(case["first"])
    st["table"], pages = _table(gen, st["ctx"], case["T"])
    st["dst_table"], dst_pages = _table(gen, st["ctx"], case["T"])
    (st["k_pool"], st["v_pool"]), (st["k_scale"], st["v_scale"]) = _fill(gen, pages, case)
    shape = (dst_pages, case["hkv"], case["T"], case["d"])
    st["k_out"] = torch.zeros(shape, dtype=DTYPES[case["dtype"]], device="cuda")
    st["v_out"] = torch.zeros_like(st["k_out"])
    st["lens"], st["from"] = _i32(st["ctx"]), _i32(st["first"])
    if own:
        import sampled_sparse_decode_gb300 as santa
        st["handle"] = santa.santa_q8_read_prepared(
            _cache(st), st["table"], st["lens"], st["k_out"], st["v_out"], st["dst_table"],
            first=st["from"])
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx = _ints(case["ctx"])
    st = dict(case=case, op=case["op"], ctx=ctx)
    if case["op"] == "attend":
        return _prepare_attend(case, gen, st)
    if case["op"] == "read":
        return _prepare_read(case, gen, st)
    dtype, hq, hkv, d, T = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"], case["T"]
    new = _ints(case["new"])
    total = [L + m for L, m in zip(ctx, new)]
    tok = sum(new) + case["pad"]
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    st.update(new=new, starts=starts, cu_q=_i32(starts))
    # the three projections of one fused product, so q, k and v are strided views
    qkv = torch.randn(tok, hq + 2 * hkv, d, generator=gen, device="cuda")
    qkv *= torch.exp2(torch.randn(tok, hq + 2 * hkv, 1, generator=gen, device="cuda"))
    st["q"], st["k"], st["v"] = qkv.to(dtype).split([hq, hkv, hkv], 1)
    st["table"], pages = _table(gen, total, T)
    (st["k_pool"], st["v_pool"]), (st["k_scale"], st["v_scale"]) = _fill(gen, pages, case)
    st["reps"] = torch.zeros(pages, hkv, d, device="cuda")
    for b, L in enumerate(ctx):
        ids = st["table"][b, :-(-L // T)].long()
        if L:
            st["reps"][ids] = _stored(st, ids).mean(2)
            st["reps"][ids[-1]] = _stored(st, ids[-1:])[0, :, :L - (len(ids) - 1) * T].mean(1)
    st["q_norm"] = st["k_norm"] = st["rope"] = None
    if case["norm"]:
        st["q_norm"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
        st["k_norm"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
    if case["rope"]:
        half = case["rope"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        ang = torch.arange(max(total), dtype=torch.float64, device="cuda")[:, None] * freq
        st["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    st["lens"] = _i32(ctx)
    st["lens_next"] = torch.zeros_like(st["lens"])
    st["q_out"] = torch.zeros(tok, hq, d, dtype=dtype, device="cuda")
    if own:
        import sampled_sparse_decode_gb300 as santa
        st["handle"] = santa.santa_append_norm_prepared(
            st["q"], st["k"], st["v"], st["cu_q"], _cache(st), st["reps"], st["table"], st["lens"],
            st["rope"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS,
            seq_lens_next=st["lens_next"], q_out=st["q_out"],
            interleaved=case["style"] == "interleaved")
    return st


# ---------------------------------------------------------------- plain forms

def _normed(x, weight):
    """fp32 rows over their root mean square, times the weight."""
    x = x.float()
    return x if weight is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _rotate(x, rows, style):
    """fp32 x [n][H][d] with its first elements rotated pair by pair."""
    if rows is None:
        return x
    half = rows.shape[1] // 2
    c, s = rows[:, None, :half], rows[:, None, half:]
    y = x.clone()
    first, second = ((slice(0, half), slice(half, 2 * half)) if style == "half" else
                     (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def _append_plain(st):
    case, T = st["case"], st["case"]["T"]
    for b, (L, m) in enumerate(zip(st["ctx"], st["new"])):
        if m == 0:
            continue
        sl = slice(st["starts"][b], st["starts"][b + 1])
        rows = None if st["rope"] is None else st["rope"][L:L + m]
        pos = torch.arange(L, L + m, device="cuda")
        page, slot = st["table"][b].long()[pos // T], pos % T
        st["q_out"][sl] = _rotate(_normed(st["q"][sl], st["q_norm"]), rows,
                                  case["style"]).to(st["q_out"].dtype)
        k = _rotate(_normed(st["k"][sl], st["k_norm"]), rows, case["style"])
        for x, pool, scale in ((k, "k_pool", "k_scale"), (st["v"][sl].float(), "v_pool", "v_scale")):
            if case["cache"] != "same":
                s = _scale(x, TOP[case["cache"]])
                st[scale][page, :, slot] = s
                x = _codes(x, s, case["cache"])
            st[pool][page, :, slot] = x.to(st[pool].dtype)
        ids = st["table"][b, L // T:(L + m - 1) // T + 1].long()
        if len(ids) > 1:
            st["reps"][ids[:-1]] = _stored(st, ids[:-1]).mean(2)
        fill = (L + m - 1) % T + 1
        st["reps"][ids[-1]] = _stored(st, ids[-1:])[0, :, :fill].mean(1)
    torch.add(st["lens"], st["cu_q"][1:] - st["cu_q"][:-1], out=st["lens_next"])


def _appended(st):
    """What an append writes.  A key that a norm's last rounding moves across a border takes the
    neighbouring 16- or 8-bit value, and the mean of its page moves with it by more than fp32
    resolves: the means of such keys are given in 16 bits."""
    reps = st["reps"]
    if st["case"]["norm"] and st["k_pool"].dtype != torch.float32:
        reps = reps.bfloat16()
    return [st["q_out"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"], reps,
            st["lens_next"]]


def _values(st, which, pages):
    """All tokens on `pages` as fp32 values, [hkv][tokens][d]."""
    x = st[which + "_pool"][pages].float() * st[which + "_scale"][pages][..., None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])


def _attend_plain(st):
    case, T, d, hkv = st["case"], st["case"]["T"], st["case"]["d"], st["case"]["hkv"]
    heads = torch.arange(hkv, device="cuda")[:, None]
    for b, L in enumerate(st["ctx"]):
        pages = st["table"][b, :-(-L // T)].long()
        q = st["q"][b].float().view(hkv, -1, d)
        if case["teams"]:
            ids, pi = (t[b, :, :min(case["teams"], len(pages))] for t in st["sel"][::2])
            page = pages[ids.long()]
            K = (st["k_pool"][page, heads].float() * st["k_scale"][page, heads][..., None]).flatten(1, 2)
            V = (st["v_pool"][page, heads].float() * st["v_scale"][page, heads][..., None]).flatten(1, 2)
            pos = (ids[..., None] * T + torch.arange(T, device="cuda")).flatten(1, 2)
            bias = -pi.log().repeat_interleave(T, 1)[:, None]
        else:
            lo = max(0, L - case["window"]) if case["window"] else 0
            K, V = _values(st, "k", pages[lo // T:]), _values(st, "v", pages[lo // T:])
            pos = (lo // T * T + torch.arange(K.shape[1], device="cuda")).expand(hkv, -1)
            bias = 0.0
        s = q @ K.transpose(1, 2) / math.sqrt(d)
        if case["cap"]:
            s = case["cap"] * torch.tanh(s / case["cap"])
        unseen = pos >= L
        if case["window"]:
            unseen = unseen | (pos < L - case["window"])
        s = (s + bias).masked_fill(unseen[:, None], -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        # slots that are not seen hold anything: they do not enter the sum
        V.masked_fill_(unseen[..., None], 0.0)
        st["out"][b] = ((p @ V) / p.sum(-1, keepdim=True)).view(-1, d)
    return st["out"]


def _read_plain(st):
    T = st["case"]["T"]
    for b, (L, f) in enumerate(zip(st["ctx"], st["first"])):
        pos = torch.arange(f, L, device="cuda")
        src, dst, slot = st["table"][b].long()[pos // T], st["dst_table"][b].long()[pos // T], pos % T
        for which in ("k", "v"):
            x = st[which + "_pool"][src, :, slot].float() * st[which + "_scale"][src, :, slot][..., None]
            st[which + "_out"][dst, :, slot] = x.to(st[which + "_out"].dtype)


def run(st):
    if own:
        st["handle"].run()
    else:
        {"append": _append_plain, "attend": _attend_plain, "read": _read_plain}[st["op"]](st)
    if st["op"] == "append":
        return _appended(st)
    return st["out"] if st["op"] == "attend" else [st["k_out"], st["v_out"]]


# ---------------------------------------------------------------- 64-bit definition

def _nearest_e4m3(y):
    """Three bits behind the leading one, exponents from -6 on, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_append(case, st):
    """Token by token position: a norm as a division, a complex product for each pair."""
    T, kind, d = case["T"], case["cache"], case["d"]
    q_out = torch.zeros(st["q_out"].shape, dtype=torch.float64, device="cuda")
    pools = [st[n].double() for n in ("k_pool", "v_pool")]
    scales = [None if kind == "same" else st[n].double() for n in ("k_scale", "v_scale")]
    reps = st["reps"].double()
    for b, (L, m) in enumerate(zip(st["ctx"], st["new"])):
        sl = slice(st["starts"][b], st["starts"][b] + m)
        done = []
        for x, w in ((st["q"][sl].double(), st["q_norm"]), (st["k"][sl].double(), st["k_norm"])):
            if w is not None:
                x = x / ((x * x).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            if case["rope"]:
                half = case["rope"] // 2
                row = st["rope"][L:L + m].double()
                turn = torch.complex(row[:, :half].contiguous(), row[:, half:].contiguous())[:, None]
                head, rest = x[..., :2 * half], x[..., 2 * half:]
                if case["style"] == "half":
                    z = torch.complex(*[t.contiguous() for t in head.chunk(2, -1)]) * turn
                    head = torch.cat([z.real, z.imag], -1)
                else:
                    z = torch.view_as_complex(head.reshape(*head.shape[:2], half, 2).contiguous()) * turn
                    head = torch.view_as_real(z).flatten(2)
                x = torch.cat([head, rest], -1)
            done.append(x)
        q_out[sl] = done[0]
        for pool, scale, x in zip(pools, scales, (done[1], st["v"][sl].double())):
            for page in range(L // T, -(-(L + m) // T)):
                p = int(st["table"][b, page])
                lo, hi = max(L, page * T), min(L + m, (page + 1) * T)
                y = x[lo - L:hi - L].transpose(0, 1)
                if kind != "same":
                    s = torch.clamp(y.abs().max(-1).values, min=TINY) / TOP[kind]
                    scale[p, :, lo - page * T:hi - page * T] = s
                    y = _nearest_e4m3(y / s[..., None])
                pool[p, :, lo - page * T:hi - page * T] = y
                if pool is pools[0] and kind == "same":
                    reps[p] = pool[p, :, :hi - page * T].sum(1) / (hi - page * T)
    lens = _i32([L + m for L, m in zip(st["ctx"], st["new"])])
    # int8 codes are whole numbers; a mean of keys that were rounded to 16 or 8 bits has no exact
    # value: it jumps with every key that stands next to a rounding border
    k, v = pools if kind != "i8" else (None, None)
    exact_mean = kind == "same" and case["dtype"] == "f32"
    return [q_out, k, v, scales[0], scales[1], reps if exact_mean else None, lens]


def _exact_attend(case, st):
    """Head by head over the list of seen tokens, with the weights as a softmax."""
    T, d, hkv, group = case["T"], case["d"], case["hkv"], case["hq"] // case["hkv"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(st["ctx"]):
        pages = st["table"][b].long()
        for h in range(hkv):
            if case["teams"]:
                ids, count, pi = st["sel"]
                n = int(count[b, h])
                pos = (ids[b, h, :n, None].long() * T + torch.arange(T, device="cuda")).flatten()
                bias = torch.log(1 / pi[b, h, :n].double()).repeat_interleave(T)
                bias, pos = bias[pos < L], pos[pos < L]
            else:
                pos = torch.arange(L, device="cuda")
                pos = pos[-case["window"]:] if case["window"] else pos
                bias = 0
            K, V = (st[n + "_pool"][pages[pos // T], h, pos % T].double() *
                    st[n + "_scale"][pages[pos // T], h, pos % T, None].double() for n in "kv")
            s = torch.mm(st["q"][b, h * group:(h + 1) * group].double(), K.T) * d ** -0.5
            if case["cap"]:
                s = torch.tanh(s / case["cap"]) * case["cap"]
            out[b, h * group:(h + 1) * group] = torch.mm(torch.softmax(s + bias, 1), V)
    return out


def _exact_read(case, st):
    outs = [st["k_out"].double(), st["v_out"].double()]
    for b, (L, f) in enumerate(zip(st["ctx"], st["first"])):
        for i in range(f // case["T"], -(-L // case["T"])):
            lo, hi = max(f - i * case["T"], 0), min(L - i * case["T"], case["T"])
            src, dst = int(st["table"][b, i]), int(st["dst_table"][b, i])
            for o, which in zip(outs, "kv"):
                o[dst, :, lo:hi] = (st[which + "_pool"][src, :, lo:hi].double() *
                                    st[which + "_scale"][src, :, lo:hi].double().unsqueeze(-1))
    return outs


def exact(case, seed):
    st = prepare(case, seed)
    st.pop("handle", None)
    return {"append": _exact_append, "attend": _exact_attend, "read": _exact_read}[case["op"]](case, st)
