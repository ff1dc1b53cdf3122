"""Operators around the target's paged cache, as measured cases: writing keys
and values while positions are rotated into keys and queries (half and
interleaved layouts, part of the head, frequencies scaled for long contexts),
a cache held in 4 bits (E2M1 codes with a bfloat16 scale for every 16 of them)
written and read back, attention over such a cache, and a step that does both.

Every case exists in two forms: `own = False` computes it with elementary
torch operations, `own = True` calls the framework."""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ROPE = ("rope", "step")
ATTEND = ("attention", "step")


# ------------------------------------------------------------------- cases

def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, rows_lo=1, rows_hi=1, ctx_lo=0, ctx_hi=0, n_q=40, n_kv=8, hd=128, page=64,
             dtype="bf16", cache="e2m1", causal=True, window=0, rot=0, layout="half", theta=1e6, stretch=1.0,
             trained=0, factor=1.0, apart=0)
    c.update(kw)
    return c


def listed():
    return [
        # ordinary decoding of one request over a cache in 4 bits: one new token, a short context; latency counts
        _case("attention one token", "attention", ctx_lo=1000, ctx_hi=1000),
        # the target scores blocks of 8 for a full batch, contexts of 8,192
        _case("attention block 8 batch 32", "attention", batch=32, rows_lo=8, rows_hi=8, ctx_lo=8192, ctx_hi=8192),
        # blocks of 16 over very unequal contexts, where 4 bits are what lets them fit
        _case("attention ragged", "attention", batch=16, rows_lo=16, rows_hi=16, ctx_lo=512, ctx_hi=131072, page=128),
        # two prompts prefilled in chunks of 2,048 behind contexts of 8k to 16k; matrix products bound it
        _case("attention prompt chunk", "attention", batch=2, rows_lo=2048, rows_hi=2048, ctx_lo=8192, ctx_hi=16384),
        # mixed chunk lengths, head dim 64, 7 query heads to a KV head, small pages, a sliding window, fp16
        _case("attention odd window f16", "attention", batch=5, rows_lo=20, rows_hi=900, ctx_lo=100, ctx_hi=9000,
              n_q=14, n_kv=2, hd=64, page=16, dtype="f16", window=1000),
        # a step's new rows of a full batch, rotated and quantised to 8 bits as they are written; latency counts
        _case("rope block 8 e4m3", "rope", batch=32, rows_lo=8, rows_hi=8, ctx_lo=4096, ctx_hi=8192, rot=128,
              cache="e4m3"),
        # the rows of prompts into a 16-bit cache; memory bounds it
        _case("rope prompts bf16", "rope", batch=6, rows_lo=900, rows_hi=8192, ctx_lo=0, ctx_hi=500, page=128,
              rot=128, cache="bf16"),
        # far positions under frequencies scaled for them, half of the head rotated in neighbouring pairs, given
        # positions apart from the cache's, fp16
        _case("rope far odd f16", "rope", batch=5, rows_lo=20, rows_hi=900, ctx_lo=100000, ctx_hi=500000, n_q=14,
              n_kv=2, hd=64, page=16, dtype="f16", cache="f16", rot=32, layout="interleaved", theta=5e5, stretch=8.0,
              trained=8192, factor=1.2, apart=300000),
        # a step's new rows of a full batch into 4 bits and back; latency counts
        _case("store block 8", "store", batch=32, rows_lo=8, rows_hi=8, ctx_lo=40, ctx_hi=900),
        # the rows of prompts into 4 bits and back, as a cache that is handed on is checked
        _case("store prompts", "store", batch=9, rows_lo=900, rows_hi=8192, ctx_lo=0, ctx_hi=500, page=128),
        # one layer's step of a batch: rows rotated, written in 4 bits and attended
        _case("step block 8 batch 16", "step", batch=16, rows_lo=8, rows_hi=8, ctx_lo=2000, ctx_hi=8192, rot=128),
        # the same of three short requests with small heads in fp16
        _case("step short f16", "step", batch=3, rows_lo=1, rows_hi=5, ctx_lo=0, ctx_hi=300, n_q=14, n_kv=2, hd=64,
              page=16, dtype="f16", rot=64, theta=1e4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rope", "rope", "store", "step"])
    hd = rng.choice([64, 128])
    n_kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "f16"])
    c = dict(op=op, n_q=n_kv * group, n_kv=n_kv, hd=hd, page=rng.choice([16, 32, 64, 128]), dtype=dtype, cache="e2m1",
             causal=True, window=0, rot=0, layout="half", theta=1e6, stretch=1.0, trained=0, factor=1.0, apart=0)
    if op in ATTEND:
        if op == "step" or rng.random() < 0.6:      # decoding and block verification
            batch, hi, ctx = _log(rng, 1, 48), _log(rng, 1, 16), _log(rng, 1, 60000)
            ctx = max(1, min(ctx, 250000 // batch))
        else:                                       # chunks of prompts, no more work than the listed one's
            batch, hi, ctx = _log(rng, 1, 4), _log(rng, 17, 2048), _log(rng, 1, 14000)
            while batch * hi * (ctx + hi) * n_kv * group * hd > 2 ** 38:
                hi, ctx = (hi + 1) // 2, (ctx + 1) // 2
        c.update(causal=rng.random() < 0.8, window=rng.choice([0, 0, _log(rng, 1, 8192)]))
        c.update(ctx_lo=max(1, ctx // rng.choice([1, 3, 20])), ctx_hi=ctx)
    else:
        batch = _log(rng, 1, 40)
        hi = max(1, min(_log(rng, 1, 16384), 30000 // batch))
        ctx = _log(rng, 1, 2000) if op == "store" else _log(rng, 1, 300000)
        c.update(ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx)
    if op in ROPE:
        c.update(rot=rng.choice([32, 64] if hd == 64 else [32, 64, 96, 128, 128]),
                 layout=rng.choice(["half", "interleaved"]), theta=rng.choice([1e4, 5e5, 1e6]),
                 stretch=rng.choice([1.0, 1.0, 4.0, 8.0]), trained=rng.choice([0, 8192]), factor=rng.choice([1.0, 1.2]),
                 apart=rng.choice([0, 0, _log(rng, 1, 500000)]))
    if op == "rope":
        c.update(cache=rng.choice([dtype, "e4m3"]))
    c.update(batch=batch, rows_lo=rng.choice([1, hi]), rows_hi=hi)
    return c


def _lengths(case):
    """New rows and earlier context of every request: part of the case (the
    values behind them come from the seed)."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))

    def pick(lo, hi):
        if hi > 10 * max(lo, 1):
            return min(hi, max(lo, _log(r, max(lo, 1), hi)))
        return r.randint(lo, hi)

    rows = [pick(case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
    ctx = [pick(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    return rows, ctx


# ------------------------------------------------------------------ inputs

def _rows16(n, heads, hd, dtype, g):
    """Rows of normal values whose magnitude differs from row to row, head to
    head and, for some columns, from the others', as keys of real models do."""
    x = torch.randn(n, heads, hd, generator=g, device="cuda", dtype=torch.float32)
    size = torch.exp(0.5 * torch.randn(n, heads, 1, generator=g, device="cuda"))
    column = torch.exp(0.4 * torch.randn(heads, hd, generator=g, device="cuda"))
    return (x * size * column).to(DTYPES[dtype])


def _magnitude(x):
    """Index into E2M1 of the nearest value of x >= 0, ties to an even index."""
    return ((x > 0.25).to(torch.uint8) + (x >= 0.75) + (x > 1.25) + (x >= 1.75) + (x > 2.5) + (x >= 3.5) + (x > 5.0))


def _pack(x):
    """Rows [..., hd] in 4 bits, uint8 [..., hd * 5 / 8]: codes, the even of
    two in the lower half of a byte, then the scales as bfloat16."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1) / 6.0).to(torch.bfloat16)
    s = torch.where(s == 0, torch.ones_like(s), s)
    code = (_magnitude(b.abs() / s.float().unsqueeze(-1)) | (torch.signbit(b).to(torch.uint8) << 3)).flatten(-2)
    return torch.cat([code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)], -1)


def _unpack(rows, hd):
    """Values of such rows, float32 [..., hd]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    code = torch.stack([rows[..., :hd // 2] & 15, rows[..., :hd // 2] >> 4], -1).flatten(-2)
    s = rows[..., hd // 2:].contiguous().view(torch.bfloat16).float()
    return (lut[code.long()].unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def _fill_pages(case, n_pages, g):
    """One side of a cache whose every row holds some earlier row's values."""
    rows = _rows16(n_pages * case["page"], case["n_kv"], case["hd"], case["dtype"], g)
    rows = rows.view(n_pages, case["page"], case["n_kv"], case["hd"]).transpose(1, 2).contiguous()
    if case["cache"] == "e2m1":
        return torch.cat([_pack(r) for r in rows.split(256)]), None
    if case["cache"] != "e4m3":
        return rows, None
    scale = rows.abs().amax(-1).float() / E4M3_MAX
    return (rows.float() / scale[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")
    rows, ctx = _lengths(case)
    total = [r + c for r, c in zip(rows, ctx)]
    page = case["page"]
    # pages that this pass touches: all of a request's for attention, else those of the new rows
    first = [0 if case["op"] in ATTEND else c // page for c in ctx]
    need = [-(-t // page) for t in total]
    n_pages = sum(n - f for n, f in zip(need, first)) + 3
    k_pages, k_scale = _fill_pages(case, n_pages, g)
    v_pages, v_scale = _fill_pages(case, n_pages, g)
    order = torch.randperm(n_pages, generator=g, **dev).cpu().tolist()
    table = torch.zeros(len(total), max(need) + 1, dtype=torch.int32)
    at = 0
    for b, (f, n) in enumerate(zip(first, need)):
        table[b, f:n] = torch.tensor(order[at:at + n - f], dtype=torch.int32)
        at += n - f
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    n = start[-1]
    s = dict(case=case, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale,
             row_start=torch.tensor(start, dtype=torch.int32, **dev),
             kv_len=torch.tensor(total, dtype=torch.int64, **dev), page_table=table.cuda(),
             max_rows=max(rows), max_len=max(total), n_rows=n, positions=None)
    if case["op"] != "attention":
        s["k"] = _rows16(n, case["n_kv"], case["hd"], case["dtype"], g)
        s["v"] = _rows16(n, case["n_kv"], case["hd"], case["dtype"], g)
    if case["op"] == "store":
        s["k_back"], s["v_back"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    else:
        s["q"] = _rows16(n, case["n_q"], case["hd"], case["dtype"], g)
    if case["op"] in ROPE:
        s["q_out"] = torch.zeros_like(s["q"])
        if case["apart"]:
            s["positions"] = torch.randint(0, case["apart"], (n,), generator=g, **dev)
    if case["op"] in ATTEND:
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(n, case["n_q"], dtype=torch.float32, **dev)
    return s


# -------------------------------------------------------------- plain forms

def _places(s):
    """Page and row in the page of every new row, and its position."""
    n = torch.arange(s["n_rows"], device="cuda")
    b = torch.searchsorted(s["row_start"][1:].long(), n, right=True)
    pos = s["kv_len"][b] - (s["row_start"].long()[b + 1] - n)
    page = s["case"]["page"]
    return s["page_table"].long()[b, pos // page], pos % page, pos


def _frequencies(case):
    """Radians per position of every pair, float64."""
    f = case["theta"] ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    if not case["trained"]:
        return f / case["stretch"]
    g = ((case["trained"] * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
    return f * (g + (1.0 - g) / case["stretch"])


def _rotate(x, pos, case):
    """Rows [n, heads, hd] with their first `rot` columns rotated, float32."""
    angle = pos.double()[:, None] * _frequencies(case)
    c, s = (angle.cos() * case["factor"]).float()[:, None], (angle.sin() * case["factor"]).float()[:, None]
    x, rot = x.float(), case["rot"]
    half = case["layout"] == "half"
    a = x[..., :rot // 2] if half else x[..., 0:rot:2]
    b = x[..., rot // 2:rot] if half else x[..., 1:rot:2]
    a, b = a * c - b * s, b * c + a * s
    turned = torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    page, at, pos = _places(s)
    k = s["k"]
    if s["case"]["op"] in ROPE:
        where = pos if s["positions"] is None else s["positions"]
        k = _rotate(k, where, s["case"])
        s["q_out"].copy_(_rotate(s["q"], where, s["case"]))
    for x, pages, scale in ((k, s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        if s["case"]["cache"] == "e2m1":
            pages[page, :, at] = _pack(x)
        elif scale is None:
            pages[page, :, at] = x.to(pages.dtype)
        else:
            amax = x.abs().amax(-1).float()
            sc = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
            codes = (x.float() / sc[..., None]).to(torch.float8_e4m3fn)
            pages.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
            scale[page, :, at] = sc


def _plain_gather(s):
    page, at, _ = _places(s)
    s["k_back"].copy_(_unpack(s["k_pages"][page, :, at], s["case"]["hd"]))
    s["v_back"].copy_(_unpack(s["v_pages"][page, :, at], s["case"]["hd"]))


def _plain_attention(s, q):
    c = s["case"]
    B, H, G, hd, page = c["batch"], c["n_kv"], c["n_q"] // c["n_kv"], c["hd"], c["page"]
    start = s["row_start"].long()
    j = torch.arange(s["max_rows"], device="cuda")
    row = (start[:-1, None] + j).clamp(max=s["n_rows"] - 1)                       # [B, R]
    real = j < (start[1:] - start[:-1])[:, None]
    pos = s["kv_len"][:, None] - (start[1:, None] - row)
    key = torch.arange(s["max_len"], device="cuda")
    there = key < s["kv_len"][:, None]                                            # [B, S]
    at_page = s["page_table"].long()[:, key // page]
    at = (key % page).expand_as(at_page)
    k = _unpack(s["k_pages"][at_page, :, at], hd)                                 # [B, S, H, hd]
    v = _unpack(s["v_pages"][at_page, :, at], hd) * there[..., None, None]
    q = q[row].float().view(B, s["max_rows"], H, G, hd)
    see = there[:, None, :].expand(B, s["max_rows"], s["max_len"])
    if c["causal"]:
        see = see & (key <= pos[..., None])
    if c["window"]:
        see = see & (key > pos[..., None] - c["window"])
    q = q.permute(0, 2, 3, 1, 4).reshape(B, H, -1, hd)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * hd ** -0.5                       # [B, H, G R, S]
    z = z.view(B, H, G, s["max_rows"], s["max_len"])
    z.masked_fill_(~see[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(m > -math.inf, m, torch.zeros_like(m))).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, -1, s["max_len"]), v.transpose(1, 2))
    o = o.view(B, H, G, s["max_rows"], hd) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + total.log()).squeeze(-1)
    s["out"][row[real]] = o.permute(0, 3, 1, 2, 4).reshape(B, s["max_rows"], H * G, hd)[real].to(s["out"].dtype)
    s["lse"][row[real]] = lse.permute(0, 3, 1, 2).reshape(B, s["max_rows"], H * G)[real]


def _plain(s):
    op = s["case"]["op"]
    if op != "attention":
        _plain_append(s)
    if op == "store":
        _plain_gather(s)
    if op in ATTEND:
        _plain_attention(s, s["q_out"] if op == "step" else s["q"])


# ---------------------------------------------------------------- one pass

def _own(s):
    import block_speculative_decoding_ctx_gb300 as dfl
    c = s["case"]
    op = c["op"]
    if "cache" not in s:
        if c["cache"] == "e2m1":
            s["cache"] = dfl.paged_cache(s["k_pages"], s["v_pages"], format=dfl.DFLASH_CACHE_E2M1)
        else:
            s["cache"] = dfl.paged_cache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        s["ws"] = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(c["n_q"], c["n_kv"], c["hd"], s["max_rows"])
                                if op in ATTEND else dfl.dflash_paged_workspace_bytes())
        if op in ROPE:
            f = dfl.dflash_rope_frequencies(c["rot"], c["theta"], stretch=c["stretch"], trained=c["trained"], slow=1.0,
                                            fast=4.0)
            layout = dfl.DFLASH_ROPE_HALF if c["layout"] == "half" else dfl.DFLASH_ROPE_INTERLEAVED
            s["rope"] = dfl.dflash_rope_init(f, layout, factor=c["factor"])
    batch = (s["row_start"], s["kv_len"], s["page_table"])
    if op in ROPE:
        dfl.dflash_paged_append_rope(s["cache"], s["k"], s["v"], *batch, s["rope"], s["ws"], q=s["q"], q_out=s["q_out"],
                                     positions=s["positions"])
    elif op == "store":
        dfl.dflash_paged_append(s["cache"], s["k"], s["v"], *batch, s["ws"])
        dfl.dflash_paged_gather(s["cache"], s["k_back"], s["v_back"], *batch, s["ws"])
    if op in ATTEND:
        dfl.dflash_paged_attention(s["cache"], s["q_out"] if op == "step" else s["q"], s["out"], *batch, s["max_rows"],
                                   s["ws"], lse=s["lse"], scale=c["hd"] ** -0.5, causal=c["causal"], window=c["window"])


def run(state):
    if own:
        _own(state)
    else:
        _plain(state)
    op = state["case"]["op"]
    if op == "store":       # what was written, as the values that it stands for
        return {"k": state["k_back"], "v": state["v_back"]}
    if op == "rope":
        return {k: state[k] for k in ("k_pages", "v_pages", "k_scale", "v_scale", "q_out") if state[k] is not None}
    # a step's rows in the cache are seen through the attention that reads them
    return {"out": state["out"], "lse": state["lse"], **({"q_out": state["q_out"]} if op == "step" else {})}


# -------------------------------------------------------------- least work

def work(case):
    rows, ctx = _lengths(case)
    T = sum(rows)
    hd, n_kv, n_q, op = case["hd"], case["n_kv"], case["n_q"], case["op"]
    # one side of one cached position
    row = n_kv * {"e2m1": hd * 5 // 8, "e4m3": hd + 4}.get(case["cache"], 2 * hd)
    by = fl = 0.0
    if op != "attention":
        by += 2.0 * T * (row + n_kv * hd * 2)
        fl += 4.0 * T * n_kv * hd
    if op == "store":
        by += 2.0 * T * (row + n_kv * hd * 2)
        fl += 2.0 * T * n_kv * hd
    if op in ROPE:
        by += T * n_q * hd * 4.0 + (T * 8 if case["apart"] else 0)
        fl += 3.0 * T * (n_q + n_kv) * case["rot"]
    if op in ATTEND:
        W = case["window"]
        keys = pairs = 0
        for r, c in zip(rows, ctx):
            first = max(0, c + 1 - W) if W else 0
            keys += r + c - first
            for j in range(r):
                last = c + j + 1 if case["causal"] else r + c
                pairs += last - (max(0, c + j + 1 - W) if W else 0)
        # of a step, the rows that it writes need not be read back, nor its queries
        new = T if op == "step" else 0
        by += 2.0 * (keys - min(keys, new)) * row + T * n_q * (hd * (2 if new else 4) + 4)
        fl += 4.0 * hd * n_q * pairs
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------ in 64 bits, by definition

def _grid():
    return torch.tensor(E2M1, dtype=torch.float64, device="cuda")


def _exact_block_scales(x):
    """What a row's scales are, [..., hd / 16] float64: they are bfloat16."""
    s = (x.unflatten(-1, (-1, BLOCK)).abs().max(-1).values / 6.0).to(torch.bfloat16).double()
    s[s == 0] = 1.0
    return s


def _exact_quantised(x):
    """Rows in float64 as a cache in 4 bits holds them."""
    out = []
    for part in x.split(2048):
        s = _exact_block_scales(part).unsqueeze(-1)
        y = part.unflatten(-1, (-1, BLOCK)) / s
        # nearest of the eight magnitudes, ties to the even index
        d = (y.abs().unsqueeze(-1) - _grid()).abs()
        near = d == d.min(-1, keepdim=True).values
        index = torch.arange(8, device="cuda")
        even = torch.where(near & (index % 2 == 0), index, -1).max(-1).values
        any_ = torch.where(near, index, -1).max(-1).values
        best = torch.where(near.sum(-1) > 1, even, any_)
        out.append((torch.copysign(_grid()[best], y) * s).flatten(-2))
    return torch.cat(out)


def _exact_read(pages, hd):
    """Values of rows of bytes in float64."""
    low, high = (pages[..., :hd // 2] % 16).long(), (pages[..., :hd // 2] // 16).long()
    code = torch.stack([low, high], -1).flatten(-2)
    value = _grid()[code % 8] * (1.0 - 2.0 * (code // 8))
    scale = pages[..., hd // 2:].contiguous().view(torch.bfloat16).double()
    return value * scale.repeat_interleave(BLOCK, -1)


def _exact_turned(x, pos, case):
    """Rows in float64, pair by pair, as products with e^(i angle)."""
    out = x.double().clone()
    for j in range(case["rot"] // 2):
        f = case["theta"] ** (-2.0 * j / case["rot"])
        share = 1.0 if not case["trained"] else min(1.0, max(0.0, (case["trained"] * f / (2 * math.pi) - 1.0) / 3.0))
        if not case["trained"]:
            f = f / case["stretch"]
        else:
            f = share * f + (1.0 - share) * f / case["stretch"]
        a, b = (j, j + case["rot"] // 2) if case["layout"] == "half" else (2 * j, 2 * j + 1)
        turn = torch.polar(torch.full_like(pos, case["factor"], dtype=torch.float64), pos.double() * f)
        z = torch.complex(x[..., a].double(), x[..., b].double()) * turn[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_requests(s):
    start, lens = s["row_start"].tolist(), s["kv_len"].tolist()
    page = s["case"]["page"]
    for b, total in enumerate(lens):
        n = start[b + 1] - start[b]
        at = torch.arange(total - n, total, device="cuda")
        yield b, start[b], n, total, s["page_table"][b].long(), at // page, at % page


def exact(case, seed):
    s = prepare(case, seed)
    op, hd, page = case["op"], case["hd"], case["page"]
    if op == "store":
        return {side: _exact_quantised(s[side].double()) for side in ("k", "v")}
    out = {}
    if op in ROPE:
        where = torch.cat([torch.arange(t - n, t, device="cuda") for _, _, n, t, _, _, _ in _exact_requests(s)])
        if s["positions"] is not None:
            where = s["positions"]
        k, out["q_out"] = _exact_turned(s["k"], where, case), _exact_turned(s["q"], where, case)
        new = {"k": k, "v": s["v"].double()}
    if op == "rope":
        for side in ("k", "v"):
            pages = s[side + "_pages"].to(torch.float32).double()
            scale = None if s[side + "_scale"] is None else s[side + "_scale"].double()
            x = new[side]
            if scale is not None:
                top = x.abs().max(-1).values / E4M3_MAX
                top[top == 0] = 1.0
                x = x / top.unsqueeze(-1)
            for _, first, n, _, of, p, r in _exact_requests(s):
                pages[of[p], :, r] = x[first:first + n]
                if scale is not None:
                    scale[of[p], :, r] = top[first:first + n]
            out[side + "_pages"] = pages
            if scale is not None:
                out[side + "_scale"] = scale
        return out
    H, G = case["n_kv"], case["n_q"] // case["n_kv"]
    q = out["q_out"].to(DTYPES[case["dtype"]]) if op == "step" else s["q"]
    if op == "step":
        new = {side: _exact_quantised(x) for side, x in new.items()}
    att = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for _, first, n, total, of, _, _ in _exact_requests(s):
        k, v = (_exact_read(s[side + "_pages"][of[:-(-total // page)]], hd).transpose(0, 1).flatten(1, 2)[:, :total]
                for side in ("k", "v"))
        if op == "step":
            k[:, total - n:], v[:, total - n:] = (new[side][first:first + n].transpose(0, 1) for side in ("k", "v"))
        p = torch.arange(total - n, total, device="cuda").unsqueeze(1)
        t = torch.arange(total, device="cuda").unsqueeze(0)
        hide = torch.zeros(n, total, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= t > p
        if case["window"]:
            hide |= t <= p - case["window"]
        for h in range(case["n_q"]):
            z = q[first:first + n, h].double() @ k[h // G].T / math.sqrt(hd)
            z[hide] = -math.inf
            all_ = torch.logsumexp(z, 1)
            w = torch.exp(z - torch.where(all_ > -math.inf, all_, 0.0).unsqueeze(1))
            att[first:first + n, h] = w @ v[h // G]
            lse[first:first + n, h] = all_
    return {**out, "out": att, "lse": lse}
