"""The operators of the target's side of a speculative cycle, as measured cases:
writing new keys and values into a paged cache (16-bit or E4M3 codes with a
float32 scale per row and head), reading a range of it back, attention of a
chunk of new rows over it, and penalties, biases and token masks on the logits
of a block.

Every case exists in two forms: `own = False` computes it with elementary
torch operations, `own = True` calls the framework."""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CACHES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------- cases

def _attention(name, **kw):
    c = dict(name=name, op="attention", batch=1, rows_lo=1, rows_hi=1, ctx_lo=1, ctx_hi=1, n_q=40, n_kv=8,
             hd=128, page=64, dtype="bf16", cache="bf16", causal=True, window=0)
    c.update(kw)
    return c


def _move(name, op, **kw):
    c = dict(name=name, op=op, batch=1, rows_lo=1, rows_hi=1, ctx_lo=0, ctx_hi=0, n_kv=8, hd=128, page=64,
             dtype="bf16", cache="bf16")
    c.update(kw)
    return c


def _logits(name, **kw):
    c = dict(name=name, op="logits", batch=1, gamma=8, vocab=151936, dtype="f32", pad=0, counted=256, biased=32,
             draft=True, mask=True, allowed=0.5)
    c.update(kw)
    return c


def listed():
    return [
        # ordinary decoding of one request: one new token, a short context; latency counts
        _attention("attention one token", ctx_lo=1000, ctx_hi=1000),
        # the target scores blocks of 8 for a full batch, contexts of 8,192
        _attention("attention block 8 batch 32", batch=32, rows_lo=8, rows_hi=8, ctx_lo=8192, ctx_hi=8192),
        # blocks of 16 over very unequal contexts, cache in 8 bits
        _attention("attention ragged e4m3", batch=16, rows_lo=16, rows_hi=16, ctx_lo=512, ctx_hi=131072, page=128,
                   cache="e4m3"),
        # two prompts prefilled in chunks of 2,048 behind contexts of 8k to 16k; matrix products bound it
        _attention("attention prompt chunk", batch=2, rows_lo=2048, rows_hi=2048, ctx_lo=8192, ctx_hi=16384),
        # mixed chunk lengths, head dim 64, 7 query heads to a KV head, small pages, a sliding window, fp16
        _attention("attention odd window f16", batch=5, rows_lo=20, rows_hi=900, ctx_lo=100, ctx_hi=9000, n_q=14,
                   n_kv=2, hd=64, page=16, dtype="f16", cache="f16", window=1000),
        # a step's new rows of a full batch, quantised as they are written; latency counts
        _move("append block 8 e4m3", "append", batch=32, rows_lo=8, rows_hi=8, ctx_lo=40, ctx_hi=900, cache="e4m3"),
        # the rows of prompts, quantised as they are written
        _move("append prompts e4m3", "append", batch=9, rows_lo=900, rows_hi=8192, ctx_lo=0, ctx_hi=500,
              page=128, cache="e4m3"),
        # long prefixes read back from 8 bits, to hand them to another process
        _move("gather prefixes e4m3", "gather", batch=7, rows_lo=5000, rows_hi=32768, page=64, cache="e4m3"),
        # a few short ranges of a 16-bit cache, head dim 64, small pages
        _move("gather short f16", "gather", batch=3, rows_lo=1, rows_hi=77, ctx_lo=5, ctx_hi=300, n_kv=2, hd=64,
              page=16, dtype="f16", cache="f16"),
        # one request's block before verification: latency counts
        _logits("logits one block"),
        # a full batch of blocks of 16 with every rule in use
        _logits("logits batch 32 block 16", batch=32, gamma=16, counted=2000, biased=200),
        # an odd vocabulary, padded bf16 rows as a target writes them, no mask
        _logits("logits odd bf16", batch=3, gamma=5, vocab=5003, dtype="bf16", pad=21, mask=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "gather", "logits"])
    hd = rng.choice([64, 128])
    n_kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    cache = rng.choice([dtype, "e4m3"])
    if op == "attention":
        if rng.random() < 0.5:      # decoding and block verification
            batch, hi, ctx = _log(rng, 1, 48), _log(rng, 1, 16), _log(rng, 1, 60000)
            ctx = max(1, min(ctx, 250000 // batch))
        else:                       # chunks of prompts, no more work than the listed one's
            batch, hi, ctx = _log(rng, 1, 4), _log(rng, 17, 2048), _log(rng, 1, 14000)
            while batch * hi * (ctx + hi) * n_kv * group * hd > 2 ** 38:
                hi, ctx = (hi + 1) // 2, (ctx + 1) // 2
        return dict(op=op, batch=batch, rows_lo=rng.choice([1, hi]), rows_hi=hi, ctx_lo=max(1, ctx // rng.choice([1, 3, 20])),
                    ctx_hi=ctx, n_q=n_kv * group, n_kv=n_kv, hd=hd, page=page, dtype=dtype, cache=cache,
                    causal=rng.random() < 0.8, window=rng.choice([0, 0, _log(rng, 1, 8192)]))
    if op in ("append", "gather"):
        batch = _log(rng, 1, 40)
        hi = max(1, min(_log(rng, 1, 16384), 100000 // batch))
        ctx = _log(rng, 1, 2000)
        return dict(op=op, batch=batch, rows_lo=rng.choice([1, hi]), rows_hi=hi, ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx,
                    n_kv=n_kv, hd=hd, page=page, dtype=dtype, cache=cache)
    batch, gamma = _log(rng, 1, 32), _log(rng, 2, 16)
    vocab = _log(rng, 1000, 151936)
    return dict(op=op, batch=batch, gamma=gamma, vocab=vocab, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                pad=rng.choice([0, rng.randrange(1, 64)]), counted=_log(rng, 1, min(3000, vocab)), biased=_log(rng, 1, 300),
                draft=rng.random() < 0.8, mask=rng.random() < 0.7, allowed=rng.choice([0.001, 0.5, 0.99]))


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

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows16(n, heads, hd, dtype, g):
    """Rows of normal values whose magnitude differs from row to row and head
    to head, as keys and values of real models do."""
    x = torch.randn(n, heads, hd, generator=g, device="cuda", dtype=torch.float32)
    size = torch.exp(0.5 * torch.randn(n, heads, 1, generator=g, device="cuda"))
    return (x * size).to(DTYPES[dtype])


def _fill_pages(case, n_pages, g):
    """One side of a cache whose every row holds some earlier row's values:
    pages [n_pages, heads, page, hd] and, in 8 bits, their scales."""
    rows = _rows16(n_pages * case["page"], case["n_kv"], case["hd"], case["dtype"], g)
    rows = rows.view(n_pages, case["page"], case["n_kv"], case["hd"]).transpose(1, 2).contiguous()
    if case["cache"] != "e4m3":
        return rows.to(CACHES[case["cache"]]), None
    scale = rows.abs().amax(-1).float() / E4M3_MAX
    return (rows.float() / scale[..., None]).to(torch.float8_e4m3fn), scale


def _prepare_paged(case, seed):
    g = _gen(seed)
    rows, ctx = _lengths(case)
    total = [r + c for r, c in zip(rows, ctx)]
    need = [-(-t // case["page"]) for t in total]
    width = max(need) + 1
    n_pages = sum(need) + 3
    k_pages, k_scale = _fill_pages(case, n_pages, g)
    v_pages, v_scale = _fill_pages(case, n_pages, g)
    order = torch.randperm(n_pages, generator=g, device="cuda").cpu().tolist()
    table = [[0] * width for _ in total]
    at = 0
    for b, n in enumerate(need):
        table[b][:n] = order[at:at + n]
        at += n
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    dev = dict(device="cuda")
    s = dict(case=case, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale,
             row_start=torch.tensor(start, dtype=torch.int32, **dev),
             kv_len=torch.tensor(total, dtype=torch.int64, **dev),
             page_table=torch.tensor(table, dtype=torch.int32, **dev),
             max_rows=max(rows), max_len=max(total), n_rows=start[-1])
    n = start[-1]
    if case["op"] == "attention":
        s["q"] = _rows16(n, case["n_q"], case["hd"], case["dtype"], g) * 1.5
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(n, case["n_q"], dtype=torch.float32, **dev)
    elif case["op"] == "append":
        s["k"] = _rows16(n, case["n_kv"], case["hd"], case["dtype"], g)
        s["v"] = _rows16(n, case["n_kv"], case["hd"], case["dtype"], g)
    else:
        s["k"] = torch.zeros(n, case["n_kv"], case["hd"], dtype=DTYPES[case["dtype"]], **dev)
        s["v"] = torch.zeros_like(s["k"])
    return s


def _prepare_logits(case, seed):
    g = _gen(seed)
    B, G, V = case["batch"], case["gamma"], case["vocab"]
    dev = dict(device="cuda")
    words = (V + 31) // 32
    padded = torch.randn(B, G, V + case["pad"], generator=g, **dev) * 3.0
    logits = padded.to(DTYPES[case["dtype"]])[:, :, :V]
    counts = torch.zeros(B, V, dtype=torch.int32, **dev)
    seen = torch.randint(0, V, (B, case["counted"]), generator=g, **dev)
    counts.scatter_add_(1, seen, torch.ones_like(seen, dtype=torch.int32))
    prompt = torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=g, **dev)
    prompt &= torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=g, **dev)
    s = dict(case=case, logits=logits, out=torch.empty(B, G, V, **dev), counts=counts, prompt_mask=prompt.to(torch.int32),
             repetition=1.0 + 0.3 * torch.rand(B, generator=g, **dev), frequency=0.5 * torch.rand(B, generator=g, **dev),
             presence=torch.rand(B, generator=g, **dev) - 0.2, draft=None, allow=None)
    n = case["biased"]
    s["bias_start"] = (torch.arange(B + 1, **dev) * n).to(torch.int32)
    s["bias_ids"] = torch.randint(0, V, (B * n,), generator=g, **dev).to(torch.int32)
    s["bias_vals"] = 2.0 * torch.randn(B * n, generator=g, **dev)
    if case["draft"]:
        # drafts repeat now and then, and fall on tokens that were seen
        d = seen[:, torch.randint(0, case["counted"], (G - 1,), generator=g, **dev)]
        fresh = torch.randint(0, V, (B, G - 1), generator=g, **dev)
        s["draft"] = torch.where(torch.rand(B, G - 1, generator=g, **dev) < 0.5, d, fresh).to(torch.int32)
    if case["mask"]:
        bits = torch.rand(B, G, words, 32, generator=g, **dev) < case["allowed"]
        weight = torch.ones(32, dtype=torch.int64, **dev) << torch.arange(32, **dev)
        s["allow"] = (bits * weight).sum(-1).to(torch.int64).to(torch.int32)
    return s


def prepare(case, seed):
    return _prepare_logits(case, seed) if case["op"] == "logits" else _prepare_paged(case, seed)


# -------------------------------------------------------------- plain forms

def _places(s):
    """Page and row in the page of every new row, and its request."""
    n = torch.arange(s["n_rows"], device="cuda")
    b = torch.searchsorted(s["row_start"][1:].long(), n, right=True)
    start = s["row_start"].long()
    pos = s["kv_len"][b] - (start[b + 1] - n)
    page = s["case"]["page"]
    return s["page_table"].long()[b, pos // page], pos % page, b, pos


def _read(pages, scale, page, at):
    x = pages[page, :, at].float() if pages.dtype != torch.float8_e4m3fn else \
        pages.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).float()
    return x if scale is None else x * scale[page, :, at][..., None]


def _plain_append(s):
    page, at, _, _ = _places(s)
    for x, pages, scale in ((s["k"], s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        if scale is None:
            pages[page, :, at] = x
        else:
            amax = x.abs().amax(-1).float()
            sc = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
            codes = (x.float() / sc[..., None]).to(torch.float8_e4m3fn)
            pages.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
            scale[page, :, at] = sc


def _plain_gather(s):
    page, at, _, _ = _places(s)
    s["k"].copy_(_read(s["k_pages"], s["k_scale"], page, at))
    s["v"].copy_(_read(s["v_pages"], s["v_scale"], page, at))


def _plain_attention(s):
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
    k = _read(s["k_pages"], s["k_scale"], at_page, at)                            # [B, S, H, hd]
    v = _read(s["v_pages"], s["v_scale"], at_page, at) * there[..., None, None]
    q = s["q"][row].float().view(B, s["max_rows"], H, G, hd)
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


def _bits(words, V):
    v = torch.arange(V, device="cuda")
    return ((words[..., v // 32] >> (v % 32)) & 1) != 0


def _plain_logits(s):
    B, G, V = s["out"].shape
    c = s["counts"][:, None, :].expand(B, G, V)
    if s["draft"] is not None:
        more = torch.zeros(B, G, V, dtype=torch.int32, device="cuda")
        more[:, 1:].scatter_add_(2, s["draft"].long()[..., None], torch.ones_like(s["draft"])[..., None])
        c = c + more.cumsum(1)
    seen = (c > 0) | _bits(s["prompt_mask"], V)[:, None]
    z = s["logits"].float()
    r = s["repetition"][:, None, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = z - (s["frequency"][:, None, None] * c + s["presence"][:, None, None] * (c > 0))
    bias = torch.zeros(B, V, dtype=torch.float64, device="cuda")
    n = torch.arange(s["bias_ids"].numel(), device="cuda")
    b = torch.searchsorted(s["bias_start"][1:].long(), n, right=True)
    bias.index_put_((b, s["bias_ids"].long()), s["bias_vals"].double(), accumulate=True)
    z = z + bias.float()[:, None]
    if s["allow"] is not None:
        z = z.masked_fill(~_bits(s["allow"], V), -math.inf)
    s["out"].copy_(z)


# ---------------------------------------------------------------- one pass

def _own(s):
    import block_speculative_decoding_ctx_gb300 as dfl
    c = s["case"]
    if c["op"] == "logits":
        if "ws" not in s:
            s["ws"] = dfl.workspace(dfl.dflash_logits_adjust_workspace_bytes())
        dfl.dflash_logits_adjust(s["logits"], s["out"], s["ws"], counts=s["counts"], prompt_mask=s["prompt_mask"],
                                 draft=s["draft"], repetition=s["repetition"], frequency=s["frequency"],
                                 presence=s["presence"], bias_start=s["bias_start"], bias_ids=s["bias_ids"],
                                 bias_vals=s["bias_vals"], allow=s["allow"])
        return
    if "cache" not in s:
        s["cache"] = dfl.paged_cache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        s["ws"] = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(c["n_q"], c["n_kv"], c["hd"], s["max_rows"])
                                if c["op"] == "attention" else dfl.dflash_paged_workspace_bytes())
    if c["op"] == "append":
        dfl.dflash_paged_append(s["cache"], s["k"], s["v"], s["row_start"], s["kv_len"], s["page_table"], s["ws"])
    elif c["op"] == "gather":
        dfl.dflash_paged_gather(s["cache"], s["k"], s["v"], s["row_start"], s["kv_len"], s["page_table"], s["ws"])
    else:
        dfl.dflash_paged_attention(s["cache"], s["q"], s["out"], s["row_start"], s["kv_len"], s["page_table"],
                                   s["max_rows"], s["ws"], lse=s["lse"], scale=c["hd"] ** -0.5, causal=c["causal"],
                                   window=c["window"])


def run(state):
    op = state["case"]["op"]
    if own:
        _own(state)
    elif op == "logits":
        _plain_logits(state)
    elif op == "append":
        _plain_append(state)
    elif op == "gather":
        _plain_gather(state)
    else:
        _plain_attention(state)
    if op == "logits":
        return {"out": state["out"]}
    if op == "attention":
        return {"out": state["out"], "lse": state["lse"]}
    if op == "gather":
        return {"k": state["k"], "v": state["v"]}
    return {k: state[k] for k in ("k_pages", "v_pages", "k_scale", "v_scale") if state[k] is not None}


# -------------------------------------------------------------- least work

def work(case):
    if case["op"] == "logits":
        B, G, V = case["batch"], case["gamma"], case["vocab"]
        n = B * G * V
        size = 4 if case["dtype"] == "f32" else 2
        by = n * (size + 4) + B * V * (4 + 0.125) + (n / 8 if case["mask"] else 0) + B * case["biased"] * 8
        return {"bytes": by, "flops": 8.0 * n}
    rows, ctx = _lengths(case)
    T = sum(rows)
    width = 1 if case["cache"] == "e4m3" else 2
    row = case["n_kv"] * (case["hd"] * width + (4 if case["cache"] == "e4m3" else 0))   # one side of one position
    if case["op"] != "attention":
        return {"bytes": 2.0 * T * (row + case["n_kv"] * case["hd"] * 2), "flops": 4.0 * T * case["n_kv"] * case["hd"]}
    W = case["window"]
    keys = pairs = 0
    for r, c in zip(rows, ctx):
        first = max(0, c + 1 - W) if W else 0
        keys += r + c - first
        for j in range(r):
            last = c + j + 1 if case["causal"] else r + c
            pairs += last - (max(0, c + j + 1 - W) if W else 0)
    by = 2.0 * keys * row + T * case["n_q"] * (case["hd"] * 4 + 4)
    return {"bytes": by, "flops": 4.0 * case["hd"] * case["n_q"] * pairs}


# ------------------------------------------------------ in 64 bits, by definition

def _exact_row_list(s):
    start, lens, table = s["row_start"].tolist(), s["kv_len"].tolist(), s["page_table"].tolist()
    page = s["case"]["page"]
    for b, total in enumerate(lens):
        n = start[b + 1] - start[b]
        yield b, start[b], n, total, torch.tensor(table[b][:-(-total // page)], device="cuda")


def _exact_request(s, side, pages, total):
    """Keys or values of one request in order, float64 [Hkv, total, hd]."""
    x = s[side + "_pages"].view(torch.uint8)[pages].view(s[side + "_pages"].dtype).to(torch.float64)
    if s[side + "_scale"] is not None:
        x *= s[side + "_scale"][pages].double().unsqueeze(-1)
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :total]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logits":
        return {"out": _exact_logits(s)}
    if case["op"] == "append":
        out = {}
        for side in ("k", "v"):
            pages = s[side + "_pages"].to(torch.float32).double()
            scale = None if s[side + "_scale"] is None else s[side + "_scale"].double()
            x = s[side].double()
            if scale is not None:
                top = x.abs().max(-1).values / E4M3_MAX
                top[top == 0] = 1.0
                x = x / top.unsqueeze(-1)
            for b, first, n, total, of in _exact_row_list(s):
                at = torch.arange(total - n, total, device="cuda")
                p, r = of[at // case["page"]], at % case["page"]
                pages[p, :, r] = x[first:first + n]
                if scale is not None:
                    scale[p, :, r] = top[first:first + n]
            out[side + "_pages"] = pages
            if scale is not None:
                out[side + "_scale"] = scale
        return out
    if case["op"] == "gather":
        out = {"k": s["k"].double(), "v": s["v"].double()}
        for b, first, n, total, of in _exact_row_list(s):
            for side in ("k", "v"):
                out[side][first:first + n] = _exact_request(s, side, of, total)[:, total - n:].transpose(0, 1)
        return out
    H, G = case["n_kv"], case["n_q"] // case["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, first, n, total, of in _exact_row_list(s):
        k, v = _exact_request(s, "k", of, total), _exact_request(s, "v", of, total)
        p = torch.arange(total - n, total, device="cuda").unsqueeze(1)
        t = torch.arange(total, device="cuda").unsqueeze(0)
        hide = torch.zeros(n, total, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= t > p
        if case["window"]:
            hide |= t <= p - case["window"]
        for h in range(case["n_q"]):
            z = s["q"][first:first + n, h].double() @ k[h // G].T / math.sqrt(case["hd"])
            z[hide] = -math.inf
            all_ = torch.logsumexp(z, 1)
            w = torch.exp(z - torch.where(all_ > -math.inf, all_, 0.0).unsqueeze(1))
            out[first:first + n, h] = w @ v[h // G]
            lse[first:first + n, h] = all_
    return {"out": out, "lse": lse}


def _exact_logits(s):
    B, G, V = s["out"].shape
    words = torch.arange(V, device="cuda")
    out = torch.empty(B, G, V, dtype=torch.float64, device="cuda")
    for b in range(B):
        c = s["counts"][b].double()
        prompt = (s["prompt_mask"][b].long()[words // 32] >> (words % 32)) % 2 == 1
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        lo, hi = s["bias_start"][b:b + 2].tolist()
        bias.index_add_(0, s["bias_ids"][lo:hi].long(), s["bias_vals"][lo:hi].double())
        r, f, p = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
        for i in range(G):
            if i and s["draft"] is not None:
                c[s["draft"][b, i - 1].long()] += 1
            z = s["logits"][b, i].double()
            hit = prompt | (c > 0)
            z[hit] = torch.where(z > 0, z / r, z * r)[hit]
            z = z - f * c - p * (c > 0).double() + bias
            if s["allow"] is not None:
                ok = (s["allow"][b, i].long()[words // 32] >> (words % 32)) % 2 == 1
                z[~ok] = -math.inf
            out[b, i] = z
    return out
