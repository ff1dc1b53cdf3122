"""Inputs and bounds shared by the tests of the target-side operators."""

import numpy as np
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import target as ot

F8 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def to64(t):
    """float64 numpy copy of a CUDA or CPU tensor (codes stay uint8)."""
    if t is None:
        return None
    if t.dtype == F8:
        t = t.view(torch.uint8)
    return t.cpu().numpy() if t.dtype == torch.uint8 else t.double().cpu().numpy()


class Paged:
    """A paged cache with requests in shuffled pages.  Whatever no request
    owns holds NaN (E4M3: NaN codes and NaN scales)."""

    def __init__(self, lens, rows, n_kv=2, hd=64, page=16, dtype=torch.bfloat16, e4m3=False, seed=0, extra=2,
                 spread=0, fill=True, garbage=True):
        assert len(lens) == len(rows)
        rng = np.random.default_rng(seed)
        self.lens, self.rows, self.page, self.dtype, self.e4m3 = list(lens), list(rows), page, dtype, e4m3
        need = [-(-n // page) for n in lens]
        self.width = max(max(need), 1) + 1
        self.n_pages = sum(need) + extra
        perm = rng.permutation(self.n_pages)
        table = np.full((len(lens), self.width), -1, dtype=np.int32)   # unneeded entries: never read
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table_np = table
        shape = (self.n_pages, n_kv, page, hd)
        cell = torch.uint8 if e4m3 else dtype
        flat = n_kv * page * hd
        self.pages, self.scale = [], []
        g = torch.Generator().manual_seed(seed)
        for _ in range(2):
            x = torch.randn(shape, generator=g) * torch.exp(0.7 * torch.randn(shape[:3] + (1,), generator=g))
            if e4m3:
                codes, scale = ot.quantize(x.to(dtype).float().numpy())
                data, scale = torch.from_numpy(codes), torch.from_numpy(scale)
            else:
                data, scale = x.to(dtype), None
            if garbage:
                owned = np.zeros(shape[:1] + shape[2:3], dtype=bool)
                for b, n in enumerate(lens):
                    for s in range(n if fill else 0):
                        owned[table[b, s // page], s % page] = True
                free = torch.from_numpy(~owned)[:, None, :].expand(shape[:3])
                data[free] = 0x7F if e4m3 else float("nan")
                if e4m3:
                    scale[free] = float("nan")
            store = torch.zeros(self.n_pages, flat + spread, dtype=cell, device="cuda")
            store[:, :flat] = data.reshape(self.n_pages, flat).cuda()
            view = store.as_strided(shape, (flat + spread, page * hd, hd, 1))
            self.pages.append(view.view(F8) if e4m3 else view)
            self.scale.append(None if scale is None else scale.cuda())
        self.cache = dfl.paged_cache(self.pages[0], self.pages[1], self.scale[0], self.scale[1])
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.start_np = start
        self.n_rows = int(start[-1])
        self.row_start = torch.from_numpy(start).cuda()
        self.kv_len = torch.tensor(self.lens, dtype=torch.int64, device="cuda")
        self.table = torch.from_numpy(table).cuda()
        self.batch = (self.row_start, self.kv_len, self.table)

    def host(self):
        """(K pages, V pages, K scales, V scales) as numpy."""
        return (to64(self.pages[0]), to64(self.pages[1]), to64(self.scale[0]), to64(self.scale[1]))


def rows_tensor(n, heads, hd, dtype, seed, extra=0, order="rhd", size=1.0):
    """Random rows [n + extra, heads, hd] on the GPU; order "hrd" lays heads
    outermost, "wide" leaves room between rows."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n + extra, heads, hd, generator=g) * size).to(dtype)
    if order == "hrd":
        return x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    if order == "wide":
        big = torch.zeros(n + extra, heads + 3, hd + 8, dtype=dtype, device="cuda")
        big[:, 1:heads + 1, :hd] = x.cuda()
        return big[:, 1:heads + 1, :hd]
    return x.cuda()


def attention_reference(p, q, causal, window, scale, only=None):
    """out, lse and the bounds on their errors (see attention_bound), numpy
    [rows, n_q, hd] and [rows, n_q]."""
    kp, vp, ks, vs = p.host()
    q64 = to64(q)
    n, n_q, hd = q64.shape
    out, lse = np.zeros((n, n_q, hd)), np.zeros((n, n_q))
    b_out, b_lse = np.zeros((n, n_q, hd)), np.zeros((n, n_q))
    for b, length in enumerate(p.lens):
        s0, s1 = p.start_np[b], p.start_np[b + 1]
        if s1 == s0 or (only is not None and b not in only):
            continue
        k = ot.sequence(kp, ks, p.table_np[b], length, p.page, p.e4m3)
        v = ot.sequence(vp, vs, p.table_np[b], length, p.page, p.e4m3)
        o, l, mean, size = ot.attention(q64[s0:s1], k, v, length, causal, window, scale)
        out[s0:s1], lse[s0:s1] = o, l
        b_out[s0:s1], b_lse[s0:s1] = attention_bound(o, l, mean, size, v, length, hd, p.dtype)
    return out, lse, b_out, b_lse


def attention_bound(out, lse, mean, size, v, length, hd, dtype):
    """Largest error the kernels' arithmetic allows, before any run of them.

    With A = sum softmax |v| per output value, u the half step of the 16-bit
    type, n keys and e = 2^-24:
      scores   products exact in float32, hd additions and one fused scale,
               each off by at most 2 e of the partial sums (2 e: the tensor
               cores may truncate): dz <= 2 (hd + 4) e Z with Z = scale * sum
               |q||k|; also the reference subtracted and 2^x (2 ulp, its
               argument off by 2 e |z|): another 4 e Z + 8 e.  A weight is
               then off by the factor 1 +- d, d = dz + ..., a softmax mean by
               at most 2 d A;
      weights  rounded to the 16-bit type before the second product: u A, and
               in fp16 an absolute 2^-25 of a weight whose reference is at
               least 1: 2^-25 sum |v|;  for E4M3 caches they carry the value
               scales relative to the largest and a factor 2^8 before they
               become fp16: 2^-33 n max |v| at most, twice that allowed;
      sums     n additions of either product, 2 e each: 2 n e A twice;
      rescaling and merging of partial results, a handful of roundings: 32 e A;
      output   rounded once: u |out|, or 2^-25 where fp16 is subnormal."""
    u, e = HALF_STEP[dtype], 2.0 ** -24
    d = 2 * (hd + 4) * e * size + 4 * e * size + 8 * e
    top_v = np.abs(v).max() if v.size else 0.0
    few = 2.0 ** -25 * np.repeat(np.abs(v).sum(0), out.shape[1] // v.shape[1], axis=0) + 2.0 ** -32 * length * top_v
    rel = u + 2 * d[..., None] + 4 * length * e + 32 * e
    b_out = (rel * mean + few + u * np.abs(out)) * 1.01 + 2.0 ** -25
    b_lse = 2 * d + 2 * length * e + 8 * e * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return b_out, b_lse


def run_attention(p, q, out=None, lse=True, max_rows=None, ws=None, **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    lse_t = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    max_rows = max(p.rows) if max_rows is None else max_rows
    if ws is None:
        ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(q.shape[1], p.pages[0].shape[1], q.shape[2], max_rows))
    dfl.dflash_paged_attention(p.cache, q, out, *p.batch, max_rows, ws, lse=lse_t, **kw)
    torch.cuda.synchronize()
    return out, lse_t, dfl.dflash_read_status(ws)


def check_attention(p, q, out, lse, causal=True, window=0, scale=None, only=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, want_l, b_out, b_lse = attention_reference(p, q, causal, window, scale, only)
    rows = np.zeros(q.shape[0], dtype=bool)
    for b in range(len(p.lens)):
        if only is None or b in only:
            rows[p.start_np[b]:p.start_np[b + 1]] = True
    got = to64(out)
    err = np.abs(got - want)[rows]
    assert np.isfinite(got[rows]).all()
    worst = (err / b_out[rows]).max() if rows.any() else 0.0
    assert worst <= 1.0, f"attention is {worst:.2f} of its bound off"
    assert (got[~rows] == 7.0).all(), "rows of no request were written"
    if lse is not None:
        got_l = to64(lse)
        empty = ~np.isfinite(want_l)
        assert (got_l[rows][empty[rows]] == -np.inf).all()
        at = rows[:, None] & ~empty
        worst = (np.abs(got_l[at] - want_l[at]) / b_lse[at]).max() if at.any() else 0.0
        assert worst <= 1.0, f"lse is {worst:.2f} of its bound off"
        assert (got_l[~rows] == 7.0).all()
