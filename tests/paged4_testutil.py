"""Inputs and bounds of the tests of caches in 4 bits and of rotary positions."""

import numpy as np
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import e2m1
from target_testutil import HALF_STEP, to64

BF, F16 = torch.bfloat16, torch.float16


class Paged4:
    """A cache in 4 bits with requests in shuffled pages.  Whatever no request owns
    holds NaN scales.  values: [requests][positions, heads, hd] float rows of K and V
    to hold instead of random ones."""

    def __init__(self, lens, rows, n_kv=2, hd=64, page=16, dtype=BF, seed=0, extra=2, spread=0, garbage=True, sizes=0.7,
                 values=None):
        rng = np.random.default_rng(seed)
        self.lens, self.rows, self.page, self.dtype, self.hd, self.n_kv = list(lens), list(rows), page, dtype, hd, n_kv
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
        shape = (self.n_pages, n_kv, page)
        rec = hd * 5 // 8
        flat = n_kv * page * rec
        self.pages = []
        for side in range(2):
            data = np.empty(shape + (rec,), dtype=np.uint8)
            for p0 in range(0, self.n_pages, 512):
                part = rng.standard_normal((min(512, self.n_pages - p0),) + shape[1:] + (hd,)) * \
                    np.exp(sizes * rng.standard_normal((min(512, self.n_pages - p0),) + shape[1:] + (1,)))
                part = torch.from_numpy(part).to(dtype).float().numpy()
                data[p0:p0 + 512] = pack_fast(part)
            if values is not None:
                for b, n in enumerate(lens):
                    s = np.arange(n)
                    data[table[b, s // page], :, s % page] = e2m1.pack(values[side][b])
            if garbage:
                owned = np.zeros((self.n_pages, page), dtype=bool)
                for b, n in enumerate(lens):
                    s = np.arange(n)
                    owned[table[b, s // page], s % page] = True
                free = np.broadcast_to(~owned[:, None, :], shape)
                data[free] = 0xFF                                     # NaN scales, all codes -6
            store = torch.zeros(self.n_pages, flat + spread, dtype=torch.uint8, device="cuda")
            store[:, :flat] = torch.from_numpy(data.reshape(self.n_pages, flat)).cuda()
            self.pages.append(store.as_strided(shape + (rec,), (flat + spread, page * rec, rec, 1)))
        self.cache = dfl.paged_cache(self.pages[0], self.pages[1], format=dfl.DFLASH_CACHE_E2M1)
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.start_np = start
        self.n_rows = int(start[-1])
        self.row_start = torch.from_numpy(start).cuda()
        self.kv_len = torch.tensor(self.lens, dtype=torch.int64, device="cuda")
        self.table = torch.from_numpy(table).cuda()
        self.batch = (self.row_start, self.kv_len, self.table)

    def host(self):
        return [t.cpu().numpy() for t in self.pages]


def pack_fast(x):
    """e2m1.pack for large inputs: the same rounding by comparisons."""
    x = np.asarray(x, dtype=np.float32)
    s = e2m1.scales(x)
    y = np.abs(x.reshape(s.shape + (e2m1.BLOCK,)) / s.astype(np.float32)[..., None])
    mids = (e2m1.MAGNITUDE[1:] + e2m1.MAGNITUDE[:-1]) / 2
    c = np.zeros(y.shape, dtype=np.uint8)
    for i, m in enumerate(mids):
        c += (y > m) if i % 2 == 0 else (y >= m)
    c = c.reshape(x.shape) | ((x < 0).astype(np.uint8) << 3)
    bits = e2m1.bf16_bits(s.astype(np.float32))
    two = np.stack([bits & 0xFF, bits >> 8], -1).astype(np.uint8).reshape(x.shape[:-1] + (-1,))
    return np.concatenate([c[..., 0::2] | (c[..., 1::2] << 4), two], -1)


def reference(p, q, causal, window, scale, only=None, max_rows=None):
    """out, lse and the bounds on their errors (see bound)."""
    together = (max_rows or max(p.rows)) * q.shape[1] // p.n_kv > 128
    kp, vp = p.host()
    q64 = to64(q)
    n, n_q, hd = q64.shape
    out, lse = np.zeros((n, n_q, hd)), np.full((n, n_q), -np.inf)
    b_out, b_lse = np.zeros((n, n_q, hd)), np.zeros((n, n_q))
    group = n_q // p.n_kv
    for b, length in enumerate(p.lens):
        s0, s1 = p.start_np[b], p.start_np[b + 1]
        if s1 == s0 or length == 0 or (only is not None and b not in only):
            continue
        k = e2m1.sequence(kp, p.table_np[b], length, p.page)
        v = e2m1.sequence(vp, p.table_np[b], length, p.page)
        at = np.arange(length)
        vs = np.abs(e2m1.split(vp[p.table_np[b][at // p.page], :, at % p.page])[1]).max(-1)      # [length, heads]
        if together:            # of 32 neighbouring positions the largest
            vs = np.repeat([vs[i:i + 32].max(0) for i in range(0, length, 32)], 32, 0)[:length]
        power = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(vs, 2.0 ** -140))), -64)
        ks = np.abs(e2m1.split(kp[p.table_np[b][at // p.page], :, at % p.page])[1]).max(-1)      # (their largest counts)
        pos = np.arange(length - (s1 - s0), length)[:, None]
        hide = np.zeros((s1 - s0, length), dtype=bool)
        if causal:
            hide |= at > pos
        if window:
            hide |= at <= pos - window
        for h in range(n_q):
            g = h // group
            x = q64[s0:s1, h]
            z = x @ k[:, g].T * scale
            size = np.abs(x) @ np.abs(k[:, g]).T * scale
            size = np.where(hide, 0, size).max(1)
            most = np.where(hide, 0, ks[None, :, g]).max(1) * np.abs(x).max(1) * scale * hd
            z[hide] = -np.inf
            m = z.max(1)
            seen = m > -np.inf
            w = np.exp(z - np.where(seen, m, 0)[:, None])
            tot = w.sum(1)
            w /= np.where(seen, tot, 1)[:, None]
            out[s0:s1, h] = w @ v[:, g]
            lse[s0:s1, h] = np.where(seen, m + np.log(np.where(seen, tot, 1)), -np.inf)
            mean = w @ np.abs(v[:, g])
            few = (w * power[None, :, g]).max(1) * (2.0 ** -4 if together else 1.0)
            bo, bl = bound(out[s0:s1, h], lse[s0:s1, h], mean, size, most, few, w @ vs[:, g], length, hd, p.dtype)
            b_out[s0:s1, h] = np.where(seen[:, None], bo, 0)
            b_lse[s0:s1, h] = np.where(seen, bl, 0)
    return out, lse, b_out, b_lse


def bound(out, lse, mean, size, most, few, mean_scale, n, hd, dtype):
    """Largest error the kernel's arithmetic allows, derived before any run of it.

    With A = sum softmax |v| per output value (mean), u the half step of the
    output's type, n keys, e = 2^-24, Z = scale * sum |q||k| (size):
      operands  q times a power of two in fp16, its largest value in [2^14, 2^15):
                off by 2^-25 of that unit, 2^-39 of the row's largest; k and v times
                a power of two, scales in [.., 2^13): off by the scale's rounding,
                2^-25 times 6, and the product's, 2^-25, of 2^12: 2^-34 of the row's
                largest scale (less where nothing is subnormal).  Scores: hd times
                either, with the other operand's largest, 6 scales: most holds scale
                * hd * max|q| * max scale, so dz <= (6 2^-38 + 2^-34) most; values:
                2^-34 of the mean of the rows' largest scales;
      scores    products exact in float32, hd additions, 2 e of the partial sums
                each (the tensor cores may truncate), the factor and its product
                with the score: 2 (hd + 4) e Z; the value row's power added, the
                reference subtracted and 2^x: their sum is at most |z| + 130 in
                log2 terms: 6 e (Z + 130); a softmax mean is then off by 2 d A;
      weights   rounded to fp16: 2^-11 A, and an absolute 2^-25 where the row's
                largest weight times its value row's power (few) is at least 2^4:
                2^-29 n few times what a value has beside its power, 12 (above 128
                packed rows 2^8 and the power of 32 neighbours: few is given so);
      sums      n additions of either product, 2 e each, twice; rescaling and
                merging of partial results: 32 e A;
      output    rounded once: u |out|, or 2^-25 where fp16 is subnormal."""
    u, e = HALF_STEP[dtype], 2.0 ** -24
    d = (2 * (hd + 4) * e * size + 6 * e * (size + 130) + 8 * e + (6 * 2.0 ** -38 + 2.0 ** -34) * most)
    rel = 2.0 ** -11 + 2 * d[:, None] + 4 * n * e + 32 * e
    b_out = (rel * mean + (12 * 2.0 ** -29 * n * few)[:, None] + 2.0 ** -34 * mean_scale[:, None] + u * np.abs(out)) * 1.01
    if dtype == F16:
        b_out = b_out + 2.0 ** -25
    b_lse = 2 * d + 2 * n * e + 8 * e * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return b_out, b_lse


def run(p, q, out=None, lse=True, max_rows=None, ws=None, **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    lse_t = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    max_rows = max(p.rows) if max_rows is None else max_rows
    if ws is None:
        ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(q.shape[1], p.n_kv, q.shape[2], max_rows))
    dfl.dflash_paged_attention(p.cache, q, out, *p.batch, max_rows, ws, lse=lse_t, **kw)
    torch.cuda.synchronize()
    return out, lse_t, dfl.dflash_read_status(ws)


def check(p, q, out, lse, causal=True, window=0, scale=None, only=None, max_rows=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, want_l, b_out, b_lse = reference(p, q, causal, window, scale, only, max_rows)
    rows = np.zeros(q.shape[0], dtype=bool)
    for b in range(len(p.lens)):
        if only is None or b in only:
            rows[p.start_np[b]:p.start_np[b + 1]] = True
    got = to64(out)
    assert np.isfinite(got[rows]).all()
    err = np.abs(got - want)[rows]
    some = b_out[rows] > 0
    assert (err[~some] == 0).all()
    worst = (err[some] / b_out[rows][some]).max() if some.any() else 0.0
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


def kv_rows(n, n_kv, hd, dtype, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(n + extra, n_kv, hd, generator=g) * torch.exp(torch.randn(n + extra, n_kv, 1, generator=g))).to(dtype).cuda())

