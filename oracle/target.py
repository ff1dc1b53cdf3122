"""The target's side of a cycle: rows of a paged cache, attention of new rows
over them, and penalties, biases and token masks on logits, in float64 with
plain loops over requests and heads.

Test infrastructure only (see the package docstring).

The pages leave the target's kernels to the serving stack ("Speculative
decoding" product doc, section "How it works": the target scores the whole
block in one pass), so the rules are the library's own: include/dflash.h
states them, and this file follows that text.
"""

import numpy as np

from . import quant


def places(row_start, kv_len, table, page):
    """(row, request, position, page id, row of the page) of every new row."""
    out = []
    for b in range(len(kv_len)):
        n = int(row_start[b + 1]) - int(row_start[b])
        for j in range(n):
            pos = int(kv_len[b]) - n + j
            if pos >= 0:
                out.append((int(row_start[b]) + j, b, pos, int(table[b][pos // page]), pos % page))
    return out


def quantize(x):
    """(codes uint8, scales float32) of the rows of x [..., hd]: the weights'
    rule per row; a row that holds a NaN or an infinity has a NaN scale (its
    codes do not matter)."""
    flat = np.asarray(x, dtype=np.float32).reshape(-1, x.shape[-1])
    bad = ~np.isfinite(flat).all(axis=1)
    codes, scale = quant.quantize_rows(np.where(bad[:, None], np.float32(0), flat))
    scale = np.where(bad, np.float32(np.nan), scale)
    return codes.reshape(x.shape), scale.reshape(x.shape[:-1])


def read(pages, scale, pid, at, e4m3):
    """Row `at` of page `pid`, [heads, hd] float64 (e4m3: pages are codes)."""
    if not e4m3:
        return np.asarray(pages[pid, :, at], dtype=np.float64)
    return quant.e4m3_value(pages[pid, :, at]) * np.asarray(scale[pid, :, at], dtype=np.float64)[:, None]


def sequence(pages, scale, table_row, length, page, e4m3):
    """Positions 0 .. length - 1 of one request, [length, heads, hd] float64."""
    rows = [read(pages, scale, int(table_row[s // page]), s % page, e4m3) for s in range(length)]
    return np.stack(rows) if rows else np.zeros((0,) + (pages.shape[1], pages.shape[3]))


def visible(pos, length, causal, window):
    """[lo, hi): the positions a row at position `pos` sees."""
    hi = min(length, pos + 1) if causal else length
    lo = max(0, pos - window + 1) if window else 0
    return lo, max(hi, lo)


def attention(q, keys, values, length, causal, window, scale):
    """out [n, n_q, hd], lse [n, n_q] and, for error bounds, the softmax mean
    of |v| and the largest scale * sum |q||k| of every row and head.  q
    [n, n_q, hd]; keys, values [length, n_kv, hd]; the rows are the last n
    positions."""
    n, n_q, hd = q.shape
    group = n_q // keys.shape[1]
    out = np.zeros((n, n_q, hd))
    lse = np.full((n, n_q), -np.inf)
    mean = np.zeros((n, n_q, hd))
    size = np.zeros((n, n_q))
    for j in range(n):
        lo, hi = visible(length - n + j, length, causal, window)
        if hi <= lo:
            continue
        for h in range(n_q):
            k, v = keys[lo:hi, h // group], values[lo:hi, h // group]
            z = k @ q[j, h] * scale
            m = z.max()
            w = np.exp(z - m)
            total = w.sum()
            out[j, h] = w @ v / total
            lse[j, h] = m + np.log(total)
            mean[j, h] = w @ np.abs(v) / total
            size[j, h] = (np.abs(k) @ np.abs(q[j, h])).max() * scale
    return out, lse, mean, size


def adjust(logits, counts=None, prompt=None, slot=None, draft=None, repetition=None, frequency=None,
           presence=None, bias=None, allow=None):
    """out [B, G, V] and the sum of the magnitudes that went into every value.
    prompt [slots, V] and allow [B, G, V] are booleans here; bias is a list of
    (request, id, value)."""
    B, G, V = logits.shape
    out = np.array(logits, dtype=np.float64)
    size = np.abs(out)
    for b in range(B):
        s = b if slot is None else int(slot[b])
        c = np.zeros(V) if counts is None else np.array(counts[s], dtype=np.float64)
        r = 1.0 if repetition is None else float(repetition[b])
        f = 0.0 if frequency is None else float(frequency[b])
        p = 0.0 if presence is None else float(presence[b])
        for i in range(G):
            if i and draft is not None and 0 <= draft[b, i - 1] < V:
                c[draft[b, i - 1]] += 1
            x = out[b, i]
            hit = c > 0
            if prompt is not None:
                hit = hit | prompt[s]
            x[hit] = np.where(x > 0, x / r, x * r)[hit]
            x -= f * c + np.where(c > 0, p, 0.0)
            size[b, i] = np.maximum(size[b, i], np.abs(x)) + abs(f) * c + abs(p)
            for rb, v, val in bias or ():
                if rb == b:
                    x[v] += val
                    size[b, i, v] += abs(val)
            if allow is not None:
                x[~allow[b, i]] = -np.inf
    return out, size
