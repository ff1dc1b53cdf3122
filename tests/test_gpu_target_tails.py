"""Attention over caches where one key takes most of a row's weight and a long
tail of keys shares the rest, as the first position of a long context does:
the tail's weights are far below the largest one and still make the output.

Every value is positive, so that an output is as large as the sum of its
parts and whatever a weight loses shows in it.  152 requests read the same
pages, so that a CTA runs over most of a request and its reference is the
dominant key's."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import quant
from oracle import target as ot
from target_testutil import HALF_STEP, Paged, check_attention, rows_tensor, run_attention, to64

pytestmark = pytest.mark.gpu
BF, FH = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


MANY, LOOK = 152, (0, 70, 151)


def share(p, rows):
    """The one request of p as MANY requests of `rows` new rows each."""
    p.table_np = np.repeat(p.table_np, MANY, axis=0)
    p.lens, p.rows = p.lens * MANY, [rows] * MANY
    p.start_np = (np.arange(MANY + 1) * rows).astype(np.int32)
    p.n_rows = MANY * rows
    p.row_start = torch.from_numpy(p.start_np).cuda()
    p.kv_len = torch.tensor(p.lens, dtype=torch.int64, device="cuda")
    p.table = torch.from_numpy(p.table_np).cuda()
    p.batch = (p.row_start, p.kv_len, p.table)


def put(p, side, x):
    """Positions 0 .. n - 1 of request 0 get the rows x [n, heads, hd] (float32
    numpy); what the cache then holds, as float64."""
    at = np.arange(x.shape[0])
    pid, row = torch.from_numpy(p.table_np[0][at // p.page].astype(np.int64)).cuda(), torch.from_numpy(at % p.page).cuda()
    x = torch.from_numpy(x).to(p.dtype)
    if not p.e4m3:
        p.pages[side][pid, :, row] = x.cuda()
        return x.double().numpy()
    codes, scale = ot.quantize(x.float().numpy())
    p.pages[side].view(torch.uint8)[pid, :, row] = torch.from_numpy(codes).cuda()
    p.scale[side][pid, :, row] = torch.from_numpy(scale).cuda()
    return quant.e4m3_value(codes) * scale.astype(np.float64)[..., None]


def bound(out, lse, mean, size, n, hd, dtype, q64, k64, e4m3):
    """Largest error of the kernels' arithmetic, e = 2^-24 and u the half step
    of the 16-bit type, A = sum softmax |v|:
      queries  over codes as 8-bit terms, 2^-20 (bf16) or 2^-23 (fp16) of a
               row's largest is what may be left of each;
      scores   hd products and one fused scale, 2 e each (the tensor cores may
               truncate) of Z = scale sum |q||k|, the reference taken off and
               2^x: d = 2 (hd + 4) e Z + 4 e Z + 8 e, a softmax mean is off by
               2 d A;
      weights  rounded to 16 bits: u A.  In fp16 (over codes, and over fp16 rows)
               a weight's last place is at most 2^-35 of the row's largest part,
               half of it is left out: over codes that largest part is a key's
               weight times its value scale, and the dominant key's values are
               small here, so that there is nothing beside u A;
      sums     an accumulator takes 16 keys at a time, 2 e of it each: n / 8 e A;
               the weights' own sum 32 at a time and e: n / 32 e A; a few joins;
      output   u of itself."""
    u, e = HALF_STEP[dtype], 2.0 ** -24
    d = (2 * (hd + 4) + 4) * e * size + 8 * e
    if e4m3:
        left = 2.0 ** -20 if dtype is BF else 2.0 ** -23
        d = d + left * np.abs(q64).max(-1) * np.abs(k64).sum(-1).max() * hd ** -0.5
    rel = u + 2 * d[..., None] + (n / 8 + n / 32 + 64) * e
    b_lse = 2 * d + (n / 32 + 64) * e + 8 * e * (1 + np.abs(lse))
    return rel * mean + u * np.abs(out) * (1 + u), b_lse


def tail_case(n, part, rows, n_q, hd, dtype, e4m3, flat, large, seed=3):
    """A request of n positions whose first key takes `part` of every row's
    weight and holds values a hundredth of the others'.  flat: all other keys
    are alike, so that their weights' roundings are, too.  large: one other
    value row is 16 times the rest."""
    p = Paged([n], [rows], 1, hd, 64, dtype, e4m3, garbage=False)
    share(p, rows)
    rng = np.random.default_rng(seed)
    q = rows_tensor(p.n_rows, n_q, hd, dtype, seed)
    q[..., 0] = 4.0
    k = rng.normal(size=(n, 1, hd)).astype(np.float32) * (0.0 if flat else 0.5)
    k[:, :, 0] = 0.0
    k[0] = 0.0
    k[0, 0, 0] = (np.log(part / (1 - part)) + np.log(n)) * hd ** 0.5 / 4
    v = rng.uniform(0.5, 1.5, size=(n, 1, hd)) * np.exp(0.5 * rng.normal(size=(n, 1, 1)))
    v[0] *= 0.01
    if large:
        v[n // 2] *= 16
    k64, v64 = put(p, 0, k), put(p, 1, v.astype(np.float32))
    return p, q, k64, v64


def compare(p, q, k64, v64, out, lse, part=None):
    n, _, hd = k64.shape
    rows = np.concatenate([np.arange(p.start_np[b], p.start_np[b + 1]) for b in LOOK])
    q64 = to64(q)[rows]
    want, want_l, mean, size = ot.attention(q64, k64, v64, n, False, 0, hd ** -0.5)
    if part:                                          # the case is what it says
        assert (np.exp((q64 @ k64[0, 0]) * hd ** -0.5 - want_l) > 0.4 * part).all()
    b_out, b_lse = bound(want, want_l, mean, size, n, hd, p.dtype, q64, k64, p.e4m3)
    if p.dtype is FH and not p.e4m3:   # the last place of a weight is at most 2^-35 of the row's largest
        b_out += 2.0 ** -36 * np.abs(v64).sum(0).max()
    worst = (np.abs(to64(out)[rows] - want) / b_out).max()
    worst_l = (np.abs(to64(lse)[rows] - want_l) / b_lse).max()
    assert worst <= 1.0 and worst_l <= 1.0, f"out {worst:.2f}, lse {worst_l:.2f} of their bounds off"


CASES = [
    # keys, share, new rows, query heads, head_dim, flat, one large value row
    (8192, 0.5, 1, 5, 128, False, False),
    (8192, 0.9, 8, 5, 128, True, False),
    (8192, 0.9, 8, 5, 64, False, True),
    (8192, 0.99, 33, 4, 128, True, True),
    (32768, 0.8, 8, 2, 128, False, False),
    (32768, 0.9, 33, 4, 64, True, False),
    (32768, 0.9, 1, 3, 64, False, True),
    (131072, 0.9, 2, 2, 128, True, False),
    (131072, 0.99, 2, 1, 128, False, True),
]


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("n,part,rows,n_q,hd,flat,large", CASES)
def test_attention_over_codes_keeps_the_tail_behind_one_dominant_key(n, part, rows, n_q, hd, flat, large, dtype):
    p, q, k64, v64 = tail_case(n, part, rows, n_q, hd, dtype, True, flat, large)
    out, lse, status = run_attention(p, q, causal=False)
    assert status == 0
    compare(p, q, k64, v64, out, lse, part)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FH])
def test_attention_returns_every_code_of_a_single_visible_row(hd, dtype):
    """One key: the output is the value row itself, all finite codes of E4M3
    under a scale that is a power of two, exactly."""
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    codes = np.resize(codes, (256 // hd, 1, hd))
    n = codes.shape[0]
    p = Paged([1] * n, [1] * n, 1, hd, 16, dtype, True, garbage=False)
    for b in range(n):
        p.pages[1].view(torch.uint8)[int(p.table_np[b, 0]), :, 0] = torch.from_numpy(codes[b]).cuda()
        p.scale[1][int(p.table_np[b, 0]), :, 0] = 0.25
    q = rows_tensor(n, 3, hd, dtype, 3)
    out, _, status = run_attention(p, q)
    assert status == 0
    want = np.repeat(quant.e4m3_value(codes) * 0.25, 3, axis=1)
    np.testing.assert_array_equal(to64(out), want)


@pytest.mark.parametrize("n,part,rows,n_q,hd,flat,large", CASES)
@pytest.mark.parametrize("dtype", [BF, FH])
def test_attention_over_16_bits_keeps_the_tail_behind_one_dominant_key(n, part, rows, n_q, hd, flat, large, dtype):
    p, q, k64, v64 = tail_case(n, part, rows, n_q, hd, dtype, False, flat, large)
    out, lse, status = run_attention(p, q, causal=False)
    assert status == 0
    compare(p, q, k64, v64, out, lse, part)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("size", [2.0 ** 112, 2.0 ** 119])
def test_attention_of_very_large_values_under_scores_that_grow(e4m3, size):
    """The second half of the keys has scores 19 above the first's, 2^27 in
    weight; sums of weights and values stay finite as the formula's do."""
    n, hd = 1536, 128
    p = Paged([n], [9], 1, hd, 64, BF, e4m3, garbage=False)
    share(p, 9)
    rng = np.random.default_rng(5)
    q = rows_tensor(p.n_rows, 4, hd, BF, 3)
    q[..., 0] = 4.0
    k = rng.normal(size=(n, 1, hd)).astype(np.float32) * 0.2
    k[:, 0, 0] = np.where(np.arange(n) < 768, 0.0, 19.0 * hd ** 0.5 / 4)
    k64 = put(p, 0, k)
    v64 = put(p, 1, (rng.uniform(0.5, 1.5, size=(n, 1, hd)) * size).astype(np.float32))
    out, lse, status = run_attention(p, q, causal=False)
    assert status == 0
    compare(p, q, k64, v64, out, lse)


@pytest.mark.parametrize("dtype", [BF, FH])
def test_attention_over_codes_takes_scales_of_any_size_and_sign(dtype):
    """value = code * scale, whoever filled the cache: zeros, negative scales,
    scales that differ by 2^40."""
    p = Paged([700, 90, 300], [8, 20, 3], 2, 128, 32, dtype, True, seed=6, garbage=False)
    g = torch.Generator().manual_seed(1)
    for i in range(2):
        kind = torch.randint(0, 6, p.scale[i].shape, generator=g).cuda()
        f = torch.tensor([1.0, -1.0, 0.0, 2.0 ** -40, -(2.0 ** -20), 2.0 ** -3], device="cuda")
        p.scale[i] *= f[kind]
    for b in range(3):                                   # a dominant key beside a value row a thousand times larger
        p.scale[0][int(p.table_np[b, 0]), :, 5] *= 4.0
        p.scale[1][int(p.table_np[b, 0]), :, 6] *= 1000.0
    q = rows_tensor(p.n_rows, 6, 128, dtype, 3, size=1.5)
    out, lse, status = run_attention(p, q)
    assert status == 0
    check_attention(p, q, out, lse)
