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
from target_testutil import HALF_STEP, Paged, rows_tensor, run_attention, to64

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
      weights  rounded to 16 bits: u A.  They have an exponent for every weight
               that counts, so there is nothing absolute beside it;
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
