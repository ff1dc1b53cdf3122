"""Attention over a paged cache in 4 bits whose rows hold blocks of zeros.  append gives
such a block a scale of 1, which says nothing of its values: bounds come from the scales
of the blocks that hold any."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from paged4_testutil import BF, F16, Paged4, reference, run
from target_testutil import rows_tensor, to64

pytestmark = pytest.mark.gpu
MANY, LOOK = 152, (0, 70, 151)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


class Held:
    """p as the oracle sees it: blocks of zeros under scales of 0, which are the same
    values and count for nothing in the bounds."""

    def __init__(self, p):
        self.__dict__.update(p.__dict__)

    def host(self):
        out = []
        for t in self.pages:
            r = t.cpu().numpy()
            for b in range(self.hd // 16):
                none = ((r[..., 8 * b:8 * b + 8] & 0x77) == 0).all(-1)
                at = self.hd // 2 + 2 * b
                r[..., at:at + 2] = np.where(none[..., None], 0, r[..., at:at + 2])
            out.append(r)
        return out


def share(p, rows):
    """The one request of p as MANY of `rows` new rows each, so that a block of threads
    runs over most of a request and its references are the dominant key's."""
    p.table_np = np.repeat(p.table_np, MANY, axis=0)
    p.lens, p.rows = p.lens * MANY, [rows] * MANY
    p.start_np = (np.arange(MANY + 1) * rows).astype(np.int32)
    p.n_rows = MANY * rows
    p.row_start = torch.from_numpy(p.start_np).cuda()
    p.kv_len = torch.tensor(p.lens, dtype=torch.int64, device="cuda")
    p.table = torch.from_numpy(p.table_np).cuda()
    p.batch = (p.row_start, p.kv_len, p.table)


def compare(p, q, out, lse, causal=False, look=LOOK):
    want, want_l, b_out, b_lse = reference(Held(p), q, causal, 0, q.shape[2] ** -0.5, look)
    rows = np.concatenate([np.arange(p.start_np[b], p.start_np[b + 1]) for b in look])
    got, got_l = to64(out)[rows], to64(lse)[rows]
    assert np.isfinite(got).all()
    worst = (np.abs(got - want[rows]) / np.maximum(b_out[rows], 1e-300)).max()
    worst_l = (np.abs(got_l - want_l[rows]) / b_lse[rows]).max()
    assert worst <= 1.0 and worst_l <= 1.0, f"out {worst:.2f}, lse {worst_l:.2f} of their bounds off"


def rounded(x, dtype):
    return torch.from_numpy(x).to(dtype).float().numpy()


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -8])
@pytest.mark.parametrize("rows,n_q", [(1, 1), (2, 2), (40, 2), (50, 2), (200, 1)])
def test_tail_behind_a_dominant_key_without_values(rows, n_q, size, dtype):
    """One key's weight is 2^22 of every other's and its values are 0, as those of a
    position that only takes what weight is left: the others are the output."""
    n, hd = 4096, 64
    rng = np.random.default_rng(2)
    k = np.zeros((n, 1, hd), dtype=np.float32)
    k[:, 0, 0] = 0.01 * rng.standard_normal(n)
    k[777, 0, 0] = 4.0
    v = size * (rng.standard_normal((n, 1, hd)).astype(np.float32) + 1.0)
    v[777] = 0
    p = Paged4([n], [rows], 1, hd, 64, dtype, values=[[rounded(k, dtype)], [rounded(v, dtype)]])
    share(p, rows)
    q = torch.zeros(p.n_rows, n_q, hd, dtype=dtype, device="cuda")
    q[..., 0] = 22 * np.log(2.0) * 8.0 / 4.0             # over sqrt(64), times the key's 4
    out, lse, status = run(p, q, causal=False)
    assert status == 0
    compare(p, q, out, lse)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 12, 70])
def test_rows_that_are_zero_in_some_blocks(rows, hd):
    """Keys and values that are tiny in some blocks and 0 in the others, other blocks for
    other rows, among whole rows, rows of zeros and rows whose largest scale is 1."""
    n, n_kv = 700, 2
    rng = np.random.default_rng(7)
    k, v = (rng.standard_normal((n, n_kv, hd)).astype(np.float32) for _ in range(2))
    k *= 2.0 ** -40
    v *= 2.0 ** -45
    for x in (k, v):
        off = rng.random((n, n_kv, hd // 16)) < 0.5
        off[::11] = False
        off[5::31] = True
        x *= np.repeat(~off, 16, -1)
    p = Paged4([n, 40], [rows, 40], n_kv, hd, 32, BF, values=[[rounded(k, BF), rounded(k[:40], BF)], [rounded(v, BF), rounded(v[:40], BF)]])
    q = rows_tensor(p.n_rows, 4, hd, BF, 4) * 2.0 ** 40
    out, lse, status = run(p, q)
    assert status == 0
    compare(p, q, out, lse, causal=True, look=(0, 1))
    ones = v.copy()                                      # some rows with a block of largest value 6, scale 1
    ones[3::7, :, :16] *= 6 / np.maximum(np.abs(ones[3::7, :, :16]).max(-1, keepdims=True), 1e-30)
    p = Paged4([n], [rows], n_kv, hd, 32, BF, values=[[rounded(k, BF)], [rounded(ones, BF)]])
    q = rows_tensor(p.n_rows, 4, hd, BF, 4) * 2.0 ** 40
    out, lse, status = run(p, q)
    assert status == 0
    compare(p, q, out, lse, causal=True, look=(0,))


@pytest.mark.parametrize("rows", [1, 12, 70])
def test_rows_of_zeros_among_huge_values_and_alone(rows):
    """Rows of zeros weigh in the sums whatever the size of the others'; a cache of zeros
    gives zeros and the logarithm of the number of keys."""
    n, n_kv, hd = 1500, 2, 128
    rng = np.random.default_rng(9)
    k, v = (rng.standard_normal((n, n_kv, hd)).astype(np.float32) for _ in range(2))
    v *= 2.0 ** 70
    v[::3] = 0
    v[64:256] = 0
    p = Paged4([n], [rows], n_kv, hd, 16, BF, values=[[rounded(k, BF)], [rounded(v, BF)]])
    q = rows_tensor(p.n_rows, 4, hd, BF, 4)
    out, lse, status = run(p, q)
    assert status == 0
    compare(p, q, out, lse, causal=True, look=(0,))
    p = Paged4([n], [rows], n_kv, hd, 16, BF, values=[[0 * k], [0 * v]])
    out, lse, status = run(p, q, causal=False)
    assert status == 0 and (out == 0).all()
    assert (np.abs(to64(lse) - np.log(n)) <= 2.0 ** -21 * np.log(n)).all()
