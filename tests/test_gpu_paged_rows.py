"""GPU: every attended row of a long cut sequence counts once, and P is held beyond bf16.

Rows are counted by construction, not within a tolerance that grows with their number.  With queries
of zero and no sink all probabilities are equal: exactly 1 (or one power of two) before they are
normalised, so that sums of one-hot values are whole numbers below 2^24 and exact in fp32 in any order,
in the pieces and where they are joined.  What is left is the division (inverse and product: 2^-23
relative) and the output's rounding: out * N must be the count of the rows with that value to
2^-8 (bf16; fp32 2^-22) relative, and a count of c <= 127 (bf16) or < 2^21 (fp32) is then known to the
row: one lost or doubled row moves it by 1 / c.  lse = log N, to 4 half steps of fp32 of its parts
(the maximum's shift, at most 6, and the logarithm): a row more or less moves it by 1 / N."""
from __future__ import annotations

import math

import pytest
import torch

from test_gpu_paged import BF, F32, R, U, entry_rows, make_idx
from test_gpu_paged_range import Plain

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import compressed_sparse_long_csa_b200 as csa

LONG = [  # dtype, H, dk, dv, lens
    (BF, 128, 576, 512, [32701]),
    (BF, 64, 576, 512, [30000, 1, 3333]),
    (BF, 65, 576, 512, [20000, 0, 17, 9000, 12345]),
    (BF, 12, 200, 128, [8000, 129, 5001]),
    (F32, 4, 64, 64, [20000, 3, 900]),
    (F32, 20, 576, 512, [9000, 33]),
]


def counts_match(c, b, code, n):
    """code [n]: the value dim in which each row holds a one."""
    dv = c.dv
    want = torch.bincount(code, minlength=dv).double()
    eps = R[c.out.dtype] + 4 * U
    assert eps * float(want.max()) < 0.5, "the case must tell a single row"
    got = c.out[b].double() * n
    off = (got - want).abs() > eps * want
    assert not bool(off.any()), (b, n, off.nonzero()[:4].tolist(), got[off][:4].tolist(), want.expand_as(got)[off][:4].tolist())


def one_hot(c, code_of, attended=None):
    """The rows' values are ones at code_of(row's place); every other dim and the logit are zero."""
    for b, n in enumerate(c.lens):
        if not n:
            continue
        ids = torch.arange(n)
        rows = torch.zeros(n, c.pages.shape[2])
        rows[ids, code_of(ids) % c.dv] = 1.0
        c.put(b, ids[:, None], torch.arange(c.pages.shape[2]).cuda(), rows.cuda())


@pytest.mark.parametrize("dtype,H,dk,dv,lens", LONG)
@pytest.mark.parametrize("code", ["tile of 64", "tile of 32", "row"])
def test_every_row_of_a_long_cache_counts_once(code, dtype, H, dk, dv, lens):
    code_of = {"tile of 64": lambda i: i // 64, "tile of 32": lambda i: i // 32, "row": lambda i: i}[code]
    c = Plain(41, dtype, H, dk, dv, lens)
    c.q.zero_()
    one_hot(c, code_of)
    c.run()
    for b, n in enumerate(lens):
        if n:
            counts_match(c, b, (code_of(torch.arange(n)) % dv).cuda(), n)
            lim = 4 * U * (6.0 + math.log(n))
            assert lim < 0.5 / n
            assert bool(((c.lse[b].double() - math.log(n)).abs() <= lim).all()), (b, n)
        else:
            assert bool((c.out[b] == 0).all()) and bool((c.lse[b] == -math.inf).all())


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (BF, 40, 576, 512), (F32, 4, 64, 64)])
@pytest.mark.parametrize("kind", ["full", "padded_holes"])
def test_every_selected_row_counts_once(kind, dtype, H, dk, dv):
    """Selections out of order, with unused slots among them."""
    B, cap, k = 3, 16000, 8000
    c = Plain(43, dtype, H, dk, dv, [cap] * B)
    c.q.zero_()
    one_hot(c, lambda i: i)
    c.idx = make_idx(47, B, k, cap, kind)
    c.ws = torch.empty(csa.attn_decode_paged_workspace_size(B, H, dv, k), dtype=torch.uint8, device="cuda")
    c.run()
    for b in range(B):
        ids = c.idx[b][c.idx[b] >= 0].long()
        counts_match(c, b, ids % dv, len(ids))
        assert bool(((c.lse[b].double() - math.log(len(ids))).abs() <= 4 * U * (6.0 + math.log(len(ids)))).all())


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (BF, 64, 576, 512), (BF, 12, 200, 128)])
@pytest.mark.parametrize("lens", [[65, 130], [9000, 500]])
def test_probabilities_are_held_beyond_bf16(lens, dtype, H, dk, dv):
    """Every tile has a row of logit 5 (and value 0) that sets its maximum; all others have probabilities
    of one mantissa just below the middle between two bf16 values, so that a P of bf16 alone would be
    off by 2^-8 in the same direction in all of them, and the output by as much: twice its own rounding.
    Sums of N terms may add N 2u relative; P's 2^-17, the exponentials and the joining 2^-15 in all."""
    c = Plain(53, dtype, H, dk, dv, lens)
    g = torch.Generator(device="cuda").manual_seed(59)
    logit = 5.0 + math.log((1.0 + 2.0 ** -8 - 2.0 ** -12) / 64.0)
    high = torch.tensor(5.0)
    # the key dims dk - 1 and dk - 2: the logit in two parts that bf16 holds, q = (1, 2^-8)
    part = torch.tensor(logit).to(BF).float()
    rest = ((logit - part) * 256.0).to(BF).float()
    c.q[..., dk - 2] = 2.0 ** -8
    for b, n in enumerate(lens):
        ids = torch.arange(n)
        c.put(b, ids[:, None], torch.arange(dv).cuda(), 1.0 + torch.randint(0, 128, (dv,), generator=g, device="cuda") / 128.0)
        c.put(b, ids, dk - 1, float(part))
        c.put(b, ids, dk - 2, float(rest))
        top = ids[ids % 32 == 7]
        c.put(b, top[:, None], torch.arange(dv).cuda(), 0.0)
        c.put(b, top, dk - 1, float(high))
        c.put(b, top, dk - 2, 0.0)
    c.run()
    p_err = []
    for b, n in enumerate(lens):
        rows = entry_rows(c.pages, c.table, b, torch.arange(n, device="cuda"))
        s = rows @ c.q[b, 0].double()
        want = torch.softmax(s, 0) @ rows[:, :dv]
        tol = want * (2.0 ** -15 + 2 * (n + 16) * 2 * U) + 2.0 ** -9 * 2.0 ** torch.floor(torch.log2(want)) * 2
        # half a bf16 step of the output: 2^-8 of the power of two below it
        assert bool(((c.out[b].double() - want).abs() <= tol).all()), (b, float(((c.out[b].double() - want).abs() / tol).max()))
        p = torch.exp(s - s.max()).float().to(BF).double()                          # a P of bf16 alone
        p_err.append(bool((((p @ rows[:, :dv]) / torch.exp(s - s.max()).sum() - want).abs() > 0.9 * 2.0 ** -8 * want).any()))
    assert all(p_err), "the case must show a P of bf16 alone"
