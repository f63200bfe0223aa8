"""GPU: the paged attention at the ends of the types' range, and what joins the pieces of a cut
sequence.

The rows here are made so that logits depend on one key dim only (the queries are zero elsewhere),
and so that the values of some dims can be set freely.  Tolerances as in test_gpu_paged.py without
its terms for rounded partials (the pieces are held in fp32), and next to the smallest normal
number: a probability or a product below 2^-126 may be taken as 0, which moves an output by
2^-126 (1 + max |v|) at most."""
from __future__ import annotations

import math

import pytest
import torch

from test_gpu_paged import BF, F32, R, U, Case, entry_rows, reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import compressed_sparse_long_csa_b200 as csa

SHAPES = [(BF, 128, 576, 512), (BF, 64, 576, 512), (BF, 12, 200, 128), (F32, 4, 64, 64)]


class Plain(Case):
    """Queries that read the last dim only; the rows' last dim is their logit (0 at first)."""

    def __init__(self, seed, dtype, H, dk, dv, lens, sink=-math.inf):
        super().__init__(seed, dtype, H, dk, dv, 64, lens, 0, sink=sink)
        self.scale = 1.0
        self.q.zero_()
        self.q[..., dk - 1] = 1.0
        for b, n in enumerate(lens):
            self.put(b, torch.arange(n), dk - 1, 0.0)

    def put(self, b, ids, dims, x):
        """rows[ids][:, dims] = x of sequence b"""
        assert all(0 <= i < self.lens[b] for i in ids.flatten().tolist())
        ids = ids.cuda()
        self.pages[self.table[b].long()[ids // 64], ids % 64, dims] = x if isinstance(x, float) else x.to(self.pages)

    def run(self):
        self.call()
        torch.cuda.synchronize()
        assert csa.read_device_error() == 0

    def check(self, what):
        for b in range(len(self.lens)):
            rows = entry_rows(self.pages, self.table, b, torch.arange(self.lens[b], device="cuda"))
            o, l, A, D, N, _ = reference(self.q[b], rows, self.sink, self.scale, self.dv)
            tol = A * (2 * D + 2.0 ** -15 + 2 * (N + 16) * 2 * U)[:, None] + R[self.out.dtype] * o.abs()
            err = (self.out[b].double() - o).abs()
            assert bool(torch.isfinite(self.out[b]).all()), (what, b)
            small = 2.0 ** -126 * (1.0 + rows[:, :self.dv].abs().amax(dim=0)) if N else 0.0
            assert bool((err <= tol + small).all()), (what, b, float((err / (tol + small)).max()))
            assert bool(((self.lse[b].double() - l).abs() <= D + (N + 16) * 2 * U + l.abs() * 2 * U).all()), (what, b)


@pytest.mark.parametrize("dtype,H,dk,dv", SHAPES)
@pytest.mark.parametrize("power", [-133, -130, -127, -120, 100, 119, 126, 127])
def test_tiny_and_huge_values(power, dtype, H, dk, dv):
    """A quarter of the dims is zero but for the row that takes all of the probability."""
    c = Plain(7, dtype, H, dk, dv, [9000, 100])
    dims = torch.arange(dv // 4, dv // 2)
    for b, at in ((0, 4321), (1, 70)):
        c.put(b, torch.arange(c.lens[b])[:, None], dims.cuda(), 0.0)
        v = (1.0 + (dims % 100) / 128.0) * (1 - 2 * (dims % 2)) * 2.0 ** power
        c.put(b, torch.tensor([at]), dims.cuda(), v)
        c.put(b, torch.tensor([at]), dk - 1, 30.0)
    c.run()
    c.check(power)


@pytest.mark.parametrize("dtype,H,dk,dv", SHAPES)
@pytest.mark.parametrize("nats", [60.0, 86.0, 88.0, 90.0, 92.0, 94.0, 120.0])
def test_sums_that_later_rows_scale_down_to_almost_nothing(nats, dtype, H, dk, dv):
    """Ordinary rows, then rows of far higher logits that are zero in a quarter of the dims."""
    c = Plain(11, dtype, H, dk, dv, [5000, 300])
    dims = torch.arange(dv // 4, dv // 2).cuda()
    for b in range(2):
        ids = torch.arange(c.lens[b])
        high = ids[(ids // 64) % 2 == 1]
        c.put(b, high[:, None], dims, 0.0)
        c.put(b, high, dk - 1, nats)
    c.run()
    c.check(nats)


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (BF, 64, 576, 512), (BF, 12, 200, 128)])
@pytest.mark.parametrize("lens", [[9000, 130], [1500] * 10])
def test_pieces_are_joined_without_another_rounding(lens, dtype, H, dk, dv):
    """Equal logits and values of 8 bits: every sum of a piece has at most 21 bits, which fp32 holds
    exactly.  The outputs are means that lie 2^-10 of a bf16 step beyond the middle between two
    values (2^-18 relative), and the joining rounds by 8 partials and 4 operations of 2^-24 each at
    most where a warp joins few pieces, by 3 such where a CTA joins many: 2^-20.  So every output is
    the mean rounded once."""
    c = Plain(13, dtype, H, dk, dv, lens)
    g = torch.Generator(device="cuda").manual_seed(17)
    for b, n in enumerate(lens):
        low = torch.randint(0, 127, (dv,), generator=g, device="cuda")
        up = torch.rand(n, dv, generator=g, device="cuda").argsort(dim=0) < n // 2 + max(1, -(-n // 1024))
        c.put(b, torch.arange(n)[:, None], torch.arange(dv).cuda(), 1.0 + (low + up) / 128.0)
    c.run()
    for b, n in enumerate(lens):
        rows = entry_rows(c.pages, c.table, b, torch.arange(n, device="cuda"))[:, :dv]
        want = rows.mean(dim=0).float().to(BF)
        assert torch.equal(c.out[b], want.expand(H, dv)), (b, int((c.out[b] != want).sum()))
        assert bool(((c.lse[b].double() - math.log(n)).abs() <= 4 * U * math.log(n)).all())


@pytest.mark.parametrize("dtype,H,dk,dv", SHAPES)
@pytest.mark.parametrize("lens", [[100, 64], [20000, 15000, 9000, 12000]])
@pytest.mark.parametrize("nats", [-3.0, 0.7, 5.4, 20.0])
def test_large_values_at_a_maximum_that_rises(nats, lens, dtype, H, dk, dv):
    """Values of 2^126 in a row behind others of lower or higher logits: the sums of p v, p <= 1, are in range."""
    c = Plain(23, dtype, H, dk, dv, lens)
    dims = torch.arange(dv // 4, dv // 2)
    for b, n in enumerate(lens):
        c.put(b, torch.arange(n)[:, None], dims.cuda(), 0.0)
        at = torch.tensor([min(n - 1, n // 2 + 30 + 64 * b)])      # (not every unit begins at that tile)
        c.put(b, at, dims.cuda(), (1.0 + (dims % 100) / 128.0) * (1 - 2 * (dims % 2)) * 2.0 ** 126)
        c.put(b, at, dk - 1, nats)
    c.run()
    c.check(nats)


@pytest.mark.parametrize("dtype,H,dk,dv", SHAPES)
@pytest.mark.parametrize("sink", [-math.inf, 0.5])
@pytest.mark.parametrize("lens", [[1, 40, 64], [9000, 70]])
def test_rows_of_nan_alone(lens, sink, dtype, H, dk, dv):
    """Every attended row is NaN: so are all outputs, with or without a sink, cut or not."""
    c = Plain(29, dtype, H, dk, dv, lens + [50], sink=sink)
    for b, n in enumerate(lens):
        c.put(b, torch.arange(n), slice(0, dk), math.nan)
    c.run()
    for b in range(len(lens)):
        assert bool(c.out[b].isnan().all()) and bool(c.lse[b].isnan().all()), b
    assert bool(c.out[-1].isfinite().all()) and bool(c.lse[-1].isfinite().all())


@pytest.mark.parametrize("dtype,H,dk,dv", SHAPES)
@pytest.mark.parametrize("lens", [[1, 40, 0, 64], [9000, 0, 70], [1500] * 10])
def test_sinks_of_infinity_and_nan(lens, dtype, H, dk, dv):
    """A sink of +inf takes all of the probability: out = 0, lse = inf.  A NaN shows in its head alone."""
    c = Plain(31, dtype, H, dk, dv, lens, sink=0.25)
    c.sink[0], c.sink[2] = math.inf, math.nan
    c.run()
    assert bool((c.out[:, 0] == 0).all()) and bool((c.lse[:, 0] == math.inf).all())
    for b, n in enumerate(lens):
        assert bool(c.lse[b, 2].isnan())
        assert bool(c.out[b, 2].isnan().all()) if n else bool((c.out[b, 2] == 0).all())
    keep = [h for h in range(H) if h not in (0, 2)]
    c.out, c.lse, c.q, c.sink = c.out[:, keep], c.lse[:, keep], c.q[:, keep], c.sink[keep]
    c.check("other heads")
