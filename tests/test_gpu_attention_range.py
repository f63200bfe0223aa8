"""GPU: the attention over contiguous caches at the ends of the types' range.

The split partials carry a power of two per head and half of the dims; a half that is zero but for
one tiny or huge value must come out as that value.  The queries read the last key dim only, so the
row with 30 there takes all of the probability but e^-30 N (8e-10 of 9000 rows).

Tolerance: the probabilities are off by 2^-15 relative, a partial by 2^-11 of a value and by 2^-25 of
the largest of its half (which is the value here), the output by its rounding 2^-8; what is below the
smallest normal number may be taken as 0: 2^-126 (1 + max |v|)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import compressed_sparse_long_csa_b200 as csa


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("B,N", [(1, 20000), (3, 4000), (8, 900)])
@pytest.mark.parametrize("power", [-133, -130, -127, -120, 100, 126, 127])
def test_tiny_and_huge_values(power, B, N, sparse):
    H, dk, dv, bf = 128, 576, 512, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(19)
    cache = torch.randn(B, N, dk, generator=g, device="cuda").to(bf)
    cache[..., dk - 1] = 0.0
    cache[..., :dv // 2] = 0.0
    at = N // 2 + 3
    cache[:, at, dk - 1] = 30.0
    d = torch.arange(dv // 2)
    cache[:, at, :dv // 2] = ((1.0 + (d % 100) / 128.0) * (1 - 2 * (d % 2)) * 2.0 ** power).to(cache)
    q = torch.zeros(B, H, dk, device="cuda", dtype=bf)
    q[..., dk - 1] = 1.0
    sink = torch.zeros(H, device="cuda")
    out, lse = torch.empty(B, H, dv, device="cuda", dtype=bf), torch.empty(B, H, device="cuda")
    ws = torch.empty(max(1, csa.attn_decode_workspace_size(B, H, dv, N)), dtype=torch.uint8, device="cuda")
    if sparse:
        idx = torch.arange(N, device="cuda", dtype=torch.int32).repeat(B, 1)
        csa.sparse_attn_decode(q, cache, idx, None, None, sink, 1.0, dv, out, lse, ws)
    else:
        n = torch.full((B,), N, dtype=torch.int32, device="cuda")
        csa.hca_attn_decode(q, cache, n, None, None, sink, 1.0, dv, out, lse, ws)
    torch.cuda.synchronize()
    assert csa.read_device_error() == 0
    rows = cache.double()
    logits = rows[..., dk - 1]
    L = torch.logsumexp(torch.cat((logits, torch.zeros(B, 1, device="cuda", dtype=torch.float64)), 1), 1)
    p = (logits - L[:, None]).exp()
    want, A = torch.einsum("bn,bnd->bd", p, rows[..., :dv]), torch.einsum("bn,bnd->bd", p, rows[..., :dv].abs())
    tol = A * (2.0 ** -15 + 2.0 ** -11) + 2.0 ** -8 * want.abs() + 2.0 ** -126 * (1.0 + rows[..., :dv].abs().amax(1))
    tol[:, dv // 2:] += 2.0 ** -24 * rows[..., dv // 2:dv].abs().amax(dim=(1, 2))[:, None]
    assert bool(torch.isfinite(out).all())
    assert bool(((out.double() - want[:, None]).abs() <= tol[:, None]).all())
    assert bool(((lse.double() - L[:, None]).abs() <= 1e-4).all())
