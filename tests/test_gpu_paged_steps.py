"""GPU: the paged calls in the order in which they are used.

* The decode steps over paged entry caches (steps.page_caches) against the same steps over the
  contiguous caches and against the oracle: the new entry in its page and the selected indices
  equal bit for bit, outputs and lse within the decode tolerances of the contiguous calls.
* A latent cache that a prompt and then single tokens are appended to with the position rotation,
  attended at every step, against a recomputation from all unrotated rows in 64 bits; the decode
  step as one captured graph that is replayed with other positions.

Tolerance of the second: a stored row and a query are rounded to bf16 once after the rotation,
2^-8 of a value each, so a logit is off by at most 2^-7 * s * sum|q||k| (and the fp32 terms, which
are 2^13 times smaller: taken as 2^-7 * 1.01), a probability by twice that relative, a value by
2^-8 of itself; the output's own rounding adds 2^-8: |out - o| <= A (2 L + 2^-8) + 2^-8 |o|, A = sum p |v|."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import csa_inputs as CI
from oracle import csa_oracle as O
from test_gpu_parity import _np, check_close

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import compressed_sparse_long_csa_b200 as csa
    from compressed_sparse_long_csa_b200 import steps


@pytest.mark.parametrize("wid,scale,page", [(1, {"B": 3, "T": 8192}, 64), (1, {"B": 2, "T": 4100, "k": 100}, 24),
                                            (2, {"B": 3, "T": 128 * 300}, 16), (4, {"B": 2, "T": 65536}, 64)])
def test_paged_decode_steps(wid, scale, page):
    wl = CI.make_workload(wid, scale=scale)
    D = wl.dims
    A, P = steps.upload(wl), steps.upload(wl)
    steps.page_caches(P, D, wl.kind, page)
    # the pages anywhere in the pool: both the pool and the table in another order
    for p in ("", "h_"):
        if p + "pages" in P:
            order = torch.randperm(P[p + "pages"].shape[0], generator=torch.Generator().manual_seed(7)).cuda()
            P[p + "pages"] = P[p + "pages"][order].contiguous()
            P[p + "block_table"] = order.argsort()[P[p + "block_table"].long()].to(torch.int32).contiguous()
    contiguous = P["cache"].clone()
    steps.run_step(wl.kind, A, D)
    steps.run_step(wl.kind, P, D)
    torch.cuda.synchronize()
    assert csa.read_device_error() == 0
    assert torch.equal(P["cache"], contiguous)             # the step went to the pages
    for p in ("", "h_"):
        if p + "pages" not in P:
            continue
        e = int(A[p + "entry0"][0])
        pid = P[p + "block_table"][:, e // page].long()
        assert torch.equal(P[p + "pages"][pid, e % page], A[p + "cache"][:, e])
    if wl.kind != "hca_decode":
        assert torch.equal(A["idx"], P["idx"]) and torch.equal(A["kI"], P["kI"]) and torch.equal(A["win"], P["win"])
        ref = O.run_csa_decode(wl)
        check_close(_np(P["out"][:, 0]), np.stack([ref["out"][b] for b in range(D["B"])]), "bf16", "csa out")
        np.testing.assert_allclose(_np(P["lse"][:, 0]), np.stack([ref["lse"][b] for b in range(D["B"])]), atol=2e-3, rtol=0)
    if wl.kind != "csa_decode":
        p = "" if wl.kind == "hca_decode" else "h_"
        ref = O.run_hca_decode(wl, prefix=p)
        check_close(_np(P[p + "out"][:, 0]), np.stack([ref["out"][b] for b in range(D["B"])]), "bf16", "hca out")
        np.testing.assert_allclose(_np(P[p + "lse"][:, 0]), np.stack([ref["lse"][b] for b in range(D["B"])]), atol=2e-3, rtol=0)


def test_first_entry_of_a_sequence_goes_without_the_block_before_it():
    """A batch in which one sequence completes its first entry and another its last."""
    wl = CI.make_workload(1, scale={"B": 2, "T": 4096})
    D = wl.dims
    A, P = steps.upload(wl), steps.upload(wl)
    for T in (A, P):
        T["entry0"].copy_(torch.tensor([0, D["N"] - 1], dtype=torch.int32))
        T["n_entries"].copy_(torch.tensor([1, D["N"]], dtype=torch.int32))
        T["q_pos"].copy_(torch.tensor([[3], [D["q_pos0"]]], dtype=torch.int32))
    steps.page_caches(P, D, wl.kind, 64)
    steps.run_step(wl.kind, A, D)
    steps.run_step(wl.kind, P, D)
    torch.cuda.synchronize()
    assert csa.read_device_error() == 0
    assert torch.equal(P["pages"][P["block_table"][0, 0].long(), 0], A["cache"][0, 0])
    e = D["N"] - 1
    assert torch.equal(P["pages"][P["block_table"][1, e // 64].long(), e % 64], A["cache"][1, e])
    assert torch.equal(A["idx"], P["idx"])
    # the same sum over the same rows by two kernels: each off by half a step of bf16
    a, b = A["out"].double(), P["out"].double()
    assert bool(((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 1e-3 * a.abs().amax()).all())


def rotate(x, pos, inv_freq):
    ang = pos.double()[..., None] * inv_freq.double()
    y = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(ang), ang)
    return torch.view_as_real(y).flatten(-2)


@pytest.mark.parametrize("H,page", [(128, 64), (16, 24)])
def test_a_rotated_latent_cache_over_a_prompt_and_single_tokens(H, page):
    g = torch.Generator(device="cuda").manual_seed(101 + H)
    lens, d, dv, dr, new = [130, 1, 77], 576, 512, 64, 5
    B, cap, pad = len(lens), 200, 9
    width = -(-cap // page)
    bf = torch.bfloat16
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(bf)          # noqa: E731
    pages = torch.full((B * width, page, d), float("nan"), device="cuda", dtype=bf)
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width).contiguous()
    inv = 10000.0 ** (-torch.arange(0, dr, 2, device="cuda", dtype=torch.float32) / dr)
    far = torch.tensor([900000, 5, 70000], device="cuda", dtype=torch.int32)     # position of entry 0
    # the prompts, in one call with padding rows behind
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)] + [torch.zeros(pad)]).to(torch.int32).cuda()
    entry = torch.cat([torch.arange(n) for n in lens] + [torch.full((pad,), -1)]).to(torch.int32).cuda()
    rows = rnd(sum(lens) + pad, d)
    csa.latent_append_paged(rows, entry, pages, table, seq=seq, pos=far[seq.long()] + entry, inv_freq=inv)
    at = np.cumsum([0] + lens)
    history = [rows[at[b]:at[b + 1]] for b in range(B)]
    # decode: static buffers and one graph
    row, q = rnd(B, d), rnd(B, H, d)
    e, pos, n = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    sink = torch.randn(H, generator=g, device="cuda")
    out, lse = torch.empty(B, H, dv, device="cuda", dtype=bf), torch.empty(B, H, device="cuda")
    q_rot = torch.empty_like(q)
    ws = torch.empty(csa.attn_decode_paged_workspace_size(B, H, dv, width * page), dtype=torch.uint8, device="cuda")
    scale = d ** -0.5

    def step():
        q_rot.copy_(q)
        csa.latent_append_paged(row, e, pages, table, pos=pos, inv_freq=inv, q_pe=q_rot[..., dv:], q=q_rot)
        csa.hca_attn_decode_paged(q_rot, pages, table, n, None, None, sink, scale, dv, out, lse, ws)

    length = list(lens)
    graph = None
    for k in range(new):
        row.copy_(rnd(B, d))
        q.copy_(rnd(B, H, d))
        e.copy_(torch.tensor(length, dtype=torch.int32))
        pos.copy_(far + e)
        n.copy_(e + 1)
        if k < 2:
            step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        assert csa.read_device_error() == 0
        for b in range(B):
            history[b] = torch.cat((history[b], row[b:b + 1].clone()))
            length[b] += 1
            p = far[b] + torch.arange(length[b], device="cuda")
            K = torch.cat((history[b][:, :dv].double(), rotate(history[b][:, dv:], p, inv)), dim=1)
            Q = torch.cat((q[b, :, :dv].double(), rotate(q[b, :, dv:], p[-1].expand(H), inv)), dim=1)
            logits = Q @ K.T * scale
            L = (Q.abs() @ K.abs().T).amax(dim=1) * scale * 2.0 ** -7 * 1.01
            want = torch.logsumexp(torch.cat((logits, sink.double()[:, None]), 1), 1)
            w = torch.exp(logits - want[:, None])
            o, A = w @ K[:, :dv], w @ K[:, :dv].abs()
            assert bool(((out[b].double() - o).abs() <= A * (2 * L + 2.0 ** -8)[:, None] + 2.0 ** -8 * o.abs()).all()), (k, b)
            assert bool(((lse[b].double() - want).abs() <= L + 1e-5).all()), (k, b)
    # what no sequence appended was not written
    written = sum(length)
    assert int(torch.isfinite(pages.float()).all(dim=2).sum()) == written
