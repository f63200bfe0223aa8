"""GPU: decode steps over pages while the position moves on, as a decode loop moves it: entry0,
n_entries and q_pos written in place between steps, eager and as a replayed graph.  After every step
the pages hold what the contiguous steps' cache holds, bit for bit."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import csa_inputs as CI

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import compressed_sparse_long_csa_b200 as csa
    from compressed_sparse_long_csa_b200 import steps

DEVERR_ENTRY = 0x10


def unpaged(T, p):
    pages, table, cache = T[p + "pages"], T[p + "block_table"], T[p + "cache"]
    return pages[table.long()].flatten(1, 2)[:, :cache.shape[1]]


def prefixes(T):
    return [p for p in ("", "h_") if p + "pages" in T]


def move(T, D, kind, entries):
    """The sequences' new tokens complete these entries (of each cache)."""
    e = torch.tensor(entries, dtype=torch.int32, device="cuda")
    for p in ("", "h_"):
        if p + "entry0" in T:
            T[p + "entry0"].copy_(e)
            T[p + "n_entries"].copy_(e + 1)
    if "q_pos" in T:
        T["q_pos"].copy_((e * D["m"] + D["m"] - 1)[:, None])


def fresh_tokens(A, P, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for k in ("Ca", "Cb", "CaI", "CbI", "C", "h_C", "raw_new", "h_raw_new"):
        if k in A:
            A[k].copy_(torch.randn(A[k].shape, generator=g, device="cuda"))
            P[k].copy_(A[k])


def same(A, P, D, kind, what):
    for p in prefixes(P):
        assert torch.equal(unpaged(P, p), A[p + "cache"]), (what, p)
        # the same sum over the same rows by two kernels: each off by half a step of bf16
        a, b = A[p + "out"].double(), P[p + "out"].double()
        assert bool(((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 1e-3 * a.abs().amax()).all()), (what, p)
    if "idx" in A:
        assert torch.equal(A["idx"], P["idx"]), what


@pytest.mark.parametrize("wid,scale,page", [(1, {"B": 2, "T": 4096, "k": 64}, 7), (2, {"B": 2, "T": 128 * 100}, 16),
                                            (4, {"B": 2, "T": 65536}, 8)])
@pytest.mark.parametrize("captured", [False, True])
def test_the_position_moves_on(wid, scale, page, captured):
    wl = CI.make_workload(wid, scale=scale)
    D = wl.dims
    A, P = steps.upload(wl), steps.upload(wl)
    steps.page_caches(P, D, wl.kind, page)
    for p in prefixes(P):
        order = torch.randperm(P[p + "pages"].shape[0], generator=torch.Generator().manual_seed(7)).cuda()
        P[p + "pages"] = P[p + "pages"][order].contiguous()
        P[p + "block_table"] = order.argsort()[P[p + "block_table"].long()].to(torch.int32).contiguous()
    graph = None
    for i, entries in enumerate([(0, 5), (1, 6), (2, 7), (3, 0), (page - 1, 1), (page, 2), (page + 1, 2 * page), (0, 0)]):
        for T in (A, P):
            move(T, D, wl.kind, entries)
        fresh_tokens(A, P, 100 + i)
        steps.run_step(wl.kind, A, D)
        if captured and i == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                steps.run_step(wl.kind, P, D)
        if graph is None:
            steps.run_step(wl.kind, P, D)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert csa.read_device_error() == 0
        same(A, P, D, wl.kind, (i, entries))


@pytest.mark.parametrize("how", ["stream", "address", "holder", "null"])
def test_on_another_stream(how):
    """The step's device operations all run on the stream that it is given: a torch stream, an address,
    an object that has one, the null stream."""
    wl = CI.make_workload(2, scale={"B": 2, "T": 128 * 100})
    D = wl.dims
    A, P = steps.upload(wl), steps.upload(wl)
    steps.page_caches(P, D, wl.kind, 16)
    s = torch.cuda.default_stream() if how == "null" else torch.cuda.Stream()
    given = {"stream": s, "address": s.cuda_stream, "holder": SimpleNamespace(cuda_stream=s.cuda_stream), "null": 0}[how]
    torch.cuda.synchronize()
    for entries in ((3, 4), (4, 16)):
        for T in (A, P):
            move(T, D, wl.kind, entries)
        steps.run_step(wl.kind, A, D)
        torch.cuda.synchronize()
        steps.run_step(wl.kind, P, D, stream=given)
        s.synchronize()
        same(A, P, D, wl.kind, entries)
    assert csa.read_device_error() == 0


@pytest.mark.parametrize("wid,scale", [(1, {"B": 2, "T": 4096, "k": 64}), (2, {"B": 2, "T": 128 * 100})])
def test_an_entry_below_zero_is_flagged_and_writes_nothing(wid, scale):
    wl = CI.make_workload(wid, scale=scale)
    D = wl.dims
    P = steps.upload(wl)
    steps.page_caches(P, D, wl.kind, 16)
    P["entry0"].copy_(torch.tensor([-3, 9], dtype=torch.int32))
    P["n_entries"].copy_(torch.tensor([4, 10], dtype=torch.int32))
    before = P["pages"].clone()
    steps.run_step(wl.kind, P, D)
    torch.cuda.synchronize()
    assert csa.read_device_error() == DEVERR_ENTRY
    now = unpaged(P, "")
    was = before[P["block_table"].long()].flatten(1, 2)[:, :now.shape[1]]
    assert torch.equal(now[0], was[0])
    assert torch.equal(now[1, :9], was[1, :9]) and torch.equal(now[1, 10:], was[1, 10:]) and not torch.equal(now[1, 9], was[1, 9])
