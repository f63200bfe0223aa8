"""GPU: the paged-cache calls (latent_append_paged, hca_attn_decode_paged,
sparse_attn_decode_paged) against their definitions in 64 bits.

Tolerances, per output value, u = 2^-24 (half a step of fp32):
* a logit is a sum of d_k products and a scale in fp32: off by at most
  D = s * sum|q||k| * (d_k + 4) * 2u (2u: a tensor-core accumulation may truncate);
* a probability is off by 2 D + 4 * 2u relative (the exponentials of the logit and of the
  normaliser), plus 2^-16 when P is carried as two bf16 parts of 8 bits each;
* with A = sum p |v| / den, the sums of N products add N * 2u * A at most (and the joined
  pieces the same again), so |out - o| <= A * (2 D + 2^-15 + 2 * (N + 16) * 2u) + r |o| with
  r the storage rounding (bf16 2^-8, fp32 2^-24);
* bf16: the partials of a sequence cut over several CTAs are rounded to fp16 before they are
  joined, each by 2^-11 of itself at most (half a step: eps / 2), and their weighted magnitudes
  sum to at most A: 2^-11 A more;
* bf16, d_v = 512: a quarter of a partial's dims shares a power of two s that puts its largest
  magnitude into [s / 2, s), and below 2^-14 s the steps of fp16 stay at 2^-24 s: what is tiny is
  rounded by 2^-25 s <= 2^-24 of the largest.  That is at most the partial's sum of p max |v| over
  the quarter, and the partials' weighted sums add up to the sequence's: 2^-24 sum p max |v| more;
* lse is off by D + (N + 16) * 2u + |lse| * 2u.
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import compressed_sparse_long_csa_b200 as csa

U = 2.0 ** -24
R = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
DEVERR_INDEX, DEVERR_ENTRY = 0x1, 0x10


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def make_cache(g, dtype, caps, page, d, spare=3, fill=float("nan")):
    """A pool whose rows hold `fill` where no sequence has an entry, and a table whose ids past
    a sequence's last page are out of range (they must not be read)."""
    B = len(caps)
    used = [-(-c // page) for c in caps]
    width = max(1, max(used)) + 1
    n_pages = sum(used) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    table = torch.full((B, width), -7, dtype=torch.int32)
    table[:, 1::2] = 2 ** 31 - 1
    pages = torch.full((n_pages, page, d), fill, device="cuda", dtype=dtype)
    for b, c in enumerate(caps):
        for i in range(used[b]):
            table[b, i] = order.pop()
            rows = min(page, c - i * page)
            pages[table[b, i], :rows] = randn(g, rows, d, dtype=dtype)
    return pages, table.cuda()


def entry_rows(pages, table, b, ids):
    page = pages.shape[1]
    ids = ids.long()
    return pages[table[b].long()[ids // page], ids % page].double()


def reference(q, rows, sink, scale, dv):
    """One sequence in 64 bits: (out, lse, A, D, N)."""
    H, dk = q.shape
    q = q.double()
    N = rows.shape[0]
    logits = q @ rows.T * scale
    mag = (q.abs() @ rows.abs().T).amax(dim=1) * abs(scale) if N else torch.zeros(H, device="cuda", dtype=torch.float64)
    every = torch.cat((logits, sink.double()[:, None]), dim=1)
    lse = torch.logsumexp(every, dim=1)
    safe = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    p = torch.exp(logits - safe[:, None])
    out = p @ rows[:, :dv]
    A = p @ rows[:, :dv].abs()
    if dv == 512 and N:
        tiny = p @ rows[:, :dv].abs().view(N, 4, 128).amax(dim=2)
        return out, lse, A, mag * (dk + 4) * 2 * U, N, 2.0 ** -24 * tiny.repeat_interleave(128, dim=1)
    return out, lse, A, mag * (dk + 4) * 2 * U, N, 0.0


def check(out, lse, q, rows_of, sink, scale, what=""):
    B, H, dv = out.shape
    for b in range(B):
        o, l, A, D, N, tiny = reference(q[b], rows_of(b), sink, scale, dv)
        cut = 2.0 ** -11 if out.dtype == BF else 0.0
        tol = A * (2 * D + 2.0 ** -15 + cut + 2 * (N + 16) * 2 * U)[:, None] + R[out.dtype] * o.abs() + (tiny if out.dtype == BF else 0.0)
        bad = (out[b].double() - o).abs() > tol
        assert not bool(bad.any()) and bool(torch.isfinite(out[b]).all()), (
            what, b, N, float(((out[b].double() - o).abs() / tol.clamp(min=1e-300)).nan_to_num(9e9).max()))
        if lse is not None:
            inf = torch.isinf(l)
            assert bool((lse[b][inf] == l[inf].float()).all()), (what, b)
            err = (lse[b].double() - l).abs()[~inf]
            lim = (D + (N + 16) * 2 * U + l.abs() * 2 * U)[~inf]
            assert bool((err <= lim).all()), (what, b, N, float((err / lim).max()))


class Case:
    """Inputs of an attention call over a paged cache."""

    def __init__(self, seed, dtype, H, dk, dv, page, lens, W, idx=None, sink=None, qstd=1.5):
        g = gen(seed)
        self.lens, self.W, self.dv = lens, W, dv
        B = len(lens)
        self.pages, self.table = make_cache(g, dtype, lens, page, dk)
        self.q = randn(g, B, H, dk, dtype=dtype, std=qstd)
        self.sink = randn(g, H) if sink is None else torch.full((H,), sink, device="cuda")
        self.scale = dk ** -0.5
        self.n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.win = self.win_len = None
        if W:
            self.win = randn(g, B, W, dk, dtype=dtype)
            wl = [(5 * b + 1) % (W + 1) for b in range(B)]
            self.win_len = torch.tensor(wl, dtype=torch.int32, device="cuda")
            for b, w in enumerate(wl):
                self.win[b, w:] = float("nan")
        self.idx = idx
        self.out = torch.full((B, H, dv), 7.0, device="cuda", dtype=dtype)
        self.lse = torch.full((B, H), 7.0, device="cuda")
        rows = (idx.shape[1] if idx is not None else self.table.shape[1] * page) + W
        self.ws = torch.full((max(1, csa.attn_decode_paged_workspace_size(B, H, dv, rows)),), 255, dtype=torch.uint8, device="cuda")

    def rows_of(self, b):
        if self.idx is None:
            ids = torch.arange(self.lens[b], device="cuda")
        else:
            ids = self.idx[b][self.idx[b] >= 0]
        rows = entry_rows(self.pages, self.table, b, ids)
        if self.W:
            rows = torch.cat((rows, self.win[b, :int(self.win_len[b])].double()))
        return rows

    def call(self, stream=None):
        if self.idx is None:
            csa.hca_attn_decode_paged(self.q, self.pages, self.table, self.n, self.win, self.win_len, self.sink, self.scale,
                                      self.dv, self.out, self.lse, self.ws, stream=stream)
        else:
            csa.sparse_attn_decode_paged(self.q, self.pages, self.table, self.idx, self.win, self.win_len, self.sink,
                                         self.scale, self.dv, self.out, self.lse, self.ws, stream=stream)

    def run_and_check(self, what=""):
        t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        t[0].record()
        self.call()
        t[1].record()
        torch.cuda.synchronize()
        assert t[0].elapsed_time(t[1]) < 1000, "a device wait gave up (after 2 s)"
        assert csa.read_device_error() == 0
        check(self.out, self.lse, self.q, self.rows_of, self.sink, self.scale, what)


EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 640]

DENSE = {
    # dtype, H, dk, dv, page, lens, W
    "bf16_edges": (BF, 128, 576, 512, 64, EDGE, 0),
    "bf16_edges_window": (BF, 128, 576, 512, 16, EDGE, 128),
    "bf16_page_1": (BF, 64, 576, 512, 1, [0, 3, 70, 200], 16),
    "bf16_page_7": (BF, 128, 576, 512, 7, [5, 64, 333], 0),
    "bf16_page_24": (BF, 100, 576, 512, 24, [129, 24, 1000], 5),
    "bf16_page_32": (BF, 128, 576, 512, 32, [31, 32, 33, 4000], 128),
    "bf16_page_48": (BF, 65, 576, 512, 48, [47, 48, 49, 1500], 0),
    "bf16_page_256": (BF, 128, 576, 512, 256, [255, 257, 3001], 7),
    "bf16_heads_1": (BF, 1, 576, 512, 64, [1, 500, 64], 3),
    "bf16_heads_16": (BF, 16, 576, 512, 64, [900, 0, 64], 0),
    "bf16_heads_33": (BF, 33, 576, 512, 128, [2000, 77], 128),
    "bf16_heads_64": (BF, 64, 576, 512, 64, [5000, 63], 128),
    "bf16_heads_127": (BF, 127, 576, 512, 64, [321], 4),
    "bf16_one_long": (BF, 128, 576, 512, 64, [50001], 128),
    "bf16_one_long_64": (BF, 64, 576, 512, 32, [100000], 0),
    "bf16_small_width": (BF, 4, 64, 64, 16, [0, 1, 100, 33], 16),
    "bf16_odd_width": (BF, 9, 200, 72, 10, [77, 400], 9),
    "f32_edges": (F32, 4, 64, 64, 24, EDGE, 16),
    "f32_wide": (F32, 20, 576, 512, 64, [100, 1, 700], 128),
    "f32_dk8": (F32, 3, 8, 4, 5, [50, 9], 0),
    "f32_dv_576": (F32, 2, 576, 576, 16, [90], 3),
    "f32_long": (F32, 8, 64, 64, 64, [20000, 3], 0),
}


@pytest.mark.parametrize("case", list(DENSE))
def test_dense(case):
    dtype, H, dk, dv, page, lens, W = DENSE[case]
    Case(sum(map(ord, case)), dtype, H, dk, dv, page, lens, W).run_and_check(case)


def make_idx(seed, B, k, cap, kind):
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((B, k), -1, dtype=torch.int32)
    for b in range(B):
        n = {"full": k, "padded": (k * (b + 1)) // (B + 1), "empty": 0 if b % 2 == 0 else k}[kind.split("_")[0]]
        n = min(n, cap)
        sel = torch.randperm(cap, generator=g)[:n].to(torch.int32)
        if "sorted" in kind:
            sel = sel.sort().values
        idx[b, :n] = sel
        if "holes" in kind:
            idx[b, ::3] = -1
    return idx.cuda()


SPARSE = {
    # dtype, H, dk, dv, page, cap, B, k, W, kind
    "bf16_512": (BF, 128, 576, 512, 64, 3000, 4, 512, 128, "full_sorted"),
    "bf16_pages_16": (BF, 128, 576, 512, 16, 2000, 3, 640, 128, "padded_sorted"),
    "bf16_k1": (BF, 128, 576, 512, 64, 100, 2, 1, 0, "full"),
    "bf16_k65_holes": (BF, 128, 576, 512, 7, 333, 5, 65, 5, "full_holes"),
    "bf16_empty": (BF, 128, 576, 512, 64, 500, 4, 100, 0, "empty"),
    "bf16_empty_window": (BF, 64, 576, 512, 64, 500, 4, 100, 128, "empty"),
    "bf16_k2048": (BF, 128, 576, 512, 32, 5000, 2, 2048, 128, "full_sorted"),
    "bf16_heads_12": (BF, 12, 576, 512, 64, 1000, 3, 300, 128, "padded"),
    "bf16_page_1": (BF, 96, 576, 512, 1, 400, 3, 128, 0, "full"),
    "f32": (F32, 4, 64, 64, 7, 600, 3, 77, 16, "padded_sorted"),
    "f32_wide": (F32, 11, 576, 512, 16, 300, 2, 150, 16, "full_holes"),
}


@pytest.mark.parametrize("case", list(SPARSE))
def test_sparse(case):
    dtype, H, dk, dv, page, cap, B, k, W, kind = SPARSE[case]
    Case(sum(map(ord, case)), dtype, H, dk, dv, page, [cap] * B, W, idx=make_idx(k, B, k, cap, kind)).run_and_check(case)


def test_sparse_counts_an_entry_twice_when_listed_twice():
    idx = make_idx(5, 2, 90, 200, "full")
    idx[:, 50:] = idx[:, :40]
    Case(91, BF, 128, 576, 512, 64, [200, 200], 16, idx=idx).run_and_check()


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (BF, 40, 576, 512), (F32, 4, 64, 64)])
def test_rows_without_anything_and_no_sink(dtype, H, dk, dv):
    c = Case(17, dtype, H, dk, dv, 64, [0, 70, 0, 1], 0, sink=-math.inf)
    c.run_and_check()
    assert bool((c.out[0] == 0).all()) and bool((c.lse[0] == -math.inf).all())
    s = Case(18, dtype, H, dk, dv, 64, [9, 70], 0, idx=torch.full((2, 33), -1, dtype=torch.int32, device="cuda"), sink=-math.inf)
    s.call()
    torch.cuda.synchronize()
    assert bool((s.out == 0).all()) and bool((s.lse == -math.inf).all())


@pytest.mark.parametrize("H", [128, 24])
def test_many_short_sequences(H):
    """More sequences than units: a unit holds many, most of them whole."""
    lens = [(37 * i) % 150 for i in range(700)]
    Case(23, BF, H, 576, 512, 16, lens, 8).run_and_check()


def test_many_sequences_small():
    lens = [(11 * i) % 40 for i in range(3000)]
    c = Case(29, F32, 2, 16, 16, 8, lens, 0)
    c.run_and_check()


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (F32, 4, 64, 64)])
def test_large_logits(dtype, H, dk, dv):
    """Logits of some hundreds: the running maximum rises along the cache, the scale of earlier
    sums falls to nothing."""
    c = Case(31, dtype, H, dk, dv, 64, [3000, 200], 16, qstd=60.0)
    ramp = torch.linspace(0.0, 1.0, 3000, device="cuda")
    for e in range(0, 3000, 64):
        n = min(64, 3000 - e)
        c.pages[c.table[0, e // 64], :n] *= ramp[e:e + n, None].to(dtype)
    c.run_and_check()


def test_same_bits_twice_and_in_any_workspace():
    c = Case(37, BF, 128, 576, 512, 64, [9000, 100, 4000], 128)
    c.call()
    first = c.out.clone(), c.lse.clone()
    c.ws.fill_(0)
    c.out.zero_()
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)


def test_lse_is_optional():
    c = Case(41, BF, 128, 576, 512, 64, [500, 20], 0)
    c.call()
    out = c.out.clone()
    csa.hca_attn_decode_paged(c.q, c.pages, c.table, c.n, None, None, c.sink, c.scale, c.dv, c.out, workspace=c.ws)
    torch.cuda.synchronize()
    assert torch.equal(out, c.out)


def test_captured_and_replayed_with_other_lengths():
    """A graph follows the lengths, tables and rows it finds when it is replayed."""
    c = Case(43, BF, 128, 576, 512, 64, [3000, 500, 64], 128)
    c.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for lens in ([10, 0, 64], [3000, 500, 1], [2999, 499, 63]):
        c.lens = lens
        c.n.copy_(torch.tensor(lens, dtype=torch.int32))
        c.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(c.out, c.lse, c.q, c.rows_of, c.sink, c.scale, str(lens))


def test_two_streams_at_once():
    a, b = Case(47, BF, 128, 576, 512, 64, [8000, 100], 128), Case(53, BF, 128, 576, 512, 32, [700, 6000], 0)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.call(stream=s)
        b.call(stream=t)
    torch.cuda.synchronize()
    for c in (a, b):
        check(c.out, c.lse, c.q, c.rows_of, c.sink, c.scale)


def test_pool_beyond_32_bit_offsets():
    """The rows lie behind 2^32 bytes and 2^31 values of the pool."""
    g = gen(59)
    page, d, n_pages = 256, 576, 16000                     # 2.36e9 values, 4.7 GB
    pages = torch.empty(n_pages, page, d, device="cuda", dtype=BF)
    c = Case(61, BF, 128, d, 512, page, [600, 300], 0)
    table = torch.tensor([[n_pages - 1, n_pages - 3, 0, 0], [15999 - 5, 0, 0, 0]], dtype=torch.int32, device="cuda")
    table[1, 1] = n_pages - 7
    for b in range(2):
        for i in range(-(-c.lens[b] // page)):
            pages[table[b, i]] = randn(g, page, d, dtype=BF)
    c.pages, c.table = pages, table
    c.ws = torch.empty(csa.attn_decode_paged_workspace_size(2, 128, 512, 4 * page), dtype=torch.uint8, device="cuda")
    c.run_and_check()
    rows = randn(g, 2, d, dtype=BF)
    csa.latent_append_paged(rows, torch.tensor([601, 256], dtype=torch.int32, device="cuda"), pages, table)
    torch.cuda.synchronize()
    assert torch.equal(pages[table[0, 2].long(), 601 - 512], rows[0]) and torch.equal(pages[table[1, 1].long(), 0], rows[1])


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (F32, 4, 64, 64)])
def test_bad_pages_and_entries_are_skipped_and_flagged(dtype, H, dk, dv):
    c = Case(67, dtype, H, dk, dv, 16, [200, 100], 0)
    good = c.table.clone()
    c.table[0, 3] = -1                                     # entries 48 .. 63 are gone
    c.table[1, 0] = c.pages.shape[0]                       # entries 0 .. 15 are gone
    c.call()
    torch.cuda.synchronize()
    assert csa.read_device_error() == DEVERR_INDEX
    keep = [torch.cat((torch.arange(0, 48), torch.arange(64, 200))).cuda(), torch.arange(16, 100).cuda()]
    check(c.out, c.lse, c.q, lambda b: entry_rows(c.pages, good, b, keep[b]), c.sink, c.scale)
    idx = torch.tensor([[0, 50, 199, 7], [16, 3, 99, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    s = Case(67, dtype, H, dk, dv, 16, [200, 100], 0, idx=idx)
    s.table.copy_(c.table)
    s.call()
    torch.cuda.synchronize()
    assert csa.read_device_error() == DEVERR_INDEX
    kept = [torch.tensor([0, 199, 7], device="cuda"), torch.tensor([16, 99], device="cuda")]
    check(s.out, s.lse, s.q, lambda b: entry_rows(s.pages, good, b, kept[b]), s.sink, s.scale)


def test_lengths_beyond_the_table_are_clamped():
    c = Case(71, BF, 128, 576, 512, 16, [160, 160], 0)
    table = c.table[:, :10].contiguous()
    c.n.copy_(torch.tensor([10 ** 6, -5], dtype=torch.int32))
    c.table, c.lens = table, [160, 0]
    c.run_and_check()


# ----------------------------------------------------------------------------- append

def rotated(x, pos, inv_freq, near):
    """x [..., d_r] in 64 bits, pos broadcastable to x[..., 0]."""
    ang = pos.double()[..., None] * inv_freq.double()
    z = torch.polar(torch.ones_like(ang), ang)
    x = x.double()
    if near:
        y = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * z
        return torch.view_as_real(y).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    y = torch.complex(a, b) * z
    return torch.cat((y.real, y.imag), dim=-1)


def check_rotated(got, x, pos, inv_freq, near, what):
    """A rotated value a c - b s: cos and sin off by 4 half steps of fp32 each (the reduced angle's
    rounding and the function's own), two products and a sum: |a| + |b| times 8u, and the storage
    rounding."""
    want = rotated(x, pos, inv_freq, near)
    size = x.double().abs().amax(dim=-1, keepdim=True) * 2
    assert bool(((got.double() - want).abs() <= size * 8 * U + R[got.dtype] * want.abs()).all()), what


APPEND = {
    # dtype, T, B, H, d, d_r, page, near
    "one": (BF, 1, 1, 128, 576, 64, 64, True),
    "batch": (BF, 33, 33, 128, 576, 64, 64, True),
    "chunk": (BF, 700, 3, 64, 576, 64, 32, True),
    "far": (BF, 41, 41, 5, 576, 64, 7, False),
    "whole_row": (BF, 9, 9, 2, 64, 64, 1, False),
    "f32": (F32, 50, 4, 4, 64, 32, 16, True),
    "f32_far": (F32, 50, 50, 3, 576, 64, 24, False),
    "no_queries": (BF, 65, 65, 0, 576, 64, 64, True),
    "wide_rotation": (F32, 5, 5, 1, 576, 576, 64, False),
}


@pytest.mark.parametrize("case", list(APPEND))
def test_append(case):
    dtype, T, B, H, d, dr, page, near = APPEND[case]
    g = gen(sum(map(ord, case)))
    per = -(-T // B)
    cap = per + 3 * page + 5
    pages, table = make_cache(g, dtype, [cap] * B, page, d, fill=3.0)
    t = torch.arange(T, device="cuda")
    seq = (t // per).to(torch.int32)
    entry = ((seq * 7) % (cap - per + 1) + t % per).to(torch.int32)
    skip = torch.zeros(T, dtype=torch.bool, device="cuda")
    if T > 4:
        skip[2] = skip[T - 1] = True
        entry[skip] = -1
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    inv = 10000.0 ** (-torch.arange(0, dr, 2, device="cuda", dtype=torch.float32) / dr)
    wide = randn(g, T, d + 32, dtype=dtype)                # rows are a slice of a wider projection
    rows = wide[:, 16:16 + d]
    q = q_pe = None
    if H:
        q = randn(g, T, H, d, dtype=dtype)
        q_pe = randn(g, T, H, dr + 16, dtype=dtype)[..., 8:8 + dr]
        q0 = q.clone()
    before = pages.clone()
    csa.latent_append_paged(rows, entry, pages, table, seq=None if T == B else seq, pos=pos, inv_freq=inv, interleaved=near,
                            q_pe=q_pe, q=q)
    torch.cuda.synchronize()
    assert csa.read_device_error() == 0
    live = (~skip).nonzero()[:, 0]
    e = entry[live].long()
    pid, off = table[seq[live].long(), e // page].long(), e % page
    got = pages[pid, off]
    assert torch.equal(got[:, :d - dr], rows[live][:, :d - dr])
    check_rotated(got[:, d - dr:], rows[live][:, d - dr:], pos[live], inv, near, case)
    pages[pid, off] = before[pid, off]
    assert torch.equal(pages, before)                      # nothing else was written
    if H:
        check_rotated(q[live][..., d - dr:], q_pe[live], pos[live][:, None].expand(-1, H), inv, near, case)
        q[live, :, d - dr:] = q0[live, :, d - dr:]
        assert torch.equal(q, q0)


def test_append_without_rotation_is_a_copy_and_position_defaults_to_the_entry():
    g = gen(73)
    pages, table = make_cache(g, BF, [100, 100], 16, 576)
    rows = randn(g, 2, 576, dtype=BF)
    rows[0, 5] = float("nan")
    entry = torch.tensor([17, 99], dtype=torch.int32, device="cuda")
    csa.latent_append_paged(rows, entry, pages, table)
    torch.cuda.synchronize()
    for t in range(2):
        got = pages[table[t, int(entry[t]) // 16].long(), int(entry[t]) % 16]
        assert torch.equal(got.view(torch.int16), rows[t].view(torch.int16))
    inv = torch.tensor([1.0, 0.5, 0.25, 0.125], device="cuda")
    csa.latent_append_paged(rows, entry, pages, table, inv_freq=inv)
    torch.cuda.synchronize()
    got = pages[table[1, 99 // 16].long(), 99 % 16]
    check_rotated(got[None, -8:], rows[1:, -8:], entry[1:], inv, True, "entry as position")


def test_queries_rotated_in_place():
    g = gen(79)
    pages, table = make_cache(g, BF, [64] * 3, 64, 576)
    q = randn(g, 3, 128, 576, dtype=BF)
    q0 = q.clone()
    inv = 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float32) / 64)
    entry = torch.tensor([3, 60, 9], dtype=torch.int32, device="cuda")
    for near in (True, False):
        q.copy_(q0)
        csa.latent_append_paged(randn(g, 3, 576, dtype=BF), entry, pages, table, inv_freq=inv, interleaved=near,
                                q_pe=q[..., 512:], q=q)
        torch.cuda.synchronize()
        check_rotated(q[..., 512:], q0[..., 512:], entry[:, None].expand(-1, 128), inv, near, near)
        assert torch.equal(q[..., :512], q0[..., :512])


def test_append_out_of_range_is_skipped_and_flagged():
    g = gen(83)
    pages, table = make_cache(g, BF, [32] * 4, 16, 576, fill=1.0)
    before = pages.clone()
    q = randn(g, 4, 2, 576, dtype=BF)
    q0 = q.clone()
    inv = torch.ones(4, device="cuda")
    width = table.shape[1]
    table[3, 0] = pages.shape[0]
    entry = torch.tensor([width * 16, 5, 5, 5], dtype=torch.int32, device="cuda")     # beyond the table
    seq = torch.tensor([0, 4, -1, 3], dtype=torch.int32, device="cuda")               # no such sequences; a bad page
    csa.latent_append_paged(randn(g, 4, 576, dtype=BF), entry, pages, table, seq=seq, inv_freq=inv, q_pe=q0[..., :8], q=q)
    torch.cuda.synchronize()
    assert csa.read_device_error() == DEVERR_ENTRY
    assert torch.equal(pages, before) and torch.equal(q, q0)


def test_binding_refuses_tensors_that_do_not_fit():
    c = Case(89, BF, 128, 576, 512, 64, [100, 50], 16)
    ok = dict(q=c.q, pages=c.pages, block_table=c.table, n_entries=c.n, win=c.win, win_len=c.win_len, sink=c.sink,
              sm_scale=c.scale, d_v=512, out=c.out, lse=c.lse, workspace=c.ws)
    before = csa.launch_count()
    for k, bad in [("q", c.q.float()), ("q", c.q[:1]), ("q", c.q.transpose(0, 1)), ("q", c.q.cpu()), ("pages", c.pages[:, :, ::2]),
                   ("pages", c.pages.half()), ("block_table", c.table.long()), ("block_table", c.table.t()), ("n_entries", c.n.long()),
                   ("n_entries", c.n[:1]), ("win", c.win[:, :, :512]), ("win_len", c.win_len.cpu()), ("win_len", c.win_len[:1]),
                   ("sink", c.sink[:64]), ("sink", c.sink.bfloat16()), ("d_v", 256), ("out", c.out.float()), ("lse", c.lse.double()),
                   ("workspace", c.ws[:64]), ("workspace", None), ("workspace", c.ws.cpu()), ("sm_scale", math.nan)]:
        with pytest.raises(csa.CsaError):
            csa.hca_attn_decode_paged(**{**ok, k: bad})
    idx = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    more = {k: v for k, v in ok.items() if k != "n_entries"}
    for bad in (idx.long(), idx[:1], idx[:, ::2], idx.cpu(), idx[0]):
        with pytest.raises(csa.CsaError):
            csa.sparse_attn_decode_paged(**{**more, "idx": bad})
    rows, entry, inv = torch.zeros(2, 576, device="cuda", dtype=BF), c.n, torch.ones(32, device="cuda")
    good = dict(rows=rows, entry=entry, pages=c.pages, block_table=c.table, inv_freq=inv, q=c.q, q_pe=c.q[..., 512:])
    for k, bad in [("rows", rows.float()), ("rows", rows[:1]), ("rows", rows[:, :512]), ("rows", torch.zeros(576, 2, device="cuda", dtype=BF).t()),
                   ("entry", entry.long()), ("entry", entry[:1]), ("seq", entry.long()), ("pos", entry[:1]), ("inv_freq", inv.double()),
                   ("inv_freq", inv.cpu()), ("inv_freq", inv[:30]), ("q", None), ("q_pe", None), ("q", c.q.float()),
                   ("q_pe", c.q[..., :32]), ("q_pe", c.q[:, :64, 512:])]:
        with pytest.raises(csa.CsaError):
            csa.latent_append_paged(**{**good, k: bad})
    assert csa.launch_count() == before
    torch.cuda.synchronize()
    assert csa.read_device_error() == 0


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 576, 512), (F32, 64, 64)])
def test_the_smallest_call(dtype, dk, dv):
    """One sequence, one head, a pool of one page of one row, a window of one row."""
    c = Case(97, dtype, 1, dk, dv, 1, [1], 1)
    row = c.pages[c.table[0, 0].long()].clone().view(1, 1, dk)
    c.pages, c.table = row.contiguous(), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    c.run_and_check()


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (BF, 7, 576, 512), (F32, 4, 64, 64)])
@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-30])
def test_scales(dtype, H, dk, dv, scale):
    c = Case(103, dtype, H, dk, dv, 64, [0, 70, 1000], 9)
    c.scale = scale
    c.run_and_check(str(scale))


def test_many_sequences_most_of_them_empty():
    lens = [0 if i % 7 else 1 + i % 90 for i in range(5000)]
    Case(107, BF, 3, 576, 512, 32, lens, 0).run_and_check()


def test_append_with_strides_that_mean_nothing():
    """A single row or head: torch gives its stride any value."""
    g = gen(109)
    pages, table = make_cache(g, BF, [64], 64, 576)
    rows = randn(g, 3, 576, dtype=BF)[1:2]
    q = randn(g, 1, 1, 576, dtype=BF)
    q_pe = randn(g, 1, 1, 64, dtype=BF).as_strided((1, 1, 64), (3, 5, 1))
    inv = 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float32) / 64)
    entry = torch.tensor([9], dtype=torch.int32, device="cuda")
    csa.latent_append_paged(rows, entry, pages, table, inv_freq=inv, q_pe=q_pe, q=q)
    torch.cuda.synchronize()
    check_rotated(q[0, :, 512:], q_pe[0], entry, inv, True, "single")
    assert torch.equal(pages[table[0, 0].long(), 9, :512], rows[0, :512])


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (BF, 7, 576, 512), (F32, 4, 64, 64), (F32, 1, 64, 36), (F32, 11, 72, 64)])
@pytest.mark.parametrize("every", [False, True])
def test_a_nan_that_is_attended_shows_and_stays_with_its_sequence(dtype, H, dk, dv, every):
    c = Case(113, dtype, H, dk, dv, 16, [40, 900, 40], 9)
    for e in range(900) if every else [517]:
        c.pages[c.table[1, e // 16].long(), e % 16] = math.nan
    if every:
        c.win[1] = math.nan
    c.call()
    torch.cuda.synchronize()
    assert csa.read_device_error() == 0
    assert bool(c.out[1].isnan().all()) and bool(c.lse[1].isnan().all())
    for b in (0, 2):
        check(c.out[b:b + 1], c.lse[b:b + 1], c.q[b:b + 1], lambda _, b=b: c.rows_of(b), c.sink, c.scale)


@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 64, 64), (F32, 8, 4), (BF, 136, 100), (F32, 576, 576), (BF, 64, 16), (F32, 320, 260)])
def test_few_heads_share_a_tile_s_rows(H, dtype, dk, dv):
    Case(127 + H, dtype, H, dk, dv, 24, [0, 1, 31, 33, 700, 4100], 9).run_and_check()


def test_out_and_rows_at_16_bytes():
    """Every address a multiple of 16 bytes, none of 32."""
    c = Case(131, BF, 128, 576, 512, 64, [100, 0, 9000, 64], 9)

    def moved(t):
        buf = torch.empty(t.numel() + 16, device="cuda", dtype=t.dtype)
        k = 16 // t.element_size()
        v = buf[k:k + t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v
    c.q, c.pages, c.win, c.out, c.lse, c.sink, c.ws = (moved(t) for t in (c.q, c.pages, c.win, c.out, c.lse, c.sink, c.ws))
    c.run_and_check()


@pytest.mark.parametrize("dtype,H,dk,dv", [(BF, 128, 576, 512), (F32, 4, 64, 64)])
def test_the_largest_pages_windows_and_selections(dtype, H, dk, dv):
    Case(137, dtype, H, dk, dv, 65536, [70001, 5], 4096).run_and_check("dense")
    g = gen(139)
    idx = torch.randint(-1, 5000, (2, 65536), generator=g, device="cuda", dtype=torch.int32)
    Case(149, dtype, H, dk, dv, 100, [5000, 5000], 4096, idx=idx).run_and_check("sparse")


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 576, 512), (F32, 64, 64)])
def test_the_most_sequences(dtype, dk, dv):
    """65 535 sequences of one row or none, pages of one row; out and lse have closed forms."""
    g, B = gen(151), 65535
    pages = randn(g, 3000, 1, dk, dtype=dtype)
    table = torch.randint(0, 3000, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    n = (torch.arange(B, device="cuda") % 3 != 1).to(torch.int32)
    q, sink, scale = randn(g, B, 1, dk, dtype=dtype), randn(g, 1), dk ** -0.5
    out, lse = torch.full((B, 1, dv), 7.0, device="cuda", dtype=dtype), torch.full((B, 1), 7.0, device="cuda")
    ws = torch.empty(csa.attn_decode_paged_workspace_size(B, 1, dv, 1), dtype=torch.uint8, device="cuda")
    csa.hca_attn_decode_paged(q, pages, table, n, None, None, sink, scale, dv, out, lse, ws)
    torch.cuda.synchronize()
    assert csa.read_device_error() == 0
    rows = pages.double()[table[:, 0].long(), 0]
    qr = q.double()[:, 0] * rows
    l = torch.where(n > 0, qr.sum(1) * scale, -math.inf)
    D = (qr.abs().sum(1) * scale) * (dk + 8) * 2 * U + l.abs().nan_to_num(0, 0, 0) * 2 * U + 2.0 ** -21
    L = torch.logaddexp(l, sink.double())
    p = (l - L).exp()
    want = p[:, None] * rows[:, :dv]
    tol = (p[:, None] * rows[:, :dv].abs()) * (2 * D + 2.0 ** -15 + 2.0 ** -11 * (dtype == BF) + 40 * U)[:, None] + R[dtype] * want.abs()
    assert bool(((out[:, 0].double() - want).abs() <= tol).all())
    assert bool(((lse[:, 0].double() - L).abs() <= D + 40 * U + L.abs() * 2 * U).all())


@pytest.mark.parametrize("H", [128, 7])
def test_tiles_without_a_row(H):
    """Selections without an entry: whole tiles of zeros, alone and between others."""
    idx = torch.full((5, 200), -1, dtype=torch.int32, device="cuda")
    idx[1, 70:75] = torch.arange(5, dtype=torch.int32, device="cuda")
    idx[3, ::3] = 7
    idx[4, 199] = 300
    Case(157, BF, H, 576, 512, 64, [400] * 5, 0, idx=idx).run_and_check("no window")
    Case(163, BF, H, 576, 512, 64, [400] * 5, 9, idx=idx).run_and_check("window")
