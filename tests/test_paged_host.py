"""Host-only checks of the paged-cache calls: arguments that the documentation rules out are
refused before any device work, with the documented status, and the binding refuses tensors
that do not fit (these calls never reach a kernel, so they run without a GPU)."""
import pytest
import torch

import compressed_sparse_long_csa_b200 as csa
from compressed_sparse_long_csa_b200 import _native as N

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_UNSUP, ERR_WS, ERR_CUDA = range(8)
FAKE = 1 << 20          # a 16-byte aligned address that is never dereferenced on the host


def append(**kw):
    a = dict(rows=FAKE, rows_ld=576, seq=None, entry=FAKE, pos=None, inv=FAKE, d_r=64, near=1, pages=FAKE, n_pages=8, page=64,
             table=FAKE, width=4, B=2, T=2, d=576, q_pe=FAKE, ld_t=8192, ld_h=64, q=FAKE, H=128, d_q=576, dtype=1)
    a.update(kw)
    return N.lib.latent_append_paged(*[a[k] for k in ("rows", "rows_ld", "seq", "entry", "pos", "inv", "d_r", "near", "pages",
                                                      "n_pages", "page", "table", "width", "B", "T", "d", "q_pe", "ld_t", "ld_h",
                                                      "q", "H", "d_q", "dtype")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), ERR_NULL), (dict(entry=None), ERR_NULL), (dict(pages=None), ERR_NULL), (dict(table=None), ERR_NULL),
    (dict(q_pe=None), ERR_NULL), (dict(inv=None), ERR_NULL), (dict(inv=None, d_r=0), ERR_NULL),
    (dict(rows=FAKE + 8), ERR_ALIGN), (dict(pages=FAKE + 2), ERR_ALIGN), (dict(q=FAKE + 4), ERR_ALIGN), (dict(q_pe=FAKE + 4), ERR_ALIGN),
    (dict(dtype=2), ERR_DTYPE), (dict(T=0), ERR_SHAPE), (dict(T=3), ERR_SHAPE), (dict(B=0), ERR_SHAPE), (dict(B=65536), ERR_SHAPE),
    (dict(d=577), ERR_SHAPE), (dict(d=580), ERR_SHAPE), (dict(d=584), ERR_SHAPE), (dict(rows_ld=568), ERR_SHAPE),
    (dict(rows_ld=580), ERR_SHAPE), (dict(d_r=60), ERR_SHAPE), (dict(d_r=584), ERR_SHAPE), (dict(d_r=72, near=0), ERR_SHAPE),
    (dict(page=0), ERR_SHAPE), (dict(page=65537), ERR_SHAPE), (dict(width=0), ERR_SHAPE), (dict(n_pages=0), ERR_SHAPE),
    (dict(width=1 << 25), ERR_SHAPE), (dict(n_pages=1 << 25), ERR_SHAPE), (dict(H=0), ERR_SHAPE), (dict(H=129), ERR_SHAPE),
    (dict(d_q=56), ERR_SHAPE), (dict(ld_t=4), ERR_SHAPE), (dict(ld_h=-64), ERR_SHAPE),
])
def test_append_refusals(kw, status):
    before = N.lib.csa_launch_count()
    assert append(**kw) == status
    assert N.lib.csa_launch_count() == before


def attend(sparse=False, **kw):
    a = dict(q=FAKE, pages=FAKE, n_pages=8, page=64, table=FAKE, width=4, sel=FAKE, k=32, win=FAKE, win_len=FAKE, sink=FAKE, B=2,
             H=128, dk=576, dv=512, W=128, scale=0.04, dtype=1, out=FAKE, lse=FAKE, ws=FAKE, wb=1 << 40)
    a.update(kw)
    head = [a[k] for k in ("q", "pages", "n_pages", "page", "table", "width", "sel")] + ([a["k"]] if sparse else [])
    tail = [a[k] for k in ("win", "win_len", "sink", "B", "H", "dk", "dv", "W", "scale", "dtype", "out", "lse", "ws", "wb")]
    return (N.lib.sparse_attn_decode_paged if sparse else N.lib.hca_attn_decode_paged)(*head, *tail, None)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ERR_NULL), (dict(pages=None), ERR_NULL), (dict(table=None), ERR_NULL), (dict(sel=None), ERR_NULL),
    (dict(win=None), ERR_NULL), (dict(win_len=None), ERR_NULL), (dict(sink=None), ERR_NULL), (dict(out=None), ERR_NULL),
    (dict(q=FAKE + 4), ERR_ALIGN), (dict(pages=FAKE + 8), ERR_ALIGN), (dict(lse=FAKE + 4), ERR_ALIGN), (dict(ws=FAKE + 8), ERR_ALIGN),
    (dict(dtype=3), ERR_DTYPE), (dict(B=0), ERR_SHAPE), (dict(H=129), ERR_SHAPE), (dict(H=0), ERR_SHAPE), (dict(dk=572), ERR_SHAPE),
    (dict(dk=584), ERR_SHAPE), (dict(dv=600), ERR_SHAPE), (dict(dv=510), ERR_SHAPE), (dict(W=-1), ERR_SHAPE), (dict(W=4097), ERR_SHAPE),
    (dict(scale=float("nan")), ERR_SHAPE), (dict(scale=float("inf")), ERR_SHAPE), (dict(page=0), ERR_SHAPE), (dict(width=0), ERR_SHAPE),
    (dict(n_pages=1 << 25), ERR_SHAPE), (dict(width=1 << 25), ERR_SHAPE), (dict(ws=None), ERR_WS), (dict(wb=1000), ERR_WS),
])
def test_attention_refusals(sparse, kw, status):
    before = N.lib.csa_launch_count()
    assert attend(sparse, **kw) == status
    assert N.lib.csa_launch_count() == before


def test_sparse_slots_are_bounded():
    assert attend(True, k=0) == ERR_SHAPE
    assert attend(True, k=65537) == ERR_SHAPE


def test_workspace_size():
    size = csa.attn_decode_paged_workspace_size
    assert size(0, 128, 512, 100) == 0 and size(1, 0, 512, 100) == 0 and size(1, 1, 0, 100) == 0 and size(1, 1, 4, -1) == 0
    assert 0 < size(1, 128, 512, 100) <= size(16, 128, 512, 100) <= size(16, 128, 512, 10 ** 6) == size(65535, 128, 512, 2 ** 31 - 1)
    # the call asks for exactly that much: one byte less is refused (and a full one would launch)
    assert attend(wb=size(2, 128, 512, 4 * 64 + 128) - 1) == ERR_WS
    assert attend(True, wb=size(2, 128, 512, 32 + 128) - 1) == ERR_WS


def test_binding_refuses_tensors_that_do_not_fit():
    pages, table = torch.zeros(4, 16, 64), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(csa.CsaError, match="current CUDA device"):
        csa.latent_append_paged(torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), pages, table)
    with pytest.raises(csa.CsaError, match="current CUDA device"):
        csa.hca_attn_decode_paged(torch.zeros(2, 4, 64), pages, table, torch.zeros(2, dtype=torch.int32), None, None,
                                  torch.zeros(4), 0.1, 64, torch.zeros(2, 4, 64))
    with pytest.raises(csa.CsaError, match="current CUDA device"):
        csa.sparse_attn_decode_paged(torch.zeros(2, 4, 64), pages, table, torch.zeros(2, 3, dtype=torch.int32), None, None,
                                     torch.zeros(4), 0.1, 64, torch.zeros(2, 4, 64))


@pytest.mark.parametrize("missing", range(4))
def test_binding_names_what_is_missing(missing):
    args = [torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(4, 16, 64), torch.zeros(2, 2, dtype=torch.int32)]
    args[missing] = None
    with pytest.raises(csa.CsaError, match="needed"):
        csa.latent_append_paged(*args)
    with pytest.raises(csa.CsaError, match="needed"):
        csa.hca_attn_decode_paged(*args, None, None, torch.zeros(4), 0.1, 64, torch.zeros(2, 4, 64))
    with pytest.raises(csa.CsaError, match="needed"):
        csa.sparse_attn_decode_paged(*[torch.zeros(2, 4, 64)] * 4, None, None, None, 0.1, 64, torch.zeros(2, 4, 64))
