"""ctypes binding of libcsa_b200.so (argument marshalling only)."""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libcsa_b200.so")
if not os.path.exists(lib_path):
    raise ImportError(f"{lib_path} is missing: build it with `python -m compressed_sparse_long_csa_b200.build`")
lib = C.CDLL(lib_path)

CSA_F32, CSA_BF16 = 0, 1
CSA_IFMT_F32, CSA_IFMT_E4M3, CSA_IFMT_MXFP4 = 0, 1, 2

_vp, _i32, _i64, _f32, _sz = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t

_SIGS = {
    "csa_abi_version": ([], _i32),
    "csa_status_string": ([_i32], C.c_char_p),
    "csa_read_device_error": ([_vp, C.POINTER(C.c_uint32)], _i32),
    "csa_launch_count": ([], C.c_uint64),
    "csa_wait_probe": ([C.c_uint64, _vp], _i32),
    "csa_tensor_peak_probe": ([_i32, _i32, _vp], _i32),
    "csa_compress": ([_vp] * 10 + [_i64, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "csa_compress_kv8": ([_vp] * 10 + [_i64, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "csa_decode_append": ([_vp] * 10 + [_i64, _i32] + [_vp] * 10 + [_i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "window_append": ([_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp], _i32),
    "index_key_compress": ([_vp] * 11 + [_i64, _i32, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "shard_topk_merge": ([_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp], _i32),
    "attn_merge_shards": ([_vp, _vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp], _i32),
    "grouped_out_proj_workspace_size": ([_i32, _i32, _i32, _i32], _sz),
    "grouped_out_proj": ([_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "hca_compress": ([_vp] * 5 + [_i64, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "lightning_index_workspace_size": ([_i32, _i32, _i64, _i32], _sz),
    "lightning_index_workspace_size_exact": ([_i32, _i32, _i64, _i32, _i32, _i32, _i32], _sz),
    "lightning_index": ([_vp] * 7 + [_i32, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "lightning_index_bf16": ([_vp] * 7 + [_i32, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _sz, _vp], _i32),
    "topk_select_workspace_size": ([_i32, _i64, _i32], _sz),
    "topk_select": ([_vp, _i64, _vp, _i32, _i64, _i32, _vp, _vp, _sz, _vp], _i32),
    "attn_decode_workspace_size": ([_i32, _i32, _i32, _i64], _sz),
    "sparse_attn_decode": ([_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _i32, _i32, _f32, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "hca_attn_decode": ([_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _i32, _f32, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "sparse_attn_decode_kv8": ([_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _i32, _i32, _f32, _vp, _vp, _vp, _sz, _vp], _i32),
    "hca_attn_decode_kv8": ([_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _i32, _f32, _vp, _vp, _vp, _sz, _vp], _i32),
    "hca_compress_attn_decode": ([_vp] * 4 + [_i32, _i32] + [_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _i32, _f32, _i32,
                                                                      _vp, _vp, _vp, _sz, _vp], _i32),
    "sparse_attn_decode_noalloc": ([_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _i32, _i32, _f32, _i32, _vp, _vp, _vp], _i32),
    "latent_append_paged": ([_vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _i64, _i32, _vp, _i32, _i32, _i32, _i32,
                             _vp, _i64, _i64, _vp, _i32, _i32, _i32, _vp], _i32),
    "attn_decode_paged_workspace_size": ([_i32, _i32, _i32, _i64], _sz),
    "hca_attn_decode_paged": ([_vp, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _vp, _vp] + [_i32] * 5 +
                              [_f32, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "sparse_attn_decode_paged": ([_vp, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _vp] + [_i32] * 5 +
                                 [_f32, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "sparse_attn_prefill": ([_vp] * 5 + [_i64, _vp, _vp] + [_i32] * 5 + [_i64, _i32, _i32, _f32, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class CsaError(RuntimeError):
    pass


def _check(status: int, name: str):
    if status != 0:
        raise CsaError(f"{name}: {lib.csa_status_string(status).decode()}")


def _p(t):
    """Device pointer of a tensor (None -> NULL)."""
    if t is None:
        return None
    return t.data_ptr()


# The current device and its current stream's address without what the public calls add (a Stream
# object a call: 3 us; a look for an initialised context).  These names are torch's own: where a
# version has no such name, the public calls serve.
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream_now = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream):
    if stream is None:
        return _stream_now(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t):
    return CSA_BF16 if t.dtype == torch.bfloat16 else CSA_F32


def csa_decode_append(Ca, Cb, Za, Zb, Ba, Bb, prev_Cb, prev_Zb, entry0, cache, keys=None, window=None, stream=None):
    """One decode step's appends in one launch (see csa.h).  keys = (CaI, CbI, ZaI, ZbI, BaI,
    BbI, prev_CbI, prev_ZbI, kI, kI_scale, ifmt) or None; window = (raw_new, win, win_slot) or None."""
    B, _, d = Ca.shape
    kp = [None] * 10
    d_I, ifmt = 0, CSA_IFMT_E4M3
    if keys is not None:
        kp = [_p(t) for t in keys[:10]]
        d_I, ifmt = keys[0].shape[-1], keys[10]
    raw_new, win, slot, W = None, None, None, 0
    if window is not None:
        raw_new, win, slot = window
        W = win.shape[1]
    _check(lib.csa_decode_append(_p(Ca), _p(Cb), _p(Za), _p(Zb), _p(Ba), _p(Bb), _p(prev_Cb), _p(prev_Zb), _p(entry0),
                                 _p(cache), cache.shape[1], d, *kp, d_I, ifmt, _p(raw_new), _p(win), _p(slot), W, B,
                                 _dtype_code(Ca), _stream(stream)), "csa_decode_append")


def window_append(raw_new, win, win_slot, stream=None):
    B, W, d = win.shape
    _check(lib.window_append(_p(raw_new), _p(win), _p(win_slot), B, W, d, _dtype_code(win), _stream(stream)),
           "window_append")


def wait_probe(limit_ns: int, stream=None):
    """One kernel whose wait can never end, bounded by limit_ns (sets CSA_DEVERR_TIMEOUT)."""
    _check(lib.csa_wait_probe(int(limit_ns), _stream(stream)), "csa_wait_probe")


def tensor_peak_probe(ifmt, iters, stream=None):
    """Dense MMA rate probe at the indexer's operand formats (see csa_tensor_peak_probe)."""
    _check(lib.csa_tensor_peak_probe(int(ifmt), int(iters), _stream(stream)), "csa_tensor_peak_probe")


def launch_count() -> int:
    """Kernels the library has enqueued in this process (a captured launch counts once)."""
    return int(lib.csa_launch_count())


def read_device_error(stream=None) -> int:
    v = C.c_uint32(0)
    _check(lib.csa_read_device_error(_stream(stream), C.byref(v)), "csa_read_device_error")
    return int(v.value)


def csa_compress(Ca, Cb, Za, Zb, Ba, Bb, prev_Cb, prev_Zb, entry0, cache, m=4, stream=None):
    B, T_new, d = Ca.shape
    _check(lib.csa_compress(_p(Ca), _p(Cb), _p(Za), _p(Zb), _p(Ba), _p(Bb), _p(prev_Cb), _p(prev_Zb),
                            _p(entry0), _p(cache), cache.shape[1], B, T_new, d, m, _dtype_code(Ca),
                            _stream(stream)), "csa_compress")


def index_key_compress(Ca, Cb, Za, Zb, Ba, Bb, prev_Cb, prev_Zb, entry0, kI, kI_scale, ifmt, m=4, stream=None):
    B, T_new, d_I = Ca.shape
    _check(lib.index_key_compress(_p(Ca), _p(Cb), _p(Za), _p(Zb), _p(Ba), _p(Bb), _p(prev_Cb), _p(prev_Zb),
                                  _p(entry0), _p(kI), _p(kI_scale), kI.shape[1], B, T_new, d_I, m,
                                  _dtype_code(Ca), ifmt, _stream(stream)), "index_key_compress")


def shard_topk_merge(idx_parts, score_parts, bounds, local_idx_out, stream=None):
    """idx_parts / score_parts [G, R, k]; bounds [G+1] int32; local_idx_out [G, R, k]."""
    G, R, k = idx_parts.shape
    _check(lib.shard_topk_merge(_p(idx_parts), _p(score_parts), _p(bounds), G, R, k, _p(local_idx_out),
                                _stream(stream)), "shard_topk_merge")


def attn_merge_shards(o_parts, lse_parts, out, lse_out=None, stream=None):
    """o_parts [G, rows, dv] (any leading shape flattened to rows); lse_parts [G, rows]."""
    G = o_parts.shape[0]
    dv = o_parts.shape[-1]
    rows = o_parts[0].numel() // dv
    _check(lib.attn_merge_shards(_p(o_parts), _p(lse_parts), G, rows, dv, _dtype_code(o_parts), _p(out),
                                 _p(lse_out), _stream(stream)), "attn_merge_shards")


def grouped_out_proj_workspace_size(T, g, d_mid, d):
    return lib.grouped_out_proj_workspace_size(T, g, d_mid, d)


def grouped_out_proj(o, W1, W2, g, u, y, workspace=None, stream=None):
    """o [T, H, dv] bf16; W1 [g*d_mid, (H/g)*dv]; W2 [d, g*d_mid]; writes u [T, g*d_mid], y [T, d]."""
    T, H, dv = o.shape
    d_mid = W1.shape[0] // g
    d = W2.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.grouped_out_proj(_p(o), T, H, dv, g, d_mid, _p(W1), _p(W2), d, _p(u), _p(y), _p(workspace), ws_bytes,
                                _stream(stream)), "grouped_out_proj")


def csa_compress_kv8(Ca, Cb, Za, Zb, Ba, Bb, prev_Cb, prev_Zb, entry0, cache8, m=4, stream=None):
    """cache8: [B, n_max, 656] uint8 FP8 rows (see csa.h)."""
    B, T_new, d = Ca.shape
    _check(lib.csa_compress_kv8(_p(Ca), _p(Cb), _p(Za), _p(Zb), _p(Ba), _p(Bb), _p(prev_Cb), _p(prev_Zb),
                                _p(entry0), _p(cache8), cache8.shape[1], B, T_new, d, m, _dtype_code(Ca),
                                _stream(stream)), "csa_compress_kv8")


def hca_compress(C_, Z, bias, entry0, cache, m_prime=128, stream=None):
    B, T_new, d = C_.shape
    _check(lib.hca_compress(_p(C_), _p(Z), _p(bias), _p(entry0), _p(cache), cache.shape[1], B, T_new, d,
                            m_prime, _dtype_code(C_), _stream(stream)), "hca_compress")


def lightning_index_workspace_size(B, Tq, n_max, k):
    return int(lib.lightning_index_workspace_size(B, Tq, n_max, k))


def lightning_index_workspace_size_exact(B, Tq, n_max, k, ifmt, H_I, d_I):
    return int(lib.lightning_index_workspace_size_exact(B, Tq, n_max, k, ifmt, H_I, d_I))


def lightning_index(qI, qI_scale, w, kI, kI_scale, n_entries, q_pos, k, ifmt, idx_out, workspace,
                    score_out=None, m=4, stream=None):
    B, Tq, H_I = w.shape
    n_max = kI.shape[1]
    d_I = qI.shape[-1] * (2 if ifmt == CSA_IFMT_MXFP4 else 1)
    _check(lib.lightning_index(_p(qI), _p(qI_scale), _p(w), _p(kI), _p(kI_scale), _p(n_entries), _p(q_pos), m,
                               B, Tq, H_I, d_I, n_max, k, ifmt, _p(idx_out), _p(score_out), _p(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)), "lightning_index")


def lightning_index_bf16(qI, qI_scale, w, kI, kI_scale, n_entries, q_pos, k, ifmt, idx_out, workspace, m=4,
                         stream=None):
    B, Tq, H_I = w.shape
    n_max = kI.shape[1]
    d_I = qI.shape[-1] * (2 if ifmt == CSA_IFMT_MXFP4 else 1)
    _check(lib.lightning_index_bf16(_p(qI), _p(qI_scale), _p(w), _p(kI), _p(kI_scale), _p(n_entries), _p(q_pos), m,
                                    B, Tq, H_I, d_I, n_max, k, ifmt, _p(idx_out), _p(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)),
           "lightning_index_bf16")


def topk_select(scores, n_valid, k, idx_out, stream=None):
    R, n = scores.shape
    _check(lib.topk_select(_p(scores), scores.stride(0), _p(n_valid), R, n, k, _p(idx_out), None, 0,
                           _stream(stream)), "topk_select")


def attn_decode_workspace_size(B, H, d_v, rows_max):
    return int(lib.attn_decode_workspace_size(B, H, d_v, rows_max))


def _ws(workspace):
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def sparse_attn_decode(q, cache, idx, win, win_len, sink, sm_scale, d_v, out, lse=None, workspace=None,
                       stream=None):
    B, H, d_k = q.shape
    W = win.shape[1] if win is not None else 0
    k = idx.shape[1] if idx is not None else 0
    wp, wb = _ws(workspace)
    _check(lib.sparse_attn_decode(_p(q), _p(cache), _p(idx), _p(win), _p(win_len), _p(sink), B, H, d_k, d_v,
                                  cache.shape[1], k, W, sm_scale, _dtype_code(q), _p(out), _p(lse), wp, wb,
                                  _stream(stream)), "sparse_attn_decode")


def hca_attn_decode(q, cache, n_entries, win, win_len, sink, sm_scale, d_v, out, lse=None, workspace=None,
                    stream=None):
    B, H, d_k = q.shape
    W = win.shape[1] if win is not None else 0
    wp, wb = _ws(workspace)
    _check(lib.hca_attn_decode(_p(q), _p(cache), _p(n_entries), _p(win), _p(win_len), _p(sink), B, H, d_k, d_v,
                               cache.shape[1], W, sm_scale, _dtype_code(q), _p(out), _p(lse), wp, wb,
                               _stream(stream)), "hca_attn_decode")


def sparse_attn_decode_kv8(q, cache8, idx, win, win_len, sink, sm_scale, d_v, out, lse=None, workspace=None,
                           stream=None):
    """cache8: [B, n_max, 656] uint8 FP8 rows (see csa.h)."""
    B, H, d_k = q.shape
    W = win.shape[1] if win is not None else 0
    k = idx.shape[1] if idx is not None else 0
    wp, wb = _ws(workspace)
    _check(lib.sparse_attn_decode_kv8(_p(q), _p(cache8), _p(idx), _p(win), _p(win_len), _p(sink), B, H, d_k, d_v,
                                      cache8.shape[1], k, W, sm_scale, _p(out), _p(lse), wp, wb, _stream(stream)),
           "sparse_attn_decode_kv8")


def hca_attn_decode_kv8(q, cache8, n_entries, win, win_len, sink, sm_scale, d_v, out, lse=None, workspace=None,
                        stream=None):
    B, H, d_k = q.shape
    W = win.shape[1] if win is not None else 0
    wp, wb = _ws(workspace)
    _check(lib.hca_attn_decode_kv8(_p(q), _p(cache8), _p(n_entries), _p(win), _p(win_len), _p(sink), B, H, d_k,
                                   d_v, cache8.shape[1], W, sm_scale, _p(out), _p(lse), wp, wb, _stream(stream)),
           "hca_attn_decode_kv8")


def hca_compress_attn_decode(C_, Z, bias, entry0, q, cache, n_entries, win, win_len, sink, sm_scale, d_v, out,
                             lse=None, workspace=None, m_prime=128, stream=None):
    """hca_compress of the fresh chunk (C_, Z) then hca_attn_decode, as one call."""
    B, H, d_k = q.shape
    T_new = C_.shape[1]
    W = win.shape[1] if win is not None else 0
    wp, wb = _ws(workspace)
    _check(lib.hca_compress_attn_decode(_p(C_), _p(Z), _p(bias), _p(entry0), T_new, m_prime, _p(q), _p(cache),
                                        _p(n_entries), _p(win), _p(win_len), _p(sink), B, H, d_k, d_v, cache.shape[1],
                                        W, sm_scale, _dtype_code(q), _p(out), _p(lse), wp, wb, _stream(stream)),
           "hca_compress_attn_decode")


def sparse_attn_prefill(q, q_pos, cache, idx, raw, raw_pos0, W, sink, sm_scale, d_v, out, lse=None,
                        workspace=None, stream=None):
    B, Tq, H, d_k = q.shape
    k = idx.shape[2] if idx is not None else 0
    wp, wb = _ws(workspace)
    _check(lib.sparse_attn_prefill(_p(q), _p(q_pos), _p(cache), _p(idx), _p(raw), raw.shape[1], _p(raw_pos0),
                                   _p(sink), B, Tq, H, d_k, d_v, cache.shape[1], k, W, sm_scale, _dtype_code(q),
                                   _p(out), _p(lse), wp, wb, _stream(stream)), "sparse_attn_prefill")


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def sparse_attn_decode_noalloc(q, cache, idx, win, win_len, sink, sm_scale, d_v, out, lse=None, stream=None):
    """sparse_attn_decode for callers that cannot allocate: the split partials use the
    library's own fixed device buffer (NOALLOC_SCRATCH_BYTES).  Calls that overlap on
    the GPU race on that buffer; the first call on a device should precede capture."""
    B, H, d_k = q.shape
    W = win.shape[1] if win is not None else 0
    k = idx.shape[1] if idx is not None else 0
    _check(lib.sparse_attn_decode_noalloc(_p(q), _p(cache), _p(idx), _p(win), _p(win_len), _p(sink), B, H, d_k,
                                          d_v, cache.shape[1], k, W, sm_scale, _dtype_code(q), _p(out), _p(lse),
                                          _stream(stream)), "sparse_attn_decode_noalloc")


# ---- paged cache.  The tensors' shapes, types, strides and device are checked here (the C
# calls see addresses only): what does not fit raises CsaError and nothing is launched.  A
# decode step makes these calls once per layer and waits for nothing else on the host, so the
# checks are plain comparisons, written out (a helper per tensor cost 2 us a call); the message
# is made when one fails.
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16


def _unfit(name, what, t, want):
    got = "None" if t is None else f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}"
    raise CsaError(f"{name}: {what} must be {want} on the pages' device, got {got}")


def _paged(name, pages, block_table):
    """Checks of the pool and its table; the device's index."""
    di = pages.get_device()
    if di < 0 or di != _device_now():
        raise CsaError(f"{name}: pages must be on the current CUDA device, got {pages.device}")
    if pages.dim() != 3 or not pages.is_contiguous() or (pages.dtype != _BF16 and pages.dtype != _F32):
        _unfit(name, "pages", pages, "a contiguous bf16 or fp32 tensor [n_pages, page_size, d]")
    if block_table.dim() != 2 or block_table.dtype != _I32 or block_table.get_device() != di or not block_table.is_contiguous():
        _unfit(name, "block_table", block_table, "a contiguous int32 tensor [B, table_width]")
    return di


def latent_append_paged(rows, entry, pages, block_table, seq=None, pos=None, inv_freq=None, interleaved=True, q_pe=None,
                        q=None, stream=None):
    """Append rows [T, d] to the paged cache, row t at entry entry[t] of sequence seq[t] (seq None:
    sequence t), the last 2 * len(inv_freq) values rotated by pos[t] (None: entry[t]) * inv_freq; the
    rotary parts q_pe [T, H, d_r] rotated into the last d_r values of q [T, H, d_q].  rows and q_pe may
    be strided in all but their last dimension.  See csa.h."""
    name = "latent_append_paged"
    if rows is None or entry is None or pages is None or block_table is None:
        raise CsaError(f"{name}: rows, entry, pages and block_table are needed")
    di = _paged(name, pages, block_table)
    n_pages, page, d = pages.shape
    B, width = block_table.shape
    dt = pages.dtype
    if entry.dim() != 1 or entry.dtype != _I32 or entry.get_device() != di or not entry.is_contiguous():
        _unfit(name, "entry", entry, "a contiguous int32 tensor [T]")
    of_T = entry.shape
    T = of_T[0]
    if rows.shape != (T, d) or rows.dtype != dt or rows.get_device() != di or (d > 1 and rows.stride(1) != 1):
        _unfit(name, "rows", rows, f"[{T}, {d}] {dt} with a dense last dimension")
    sp = pp = fp = qp = qo = d_r = H = d_q = ld_t = ld_h = 0
    if seq is not None:
        if seq.dtype != _I32 or seq.shape != of_T or seq.get_device() != di or not seq.is_contiguous():
            _unfit(name, "seq", seq, f"a contiguous int32 tensor [{T}]")
        sp = seq.data_ptr()
    if pos is not None:
        if pos.dtype != _I32 or pos.shape != of_T or pos.get_device() != di or not pos.is_contiguous():
            _unfit(name, "pos", pos, f"a contiguous int32 tensor [{T}]")
        pp = pos.data_ptr()
    if inv_freq is not None:
        if inv_freq.dim() != 1 or inv_freq.dtype != _F32 or inv_freq.get_device() != di or not inv_freq.is_contiguous():
            _unfit(name, "inv_freq", inv_freq, "a contiguous fp32 tensor [d_r / 2]")
        d_r = 2 * inv_freq.shape[0]
        fp = inv_freq.data_ptr()
    if q is not None and q_pe is not None:
        if q.dim() != 3 or q.dtype != dt or q.shape[0] != T or q.get_device() != di or not q.is_contiguous():
            _unfit(name, "q", q, f"a contiguous {dt} tensor [{T}, H, d_q]")
        _, H, d_q = q.shape
        if q_pe.shape != (T, H, d_r) or q_pe.dtype != dt or q_pe.get_device() != di or q_pe.stride(2) != 1:
            _unfit(name, "q_pe", q_pe, f"[{T}, {H}, {d_r}] {dt} with a dense last dimension")
        ld_t, ld_h, _ = q_pe.stride()
        if T == 1:
            ld_t = 0                       # the stride of a single row or head means nothing
        if H == 1:
            ld_h = 0
        qp, qo = q_pe.data_ptr(), q.data_ptr()
    elif q is not None or q_pe is not None:
        raise CsaError(f"{name}: q and q_pe come together")
    st = lib.latent_append_paged(rows.data_ptr(), rows.stride(0) if T > 1 else d, sp, entry.data_ptr(), pp, fp, d_r,
                                 1 if interleaved else 0, pages.data_ptr(), n_pages, page, block_table.data_ptr(), width, B,
                                 T, d, qp, ld_t, ld_h, qo, H, d_q, CSA_BF16 if dt == _BF16 else CSA_F32,
                                 _stream_now(di) if stream is None else _stream(stream))
    if st:
        _check(st, name)


def attn_decode_paged_workspace_size(B, H, d_v, rows_max):
    return int(lib.attn_decode_paged_workspace_size(B, H, d_v, rows_max))


def _paged_attn(name, call, q, pages, block_table, sel, sparse, win, win_len, sink, sm_scale, d_v, out, lse, workspace, stream):
    if q is None or pages is None or block_table is None or sel is None or sink is None or out is None:
        raise CsaError(f"{name}: q, pages, block_table, {'idx' if sparse else 'n_entries'}, sink and out are needed")
    di = _paged(name, pages, block_table)
    n_pages, page, d_k = pages.shape
    B, width = block_table.shape
    dt = pages.dtype
    if q.dim() != 3 or q.dtype != dt or q.shape[0] != B or q.shape[2] != d_k or q.get_device() != di or not q.is_contiguous():
        _unfit(name, "q", q, f"a contiguous {dt} tensor [{B}, H, {d_k}]")
    H = q.shape[1]
    if out.dtype != dt or out.shape != (B, H, d_v) or out.get_device() != di or not out.is_contiguous():
        _unfit(name, "out", out, f"a contiguous {dt} tensor [{B}, {H}, {d_v}]")
    if sink.dtype != _F32 or sink.shape != (H,) or sink.get_device() != di or not sink.is_contiguous():
        _unfit(name, "sink", sink, f"a contiguous fp32 tensor [{H}]")
    if sparse:
        if sel.dim() != 2 or sel.dtype != _I32 or sel.shape[0] != B or sel.get_device() != di or not sel.is_contiguous():
            _unfit(name, "idx", sel, f"a contiguous int32 tensor [{B}, k]")
        picked = (sel.data_ptr(), sel.shape[1])
    else:
        if sel.dtype != _I32 or sel.shape != (B,) or sel.get_device() != di or not sel.is_contiguous():
            _unfit(name, "n_entries", sel, f"a contiguous int32 tensor [{B}]")
        picked = (sel.data_ptr(),)
    W = wp = lp = ep = 0
    if win is not None:
        if win.dim() != 3 or win.dtype != dt or win.shape[0] != B or win.shape[2] != d_k or win.get_device() != di or not win.is_contiguous():
            _unfit(name, "win", win, f"a contiguous {dt} tensor [{B}, W, {d_k}]")
        if win_len is None or win_len.dtype != _I32 or win_len.shape != (B,) or win_len.get_device() != di or not win_len.is_contiguous():
            _unfit(name, "win_len", win_len, f"a contiguous int32 tensor [{B}]")
        W, wp, lp = win.shape[1], win.data_ptr(), win_len.data_ptr()
    if lse is not None:
        if lse.dtype != _F32 or lse.shape != (B, H) or lse.get_device() != di or not lse.is_contiguous():
            _unfit(name, "lse", lse, f"a contiguous fp32 tensor [{B}, {H}]")
        ep = lse.data_ptr()
    if workspace is None or workspace.get_device() != di or not workspace.is_contiguous():
        _unfit(name, "workspace", workspace, "a contiguous tensor")
    st = call(q.data_ptr(), pages.data_ptr(), n_pages, page, block_table.data_ptr(), width, *picked, wp, lp,
              sink.data_ptr(), B, H, d_k, d_v, W, sm_scale, CSA_BF16 if dt == _BF16 else CSA_F32, out.data_ptr(), ep,
              workspace.data_ptr(), workspace.nbytes, _stream_now(di) if stream is None else _stream(stream))
    if st:
        _check(st, name)


def hca_attn_decode_paged(q, pages, block_table, n_entries, win, win_len, sink, sm_scale, d_v, out, lse=None,
                          workspace=None, stream=None):
    """hca_attn_decode over a paged cache: pages [n_pages, page_size, d_k], block_table [B, table_width]."""
    _paged_attn("hca_attn_decode_paged", lib.hca_attn_decode_paged, q, pages, block_table, n_entries, False, win, win_len,
                sink, sm_scale, d_v, out, lse, workspace, stream)


def sparse_attn_decode_paged(q, pages, block_table, idx, win, win_len, sink, sm_scale, d_v, out, lse=None,
                             workspace=None, stream=None):
    """sparse_attn_decode over a paged cache: idx [B, k] entry ids (-1 = unused slot)."""
    _paged_attn("sparse_attn_decode_paged", lib.sparse_attn_decode_paged, q, pages, block_table, idx, True, win, win_len,
                sink, sm_scale, d_v, out, lse, workspace, stream)
