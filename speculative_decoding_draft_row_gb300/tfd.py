"""Thin ctypes binding of libtfd.so: one function per C entry point, same names.

Arguments are torch tensors on the current CUDA device (or None for nullable pointers); the binding
only checks dtypes/devices, passes ``data_ptr()`` and sizes, and raises ``TfdError`` on a non-zero
status. Every step of the computation runs in the library's kernels; there is no fallback: if the
library cannot be loaded the import of a function fails with an error.
"""
import ctypes
import os

import torch

from . import build as _build

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_DATA, ERR_TIMEOUT = range(7)
W_BF16, W_FP8_ROW, W_FP8_BLOCK32, W_FP8_BLOCK32_IL = 0, 1, 2, 3
X_BF16, X_F32, X_BF16_E4M3 = 0, 1, 2
OUT_NONE, OUT_F32, OUT_BF16, OUT_ADD_BF16 = 0, 1, 2, 3
MAX_ROWS, MAX_TOPK, MAX_WINDOW = 32, 512, 511

_c = ctypes
_vp, _i64, _i32, _sz, _f32 = _c.c_void_p, _c.c_int64, _c.c_int, _c.c_size_t, _c.c_float

SIGNATURES = {
    "tfd_status_string": (_c.c_char_p, [_i32]),
    "tfd_version": (_i32, []),
    "tfd_quant_fp8": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "tfd_head_gemv_workspace": (_sz, [_i32, _i64, _i32, _i32]),
    "tfd_head_gemv_max_k": (_i64, [_i32, _i32]),
    "tfd_head_gemv": (_i32, [_vp, _i32, _vp, _i64, _i64, _vp, _i32, _i32, _i64, _i32, _vp, _i64,
                             _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp, _vp]),
    "tfd_head_gemv_noalloc": (_i32, [_vp, _i32, _vp, _i64, _i64, _vp, _i32, _i32, _i64, _i32,
                                     _vp, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp]),
    "tfd_topk_workspace": (_sz, [_i32, _i64, _i32]),
    "tfd_topk": (_i32, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "tfd_rescore_workspace": (_sz, [_i32, _i32]),
    "tfd_rescore": (_i32, [_vp, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp,
                           _vp]),
    "tfd_window_attn": (_i32, [_vp, _vp, _vp, _vp, _vp, _f32, _f32, _vp, _vp, _vp, _i32, _i32,
                               _i32, _i32, _i32, _vp, _vp, _vp]),
    "tfd_accept": (_i32, [_vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "tfd_fp8_block32_relayout": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp]),
    "tfd_rmsnorm": (_i32, [_vp, _i64, _vp, _f32, _i32, _i64, _vp, _i64, _vp]),
    "tfd_swiglu": (_i32, [_vp, _vp, _i64, _i32, _i64, _vp, _i64, _vp]),
    "tfd_sample": (_i32, [_vp, _i32, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                          _i64, _vp, _i64, _vp, _vp]),
    "tfd_accept_sampled": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i32,
                                  _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "tfd_lora": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _i32, _i32, _i64, _vp, _vp, _i32, _vp, _i64,
                        _vp, _i64, _vp, _vp]),
    "tfd_absorb": (_i32, [_vp, _vp, _vp, _f32, _f32, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32,
                          _vp, _vp]),
}

_lib = None


class TfdError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: status {status} ({status_string(status)})")


def library(build=True):
    """The loaded libtfd.so (built first when missing or stale). The environment variable
    TFD_LIBRARY names another build of the library to load instead (it must exist)."""
    global _lib
    if _lib is None:
        path = os.environ.get("TFD_LIBRARY")
        if not path:
            path = _build.build_library() if build else _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"libtfd.so not found at {path}")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def status_string(status):
    return library().tfd_status_string(int(status)).decode()


def _p(t):
    return None if t is None else t.data_ptr()


# The raw handle of the current stream; building a Stream object costs microseconds a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, dev=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device() if dev is None else dev)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, st):
    if st != OK:
        raise TfdError(fn, st)


def _dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tfd tensors must be CUDA tensors")


def zeroed_workspace(nbytes, device=None):
    """A zero-filled device workspace (the calls leave it zeroed again)."""
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device or "cuda")


# ---- entry points ---------------------------------------------------------------------------

def tfd_quant_fp8(w, mode, codes=None, scales=None, stream=None):
    """FP8 codes of a bf16 weight [n][k]: mode W_FP8_ROW (float scales [n]), W_FP8_BLOCK32 or
    W_FP8_BLOCK32_IL (uint8 scales [n/32][k/32]; IL writes the interleaved code layout).
    Returns (codes, scales)."""
    _dev(w)
    n, k = w.shape
    if codes is None:
        codes = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = (torch.empty(n, dtype=torch.float32, device=w.device) if mode == W_FP8_ROW else
                  torch.empty((max(n // 32, 1), max(k // 32, 1)), dtype=torch.uint8,
                              device=w.device))
    st = library().tfd_quant_fp8(_p(w), n, k, mode, _p(codes), _p(scales), _stream(stream))
    _check("tfd_quant_fp8", st)
    return codes, scales


def tfd_head_gemv_workspace(rows, n, topk, parts=0):
    return library().tfd_head_gemv_workspace(rows, n, topk, parts)


def tfd_head_gemv_max_k(rows, xfmt=X_BF16):
    return library().tfd_head_gemv_max_k(rows, xfmt)


def tfd_head_gemv(w, wfmt, w_scales, x, out_mode=OUT_F32, y=None, topk=0, parts=0, id_map=None,
                  top_vals=None, top_ids=None, ws=None, dev_status=None, n=None, top1_conf=None,
                  stream=None, act_e4m3=False):
    """Few-row head GEMV with optional output and fused top-k (top-1 optionally with its softmax
    probability in ``top1_conf`` [rows]). ``act_e4m3`` (FP8 weights, bf16 x): quantise the
    activation rows to E4M3 in the call (W8A8). Returns (y, top_vals, top_ids)."""
    _dev(w, x, y, id_map, ws)
    n = w.shape[0] if n is None else n
    k = w.shape[1]
    rows = x.shape[0]
    xfmt = X_F32 if x.dtype == torch.float32 else (X_BF16_E4M3 if act_e4m3 else X_BF16)
    if y is None and out_mode != OUT_NONE:
        dt = torch.float32 if out_mode == OUT_F32 else torch.bfloat16
        y = torch.empty((rows, n), dtype=dt, device=x.device)
    ldy = y.stride(0) if y is not None else 0
    if topk > 0 and top_vals is None:
        top_vals = torch.empty((rows, topk), dtype=torch.float32, device=x.device)
        top_ids = torch.empty((rows, topk), dtype=torch.int32, device=x.device)
    if ws is None and topk > 0:
        ws = zeroed_workspace(tfd_head_gemv_workspace(rows, n, topk, parts), x.device)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    ldt = top_ids.stride(0) if (topk > 0 and top_ids.dim() == 2) else topk
    if topk > 0 and top_vals.stride(0) != ldt:
        raise ValueError("top_vals and top_ids must share their row stride")
    st = library().tfd_head_gemv(_p(w), wfmt, _p(w_scales), n, k, _p(x), xfmt, rows, x.stride(0),
                                 out_mode, _p(y), ldy, topk, parts, _p(id_map), _p(top_vals),
                                 _p(top_ids), ldt, _p(top1_conf), _p(ws), ws_bytes,
                                 _p(dev_status), _stream(stream))
    _check("tfd_head_gemv", st)
    return y, top_vals, top_ids


NOALLOC_SCRATCH_BYTES = 1048576


def tfd_head_gemv_noalloc(w, wfmt, w_scales, x, out_mode=OUT_F32, y=None, topk=0, parts=0,
                          id_map=None, top_vals=None, top_ids=None, dev_status=None,
                          top1_conf=None, stream=None):
    """tfd_head_gemv on the library's fixed scratch (no workspace argument): for callers that
    cannot allocate device memory. Outputs must be passed in by such callers; the defaults here
    allocate them only for convenience. Returns (y, top_vals, top_ids)."""
    _dev(w, x, y, id_map)
    n, k = w.shape[0], w.shape[1]
    rows = x.shape[0]
    xfmt = X_F32 if x.dtype == torch.float32 else X_BF16
    if y is None and out_mode != OUT_NONE:
        dt = torch.float32 if out_mode == OUT_F32 else torch.bfloat16
        y = torch.empty((rows, n), dtype=dt, device=x.device)
    if topk > 0 and top_vals is None:
        top_vals = torch.empty((rows, topk), dtype=torch.float32, device=x.device)
        top_ids = torch.empty((rows, topk), dtype=torch.int32, device=x.device)
    ldt = top_ids.stride(0) if topk > 0 else 0
    st = library().tfd_head_gemv_noalloc(_p(w), wfmt, _p(w_scales), n, k, _p(x), xfmt, rows,
                                         x.stride(0), out_mode, _p(y),
                                         y.stride(0) if y is not None else 0, topk, parts,
                                         _p(id_map), _p(top_vals), _p(top_ids), ldt,
                                         _p(top1_conf), _p(dev_status), _stream(stream))
    _check("tfd_head_gemv_noalloc", st)
    return y, top_vals, top_ids


def tfd_topk_workspace(rows, n, k):
    return library().tfd_topk_workspace(rows, n, k)


def tfd_topk(logits, k, id_map=None, vals=None, ids=None, ws=None, n=None, stream=None):
    """Top-k of fp32 logits [rows][>= n]. Returns (vals, ids)."""
    _dev(logits, id_map, ws)
    rows = logits.shape[0]
    n = logits.shape[1] if n is None else n
    if vals is None:
        vals = torch.empty((rows, k), dtype=torch.float32, device=logits.device)
        ids = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    if ws is None:
        ws = zeroed_workspace(tfd_topk_workspace(rows, n, k), logits.device)
    st = library().tfd_topk(_p(logits), rows, n, logits.stride(0), k, _p(id_map), _p(vals),
                            _p(ids), _p(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check("tfd_topk", st)
    return vals, ids


def tfd_rescore_workspace(rows, cand_k):
    return library().tfd_rescore_workspace(rows, cand_k)


def tfd_rescore(w_exact, x, cand, cand_logits=None, out_ids=None, out_vals=None, ws=None,
                dev_status=None, want_logits=True, stream=None):
    """Exact logits of the candidates [rows][cand_k] and their argmax. Returns
    (cand_logits, out_ids, out_vals)."""
    _dev(w_exact, x, cand, ws)
    vocab, k = w_exact.shape
    rows, cand_k = cand.shape
    dev = x.device
    if cand_logits is None and want_logits:
        cand_logits = torch.empty((rows, cand_k), dtype=torch.float32, device=dev)
    if out_ids is None:
        out_ids = torch.empty(rows, dtype=torch.int32, device=dev)
        out_vals = torch.empty(rows, dtype=torch.float32, device=dev)
    if ws is None:
        ws = zeroed_workspace(tfd_rescore_workspace(rows, cand_k), dev)
    st = library().tfd_rescore(_p(w_exact), vocab, k, _p(x), rows, _p(cand), cand_k,
                               _p(cand_logits), _p(out_ids), _p(out_vals), _p(ws),
                               ws.numel() * ws.element_size(), _p(dev_status), _stream(stream))
    _check("tfd_rescore", st)
    return cand_logits, out_ids, out_vals


def tfd_window_attn(q, k_new, v_new, pos, k_ring, v_ring, window, q_gamma=None, k_gamma=None,
                    eps=1e-6, rope_base=10000.0, out=None, dev_status=None, stream=None):
    """qk_norm + RoPE + ring write + window attention. Returns out [streams][heads*dim]."""
    _dev(q, k_new, v_new, pos, k_ring, v_ring)
    streams, heads, dim = q.shape
    ring = k_ring.shape[1]
    if out is None:
        out = torch.empty((streams, heads * dim), dtype=torch.bfloat16, device=q.device)
    st = library().tfd_window_attn(_p(q), _p(k_new), _p(v_new), _p(q_gamma), _p(k_gamma),
                                   float(eps), float(rope_base), _p(pos), _p(k_ring), _p(v_ring),
                                   ring, window, streams, heads, dim, _p(out), _p(dev_status),
                                   _stream(stream))
    _check("tfd_window_attn", st)
    return out


def tfd_accept(drafts, n_asked, draws, n_kept=None, asked_hist=None, kept_hist=None,
               dev_status=None, stream=None):
    """Accept-prefix count. Returns n_kept [streams]."""
    _dev(drafts, n_asked, draws)
    streams, win = drafts.shape
    if n_kept is None:
        n_kept = torch.empty(streams, dtype=torch.int32, device=drafts.device)
    st = library().tfd_accept(_p(drafts), _p(n_asked), _p(draws), streams, win, _p(n_kept),
                              _p(asked_hist), _p(kept_hist), _p(dev_status), _stream(stream))
    _check("tfd_accept", st)
    return n_kept


def tfd_rmsnorm(x, gamma=None, eps=1e-6, out=None, stream=None):
    """RMSNorm of the rows of x [rows][hidden] (bf16). out may be x (in place). Returns out."""
    _dev(x, gamma, out)
    rows, hidden = x.shape
    if out is None:
        out = torch.empty_like(x)
    st = library().tfd_rmsnorm(_p(x), x.stride(0), _p(gamma), float(eps), rows, hidden, _p(out),
                               out.stride(0), _stream(stream))
    _check("tfd_rmsnorm", st)
    return out


def tfd_swiglu(g, u, out=None, stream=None):
    """bf16(bf16(SiLU(g)) * u) of two [rows][cols] bf16 tensors with the same row stride."""
    _dev(g, u, out)
    rows, cols = g.shape
    if u.shape != g.shape or u.stride(0) != g.stride(0):
        raise ValueError("g and u must have the same shape and row stride")
    if out is None:
        out = torch.empty_like(g)
    st = library().tfd_swiglu(_p(g), _p(u), g.stride(0), rows, cols, _p(out), out.stride(0),
                              _stream(stream))
    _check("tfd_swiglu", st)
    return out


def tfd_absorb(k_rows, v_rows, p0, k_ring, v_ring, k_gamma=None, eps=1e-6, rope_base=10000.0,
               dev_status=None, stream=None):
    """Write n rows per stream (k_rows, v_rows [streams][n][heads][dim]) into the rings at positions
    p0[s] .. p0[s] + n - 1. Refuses n > ring."""
    _dev(k_rows, v_rows, p0, k_ring, v_ring, k_gamma)
    streams, n, heads, dim = k_rows.shape
    ring = k_ring.shape[1]
    st = library().tfd_absorb(_p(k_rows), _p(v_rows), _p(k_gamma), float(eps), float(rope_base),
                              _p(p0), n, _p(k_ring), _p(v_ring), ring, streams, heads, dim,
                              _p(dev_status), _stream(stream))
    _check("tfd_absorb", st)


def tfd_fp8_block32_relayout(codes, to_interleaved=True, out=None, stream=None):
    """Block-32 FP8 codes [n][k] between the plain and the interleaved layout. Returns out."""
    _dev(codes, out)
    n, k = codes.shape
    if out is None:
        out = torch.empty_like(codes)
    st = library().tfd_fp8_block32_relayout(_p(codes), n, k, 1 if to_interleaved else 0, _p(out),
                                            _stream(stream))
    _check("tfd_fp8_block32_relayout", st)
    return out


def _vec(t, dtype, count, dev, name):
    """A contiguous vector (or matrix) of ``count`` elements of one type on the device: its address
    (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != count or t.get_device() != dev or \
            not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor of {count} {dtype} on the current CUDA "
                         "device is wanted")
    return t.data_ptr()


def _rows_of(t, rows, cols, dtype, dev, name):
    """Row stride of a matrix [rows][cols] with contiguous columns on the device."""
    stride, step = t.stride()
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, cols) or \
            (step != 1 and cols > 1):
        raise ValueError(f"{name}: {dtype} [{rows}][{cols}] with contiguous columns on the current "
                         "CUDA device is wanted")
    return stride if rows > 1 else max(cols, stride)


def tfd_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, id_map=None,
               ids=None, prob=None, probs=None, want_probs=False, dev_status=None, n=None,
               stream=None):
    """One token a row of logits [rows][>= n] (bf16 or float32), drawn with the random numbers
    u [rows] after temperature, top_k, top_p and min_p (each [rows] or None). ``ids`` [rows] may be
    a column of a larger array (``prob`` then with the same stride); ``probs`` [rows][n] (or
    want_probs) receives the filtered distribution. Returns (ids, prob, probs)."""
    f32, i32, dev, vec = torch.float32, torch.int32, _current_device(), _vec
    rows, cols = logits.shape
    kind = logits.dtype
    if kind is not f32 and kind is not torch.bfloat16:
        raise ValueError("logits: float32 or bfloat16 is wanted")
    ld = _rows_of(logits, rows, cols, kind, dev, "logits")
    if n is None:
        n = cols
    elif n > cols:
        raise ValueError("logits have fewer than n columns")
    if ids is None:
        ids = torch.empty(rows, dtype=i32, device=logits.device)
        if prob is None:
            prob = torch.empty(rows, dtype=f32, device=logits.device)
    ldt, = ids.stride() if ids.dim() == 1 else (0,)
    if ids.dtype is not i32 or ids.shape != (rows,) or ids.get_device() != dev or \
            (ldt < 1 and rows > 1):
        raise ValueError("ids: an int32 vector of one id a row is wanted")
    if prob is not None and (prob.dtype is not f32 or prob.shape != (rows,) or
                             prob.get_device() != dev or (rows > 1 and prob.stride(0) != ldt)):
        raise ValueError("prob: a float32 vector with the stride of ids is wanted")
    if probs is None and want_probs:
        probs = torch.empty((rows, n), dtype=f32, device=logits.device)
    ldp = 0 if probs is None else _rows_of(probs, rows, n, f32, dev, "probs")
    st = (_lib or library()).tfd_sample(
        logits.data_ptr(), X_F32 if kind is f32 else X_BF16, rows, n, ld,
        vec(temperature, f32, rows, dev, "temperature"), vec(top_k, i32, rows, dev, "top_k"),
        vec(top_p, f32, rows, dev, "top_p"), vec(min_p, f32, rows, dev, "min_p"),
        vec(u, f32, rows, dev, "u"), vec(id_map, i32, n, dev, "id_map"), ids.data_ptr(),
        None if prob is None else prob.data_ptr(), ldt if rows > 1 else 1,
        None if probs is None else probs.data_ptr(), ldp,
        vec(dev_status, i32, 1, dev, "dev_status"), _stream(stream, dev))
    if st:
        _check("tfd_sample", st)
    return ids, prob, probs


def tfd_accept_sampled(p, q, drafts, n_asked, u, u_next, q_map=None, n_kept=None, next_ids=None,
                       next_prob=None, asked_hist=None, kept_hist=None, dev_status=None,
                       stream=None):
    """The rejection accept of drafts [streams][win] drawn from q [streams][win][nq] against the
    target's p [streams][win + 1][n], with the random numbers u [streams][win], and the next token
    drawn with u_next [streams]. q_map [n] gives a token's column in q (-1: none). The streams and
    steps of p and q are contiguous but for the row stride. Returns (n_kept, next_ids, next_prob)."""
    f32, i32, dev, vec = torch.float32, torch.int32, _current_device(), _vec
    streams, win = drafts.shape
    ps, pw, n = p.shape
    qs, qw, nq = q.shape
    p0, ldp, p2 = p.stride()
    q0, ldq, q2 = q.stride()
    if win == 1 and streams > 1:                         # one row a stream: theirs is the row stride
        ldq = q0
    if p.dtype is not f32 or p.get_device() != dev or ps != streams or pw != win + 1 or \
            (p2 != 1 and n > 1) or (p0 != pw * ldp and streams > 1):
        raise ValueError(f"p: float32 [{streams}][{win + 1}][columns] with evenly spaced rows on the "
                         "current CUDA device is wanted")
    if q.dtype is not f32 or q.get_device() != dev or qs != streams or qw != win or \
            (q2 != 1 and nq > 1) or (q0 != qw * ldq and streams > 1):
        raise ValueError(f"q: float32 [{streams}][{win}][columns] with evenly spaced rows on the "
                         "current CUDA device is wanted")
    if streams * win == 1:                               # a stride of one row says nothing
        ldq = max(ldq, nq)
    if n_kept is None:
        n_kept = torch.empty(streams, dtype=i32, device=p.device)
    if next_ids is None:
        next_ids = torch.empty(streams, dtype=i32, device=p.device)
        if next_prob is None:
            next_prob = torch.empty(streams, dtype=f32, device=p.device)
    st = (_lib or library()).tfd_accept_sampled(
        p.data_ptr(), ldp, q.data_ptr(), ldq, n, nq, vec(q_map, i32, n, dev, "q_map"),
        vec(drafts, i32, streams * win, dev, "drafts"), vec(n_asked, i32, streams, dev, "n_asked"),
        vec(u, f32, streams * win, dev, "u"), vec(u_next, f32, streams, dev, "u_next"), streams, win,
        vec(n_kept, i32, streams, dev, "n_kept"), vec(next_ids, i32, streams, dev, "next_ids"),
        vec(next_prob, f32, streams, dev, "next_prob"),
        vec(asked_hist, torch.int64, win, dev, "asked_hist"),
        vec(kept_hist, torch.int64, win, dev, "kept_hist"),
        vec(dev_status, i32, 1, dev, "dev_status"), _stream(stream, dev))
    if st:
        _check("tfd_accept_sampled", st)
    return n_kept, next_ids, next_prob


def tfd_lora(x, a, b, adapter_ids, base=None, y=None, scales=None, out_mode=OUT_BF16,
             dev_status=None, stream=None):
    """y[r] = base[r] + scales[i] * b[i] (a[i] x[r]), i = adapter_ids[r] (-1: none), for bf16 x
    [rows][k], a [adapters][rank][k], b [adapters][n][rank]. base (or None for zeros) and y have one
    type, float32 or bfloat16 (base's or y's, else out_mode); y may be base. Returns y."""
    f32, bf, dev, vec = torch.float32, torch.bfloat16, _current_device(), _vec
    rows, k = x.shape
    na, rank, ka = a.shape
    nb, n, rb = b.shape
    if ka != k or nb != na or rb != rank:
        raise ValueError("a [adapters][rank][k] and b [adapters][n][rank] do not fit x")
    like = y if y is not None else base
    if like is not None:
        out_mode = OUT_F32 if like.dtype is f32 else OUT_BF16
    dt = f32 if out_mode == OUT_F32 else bf
    ldx = _rows_of(x, rows, k, bf, dev, "x")
    if y is None:
        y = torch.empty((rows, n), dtype=dt, device=x.device)
    ldy = _rows_of(y, rows, n, dt, dev, "y")
    ldb = 0 if base is None else ldy if base is y else _rows_of(base, rows, n, dt, dev, "base")
    st = (_lib or library()).tfd_lora(
        x.data_ptr(), rows, k, ldx, vec(a, bf, na * rank * k, dev, "a"),
        vec(b, bf, na * n * rank, dev, "b"), na, rank, n,
        vec(adapter_ids, torch.int32, rows, dev, "adapter_ids"), vec(scales, f32, na, dev, "scales"),
        out_mode, None if base is None else base.data_ptr(), ldb, y.data_ptr(), ldy,
        vec(dev_status, torch.int32, 1, dev, "dev_status"), _stream(stream, dev))
    if st:
        _check("tfd_lora", st)
    return y
