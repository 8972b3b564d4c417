"""ctypes binding of libcsa_b200.so (declared in include/csa.h).

Argument marshalling only: every function takes torch tensors that already live
on the GPU, passes their data pointers and the current CUDA stream, and raises
``CsaError`` on a non-zero status.  There is no CPU fallback: if the library
is missing the import of this module fails.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa_b200.so")

CSA_F32, CSA_BF16 = 0, 1
STATUS = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_ALIGNMENT",
          4: "CSA_ERR_CUDA", 5: "CSA_ERR_TIMEOUT", 6: "CSA_ERR_NO_SPACE"}
NORM, ROPE_INVERSE, ROPE_HALF = 1, 2, 4


class CsaError(RuntimeError):
    def __init__(self, fn, status, cuda_err=0):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}"
                         + (f" (cudaError {cuda_err})" if status == 4 else ""))
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run long_context_compressed_compress_b200.build")
lib = ctypes.CDLL(LIB_PATH)

P = ctypes.c_void_p
I = ctypes.c_int
F = ctypes.c_float
I64 = ctypes.c_int64
SZ = ctypes.c_size_t

_SIGS = {
    "csa_status_string": ([I], ctypes.c_char_p),
    "csa_last_cuda_error": ([], I),
    "csa_version": ([], I),
    "csa_device_status": ([ctypes.POINTER(I)], I),
    "csa_set_wait_timeout_ns": ([ctypes.c_uint64], I),
    "csa_compress": ([P, P, P, I, I, I, I, I, I, P, I, P, I, P, P, F, P], I),
    "hca_compress": ([P, P, I, I, I, I, I, P, I, P], I),
    "nvfp4_quantize": ([P, I, I64, I, F, P, P, P], I),
    "indexer_score": ([P, P, F, P, P, F, P, I, I, I, I, I, I, I, I, I, P, P, I, I, P, P], I),
    "topk_select": ([P, I, I, I, I, I, I, I, I, P, P, P, SZ, P], I),
    "indexer_topk": ([P, P, F, P, P, F, P, I, I, I, I, I, I, I, I, I, P, P, I, P, P], I),
    "indexer_topk_max_entries": ([I, I], I),
    "csa_validate_indices": ([P, I, I, I, I, I, I, P, P, P], I),
    "topk_workspace_size": ([I, I, I, I], SZ),
    "topk_select_noalloc": ([P, I, I, I, I, I, I, I, I, P, P, P], I),
    "sparse_attn_fwd": ([P, P, P, P, P, F, I, I, I, I, I, I, I, I, I, I, P, P, P, I, P, P], I),
    "hca_dense_attn_fwd": ([P, P, P, P, F, I, I, I, I, I, I, I, I, I, I, I, P, P, P, I, P, P], I),
    "swa_sink_merge": ([P, P, P, P, P, F, I, I, I, I, I, I, I, I, P, P, I, P], I),
    "csa_ring_append": ([P, I, I, I, P, I, P, P], I),
    "csa_pos_advance": ([P, I, I, P], I),
    "csa_pos_advance_rows": ([P, I, P, P], I),
    "csa_decode_update": ([P] * 8 + [I] * 8 + [P] * 12 + [F, P, P], I),
    "csa_state_gather": ([P, I, I, I, I, P, I, I, I, P, I, P], I),
    "qk_norm_rope": ([P, I64, I64, P, I64, I64, I, I, I, I, I, P, P, I, P, I, P, P, F, I, P, P, I, P], I),
    "hca_paged_append": ([P, P, I, I, I, I, I, P, P, P, P, P, I, I, P, P, I, P, F, P, I, I, P, P], I),
    "hca_prefix_attn_fwd": ([P, P, I, I, P, P, I, P, P, P, I, I, P, P, F, I, I, I, I, I, I, I, P, P, P, I, P, P], I),
    "kv_pages_workspace_size": ([I, I], SZ),
    "kv_pages_reserve": ([P, P, I, I, P, P, I, I, P, I, P, SZ, P, P], I),
    "kv_pages_fork": ([P, P, P, I, I, P, P, I, I, P, I, P, I, I64, P, SZ, P, P], I),
    "kv_pages_free": ([P, I, P, P, I, I, P, I, P, P], I),
    "kv_pages_compact": ([P, P, I, I, P, I, P, I, I64, P, P, P, P, SZ, P], I),
    "grouped_out_proj": ([P, I, I, I, I, I, P, P, I, P, P, P, P], I),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTS = tuple(_SIGS)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _dt(t_or_dtype):
    d = t_or_dtype.dtype if isinstance(t_or_dtype, torch.Tensor) else t_or_dtype
    if d == torch.float32:
        return CSA_F32
    if d == torch.bfloat16:
        return CSA_BF16
    raise ValueError(f"unsupported dtype {d}")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(fn, st):
    if st != 0:
        raise CsaError(fn, st, lib.csa_last_cuda_error())


def device_status():
    """Read and clear the library's per-device status word (calls given no
    status word of their own report a timed-out wait there)."""
    v = I(0)
    _check("csa_device_status", lib.csa_device_status(ctypes.byref(v)))
    return v.value


def set_wait_timeout_ns(ns):
    """Wall-time limit of the kernels' bounded waits (0 = the default 2 s)."""
    _check("csa_set_wait_timeout_ns", lib.csa_set_wait_timeout_ns(int(ns)))


def csa_compress(a, b, z, m, out=None, out_fp4=None, out_sf=None, gscale=1.0, first_has_pred=0,
                 ring_pos=None, out_bstride=0, out_dtype=None, stream=None):
    B, T, D = a.shape[-3], a.shape[-2], a.shape[-1]
    od = _dt(out) if out is not None else _dt(out_dtype if out_dtype is not None else a.dtype)
    _check("csa_compress", lib.csa_compress(
        _ptr(a), _ptr(b), _ptr(z), _dt(a), B, T, D, m, first_has_pred, _ptr(ring_pos), out_bstride,
        _ptr(out), od, _ptr(out_fp4), _ptr(out_sf), gscale, _stream(stream)))


def hca_compress(a, z, m, out, stream=None):
    B, T, D = a.shape
    _check("hca_compress", lib.hca_compress(_ptr(a), _ptr(z), _dt(a), B, T, D, m, _ptr(out), _dt(out),
                                            _stream(stream)))


def nvfp4_quantize(x, packed, sf, gscale=1.0, stream=None):
    D = x.shape[-1]
    rows = x.numel() // D
    _check("nvfp4_quantize", lib.nvfp4_quantize(_ptr(x), _dt(x), rows, D, gscale, _ptr(packed), _ptr(sf),
                                                _stream(stream)))


def indexer_score(q_fp4, q_sf, k_fp4, k_sf, w, q_pos0, score, S, m, row0=0, T_chunk=None, q_gscale=1.0,
                  k_gscale=1.0, status=None, stream=None):
    """q_fp4 [B,T,HI,DI/2], k_fp4 [B,k_bstride,DI/2], w [B,T,HI], score [B,T_chunk,ld]."""
    B, T, HI, half = q_fp4.shape
    DI = half * 2
    T_chunk = T - row0 if T_chunk is None else T_chunk
    _check("indexer_score", lib.indexer_score(
        _ptr(q_fp4), _ptr(q_sf), q_gscale, _ptr(k_fp4), _ptr(k_sf), k_gscale, _ptr(w), B, T, row0, T_chunk,
        S, k_fp4.shape[1], HI, DI, m, _ptr(q_pos0), _ptr(score), _dt(score), score.shape[-1],
        _ptr(status), _stream(stream)))


def topk_select(score, idx, S, m, q_pos0, row0=0, workspace=None, stream=None):
    B, T_chunk, ld = score.shape
    k = idx.shape[-1]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("topk_select", lib.topk_select(_ptr(score), _dt(score), B, T_chunk, S, ld, k, m, row0,
                                          _ptr(q_pos0), _ptr(idx), _ptr(workspace), ws, _stream(stream)))


def indexer_topk(q_fp4, q_sf, k_fp4, k_sf, w, q_pos0, idx, S, m, row0=0, T_chunk=None, q_gscale=1.0,
                 k_gscale=1.0, status=None, stream=None):
    """Indexer score and top-k in one kernel: idx [B,T_chunk,k] equals
    topk_select of the BF16 scores indexer_score would write."""
    B, T, HI, half = q_fp4.shape
    DI = half * 2
    T_chunk = T - row0 if T_chunk is None else T_chunk
    _check("indexer_topk", lib.indexer_topk(
        _ptr(q_fp4), _ptr(q_sf), q_gscale, _ptr(k_fp4), _ptr(k_sf), k_gscale, _ptr(w), B, T, row0, T_chunk,
        S, k_fp4.shape[1], HI, DI, m, _ptr(q_pos0), _ptr(idx), idx.shape[-1], _ptr(status), _stream(stream)))


def indexer_topk_max_entries(HI, DI):
    return int(lib.indexer_topk_max_entries(HI, DI))


def validate_indices(idx, S, m, q_pos0, status, row0=0, stream=None):
    """Check idx [B, T_chunk, k] (entries in [0, visible), ascending, then -1);
    a violation is recorded in the device word ``status`` (int32 [1])."""
    B, T_chunk, k = idx.shape
    _check("csa_validate_indices", lib.csa_validate_indices(_ptr(idx), B, T_chunk, k, S, m, row0, _ptr(q_pos0),
                                                            _ptr(status), _stream(stream)))


def topk_select_noalloc(score, idx, S, m, q_pos0, row0=0, stream=None):
    """topk_select without a workspace: the library's fixed scratch serves the
    multi-CTA path (see the C header for its size limit and concurrency rule)."""
    B, T_chunk, ld = score.shape
    k = idx.shape[-1]
    _check("topk_select_noalloc", lib.topk_select_noalloc(_ptr(score), _dt(score), B, T_chunk, S, ld, k, m, row0,
                                                          _ptr(q_pos0), _ptr(idx), _stream(stream)))


def topk_workspace_size(B, T_chunk, S, k):
    return int(lib.topk_workspace_size(B, T_chunk, S, k))


def sparse_attn_fwd(q, kv_c, idx, kv_raw, sink, tau, W, q_pos0, out, lse=None, row0=0, T_chunk=None,
                    raw_cap=None, status=None, stream=None):
    B, T, H, D = q.shape
    T_chunk = T - row0 if T_chunk is None else T_chunk
    raw_cap = (kv_raw.shape[1] if kv_raw is not None else 1) if raw_cap is None else raw_cap
    _check("sparse_attn_fwd", lib.sparse_attn_fwd(
        _ptr(q), _ptr(kv_c), _ptr(idx), _ptr(kv_raw), _ptr(sink), tau, W, B, T, row0, T_chunk, H, D,
        kv_c.shape[1], idx.shape[-1], raw_cap, _ptr(q_pos0), _ptr(out), _ptr(lse), _dt(q), _ptr(status),
        _stream(stream)))


def hca_dense_attn_fwd(q, kv_c, kv_raw, sink, tau, W, q_pos0, out, m, S=None, lse=None, row0=0, T_chunk=None,
                       raw_cap=None, status=None, stream=None):
    B, T, H, D = q.shape
    T_chunk = T - row0 if T_chunk is None else T_chunk
    S = kv_c.shape[1] if S is None else S
    raw_cap = (kv_raw.shape[1] if kv_raw is not None else 1) if raw_cap is None else raw_cap
    _check("hca_dense_attn_fwd", lib.hca_dense_attn_fwd(
        _ptr(q), _ptr(kv_c), _ptr(kv_raw), _ptr(sink), tau, W, B, T, row0, T_chunk, H, D, kv_c.shape[1], S, m,
        raw_cap, _ptr(q_pos0), _ptr(out), _ptr(lse), _dt(q), _ptr(status), _stream(stream)))


def swa_sink_merge(o_c, lse_c, q, kv_raw, sink, tau, W, q_pos0, out, row0=0, T_chunk=None, raw_cap=None,
                   stream=None):
    B, T, H, D = q.shape
    T_chunk = T - row0 if T_chunk is None else T_chunk
    raw_cap = kv_raw.shape[1] if raw_cap is None else raw_cap
    _check("swa_sink_merge", lib.swa_sink_merge(
        _ptr(o_c), _ptr(lse_c), _ptr(q), _ptr(kv_raw), _ptr(sink), tau, W, B, T, row0, T_chunk, H, D, raw_cap,
        _ptr(q_pos0), _ptr(out), _dt(q), _stream(stream)))


def csa_ring_append(rows, ring, pos, stream=None):
    B, D = rows.shape
    _check("csa_ring_append", lib.csa_ring_append(_ptr(rows), _dt(rows), B, D, _ptr(ring), ring.shape[1],
                                                  _ptr(pos), _stream(stream)))


def csa_decode_update(x, carry, ring, kv_c, k_fp4, k_sf, q_fp4, q_sf, pos, m, gscale=1.0, stream=None):
    """One decode step's cache update in one launch (see the C header):
    ``x`` holds this step's rows a, b, z, a_I, b_I, z_I, kv_raw [B, .] and
    q_I [B, HI, DI]; ``carry`` the six 2m-slot carry rings by name."""
    B, D = x["a"].shape[0], x["a"].shape[-1]
    DI = x["a_I"].shape[-1]
    HI = x["q_I"].shape[-2]
    names = ("a", "b", "z", "a_I", "b_I", "z_I")
    _check("csa_decode_update", lib.csa_decode_update(
        *[_ptr(x[n]) for n in names], _ptr(x["kv_raw"]), _ptr(x["q_I"]), _dt(x["a"]), B, D, DI, HI, m,
        ring.shape[1], kv_c.shape[1], *[_ptr(carry[n]) for n in names], _ptr(ring), _ptr(kv_c), _ptr(k_fp4),
        _ptr(k_sf), _ptr(q_fp4), _ptr(q_sf), gscale, _ptr(pos), _stream(stream)))


def csa_pos_advance(pos, delta=1, stream=None):
    """pos [B] += delta, a number or an int32 [B] tensor."""
    if torch.is_tensor(delta):
        dev, n = _home(pos), pos.numel()
        _check("csa_pos_advance_rows", lib.csa_pos_advance_rows(
            _arg(pos, "pos", torch.int32, (n,), dev), n, _arg(delta, "delta", torch.int32, (n,), dev), _on(stream, dev)))
        return
    _check("csa_pos_advance", lib.csa_pos_advance(_ptr(pos), pos.numel(), delta, _stream(stream)))


def csa_state_gather(src, pos, dst, m=0, nrows=0, src_cap=None, stream=None):
    """Snapshot rows of a ring or a [B, T, D] stream into dst [B, npos, cap, D]
    (see include/csa.h): window mode (m = 0, the last ``nrows`` tokens up to
    pos) or carry mode (m >= 1, the last complete block and the one in
    progress).  pos: int32 [B, npos] on the device."""
    B, cap_src, D = src.shape
    npos = pos.shape[-1]
    dst_cap = dst.shape[-2]
    _check("csa_state_gather", lib.csa_state_gather(
        _ptr(src), _dt(src), B, D, cap_src if src_cap is None else src_cap, _ptr(pos), npos, m, nrows,
        _ptr(dst), dst_cap, _stream(stream)))


def grouped_out_proj(o, w1, w2, y, out, status=None, stream=None):
    """o [..., H, D] bf16 -> y [M, g*d_g], out [M, d_model] (see include/csa.h);
    w1 [g, d_g, (H/g)*D], w2 [d_model, g*d_g]."""
    H, D = o.shape[-2], o.shape[-1]
    M = o.numel() // (H * D)
    g, d_g, _ = w1.shape
    _check("grouped_out_proj", lib.grouped_out_proj(
        _ptr(o), M, H, D, g, d_g, _ptr(w1), _ptr(w2), w2.shape[0], _ptr(y), _ptr(out), _ptr(status),
        _stream(stream)))


# The serving calls below run for microseconds, so their checks take each tensor once
# and the current device and stream by their raw handles (torch's own accessors
# for these build Python objects).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _home(t):
    """The device index of a call's tensors: that of ``t``, which has to be the
    current device (the library launches there)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensor must be on the GPU")
    if dev != _raw_device():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is cuda:{_raw_device()}")
    return dev


def _arg(t, name, dtype, shape, dev):
    """The pointer of a contiguous tensor of that dtype, shape (None: any) and device;
    None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on(stream, dev):
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _code(dtype):
    if dtype is torch.bfloat16:
        return CSA_BF16
    if dtype is torch.float32:
        return CSA_F32
    raise ValueError(f"unsupported dtype {dtype}")


def _rope_args(inv_freq, norm, interleaved, inverse, dev):
    """(pointer of the frequencies, rotated dims, flags)"""
    flags = (NORM if norm else 0) | (0 if interleaved else ROPE_HALF) | (ROPE_INVERSE if inverse else 0)
    if inv_freq is None:
        return None, 0, flags
    return _arg(inv_freq, "inv_freq", torch.float64, None, dev), 2 * inv_freq.numel(), flags


def qk_norm_rope(q, kv, q_out, kv_out, q_pos0, inv_freq=None, q_weight=None, kv_weight=None, eps=1e-6, norm=True,
                 interleaved=True, inverse=False, pos_step=1, lens=None, stream=None):
    """RMS norm per head and position rotation of the queries q [B, T, H, D] and
    the shared key kv [B, T, D] in one pass (either pair may be None).  Token t
    is at j = q_pos0[b] + t and is rotated by j * pos_step * inv_freq (float64
    [R / 2]; the last R dims); its key goes to slot j % cap of kv_out [B, cap, D].
    q and kv may be views with free batch and token strides (slices of one
    projection's output).  Tokens from lens[b] on are left alone."""
    if (q is None) != (q_out is None) or (kv is None) != (kv_out is None) or (q is None and kv is None):
        raise ValueError("q with q_out, kv with kv_out, at least one pair")
    x = q if q is not None else kv
    dev, dt = _home(x), x.dtype
    B, T, D = x.shape[0], x.shape[1], x.shape[-1]
    if q is not None and not q.numel():
        if kv is None:
            return
        q = None                     # no heads: the key alone
    if not B or not T:
        return
    H = cap = qb = qt = kb = kt = 0
    qp = qop = kp = kop = None
    if q is not None:
        _, _, H, _ = q.shape
        qb, qt, sh, sd = q.stride()
        if (sd != 1 and D > 1) or (sh != D and H > 1):
            raise ValueError("the heads of a token of q must be contiguous")
        qt = qt if T > 1 else H * D
        qb = qb if B > 1 else T * qt
        qp, qop = q.data_ptr(), _arg(q_out, "q_out", dt, q.shape, dev)
    if kv is not None:
        if kv.shape != (B, T, D) or kv.dtype is not dt or kv.get_device() != dev:
            raise ValueError("kv must be [B, T, D], of q's dtype and device")
        kb, kt, sd = kv.stride()
        if sd != 1 and D > 1:
            raise ValueError("the values of a token of kv must be contiguous")
        kt = kt if T > 1 else D
        kb = kb if B > 1 else T * kt
        cap = kv_out.shape[1]
        kp, kop = kv.data_ptr(), _arg(kv_out, "kv_out", dt, (B, cap, D), dev)
    fp, R, flags = _rope_args(inv_freq, norm, interleaved, inverse, dev)
    _check("qk_norm_rope", lib.qk_norm_rope(
        qp, qb, qt, kp, kb, kt, _code(dt), B, T, H, D, _arg(q_pos0, "q_pos0", torch.int32, (B,), dev),
        _arg(lens, "lens", torch.int32, (B,), dev), pos_step, fp, R,
        _arg(q_weight, "q_weight", torch.float32, (D,), dev), _arg(kv_weight, "kv_weight", torch.float32, (D,), dev),
        eps, flags, qop, kop, cap, _on(stream, dev)))


def hca_paged_append(a, z, pos0, carry, pool, table, held, m, carry_out=None, lens=None, norm=False, weight=None,
                     eps=1e-6, inv_freq=None, interleaved=True, inverse=False, status=None, stream=None):
    """Pool new tokens a, z [B, T, D] (gates z) into paged entries pool [N, P, D];
    carry [B, 2, 3, D] float32 holds the open blocks and is updated in place, or
    into carry_out.  Entries are optionally normalised and rotated at m * index."""
    dev, dt = _home(a), a.dtype
    B, T, D = a.shape
    if not B:
        return                       # (its tensors have no addresses)
    N, P_, _ = pool.shape
    maxp = table.shape[1]
    state = (B, 2, 3, D)
    cp = _arg(carry, "carry", torch.float32, state, dev)
    fp, R, flags = _rope_args(inv_freq, norm, interleaved, inverse, dev)
    _check("hca_paged_append", lib.hca_paged_append(
        _arg(a, "a", dt, None, dev), _arg(z, "z", dt, (B, T, D), dev), _code(dt), B, T, D, m,
        _arg(pos0, "pos0", torch.int32, (B,), dev), _arg(lens, "lens", torch.int32, (B,), dev), cp,
        cp if carry_out is None else _arg(carry_out, "carry_out", torch.float32, state, dev),
        _arg(pool, "pool", dt, (N, P_, D), dev), N, P_, _arg(table, "table", torch.int32, (B, maxp), dev),
        _arg(held, "held", torch.int32, (B,), dev), maxp, _arg(weight, "weight", torch.float32, (D,), dev), eps, fp, R,
        flags, _arg(status, "status", torch.int32, None, dev), _on(stream, dev)))


def hca_prefix_attn_fwd(q, pool, table, held, groups, kv_raw, sink, tau, W, q_pos0, out, m, lse=None, status=None,
                        stream=None):
    """HCA attention of q [B, T, H, D] over paged entries pool [N, P, D], the raw
    window kv_raw [B, raw_cap, D] and the sink; ``groups`` (paged.PrefixGroups)
    names the sequences that share their first pages."""
    dev, dt = _home(q), q.dtype
    if not q.numel():
        return
    B, T, H, D = q.shape
    N, P_, _ = pool.shape
    maxp = table.shape[1]
    if groups.B != B or groups.dev != dev:
        raise ValueError("groups must be those of the batch, on its device")
    raw_cap = 1 if kv_raw is None else kv_raw.shape[1]
    _check("hca_prefix_attn_fwd", lib.hca_prefix_attn_fwd(
        _arg(q, "q", dt, None, dev), _arg(pool, "pool", dt, (N, P_, D), dev), N, P_,
        _arg(table, "table", torch.int32, (B, maxp), dev), _arg(held, "held", torch.int32, (B,), dev), maxp,
        groups.off_ptr, groups.seq_ptr, groups.shared_ptr, groups.G, groups.n_seq,
        _arg(kv_raw, "kv_raw", dt, (B, raw_cap, D), dev), _arg(sink, "sink", torch.float32, (H,), dev), tau, W, B, T, H,
        D, m, raw_cap, _arg(q_pos0, "q_pos0", torch.int32, (B,), dev), _arg(out, "out", dt, (B, T, H, D), dev),
        _arg(lse, "lse", torch.float32, (B, T, H), dev), _code(dt), _arg(status, "status", torch.int32, None, dev),
        _on(stream, dev)))


def kv_pages_workspace_size(N, n):
    """Bytes of workspace for a cache of N pages and lists of n rows (0 for compact)."""
    return int(lib.kv_pages_workspace_size(N, n))


def _cache_args(table, held, refcount, dev):
    R, maxp = table.shape
    return (_arg(table, "table", torch.int32, None, dev), _arg(held, "held", torch.int32, (R,), dev), R, maxp,
            _arg(refcount, "refcount", torch.int32, None, dev), refcount.numel())


def _ws(workspace, dev):
    return _arg(workspace, "workspace", torch.int32, None, dev), workspace.numel() * 4


def _layers(pool, N, dev):
    """(pointer, L, bytes of one layer's page) of pool [L, N, P, D]."""
    L, n, P_, D = pool.shape
    if n != N:
        raise ValueError("pool must be [L, N, P, D] with refcount [N]")
    return _arg(pool, "pool", pool.dtype, None, dev), L, P_ * D * pool.element_size()


def kv_pages_reserve(rows, n_entries, P, table, held, refcount, workspace, status=None, stream=None):
    """Grow the listed rows to hold n_entries entries each (pages of P)."""
    dev, n = _home(table), rows.numel()
    tp, hp, R, maxp, rp, N = _cache_args(table, held, refcount, dev)
    _check("kv_pages_reserve", lib.kv_pages_reserve(
        _arg(rows, "rows", torch.int32, (n,), dev), _arg(n_entries, "n_entries", torch.int32, (n,), dev), n, P, tp, hp,
        R, maxp, rp, N, *_ws(workspace, dev), _arg(status, "status", torch.int32, None, dev), _on(stream, dev)))


def kv_pages_fork(src, dst, n_entries, pool, table, held, refcount, workspace, status=None, stream=None):
    """Make each empty row dst[i] share the first n_entries[i] entries of src[i];
    pool [L, N, P, D] (a partial last page is copied in every layer)."""
    dev, n = _home(table), dst.numel()
    tp, hp, R, maxp, rp, N = _cache_args(table, held, refcount, dev)
    pp, L, page = _layers(pool, N, dev)
    _check("kv_pages_fork", lib.kv_pages_fork(
        _arg(src, "src", torch.int32, (n,), dev), _arg(dst, "dst", torch.int32, (n,), dev),
        _arg(n_entries, "n_entries", torch.int32, (n,), dev), n, pool.shape[2], tp, hp, R, maxp, rp, N, pp, L, page,
        *_ws(workspace, dev), _arg(status, "status", torch.int32, None, dev), _on(stream, dev)))


def kv_pages_free(rows, table, held, refcount, status=None, stream=None):
    """Give up the pages of the listed rows."""
    dev, n = _home(table), rows.numel()
    tp, hp, R, maxp, rp, N = _cache_args(table, held, refcount, dev)
    _check("kv_pages_free", lib.kv_pages_free(
        _arg(rows, "rows", torch.int32, (n,), dev), n, tp, hp, R, maxp, rp, N,
        _arg(status, "status", torch.int32, None, dev), _on(stream, dev)))


def kv_pages_compact(pool, table, held, refcount, n_live, workspace, table_out=None, refcount_out=None, stream=None):
    """Move the pages in use to the ids [0, n_live) (pool [L, N, P, D] in place);
    the new metadata goes to table_out / refcount_out (default: in place) and
    the number of pages in use to n_live int32 [1]."""
    dev = _home(table)
    tp, hp, R, maxp, rp, N = _cache_args(table, held, refcount, dev)
    pp, L, page = _layers(pool, N, dev)
    _check("kv_pages_compact", lib.kv_pages_compact(
        tp, hp, R, maxp, rp, N, pp, L, page,
        tp if table_out is None else _arg(table_out, "table_out", torch.int32, (R, maxp), dev),
        rp if refcount_out is None else _arg(refcount_out, "refcount_out", torch.int32, (N,), dev),
        _arg(n_live, "n_live", torch.int32, (1,), dev), *_ws(workspace, dev), _on(stream, dev)))
