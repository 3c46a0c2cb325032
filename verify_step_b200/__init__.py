"""B200-native speculative-decoding verify step: Python binding of include/sd_verify.h.

Argument marshalling only.  Every step of the path runs in the CUDA kernels of
libsdverify.so (built in-tree by ``python -m verify_step_b200.build``); torch supplies device
memory and streams.  There is no fallback: if the library is missing or a call fails, the
binding raises.

Functions carry the C names (sd_verify_attn, sd_draft_xattn, sd_lm_head, sd_accept,
sd_commit, sd_linear, sd_rope, sd_append_kv, sd_verify_attn_q8, sd_draft_xattn_q8, sd_logprobs and
the *_workspace_size / status helpers).  Tensors are passed as torch CUDA
tensors (their data_ptr is used; they must be contiguous), descriptors as the ctypes
structures below, ``stream`` as a torch.cuda.Stream (default: the current stream).
Row tensors whose descriptor has a row stride (sd_rope, sd_append_kv) may be strided views whose
rows are contiguous; a cache in 8 bits is a torch.float8_e4m3fn (or uint8) tensor.
The calls from sd_rope_freqs on refuse tensors of another device than the current one.
"""
from __future__ import annotations

import ctypes
import os

from .telemetry import acceptance_telemetry  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsdverify.so")

SD_OK, SD_ERR_INVALID_ARG, SD_ERR_UNSUPPORTED, SD_ERR_WORKSPACE = 0, 1, 2, 3
SD_ERR_CUDA, SD_ERR_TIMEOUT, SD_ERR_DEVICE = 4, 5, 6
SD_F32, SD_BF16, SD_E4M3 = 0, 1, 2


class SdError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_q", ctypes.c_int), ("h_q", ctypes.c_int),
                ("h_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("block_size", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("window", ctypes.c_int),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int),
                ("q_offset", ctypes.c_int)]


class HeadDesc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int), ("d", ctypes.c_int), ("vocab", ctypes.c_int),
                ("ld_logits", ctypes.c_int), ("n_clusters", ctypes.c_int),
                ("cluster_size", ctypes.c_int), ("top_c", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class AcceptDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("k", ctypes.c_int), ("vocab", ctypes.c_int),
                ("temperature", ctypes.c_float), ("seed", ctypes.c_uint64),
                ("step", ctypes.c_uint64), ("purpose", ctypes.c_int),
                ("ld_target", ctypes.c_int), ("ld_draft", ctypes.c_int),
                ("ld_out", ctypes.c_int), ("step_ptr", ctypes.c_void_p)]


class PoisonCache(ctypes.Structure):
    _fields_ = [("cache", ctypes.c_void_p), ("h_kv", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int)]


class CommitDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("k", ctypes.c_int), ("block_size", ctypes.c_int),
                ("max_blocks_per_seq", ctypes.c_int), ("num_blocks", ctypes.c_int),
                ("d", ctypes.c_int), ("hidden_dtype", ctypes.c_int),
                ("n_poison", ctypes.c_int), ("poison", ctypes.POINTER(PoisonCache)),
                ("step_ptr", ctypes.c_void_p)]


SD_EPI_STORE, SD_EPI_ADD, SD_EPI_GEGLU = 0, 1, 2


class LinearDesc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int), ("n", ctypes.c_int), ("k", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("ld_x", ctypes.c_int64), ("k_gather", ctypes.c_int),
                ("ld_table", ctypes.c_int64), ("table_rows", ctypes.c_int64),
                ("ld_tokens", ctypes.c_int64), ("norm_gain", ctypes.c_void_p),
                ("norm_eps", ctypes.c_float), ("epilogue", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("ld_out", ctypes.c_int64),
                ("norm_out", ctypes.c_void_p), ("ld_norm_out", ctypes.c_int64),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


SD_ROPE_HALF, SD_ROPE_INTERLEAVED = 0, 1
SD_ROPE_PLAIN, SD_ROPE_LINEAR, SD_ROPE_BY_PARTS = 0, 1, 2


class RopeFreqDesc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("base", ctypes.c_double), ("scaling", ctypes.c_int),
                ("factor", ctypes.c_double), ("orig_ctx", ctypes.c_int),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


class Rotary(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("amplitude", ctypes.c_float)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("ld_x", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("rows_per_seq", ctypes.c_int), ("q_offset", ctypes.c_int)]


class AppendDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_new", ctypes.c_int), ("n_rows", ctypes.c_int),
                ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("block_size", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64),
                ("ld_q", ctypes.c_int64), ("ld_q_out", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("cache_dtype", ctypes.c_int)]


class LogprobsDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("vocab", ctypes.c_int), ("ld_logits", ctypes.c_int),
                ("temperature", ctypes.c_float), ("top_n", ctypes.c_int)]


_lib = None

_P = ctypes.c_void_p
_SIGS = {
    "sd_verify_attn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(AttnDesc)]),
    "sd_verify_attn": (ctypes.c_int, [ctypes.POINTER(AttnDesc), _P, _P, _P, _P, _P, _P, _P, _P,
                                      _P, ctypes.c_size_t, _P]),
    "sd_draft_xattn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(AttnDesc)]),
    "sd_draft_xattn": (ctypes.c_int, [ctypes.POINTER(AttnDesc), _P, _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "sd_lm_head_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(HeadDesc)]),
    "sd_lm_head": (ctypes.c_int, [ctypes.POINTER(HeadDesc), _P, _P, _P, _P, _P, _P, _P,
                                  ctypes.c_size_t, _P]),
    "sd_accept_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(AcceptDesc)]),
    "sd_accept": (ctypes.c_int, [ctypes.POINTER(AcceptDesc), _P, _P, _P, _P, _P, _P, _P,
                                 ctypes.c_size_t, _P]),
    "sd_accept_noalloc": (ctypes.c_int, [ctypes.POINTER(AcceptDesc), _P, _P, _P, _P, _P, _P,
                                         _P]),
    "sd_commit": (ctypes.c_int, [ctypes.POINTER(CommitDesc), _P, _P, _P, _P, _P, _P, _P]),
    "sd_linear_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LinearDesc)]),
    "sd_linear": (ctypes.c_int, [ctypes.POINTER(LinearDesc), _P, _P, _P, _P, _P, _P, _P]),
    "sd_rope_freqs": (ctypes.c_int, [ctypes.POINTER(RopeFreqDesc), _P,
                                     ctypes.POINTER(ctypes.c_float), _P]),
    "sd_rope": (ctypes.c_int, [ctypes.POINTER(RopeDesc), ctypes.POINTER(Rotary), _P, _P, _P, _P,
                               _P]),
    "sd_append_kv": (ctypes.c_int, [ctypes.POINTER(AppendDesc), ctypes.POINTER(Rotary)] +
                     [_P] * 12),
    "sd_verify_attn_q8_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(AttnDesc)]),
    "sd_verify_attn_q8": (ctypes.c_int, [ctypes.POINTER(AttnDesc)] + [_P] * 9 +
                          [ctypes.c_size_t, _P]),
    "sd_draft_xattn_q8_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(AttnDesc)]),
    "sd_draft_xattn_q8": (ctypes.c_int, [ctypes.POINTER(AttnDesc)] + [_P] * 10 +
                          [ctypes.c_size_t, _P]),
    "sd_logprobs_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LogprobsDesc)]),
    "sd_logprobs": (ctypes.c_int, [ctypes.POINTER(LogprobsDesc)] + [_P] * 7 +
                    [ctypes.c_size_t, _P]),
    "sd_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sd_device_status_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int), _P]),
    "sd_device_status_clear": (ctypes.c_int, [_P]),
    "sd_selftest_bounded_wait": (ctypes.c_int, [_P]),
    "sd_version": (ctypes.c_int, []),
}


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m verify_step_b200.build` (no fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def status_string(status: int) -> str:
    return lib().sd_status_string(int(status)).decode()


def _refuse(t, dev):
    """What is wrong with a tensor that _ptr or _rows_ptr does not take as it is."""
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on a CUDA device")
    if dev is not None and t.get_device() != dev:
        raise ValueError("tensors must live on the current device")
    raise ValueError("tensor arguments must be contiguous")


def _ptr(t, dev=None):
    """Address of a contiguous CUDA tensor; with ``dev``, of that device (the current one, where the
    call would run)."""
    if t is None or isinstance(t, int):
        return t
    if (t.is_cuda if dev is None else t.get_device() == dev) and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dev)


def _rows_ptr(t, ld, rows, width, dev=None):
    """Address of row data [rows, ...] whose rows of ``width`` elements are contiguous and ``ld``
    elements apart (a view of a wider buffer is fine)."""
    if t is None or isinstance(t, int):
        return t
    if not (t.is_cuda if dev is None else t.get_device() == dev):
        _refuse(t, dev)
    if t.is_contiguous() and t.numel() >= (rows - 1) * ld + width:
        return t.data_ptr()
    inner = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != inner:
            raise ValueError("a row's elements must be contiguous")
        inner *= n
    if inner < width or t.shape[0] < rows or (rows > 1 and t.stride(0) != ld):
        raise ValueError("row tensor does not fit the descriptor's rows, width and row stride")
    return t.data_ptr()


_cuda = None  # torch's calls for the current device and for its stream's address


def _torch_cuda():
    global _cuda
    if _cuda is None:
        import torch
        torch.cuda.current_device()  # initialises CUDA
        # the raw calls build no object; a torch without them has the public ones
        _cuda = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                 getattr(torch._C, "_cuda_getCurrentRawStream",
                         lambda device: torch.cuda.current_stream(device).cuda_stream))
    return _cuda


def _current_device():
    return _torch_cuda()[0]()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    device, raw_stream = _torch_cuda()
    return raw_stream(device())


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _check(fn, status):
    if status != SD_OK:
        raise SdError(fn, status)


def sd_verify_attn_workspace_size(desc: AttnDesc) -> int:
    return lib().sd_verify_attn_workspace_size(ctypes.byref(desc))


def sd_draft_xattn_workspace_size(desc: AttnDesc) -> int:
    return lib().sd_draft_xattn_workspace_size(ctypes.byref(desc))


def sd_lm_head_workspace_size(desc: HeadDesc) -> int:
    return lib().sd_lm_head_workspace_size(ctypes.byref(desc))


def sd_accept_workspace_size(desc: AcceptDesc) -> int:
    return lib().sd_accept_workspace_size(ctypes.byref(desc))


def sd_verify_attn(desc, q, k_new, v_new, k_cache, v_cache, block_table, ctx_len, out, ws,
                   stream=None):
    _check("sd_verify_attn", lib().sd_verify_attn(
        ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_table), _ptr(ctx_len), _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)))


def sd_draft_xattn(desc, q, k_cache, v_cache, block_table, ctx_len, q_pos, out, ws,
                   stream=None):
    _check("sd_draft_xattn", lib().sd_draft_xattn(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(ctx_len), _ptr(q_pos), _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)))


def sd_lm_head(desc, h, w, logits, centroids=None, cluster_tokens=None, sel_clusters=None,
               ws=None, stream=None):
    _check("sd_lm_head", lib().sd_lm_head(
        ctypes.byref(desc), _ptr(h), _ptr(w), _ptr(centroids), _ptr(cluster_tokens),
        _ptr(logits), _ptr(sel_clusters), _ptr(ws), _nbytes(ws), _stream(stream)))


def sd_accept(desc, target_logits, draft_logits, draft_tokens, n_accepted, out_tokens,
              margin_flags, ws, stream=None):
    _check("sd_accept", lib().sd_accept(
        ctypes.byref(desc), _ptr(target_logits), _ptr(draft_logits), _ptr(draft_tokens),
        _ptr(n_accepted), _ptr(out_tokens), _ptr(margin_flags), _ptr(ws), _nbytes(ws),
        _stream(stream)))


def sd_accept_noalloc(desc, target_logits, draft_logits, draft_tokens, n_accepted, out_tokens,
                      margin_flags, stream=None):
    """sd_accept without a caller workspace: the library's fixed scratch array is used (see
    include/sd_verify.h for its size limit and the rule that overlapping calls race)."""
    _check("sd_accept_noalloc", lib().sd_accept_noalloc(
        ctypes.byref(desc), _ptr(target_logits), _ptr(draft_logits), _ptr(draft_tokens),
        _ptr(n_accepted), _ptr(out_tokens), _ptr(margin_flags), _stream(stream)))


def sd_commit(desc, block_table, ctx_len, n_accepted, committed_slots, hidden=None,
              next_hidden=None, stream=None):
    _check("sd_commit", lib().sd_commit(
        ctypes.byref(desc), _ptr(block_table), _ptr(ctx_len), _ptr(n_accepted),
        _ptr(committed_slots), _ptr(hidden), _ptr(next_hidden), _stream(stream)))


def sd_linear_workspace_size(desc: LinearDesc) -> int:
    return lib().sd_linear_workspace_size(ctypes.byref(desc))


def sd_linear(desc, x, w, out, table=None, tokens=None, token_sel=None, stream=None, ws=None):
    """One projection; ``ws`` (a device tensor or address), when given, is set as the
    descriptor's workspace (its size in bytes from the tensor)."""
    if ws is not None:
        desc.ws = _ptr(ws)
        desc.ws_bytes = ws.numel() * ws.element_size() if hasattr(ws, "numel") else desc.ws_bytes
    _check("sd_linear", lib().sd_linear(
        ctypes.byref(desc), _ptr(x), _ptr(w), _ptr(out), _ptr(table), _ptr(tokens),
        _ptr(token_sel), _stream(stream)))


def sd_rope_freqs(desc, freqs, stream=None) -> float:
    """Fills ``freqs`` (int64 [rot_dim / 2]: 64-bit fractions of a turn); returns the amplitude."""
    amp = ctypes.c_float(1.0)
    at = _ptr(freqs, _current_device())
    _check("sd_rope_freqs", lib().sd_rope_freqs(ctypes.byref(desc), at, ctypes.byref(amp),
                                                _stream(stream)))
    return amp.value


def rotary(freqs, layout=SD_ROPE_HALF, amplitude=1.0) -> Rotary:
    """The rotation argument of sd_rope and sd_append_kv; it keeps ``freqs`` alive."""
    r = Rotary(_ptr(freqs), 2 * freqs.numel(), layout, amplitude)
    r.table = freqs
    return r


def _rot(rot, dev):
    if rot is None:
        return None
    _ptr(getattr(rot, "table", None), dev)
    return ctypes.byref(rot)


def sd_rope(desc, rot, x, pos, ctx_len, out, stream=None):
    dev, width = _current_device(), desc.heads * desc.head_dim
    args = (_rot(rot, dev), _rows_ptr(x, desc.ld_x, desc.rows, width, dev), _ptr(pos, dev),
            _ptr(ctx_len, dev), _rows_ptr(out, desc.ld_out, desc.rows, width, dev))
    _check("sd_rope", lib().sd_rope(ctypes.byref(desc), *args, _stream(stream)))


def sd_append_kv(desc, rot, k_new, v_new, q, k_cache, v_cache, k_scale, v_scale, block_table,
                 ctx_len, cu_new=None, q_out=None, stream=None):
    dev = _current_device()
    n, kv, w = desc.n_rows, desc.h_kv * desc.head_dim, desc.h_q * desc.head_dim
    args = (_rot(rot, dev), _rows_ptr(k_new, desc.ld_k, n, kv, dev),
            _rows_ptr(v_new, desc.ld_v, n, kv, dev), _rows_ptr(q, desc.ld_q, n, w, dev),
            _ptr(k_cache, dev), _ptr(v_cache, dev), _ptr(k_scale, dev), _ptr(v_scale, dev),
            _ptr(block_table, dev), _ptr(ctx_len, dev), _ptr(cu_new, dev),
            _rows_ptr(q_out, desc.ld_q_out, n, w, dev))
    _check("sd_append_kv", lib().sd_append_kv(ctypes.byref(desc), *args, _stream(stream)))


def sd_verify_attn_q8_workspace_size(desc: AttnDesc) -> int:
    return lib().sd_verify_attn_q8_workspace_size(ctypes.byref(desc))


def sd_verify_attn_q8(desc, q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_len, out, ws,
                      stream=None):
    dev = _current_device()
    args = (_ptr(q, dev), _ptr(k_cache, dev), _ptr(v_cache, dev), _ptr(k_scale, dev),
            _ptr(v_scale, dev), _ptr(block_table, dev), _ptr(ctx_len, dev), _ptr(out, dev),
            _ptr(ws, dev), _nbytes(ws))
    _check("sd_verify_attn_q8",
           lib().sd_verify_attn_q8(ctypes.byref(desc), *args, _stream(stream)))


def sd_draft_xattn_q8_workspace_size(desc: AttnDesc) -> int:
    return lib().sd_draft_xattn_q8_workspace_size(ctypes.byref(desc))


def sd_draft_xattn_q8(desc, q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_len, q_pos,
                      out, ws, stream=None):
    dev = _current_device()
    args = (_ptr(q, dev), _ptr(k_cache, dev), _ptr(v_cache, dev), _ptr(k_scale, dev),
            _ptr(v_scale, dev), _ptr(block_table, dev), _ptr(ctx_len, dev), _ptr(q_pos, dev),
            _ptr(out, dev), _ptr(ws, dev), _nbytes(ws))
    _check("sd_draft_xattn_q8",
           lib().sd_draft_xattn_q8(ctypes.byref(desc), *args, _stream(stream)))


def sd_logprobs_workspace_size(desc: LogprobsDesc) -> int:
    return lib().sd_logprobs_workspace_size(ctypes.byref(desc))


def sd_logprobs(desc, logits, tokens, logprob, entropy=None, top_ids=None, top_logprobs=None,
                ws=None, stream=None):
    dev = _current_device()
    args = (_ptr(logits, dev), _ptr(tokens, dev), _ptr(logprob, dev), _ptr(entropy, dev),
            _ptr(top_ids, dev), _ptr(top_logprobs, dev), _ptr(ws, dev), _nbytes(ws))
    _check("sd_logprobs", lib().sd_logprobs(ctypes.byref(desc), *args, _stream(stream)))


def sd_device_status_read(stream=None) -> int:
    v = ctypes.c_int(0)
    _check("sd_device_status_read", lib().sd_device_status_read(ctypes.byref(v),
                                                                _stream(stream)))
    return v.value


def sd_device_status_clear(stream=None):
    _check("sd_device_status_clear", lib().sd_device_status_clear(_stream(stream)))


def sd_selftest_bounded_wait(stream=None):
    _check("sd_selftest_bounded_wait", lib().sd_selftest_bounded_wait(_stream(stream)))


def sd_version() -> int:
    return lib().sd_version()


def poison_list(caches):
    """ctypes array of PoisonCache for sd_commit from (tensor, h_kv, head_dim, dtype) tuples."""
    arr = (PoisonCache * len(caches))()
    for i, (t, h_kv, hd, dt) in enumerate(caches):
        arr[i] = PoisonCache(_ptr(t), h_kv, hd, dt)
    return arr
