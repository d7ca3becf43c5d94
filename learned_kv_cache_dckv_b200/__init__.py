"""B200-native DCKV codec: Python binding of the C ABI in include/*.h.

The binding only marshals arguments: every step of encode and decode runs in the
CUDA library ``libdckv_b200.so`` (sm_100a).  PyTorch supplies device memory and
streams.  If the library is missing the import of any entry point raises; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdckv_b200.so")
INCLUDE_DIR = os.path.join(os.path.dirname(_HERE), "include")

ROW_DIM = 6144
N_COEF = 2048
N_HIDDEN = 256
HEAD_KEPT = 4
TAIL_KEPT = 128

DCKV_OK, DCKV_EINVAL, DCKV_ECAPACITY, DCKV_ECUDA, DCKV_ECORRUPT, DCKV_ETIMEOUT, DCKV_ERANGE, DCKV_ESINGULAR = range(8)
STATUS_NAMES = {0: "OK", 1: "EINVAL", 2: "ECAPACITY", 3: "ECUDA", 4: "ECORRUPT", 5: "ETIMEOUT", 6: "ERANGE",
                7: "ESINGULAR"}

# fp64 layout of the closed-form fit's sums (include/dckv_fit.h)
FIT_OFF_GE = 0
FIT_OFF_CE = 2048 * 2048
FIT_OFF_GO = 2 * 2048 * 2048
FIT_OFF_CO = FIT_OFF_GO + 6144 * 6144
FIT_OFF_N = FIT_OFF_CO + 6144 * 2048
FIT_STATS_DOUBLES = FIT_OFF_N + 8

# element types, rotary layouts, scalings and modes (include/dckv_cache.h)
DCKV_BF16, DCKV_FP16, DCKV_FP32 = range(3)
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}
ROPE_MODES = {"forward": 0, "gradient": 1, "inverse": 2}

_lib = None


class DckvError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)} ({code})")
        self.code = code


class _Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("mu", "basis", "w1", "w2", "delta", "laplace_b", "embed", "w_even", "w_odd")] + [
                   ("vocab", ctypes.c_int32), ("v1", ctypes.c_void_p), ("v2", ctypes.c_void_p)]


class ByteReport(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("total", "header_tables", "kept_rows", "states", "esc_counts", "esc_values", "words",
                 "padding", "payload")] + [(n, ctypes.c_uint32) for n in
                                           ("n_prompts", "n_chunks", "n_coded_rows", "n_escapes",
                                            "chunk_rows", "k_eff")]

    def as_dict(self):
        return {k: int(getattr(self, k)) for k, _ in self._fields_}


class WsView(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("q32", "qe", "cen8", "row_slot", "sym16", "q16", "x16", "g16", "counters")] + [
        ("n_rows", ctypes.c_int64), ("ne_pad", ctypes.c_int64), ("n_chunks", ctypes.c_int32),
        ("total", ctypes.c_uint64), ("code_width", ctypes.c_int32)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("magnitude", ctypes.c_double),
                ("freq", ctypes.c_double * 128)]


class _RopeArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("x_token_stride", "x_head_stride", "out_token_stride", "out_head_stride",
                                      "n_tokens")] + [
        ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("positions", ctypes.c_void_p),
        ("dtype", ctypes.c_int32), ("device", ctypes.c_int32)]


class KvPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_int32) for n in ("device", "dtype", "n_layers", "n_kv_heads", "head_dim", "page_size")] + [
        (n, ctypes.c_int64) for n in ("n_pages", "k_layer_stride", "k_page_stride", "k_row_stride", "k_head_stride",
                                      "v_layer_stride", "v_page_stride", "v_row_stride", "v_head_stride")]


class CacheBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "max_new", "max_pages", "reserved")] + [
        (n, ctypes.c_void_p) for n in ("offsets", "kv_lens", "page_table")] + [("table_stride", ctypes.c_int64)]


class _AppendArgs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("k_layer_stride", "k_token_stride", "k_head_stride", "v_layer_stride",
                                      "v_token_stride", "v_head_stride")] + [
        ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("q_token_stride", "q_head_stride", "q_out_token_stride", "q_out_head_stride",
                                      "n_tokens")] + [
        ("n_q_heads", ctypes.c_int32), ("reserved", ctypes.c_int32), ("positions", ctypes.c_void_p)]


class _AttentionArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "out", "lse")] + [
        (n, ctypes.c_int64) for n in ("q_token_stride", "q_head_stride", "out_token_stride", "out_head_stride",
                                      "n_tokens")] + [
        (n, ctypes.c_int32) for n in ("n_q_heads", "layer", "causal")] + [("scale", ctypes.c_float)]


def lib():
    """Load libdckv_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m learned_kv_cache_dckv_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "dckv_codec_create": (I, [ctypes.POINTER(_Params), I, I, ctypes.POINTER(P)]),
        "dckv_codec_destroy": (None, [P]),
        "dckv_codec_k_eff": (I, [P]),
        "dckv_workspace_bytes": (Z, [P, P, I]),
        "dckv_blob_bound": (Z, [P, P, I]),
        "dckv_encode": (I, [P, P, P, P, I, P, Z, P, P, P, Z, P]),
        "dckv_decode": (I, [P, P, Z, P, P, I, P, P, P, P, Z, P]),
        "dckv_decode_static": (I, [P, P, Z, P, P, I, P, P, P, P]),
        "dckv_bytes": (I, [P, Z, ctypes.POINTER(ByteReport)]),
        "dckv_last_error": (ctypes.c_char_p, []),
        "dckv_ws_offsets": (I, [P, P, I, I, ctypes.POINTER(WsView)]),
        "dckv_codec_export": (I, [P, P, P, P, P]),
        "dckv_codec_tables": (I, [P, ctypes.POINTER(P), ctypes.POINTER(P)]),
        "dckv_set_timing": (I, [P, I]),
        "dckv_get_timing": (I, [P, P, P, I]),
        "dckv_debug_gemm": (I, [I, P, I, P, I, I, I, P, I, I, P]),
        "dckv_debug_ratio": (I, [P, P]),
        "dckv_codec_info": (I, [P, P, P]),
        "dckv_codec_gemm_shape": (I, [P, P]),
        "dckv_launch_count": (ctypes.c_longlong, []),
        "dckv_fit_workspace_bytes": (Z, [P, P, I]),
        "dckv_fit_accumulate": (I, [P, P, ctypes.c_int32, P, P, P, I, P, P, P, Z, P]),
        "dckv_fit_solve_workspace_bytes": (Z, []),
        "dckv_fit_solve": (I, [P, ctypes.c_double, P, P, P, P, Z, P]),
        "dckv_fit_to_bf16": (I, [P, ctypes.c_int64, P, P]),
        "dckv_fit_scales_accumulate": (I, [P, P, P, P, I, P, P, P, Z, P]),
        "dckv_fit_scales_finish": (I, [P, P, P, P]),
        "dckv_rope_init": (I, [P, I, I, ctypes.c_double, I] + [ctypes.c_double] * 5),
        "dckv_rope": (I, [P, I, P, P]),
        "dckv_cache_append": (I, [P, P, P, P, P, P]),
        "dckv_cache_rows": (I, [P, P, P, P, ctypes.c_int64, ctypes.c_int64, P, P, P]),
        "dckv_attention_workspace_bytes": (Z, [P, P, I]),
        "dckv_attention": (I, [P, P, P, P, P, Z, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def header_functions():
    """Names of every function declared in include/*.h."""
    names = []
    for fn in sorted(os.listdir(INCLUDE_DIR)):
        if fn.endswith(".h"):
            txt = open(os.path.join(INCLUDE_DIR, fn)).read()
            txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
            names += re.findall(r"\b(dckv_[a-z0-9_]+)\s*\(", txt)
    return sorted(set(names))


def last_error() -> str:
    return lib().dckv_last_error().decode()


def _check(code, what):
    if code != DCKV_OK:
        raise DckvError(code, f"{what} ({last_error()})")


def _offs(seq_offsets):
    a = np.ascontiguousarray(np.asarray(seq_offsets, dtype=np.int64))
    return a, a.ctypes.data_as(ctypes.c_void_p), a.size - 1


def _ptr(t):
    """Device address of a tensor, or NULL for None (token ids of a codec without mean models)."""
    return None if t is None else t.data_ptr()


def _stream_ptr(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ---------------------------------------------------------------------------------- C ABI
def dckv_codec_create(params: dict, device: int = 0, chunk_rows: int = 0):
    """params: device tensors mu, basis, w1, w2, delta, laplace_b (fp32), embed, w_even,
    w_odd (bf16 or int16 holding bf16 bits), v1, v2 (fp32, optional); w1 / w2 None for a
    linear codec, embed / w_even / w_odd None for unconditional tables, v1 / v2 None for a
    linear synthesis.  Returns an opaque handle."""
    p = _Params()
    for k in ("mu", "basis", "w1", "w2", "delta", "laplace_b", "embed", "w_even", "w_odd", "v1", "v2"):
        v = params.get(k)
        setattr(p, k, None if v is None else v.data_ptr())
    p.vocab = 0 if params.get("embed") is None else int(params["embed"].shape[0])
    h = ctypes.c_void_p()
    _check(lib().dckv_codec_create(ctypes.byref(p), int(device), int(chunk_rows), ctypes.byref(h)),
           "dckv_codec_create")
    return h


def dckv_codec_destroy(handle):
    lib().dckv_codec_destroy(handle)


def dckv_codec_k_eff(handle) -> int:
    return int(lib().dckv_codec_k_eff(handle))


def dckv_workspace_bytes(handle, seq_offsets) -> int:
    a, ptr, b = _offs(seq_offsets)
    return int(lib().dckv_workspace_bytes(handle, ptr, b))


def dckv_blob_bound(handle, seq_offsets) -> int:
    a, ptr, b = _offs(seq_offsets)
    return int(lib().dckv_blob_bound(handle, ptr, b))


def dckv_encode(handle, rows, token_ids, seq_offsets, blob, blob_size, status, workspace, stream=None):
    """rows bf16 [sum N, 6144], token_ids int32 [sum N], blob uint8 (device), blob_size
    uint64[1]/int64[1] (device), status int32[1] (device), workspace uint8 (device)."""
    a, ptr, b = _offs(seq_offsets)
    _check(lib().dckv_encode(handle, rows.data_ptr(), _ptr(token_ids), ptr, b, blob.data_ptr(),
                             blob.numel() * blob.element_size(), blob_size.data_ptr(), status.data_ptr(),
                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                             _stream_ptr(stream)), "dckv_encode")


def dckv_decode(handle, blob, blob_bytes, token_ids, seq_offsets, k_out, v_out, status, workspace, stream=None):
    a, ptr, b = _offs(seq_offsets)
    _check(lib().dckv_decode(handle, blob.data_ptr(), int(blob_bytes), _ptr(token_ids), ptr, b,
                             k_out.data_ptr(), v_out.data_ptr(), status.data_ptr(), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream_ptr(stream)), "dckv_decode")


def dckv_decode_static(handle, blob, blob_bytes, token_ids, seq_offsets, k_out, v_out, status, stream=None):
    """dckv_decode on the library's static per-device scratch (no workspace argument)."""
    a, ptr, b = _offs(seq_offsets)
    _check(lib().dckv_decode_static(handle, blob.data_ptr(), int(blob_bytes), _ptr(token_ids), ptr, b,
                                    k_out.data_ptr(), v_out.data_ptr(), status.data_ptr(), _stream_ptr(stream)),
           "dckv_decode_static")


def dckv_launch_count() -> int:
    return int(lib().dckv_launch_count())


def dckv_bytes(blob_host: bytes) -> dict:
    buf = ctypes.create_string_buffer(bytes(blob_host), len(blob_host))
    rep = ByteReport()
    _check(lib().dckv_bytes(buf, len(blob_host), ctypes.byref(rep)), "dckv_bytes")
    return rep.as_dict()


def dckv_ws_offsets(handle, seq_offsets, which: int) -> dict:
    a, ptr, b = _offs(seq_offsets)
    v = WsView()
    _check(lib().dckv_ws_offsets(handle, ptr, b, int(which), ctypes.byref(v)), "dckv_ws_offsets")
    return {k: int(getattr(v, k)) for k, _ in WsView._fields_}


def dckv_codec_export(handle):
    cdf = np.zeros((64, 510), np.uint16)
    scale = np.zeros(2048, np.uint8)
    keep = np.zeros(2048, np.uint8)
    exps = np.zeros(3, np.int32)
    _check(lib().dckv_codec_export(handle, cdf.ctypes.data_as(ctypes.c_void_p), scale.ctypes.data_as(ctypes.c_void_p),
                                   keep.ctypes.data_as(ctypes.c_void_p), exps.ctypes.data_as(ctypes.c_void_p)),
           "dckv_codec_export")
    return cdf, scale, keep, exps


def dckv_codec_tables(handle):
    te, to = ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib().dckv_codec_tables(handle, ctypes.byref(te), ctypes.byref(to)), "dckv_codec_tables")
    return te.value, to.value


def dckv_debug_ratio(handle, ratio_dev):
    _check(lib().dckv_debug_ratio(handle, None if ratio_dev is None else ratio_dev.data_ptr()), "dckv_debug_ratio")


def dckv_codec_info(handle):
    g = ctypes.c_int32()
    bits = ctypes.c_double()
    _check(lib().dckv_codec_info(handle, ctypes.byref(g), ctypes.byref(bits)), "dckv_codec_info")
    return {"chunk_rows": int(g.value), "model_bits_per_row": float(bits.value)}


def dckv_codec_gemm_shape(handle):
    a = (ctypes.c_int32 * 4)()
    _check(lib().dckv_codec_gemm_shape(handle, a), "dckv_codec_gemm_shape")
    return {"k_eff": a[0], "kw": a[1], "mp": a[2], "inv_lo_k": a[3]}


def dckv_set_timing(handle, enable: bool):
    _check(lib().dckv_set_timing(handle, 1 if enable else 0), "dckv_set_timing")


def dckv_get_timing(handle, max_stages: int = 24):
    ms = (ctypes.c_float * max_stages)()
    names = (ctypes.c_char_p * max_stages)()
    n = lib().dckv_get_timing(handle, ms, names, max_stages)
    return [(names[i].decode(), float(ms[i])) for i in range(max(0, n))]


def dckv_debug_gemm(bf16: bool, A, slabs: int, B, M: int, N: int, K: int, D, bn: int = 256, pair: bool = False,
                    stream=None):
    _check(lib().dckv_debug_gemm(1 if bf16 else 0, A.data_ptr(), int(slabs), B.data_ptr(), int(M), int(N), int(K),
                                 D.data_ptr(), int(bn), 1 if pair else 0, _stream_ptr(stream)), "dckv_debug_gemm")


# ---------------------------------------------------------------------------------- helpers
# ------------------------------------------------------------- closed-form fit (dckv_fit.h)
def dckv_fit_workspace_bytes(handle, seq_offsets) -> int:
    a, ptr, b = _offs(seq_offsets)
    return int(lib().dckv_fit_workspace_bytes(handle, ptr, b))


def dckv_fit_accumulate(handle, embed, rows, token_ids, seq_offsets, stats, status, workspace, stream=None):
    """embed bf16 [vocab, 2048] (device), rows bf16 [sum N, 6144], token_ids int32, stats fp64
    [FIT_STATS_DOUBLES] (accumulated into), status int32[1], workspace uint8 (device)."""
    a, ptr, b = _offs(seq_offsets)
    _check(lib().dckv_fit_accumulate(handle, embed.data_ptr(), int(embed.shape[0]), rows.data_ptr(),
                                     token_ids.data_ptr(), ptr, b, stats.data_ptr(), status.data_ptr(),
                                     workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _stream_ptr(stream)), "dckv_fit_accumulate")


def dckv_fit_solve_workspace_bytes() -> int:
    return int(lib().dckv_fit_solve_workspace_bytes())


def dckv_fit_solve(stats, ridge, w_even, w_odd, status, workspace, stream=None):
    """w_even fp64 [2048, 2048] and w_odd fp64 [6144, 2048] (device) receive the weights."""
    _check(lib().dckv_fit_solve(stats.data_ptr(), float(ridge), w_even.data_ptr(), w_odd.data_ptr(),
                                status.data_ptr(), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "dckv_fit_solve")


def dckv_fit_to_bf16(w, out, stream=None):
    """bf16 bits (out: int16/uint16-sized device tensor) of fp64 w, one RNE step."""
    _check(lib().dckv_fit_to_bf16(w.data_ptr(), int(w.numel()), out.data_ptr(), _stream_ptr(stream)),
           "dckv_fit_to_bf16")


def dckv_fit_scales_accumulate(handle, rows, token_ids, seq_offsets, abs_sum, status, workspace, stream=None):
    """abs_sum int64 [2049] (device), accumulated into."""
    a, ptr, b = _offs(seq_offsets)
    _check(lib().dckv_fit_scales_accumulate(handle, rows.data_ptr(), _ptr(token_ids), ptr, b, abs_sum.data_ptr(),
                                            status.data_ptr(), workspace.data_ptr(),
                                            workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "dckv_fit_scales_accumulate")


def dckv_fit_scales_finish(handle, abs_sum, laplace_b, stream=None):
    _check(lib().dckv_fit_scales_finish(handle, abs_sum.data_ptr(), laplace_b.data_ptr(), _stream_ptr(stream)),
           "dckv_fit_scales_finish")


# ---------------------------------------------------- paged cache and attention (dckv_cache.h)
# These calls run once per layer and step, so the checks below read each tensor's properties once.
_CODES = {}  # torch types by element type code, filled on first use


def _bad(what):
    raise DckvError(DCKV_EINVAL, what)


def _dtype_code(t):
    if not _CODES:
        import torch

        _CODES.update({torch.bfloat16: DCKV_BF16, torch.float16: DCKV_FP16, torch.float32: DCKV_FP32,
                       torch.int32: "int32"})
    code = _CODES.get(t.dtype)
    if code is None:
        _bad(f"type {t.dtype} is not supported")
    return code


def _on(device, name, t):
    """t's strides, having checked that it sits on that CUDA device and that its last dimension is
    contiguous."""
    st = t.stride()
    if t.get_device() != device or device < 0:
        _bad(f"{name} is on {t.device}, not on cuda:{max(device, 0)}")
    if st[-1] != 1 and t.shape[-1] > 1:
        _bad(f"the last dimension of {name} must be contiguous")
    return st


def _int32_on(device, name, t):
    if t.get_device() != device or device < 0:
        _bad(f"{name} is on {t.device}, not on cuda:{max(device, 0)}")
    if _CODES.get(t.dtype) != "int32" and _dtype_code(t) != "int32":
        _bad(f"{name} must be int32, not {t.dtype}")
    if not t.is_contiguous():
        _bad(f"{name} must be contiguous")
    return t.data_ptr()


_raw_stream = None


def _device_stream(device, stream):
    """The given stream, or the current one of that device (not of the current device)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch

        # the handle without a Stream object around it, where this torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def rope_spec(rotary_dim, layout="half", base=1.0e7, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0,
              magnitude=1.0) -> RopeSpec:
    """A rotation (dckv_rope_init): layout "half" or "interleaved"; scaling "none", "linear",
    "ntk" or "parts".  The codec's own is rope_spec(256)."""
    for what, name, known in (("layout", layout, ROPE_LAYOUTS), ("scaling", scaling, ROPE_SCALINGS)):
        if name not in known:
            _bad(f"unknown rotary {what} {name!r}")
    s = RopeSpec()
    _check(lib().dckv_rope_init(ctypes.byref(s), int(rotary_dim), ROPE_LAYOUTS[layout], float(base),
                                ROPE_SCALINGS[scaling], float(factor), float(original_len), float(low), float(high),
                                float(magnitude)), "dckv_rope_init")
    return s


def dckv_rope(spec, x, positions, out, mode="forward", stream=None):
    """Rotates x [n, heads, dim] (bf16, fp16 or fp32) by positions int32 [n] into out (which may
    be x).  mode "forward", "gradient" (the transpose) or "inverse"."""
    shape = x.shape
    if len(shape) != 3 or out.shape != shape or positions.dim() != 1 or len(positions) != shape[0]:
        _bad("x and out must be [n, heads, dim] alike and positions [n]")
    dt = x.dtype
    code = _CODES.get(dt)
    if code is None:
        code = _dtype_code(x)
    if out.dtype is not dt or code == "int32":
        _bad("x and out must have one type, bf16, fp16 or fp32")
    m = ROPE_MODES.get(mode)
    if m is None:
        _bad(f"unknown rotary mode {mode!r}")
    dev = x.get_device()
    xs, os_ = _on(dev, "x", x), _on(dev, "out", out)
    pos = _int32_on(dev, "positions", positions)
    if shape[0] == 0:
        return out
    a = _RopeArgs(x.data_ptr(), out.data_ptr(), xs[0], xs[1], os_[0], os_[1], *shape, pos, code, dev)
    r = lib().dckv_rope(ctypes.byref(spec), m, ctypes.byref(a), _device_stream(dev, stream))
    if r:
        _check(r, "dckv_rope")
    return out


def kv_pool(k, v) -> KvPool:
    """Describes page pools k, v [layers, pages, rows, heads, dim] (or one layer's four
    dimensions), any strides with a contiguous last dimension.  Keeps the tensors alive."""
    if k.dim() == 4:
        k, v = k[None], v[None]
    if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype:
        _bad("k and v must be [layers, pages, rows, heads, dim] alike")
    dev, code = k.get_device(), _dtype_code(k)
    ks, vs = _on(dev, "k", k), _on(dev, "v", v)
    if code not in (DCKV_BF16, DCKV_FP16):
        _bad("pool type must be bf16 or fp16")
    L, pages, rows, heads, dim = k.shape
    p = KvPool(k.data_ptr(), v.data_ptr(), dev, code, L, heads, dim, rows, pages, *ks[:4], *vs[:4])
    p.tensors = (k, v)
    # what the calls below compare with and pass on (a ctypes field is slower to read; a byref kept here
    # would hold p, which holds it: the tensors would live until a collection of cycles)
    p.dev, p.dt, p.kv_shape, p.dim, p.ref = dev, k.dtype, (L, heads, dim), dim, ctypes.addressof(p)
    return p


def cache_batch(offsets, kv_lens, page_table, max_new) -> CacheBatch:
    """Describes the sequences of a call: int32 offsets [batch + 1], kv_lens [batch] and
    page_table [batch, pages] on the pool's device; max_new bounds any sequence's new tokens.
    Keeps the tensors alive; their contents may change between calls (and graph replays: keep the
    batch as long as a graph that was captured with it)."""
    if kv_lens.dim() != 1 or offsets.shape != (kv_lens.shape[0] + 1,) or page_table.dim() != 2 or \
            page_table.shape[0] != kv_lens.shape[0]:
        _bad("offsets, kv_lens and page_table must be [batch + 1], [batch] and [batch, pages]")
    dev = offsets.get_device()
    st = _on(dev, "page_table", page_table)
    if _dtype_code(page_table) != "int32":
        _bad("page_table must be int32")
    b = CacheBatch(kv_lens.shape[0], int(max_new), page_table.shape[1], 0, _int32_on(dev, "offsets", offsets),
                   _int32_on(dev, "kv_lens", kv_lens), page_table.data_ptr(), st[0])
    b.tensors = (offsets, kv_lens, page_table)
    b.dev, b.ref = dev, ctypes.addressof(b)
    return b


def _same_device(pool, batch, status):
    if batch.dev != pool.dev:
        _bad(f"the batch is on cuda:{batch.dev}, the pool on cuda:{pool.dev}")
    return _int32_on(pool.dev, "status", status)


def dckv_cache_append(pool, batch, k, v, status, rope=None, positions=None, q=None, q_out=None, stream=None):
    """k, v [layers, n, heads, dim] (or one layer's three dimensions) into the pages, keys rotated
    by `rope` if given; q [n, q heads, dim] rotated into q_out beside them."""
    if k.dim() == 3:
        k, v = k[None], v[None]
    shape, dev, dt = k.shape, pool.dev, pool.dt
    if len(shape) != 4 or v.shape != shape:
        _bad("k and v must be [layers, n, heads, dim] of the pool")
    layers, n, heads, dim = shape
    if (layers, heads, dim) != pool.kv_shape:
        _bad("k and v must be [layers, n, heads, dim] of the pool")
    if k.dtype is not dt or v.dtype is not dt:
        _bad("k and v must have the pool's type")
    st = _same_device(pool, batch, status)
    ks, vs = _on(dev, "k", k), _on(dev, "v", v)
    qp = op = pos = None
    qs = os_ = (0, 0)
    hq = 0
    if q is not None:
        qshape = q.shape
        if q_out is None or len(qshape) != 3 or q_out.shape != qshape:
            _bad("q and q_out must be [n, q heads, dim]")
        nq, hq, dq = qshape
        if nq != n or dq != dim:
            _bad("q and q_out must be [n, q heads, dim]")
        if q.dtype is not dt or q_out.dtype is not dt:
            _bad("q and q_out must have the pool's type")
        qs, os_ = _on(dev, "q", q), _on(dev, "q_out", q_out)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        _bad("q_out without q")
    if positions is not None:
        if positions.shape != (n,):
            _bad("positions must be [n]")
        pos = _int32_on(dev, "positions", positions)
    if n == 0:
        return
    a = _AppendArgs(k.data_ptr(), v.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], qp, op, qs[0], qs[1], os_[0],
                    os_[1], n, hq, 0, pos)
    r = lib().dckv_cache_append(pool.ref, batch.ref, None if rope is None else ctypes.byref(rope), ctypes.byref(a), st,
                                _device_stream(dev, stream))
    if r:
        _check(r, "dckv_cache_append")


def dckv_cache_rows(pool, batch, rows, status, rope=None, positions=None, stream=None):
    """The sequences' first slots as rows [n, layers * 2 * heads * dim], keys rotated back by
    `rope` if given."""
    L, H, dim = pool.kv_shape
    if rows.dim() != 2 or rows.shape[1] != 2 * L * H * dim:
        _bad("rows must be [n, layers * 2 * heads * dim]")
    if rows.dtype is not pool.dt:
        _bad("rows must have the pool's type")
    st = _same_device(pool, batch, status)
    rs = _on(pool.dev, "rows", rows)
    n, pos = rows.shape[0], None
    if positions is not None:
        if positions.shape != (n,):
            _bad("positions must be [n]")
        pos = _int32_on(pool.dev, "positions", positions)
    if n == 0:
        return rows
    r = lib().dckv_cache_rows(pool.ref, batch.ref, None if rope is None else ctypes.byref(rope), rows.data_ptr(), rs[0],
                              n, pos, st, _device_stream(pool.dev, stream))
    if r:
        _check(r, "dckv_cache_rows")
    return rows


def dckv_attention_workspace_bytes(pool, batch, n_q_heads) -> int:
    n = int(lib().dckv_attention_workspace_bytes(pool.ref, batch.ref, int(n_q_heads)))
    if n == 0:
        _bad(f"dckv_attention_workspace_bytes ({last_error()})")
    return n


def dckv_attention(pool, layer, batch, q, out, status, workspace, scale=None, causal=True, lse=None, stream=None):
    """Attention of q [n, q heads, dim] over the sequences' slots in `layer` into out (same shape)
    and, if given, lse fp32 [n, q heads].  scale: dim ** -0.5 unless given."""
    shape, dev, dt = q.shape, pool.dev, pool.dt
    if len(shape) != 3 or out.shape != shape:
        _bad("q and out must be [n, q heads, dim]")
    n, hq, dim = shape
    if dim != pool.dim:
        _bad("q and out must be [n, q heads, dim] of the pool")
    if q.dtype is not dt or out.dtype is not dt:
        _bad("q and out must have the pool's type")
    st = _same_device(pool, batch, status)
    qs, os_ = _on(dev, "q", q), _on(dev, "out", out)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _bad("the workspace must be contiguous, on the pool's device")
    lp = None
    if lse is not None:
        if lse.shape != shape[:2] or _dtype_code(lse) != DCKV_FP32 or lse.get_device() != dev or \
                not lse.is_contiguous():
            _bad("lse must be contiguous fp32 [n, q heads] on the pool's device")
        lp = lse.data_ptr()
    if n == 0:
        return out
    a = _AttentionArgs(q.data_ptr(), out.data_ptr(), lp, qs[0], qs[1], os_[0], os_[1], n, hq, int(layer),
                       1 if causal else 0, dim ** -0.5 if scale is None else float(scale))
    r = lib().dckv_attention(pool.ref, batch.ref, ctypes.byref(a), st, workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _device_stream(dev, stream))
    if r:
        _check(r, "dckv_attention")
    return out


def upload_params(codec, device="cuda"):
    """Device tensors for dckv_codec_create from an object with numpy attributes mu, basis,
    w1, w2, delta, laplace_b (float32), embed, w_even, w_odd (bf16 bits as uint16) and,
    optionally, v1, v2 (float32)."""
    import torch

    out = {}
    for k in ("mu", "basis", "w1", "w2", "delta", "laplace_b", "v1", "v2"):
        v = getattr(codec, k, None)
        out[k] = None if v is None else torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(device)
    for k in ("embed", "w_even", "w_odd"):
        v = getattr(codec, k)
        if v is None:
            out[k] = None
            continue
        a = np.ascontiguousarray(v, np.uint16).view(np.int16)
        out[k] = torch.from_numpy(a).to(device).view(torch.bfloat16)
    return out


class Codec:
    """Owns a codec handle plus reusable workspace / blob / output buffers (torch)."""

    def __init__(self, params: dict, device: int = 0, chunk_rows: int = 0):
        import torch

        self.torch = torch
        self.device = torch.device("cuda", device)
        self.handle = dckv_codec_create(params, device, chunk_rows)
        self.params = params  # the library copies what it needs; kept alive for clarity
        self._ws = None
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.blob_size = torch.zeros(1, dtype=torch.int64, device=self.device)

    @property
    def k_eff(self):
        return dckv_codec_k_eff(self.handle)

    def workspace(self, seq_offsets):
        n = dckv_workspace_bytes(self.handle, seq_offsets)
        if n == 0:
            raise DckvError(DCKV_EINVAL, "dckv_workspace_bytes")
        if self._ws is None or self._ws.numel() < n:
            self._ws = self.torch.empty(n, dtype=self.torch.uint8, device=self.device)
        return self._ws

    def encode(self, rows, token_ids, seq_offsets, blob=None, stream=None):
        if blob is None:
            blob = self.torch.empty(dckv_blob_bound(self.handle, seq_offsets), dtype=self.torch.uint8,
                                    device=self.device)
        ws = self.workspace(seq_offsets)
        dckv_encode(self.handle, rows, token_ids, seq_offsets, blob, self.blob_size, self.status, ws, stream)
        return blob

    def decode(self, blob, blob_bytes, token_ids, seq_offsets, k_out=None, v_out=None, stream=None):
        n_tok = int(np.asarray(seq_offsets)[-1])
        if k_out is None:
            k_out = self.torch.empty((6, n_tok, 2, 256), dtype=self.torch.bfloat16, device=self.device)
        if v_out is None:
            v_out = self.torch.empty((6, n_tok, 2, 256), dtype=self.torch.bfloat16, device=self.device)
        ws = self.workspace(seq_offsets)
        dckv_decode(self.handle, blob, blob_bytes, token_ids, seq_offsets, k_out, v_out, self.status, ws, stream)
        return k_out, v_out

    def workspace_codes(self, seq_offsets, which: int = 0, rows=None):
        """Codes the last encode (which=0: q32, int32) or decode (which=1: q16, fp16 as float32)
        left in the workspace, as numpy [rows][2048] by component (the library keeps kept
        components only, compact; dropped components are 0).  rows: coded-row indices (all
        if None)."""
        torch = self.torch
        v = dckv_ws_offsets(self.handle, seq_offsets, which)
        n, k = v["n_rows"], self.k_eff
        if which == 0:
            c = self._ws[v["q32"]: v["q32"] + 4 * n * 2048].view(torch.int32).reshape(n, 2048)
        else:
            c = self._ws[v["q16"]: v["q16"] + 2 * n * 2048].view(torch.float16).reshape(n, 2048).float()
        if rows is not None:
            c = c[torch.as_tensor(np.asarray(rows, np.int64), device=c.device)]
        c = c[:, :k].cpu().numpy()
        keep = dckv_codec_export(self.handle)[2].astype(bool)
        out = np.zeros((c.shape[0], 2048), c.dtype)
        out[:, keep] = c
        return out

    def close(self):
        if self.handle is not None:
            dckv_codec_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedCache:
    """A paged cache beside a codec: owns the page pools, a list of free pages and each
    sequence's pages and length (on the host), and makes the calls of dckv_cache.h on them.

    A step: ``batch = cache.extend(seqs, counts)`` gives the sequences room for their new tokens;
    then, layer by layer, ``cache.append(batch, k, v, q=q, q_out=q_rot, layer=layer)`` and
    ``cache.attend(layer, batch, q_rot)`` (without `layer`, append takes all layers' at once).
    ``restore`` and ``store`` move whole prompts between blobs of a Codec and the pages.  Everything
    runs on the current stream of the cache's device; calls on one cache that overlap in time (two
    streams) need ordering between them."""

    def __init__(self, n_pages, page_size=64, n_layers=6, n_kv_heads=2, head_dim=256, dtype=None, device=0, rope=None):
        import torch

        self.torch = torch
        self.device = torch.device("cuda", device)
        shape = (n_layers, n_pages, page_size, n_kv_heads, head_dim)
        self.k = torch.empty(shape, dtype=dtype or torch.bfloat16, device=self.device)
        self.v = torch.empty_like(self.k)
        self.pool = kv_pool(self.k, self.v)
        self._layers = [kv_pool(self.k[l], self.v[l]) for l in range(n_layers)]
        self.rope = rope_spec(head_dim) if rope is None else rope
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._free = list(range(n_pages - 1, -1, -1))
        self._pages, self._len = {}, {}
        self._odd = {}  # sequences with keys that are not rotated at their slots: the first such slot
        self._ws = []  # growing sizes, none given back: a captured graph may write any of them
        self._next = 0

    def add(self) -> int:
        """A new, empty sequence."""
        s = self._next
        self._next += 1
        self._pages[s], self._len[s] = [], 0
        return s

    def length(self, seq) -> int:
        return self._len[seq]

    def drop(self, seq):
        """Gives a sequence's pages back (work already queued on the current stream still reads
        them in order)."""
        self._free += reversed(self._pages.pop(seq))
        del self._len[seq]
        self._odd.pop(seq, None)

    def _batch(self, seqs, counts):
        torch = self.torch
        width = max(1, max(len(self._pages[s]) for s in seqs))
        table = np.zeros((len(seqs), width), np.int32)
        for i, s in enumerate(seqs):
            table[i, : len(self._pages[s])] = self._pages[s]
        offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        lens = np.array([self._len[s] for s in seqs], np.int32)
        dev = [torch.from_numpy(a).to(self.device) for a in (offs, lens, table)]
        batch = cache_batch(*dev, max(1, max(counts)))
        batch.firsts = {s: self._len[s] - c for s, c in zip(seqs, counts) if c}  # slots of an append's first tokens
        return batch

    def extend(self, seqs, counts) -> CacheBatch:
        """Room for counts[i] more tokens of seqs[i]; the batch of a call that appends them."""
        seqs, counts = list(seqs), [int(c) for c in counts]
        if not seqs or len(seqs) != len(counts) or len(set(seqs)) != len(seqs) or min(counts) < 0:
            _bad("extend takes different sequences and one count of at least 0 for each")
        rows = self.pool.page_size
        need = [-(-(self._len[s] + c) // rows) - len(self._pages[s]) for s, c in zip(seqs, counts)]
        if sum(need) > len(self._free):
            raise DckvError(DCKV_ECAPACITY, f"{sum(need)} pages needed, {len(self._free)} free")
        for s, c, m in zip(seqs, counts, need):
            self._pages[s] += [self._free.pop() for _ in range(m)]
            self._len[s] += c
        try:
            return self._batch(seqs, counts)
        except BaseException:
            for s, c, m in reversed(list(zip(seqs, counts, need))):
                self._free += [self._pages[s].pop() for _ in range(m)]
                self._len[s] -= c
            raise

    def append(self, batch, k, v, q=None, q_out=None, rotate=True, positions=None, layer=None):
        """dckv_cache_append with the cache's rotation (rotate=False: keys come rotated): k and v of all
        layers [layers, n, heads, dim] or, with `layer`, of that one [n, heads, dim].  Keys that it
        did not rotate at their slots (rotate=False, or positions given) come back by `rows` and
        `store` only where these are given positions; a replayed graph is judged by its capture."""
        if layer is not None and not 0 <= layer < self.pool.n_layers:
            _bad(f"layer {layer} out of range")
        dckv_cache_append(self.pool if layer is None else self._layers[layer], batch, k, v, self.status,
                          rope=self.rope if rotate else None, positions=positions, q=q, q_out=q_out)
        if not rotate or positions is not None:
            # a batch that extend did not make does not say whose slots it writes
            for s, first in getattr(batch, "firsts", dict.fromkeys(self._len, 0)).items():
                if s in self._len:
                    self._odd[s] = min(first, self._odd.get(s, first))

    def attend(self, layer, batch, q, out=None, scale=None, causal=True, lse=None):
        """dckv_attention on the cache's workspace; out is a new tensor unless given.  Keep the cache as
        long as a graph that was captured with it."""
        need = dckv_attention_workspace_bytes(self.pool, batch, q.shape[1])
        ws = next((w for w in self._ws if w.numel() >= need), None)
        if ws is None:
            ws = self.torch.empty(need, dtype=self.torch.uint8, device=self.device)
            self._ws.append(ws)
        if out is None:
            out = self.torch.empty(q.shape, dtype=q.dtype, device=q.device)
        return dckv_attention(self.pool, layer, batch, q, out, self.status, ws, scale=scale, causal=causal, lse=lse)

    def _check_codec(self, codec, token_ids, n_tokens):
        """The codec's calls take rows of its own shape and type, and the tokens' ids, on trust."""
        p = self.pool
        if (p.n_layers, p.n_kv_heads, p.head_dim) != (6, 2, 256) or self.k.dtype != self.torch.bfloat16:
            _bad("a codec's prompts need a cache of 6 layers, 2 KV heads and 256 dims in bf16")
        if codec.device != self.device:
            _bad(f"the codec is on {codec.device}, the cache on {self.device}")
        if token_ids is not None and (token_ids.dtype != self.torch.int32 or token_ids.device != self.device or
                                      not token_ids.is_contiguous() or token_ids.numel() < n_tokens):
            _bad(f"token ids must be {n_tokens} contiguous int32 on {self.device}")

    def restore(self, codec, blob, blob_bytes, token_ids, seq_offsets):
        """Decodes a blob's prompts into new sequences of the pages (the decoder rotates the keys
        as the codec's own rotation does).  The cache must have the codec's layers, heads, dims, type,
        device and rotation.  Returns the sequences; codec.status has the decoder's status."""
        counts = [int(c) for c in np.diff(np.asarray(seq_offsets, np.int64))]
        self._check_codec(codec, token_ids, sum(counts))
        if bytes(self.rope) != bytes(rope_spec(256)):
            _bad("the cache's rotation is not the codec's (rope_spec(256)), which decoded keys come with")
        if not counts or min(counts) < 1:
            _bad("restore takes prompts of at least one token")
        stream = self.torch.cuda.current_stream(self.device)
        k, v = codec.decode(blob, blob_bytes, token_ids, seq_offsets, stream=stream)
        seqs = [self.add() for _ in counts]
        try:
            dckv_cache_append(self.pool, self.extend(seqs, counts), k, v, self.status)
        except BaseException:
            for s in seqs:
                self.drop(s)
            raise
        return seqs

    def _counts(self, seqs, counts):
        lens = [self._len[s] for s in seqs]
        counts = lens if counts is None else [int(c) for c in counts]
        if not lens or len(counts) != len(lens) or any(not 0 <= c <= n for c, n in zip(counts, lens)):
            _bad(f"counts {counts} are not within the sequences' lengths {lens}")
        return counts

    def rows(self, seqs, counts=None, positions=None):
        """The first counts[i] (default: all) tokens of each sequence as pre-RoPE rows, and their
        offsets: the arguments of Codec.encode.  Keys are rotated back from their slots or, if given,
        from positions (device int32, one per row); a key that `append` did not rotate at its slot
        needs them."""
        counts = self._counts(seqs, counts)
        for s, c in zip(seqs, counts):
            if positions is None and c > self._odd.get(s, c):
                _bad(f"keys of sequence {s} are not rotated at their slots from slot {self._odd[s]} on: "
                     "their rows need positions")
        n = sum(counts)
        rows = self.torch.empty((n, 2 * self.pool.n_layers * self.pool.n_kv_heads * self.pool.head_dim),
                                dtype=self.k.dtype, device=self.device)
        dckv_cache_rows(self.pool, self._batch(seqs, counts), rows, self.status, rope=self.rope, positions=positions)
        return rows, np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)

    def store(self, codec, seqs, token_ids, counts=None, positions=None):
        """Encodes the sequences' first tokens with a codec: (blob, seq_offsets); codec.blob_size
        and codec.status as after Codec.encode.  The cache must have the codec's layers, heads, dims,
        type and device; token_ids has an id for each of those tokens (None for a codec that takes
        none); positions as for `rows`."""
        counts = self._counts(seqs, counts)
        self._check_codec(codec, token_ids, sum(counts))
        rows, offsets = self.rows(seqs, counts, positions)
        stream = self.torch.cuda.current_stream(self.device)
        return codec.encode(rows, token_ids, offsets, stream=stream), offsets
