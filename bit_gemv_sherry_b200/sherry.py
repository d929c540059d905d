"""Python binding of libsherry.so (argument marshalling only).

Every step of the path runs in the library's CUDA kernels; this module only
checks tensor properties, passes raw device pointers and the current CUDA
stream, and turns status codes into exceptions.  PyTorch provides device
memory and streams.  There is no CPU fallback: if the library cannot be
loaded, importing the functions raises.
"""
import ctypes
import functools
import os
import struct

import torch

from . import build as _build

_lib = None

STATUS = {
    0: "SHERRY_OK", 1: "SHERRY_ERR_NULL", 2: "SHERRY_ERR_SHAPE", 3: "SHERRY_ERR_ALIGN",
    4: "SHERRY_ERR_UNSUPPORTED", 5: "SHERRY_ERR_CUDA", 6: "SHERRY_ERR_TIMEOUT",
    7: "SHERRY_ERR_WORKSPACE", 8: "SHERRY_ERR_INDEX",
}
TILE_K = 128
MAX_GEMV_BATCH = 16
MAX_GROUP = 128


class SherryError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = "%s: %s (%s)" % (where, STATUS.get(status, status),
                               lib().sherry_status_string(status).decode())
        if status == 5:
            msg += ": " + lib().sherry_last_error().decode()
        super().__init__(msg)


class PackDesc(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class GemvDesc(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class F32Desc(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("u", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("k_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("T", ctypes.c_int64),
                ("Hq", ctypes.c_int), ("Hk", ctypes.c_int), ("D", ctypes.c_int), ("R", ctypes.c_int),
                ("in_type", ctypes.c_int), ("out_type", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("eps", ctypes.c_float)]


class Kv4Args(ctypes.Structure):
    _fields_ = [("cache", ctypes.c_void_p), ("pages", ctypes.c_int64), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("page_table", ctypes.c_void_p), ("width", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("ctx_lens", ctypes.c_void_p),
                ("cu_q", ctypes.c_void_p), ("B", ctypes.c_int64), ("T", ctypes.c_int64)]


def library_path():
    return _build.LIB


def lib():
    """Load libsherry.so (built in-tree).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        raise RuntimeError("libsherry.so not built: run `python -m bit_gemv_sherry_b200.build` "
                           "(expected at %s)" % path)
    L = ctypes.CDLL(path)
    p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "sherry_packed_bytes": ([i64, i64], sz),
        "sherry_pack": ([p, i64, i64, p, p, p], i32),
        "sherry_pack_grouped": ([p, i32, p], i32),
        "sherry_gemv_workspace_bytes": ([i64, i64, i32], sz),
        "sherry_gemv": ([p, p, p, p, i64, i64, i32, p, sz, p], i32),
        "sherry_gemv_acc": ([p, p, p, i64, i64, i32, p, sz, p], i32),
        "sherry_gemv_static": ([p, p, p, p, i64, i64, i32, p], i32),
        "sherry_quantize_act": ([p, i64, i64, p, p, p], i32),
        "sherry_gemv_bf16_workspace_bytes": ([i64, i64, i32], sz),
        "sherry_gemv_bf16": ([p, p, p, p, i64, i64, i32, p, sz, p], i32),
        "sherry_gemv_bf16_grouped": ([p, i32, i32, p, sz, p], i32),
        "sherry_quantize_f32": ([p, i64, i64, p, p, p], i32),
        "sherry_quantize_swiglu": ([p, p, i64, i64, p, p, p], i32),
        "sherry_gemv_f32_workspace_bytes": ([i64, i64, i32], sz),
        "sherry_gemv_f32": ([p, p, p, p, i64, i64, i32, p, sz, p], i32),
        "sherry_gemv_swiglu": ([p, p, p, p, p, i64, i64, i32, p, sz, p], i32),
        "sherry_gemv_f32_grouped": ([p, i32, i32, p, sz, p], i32),
        "sherry_gemv_grouped": ([p, i32, i32, p, sz, p], i32),
        "sherry_gemv_prepare": ([p, i32, i32, p, sz, p], i32),
        "sherry_gemv_run": ([p, i32, i32, p, sz, p], i32),
        "sherry_gemm": ([p, p, p, p, i64, i64, i64, p], i32),
        "sherry_gemm_acc": ([p, p, p, i64, i64, i64, p], i32),
        "sherry_cmp_packed_bytes": ([i32, i64, i64], sz),
        "sherry_cmp_workspace_bytes": ([i32, i64, i64, i32], sz),
        "sherry_cmp_transcode": ([i32, p, i64, i64, p, p], i32),
        "sherry_cmp_gemv_grouped": ([i32, p, i32, i32, p, sz, p], i32),
        "sherry_cmp_gemv_acc": ([i32, p, p, p, i64, i64, i32, p, sz, p], i32),
        "sherry_qk_norm_rope": ([p, p], i32),
        "sherry_kv4_bytes": ([i64, i32, i32], sz),
        "sherry_kv4_write": ([p, p, p, i32, i64, i64, p], i32),
        "sherry_kv4_read": ([p, p, p, i32, i64, i64, p], i32),
        "sherry_attn_kv4_workspace_bytes": ([i64, i32, i32], sz),
        "sherry_attn_kv4": ([p, p, i64, p, i64, i32, i64, ctypes.c_float, p, sz, p], i32),
        "sherry_probe_mma_i8": ([i32, p, p], i32),
        "sherry_device_error": ([], i32),
        "sherry_set_wait_limit": ([i64], i32),
        "sherry_status_string": ([i32], ctypes.c_char_p),
        "sherry_last_error": ([], ctypes.c_char_p),
        "sherry_version": ([], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _check(status, where):
    if status != 0:
        raise SherryError(status, where)


# The raw handle of a device's current stream.  torch's private accessor skips
# building a Stream object (about 2 us per call on the host); the public one is
# the fallback.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device):
    if _raw_stream is not None:
        idx = device.index if device.index is not None else torch.cuda.current_device()
        return _raw_stream(idx)
    return torch.cuda.current_stream(device).cuda_stream


def _stream(t):
    return ctypes.c_void_p(_stream_handle(t.device))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


_workspaces = {}


def workspace(nbytes, device):
    """A cached device scratch buffer of at least `nbytes` for (device, current stream)."""
    device = torch.device(device)
    key = (device.index, _stream_handle(device))
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=device)
        _workspaces[key] = buf
    return buf


def packed_bytes(N, K):
    return int(lib().sherry_packed_bytes(N, K))


def gemv_workspace_bytes(N, K, B):
    return int(lib().sherry_gemv_workspace_bytes(N, K, B))


GROUP = 32  # rows per group of the code layout


def codes_shape(N, K):
    """Shape of the int32 tensor holding the codes of an N x K matrix."""
    return ((N + GROUP - 1) // GROUP, K // TILE_K, 5, GROUP)


def pack(w, codes=None, scales=None):
    """w: float32 [N, K] CUDA -> (codes int32 [ceil(N/32), K/128, 5, 32] holding the
    uint32 words, scales float32 [N])."""
    _need(w, torch.float32, "w")
    N, K = w.shape
    if codes is None:
        codes = torch.empty(codes_shape(N, max(K, TILE_K)), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty(N, dtype=torch.float32, device=w.device)
    _check(lib().sherry_pack(_ptr(w), N, K, _ptr(codes), _ptr(scales), _stream(w)), "sherry_pack")
    return codes, scales


class GroupedPack:
    """Pre-marshalled grouped pack (sherry_pack_grouped): items are
    (w float32 [N, K], codes, scales) with codes/scales shaped as pack() makes them."""

    def __init__(self, items):
        n = len(items)
        self.descs = (PackDesc * n)()
        for i, (w, codes, scales) in enumerate(items):
            _need(w, torch.float32, "w")
            N, K = w.shape
            _need(scales, torch.float32, "scales")
            if tuple(codes.shape) != codes_shape(N, max(K, TILE_K)) or scales.numel() != N:
                raise ValueError("codes/scales do not match w of shape %s" % (tuple(w.shape),))
            self.descs[i] = PackDesc(w.data_ptr(), codes.data_ptr(), scales.data_ptr(), N, K)
        self.items = items
        self.n = n
        self.device = items[0][0].device

    def __call__(self, stream=None):
        s = ctypes.c_void_p(stream if stream is not None
                            else _stream_handle(self.device))
        _check(lib().sherry_pack_grouped(ctypes.cast(self.descs, ctypes.c_void_p), self.n, s),
               "sherry_pack_grouped")


def pack_grouped(ws):
    """Packs a list of float32 [N, K] CUDA matrices in one launch; returns
    [(codes, scales)] as pack() would."""
    outs = [(torch.empty(codes_shape(w.shape[0], max(w.shape[1], TILE_K)), dtype=torch.int32,
                         device=w.device),
             torch.empty(w.shape[0], dtype=torch.float32, device=w.device)) for w in ws]
    GroupedPack([(w, c, s) for w, (c, s) in zip(ws, outs)])()
    return outs


def _codes_shape(codes, N):
    _need(codes, torch.int32, "codes")
    if codes.dim() != 4 or codes.shape[2] != 5 or codes.shape[3] != GROUP:
        raise ValueError("codes must have shape [ceil(N/32), K/128, 5, 32]")
    if codes.shape[0] != (N + GROUP - 1) // GROUP:
        raise ValueError("codes hold %d row groups, N = %d needs %d"
                         % (codes.shape[0], N, (N + GROUP - 1) // GROUP))
    return N, codes.shape[1] * TILE_K


def gemv(codes, scales, x, y=None, ws=None):
    """y[B, N] = scales * (W . x^T); x int8 [B, K] (or [K])."""
    _need(scales, torch.float32, "scales")
    N, K = _codes_shape(codes, scales.numel())
    _need(x, torch.int8, "x")
    x2 = x.view(1, -1) if x.dim() == 1 else x
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, N), dtype=torch.float32, device=x.device)
    nb = gemv_workspace_bytes(N, K, B)
    ws = workspace(nb, x.device) if ws is None else ws
    _check(lib().sherry_gemv(_ptr(codes), _ptr(scales), _ptr(x2), _ptr(y), N, K, B, _ptr(ws),
                             ws.numel(), _stream(x)), "sherry_gemv")
    return y


STATIC_SCRATCH_BYTES = 4 << 20


def gemv_static(codes, scales, x, y=None):
    """As gemv, with the library's fixed scratch array instead of a workspace
    (sherry_gemv_static: the C call allocates nothing; y is allocated here
    only when not given)."""
    _need(scales, torch.float32, "scales")
    N, K = _codes_shape(codes, scales.numel())
    _need(x, torch.int8, "x")
    x2 = x.view(1, -1) if x.dim() == 1 else x
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, N), dtype=torch.float32, device=x.device)
    _check(lib().sherry_gemv_static(_ptr(codes), _ptr(scales), _ptr(x2), _ptr(y), N, K, B,
                                    _stream(x)), "sherry_gemv_static")
    return y


def gemv_acc(codes, x, N, acc=None, ws=None):
    """Exact int32 accumulators acc[B, N] = W . x^T."""
    N, K = _codes_shape(codes, N)
    _need(x, torch.int8, "x")
    x2 = x.view(1, -1) if x.dim() == 1 else x
    B = x2.shape[0]
    if acc is None:
        acc = torch.empty((B, N), dtype=torch.int32, device=x.device)
    nb = gemv_workspace_bytes(N, K, B)
    ws = workspace(nb, x.device) if ws is None else ws
    _check(lib().sherry_gemv_acc(_ptr(codes), _ptr(x2), _ptr(acc), N, K, B, _ptr(ws), ws.numel(),
                                 _stream(x)), "sherry_gemv_acc")
    return acc


def gemv_grouped(items, B, ws=None):
    """items: list of (codes, scales, x [B, K], y [B, N]); runs every GEMV in one pass."""
    n = len(items)
    descs = (GemvDesc * n)()
    total = 0
    dev = None
    for i, (codes, scales, x, y) in enumerate(items):
        _need(scales, torch.float32, "scales")
        N, K = _codes_shape(codes, scales.numel())
        _need(x, torch.int8, "x")
        _need(y, torch.float32, "y")
        descs[i] = GemvDesc(codes.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(), N, K)
        total += gemv_workspace_bytes(N, K, B)
        dev = x.device
    ws = workspace(total, dev) if ws is None else ws
    _check(lib().sherry_gemv_grouped(ctypes.cast(descs, ctypes.c_void_p), n, B, _ptr(ws),
                                     ws.numel(), _stream(items[0][2])), "sherry_gemv_grouped")


def quantize_act(x, q=None, s=None):
    """Per-token absmax int8 quantization of bf16 activations x [B, K]:
    returns (q int8 [B, K], s fp32 [B]) with x ~ s[:, None] * q."""
    _need(x, torch.bfloat16, "x")
    x2 = x.view(1, -1) if x.dim() == 1 else x
    B, K = x2.shape
    if q is None:
        q = torch.empty((B, K), dtype=torch.int8, device=x.device)
    if s is None:
        s = torch.empty((B,), dtype=torch.float32, device=x.device)
    _check(lib().sherry_quantize_act(_ptr(x2), B, K, _ptr(q), _ptr(s), _stream(x)),
           "sherry_quantize_act")
    return q, s


def gemv_bf16_workspace_bytes(N, K, B):
    return int(lib().sherry_gemv_bf16_workspace_bytes(N, K, B))


def gemv_bf16(codes, scales, x, y=None, ws=None):
    """y[B, N] = scales * s_x * (W . q^T) for bf16 activations x [B, K] quantized per token."""
    _need(scales, torch.float32, "scales")
    N, K = _codes_shape(codes, scales.numel())
    _need(x, torch.bfloat16, "x")
    x2 = x.view(1, -1) if x.dim() == 1 else x
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, N), dtype=torch.float32, device=x.device)
    nb = gemv_bf16_workspace_bytes(N, K, B)
    ws = workspace(nb, x.device) if ws is None else ws
    _check(lib().sherry_gemv_bf16(_ptr(codes), _ptr(scales), _ptr(x2), _ptr(y), N, K, B, _ptr(ws),
                                  ws.numel(), _stream(x)), "sherry_gemv_bf16")
    return y


def gemv_bf16_grouped(items, B, ws=None):
    """items: list of (codes, scales, x bf16 [B, K], y [B, N]); one pass over all GEMVs."""
    n = len(items)
    descs = (GemvDesc * n)()  # same field layout as sherry_gemv_bf16_desc
    total = 0
    dev = None
    for i, (codes, scales, x, y) in enumerate(items):
        _need(scales, torch.float32, "scales")
        N, K = _codes_shape(codes, scales.numel())
        _need(x, torch.bfloat16, "x")
        _need(y, torch.float32, "y")
        descs[i] = GemvDesc(codes.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(), N, K)
        total += gemv_bf16_workspace_bytes(N, K, B)
        dev = x.device
    ws = workspace(total, dev) if ws is None else ws
    _check(lib().sherry_gemv_bf16_grouped(ctypes.cast(descs, ctypes.c_void_p), n, B, _ptr(ws),
                                          ws.numel(), _stream(items[0][2])),
           "sherry_gemv_bf16_grouped")


def _rows(t, name):
    _need(t, torch.float32, name)
    return t.view(1, -1) if t.dim() == 1 else t


def quantize_f32(x, q=None, s=None):
    """Per-token absmax int8 quantization of fp32 activations x [B, K]
    (K a multiple of 128): returns (q int8 [B, K], s fp32 [B])."""
    x2 = _rows(x, "x")
    B, K = x2.shape
    q = torch.empty((B, K), dtype=torch.int8, device=x.device) if q is None else q
    s = torch.empty((B,), dtype=torch.float32, device=x.device) if s is None else s
    _check(lib().sherry_quantize_f32(_ptr(x2), B, K, _ptr(q), _ptr(s), _stream(x)),
           "sherry_quantize_f32")
    return q, s


def quantize_swiglu(g, u, q=None, s=None):
    """quantize_f32 of h = silu(g) * u, formed inside the front-end."""
    g2, u2 = _rows(g, "g"), _rows(u, "u")
    if g2.shape != u2.shape:
        raise ValueError("g and u differ in shape")
    B, K = g2.shape
    q = torch.empty((B, K), dtype=torch.int8, device=g.device) if q is None else q
    s = torch.empty((B,), dtype=torch.float32, device=g.device) if s is None else s
    _check(lib().sherry_quantize_swiglu(_ptr(g2), _ptr(u2), B, K, _ptr(q), _ptr(s), _stream(g)),
           "sherry_quantize_swiglu")
    return q, s


def gemv_f32_workspace_bytes(N, K, B):
    return int(lib().sherry_gemv_f32_workspace_bytes(N, K, B))


def gemv_f32(codes, scales, x, y=None, ws=None):
    """y[B, N] = scales * s_x * (W . q^T) for fp32 activations x [B, K] quantized per token."""
    _need(scales, torch.float32, "scales")
    N, K = _codes_shape(codes, scales.numel())
    x2 = _rows(x, "x")
    B = x2.shape[0]
    y = torch.empty((B, N), dtype=torch.float32, device=x.device) if y is None else y
    ws = workspace(gemv_f32_workspace_bytes(N, K, B), x.device) if ws is None else ws
    _check(lib().sherry_gemv_f32(_ptr(codes), _ptr(scales), _ptr(x2), _ptr(y), N, K, B, _ptr(ws),
                                 ws.numel(), _stream(x)), "sherry_gemv_f32")
    return y


def gemv_swiglu(codes, scales, g, u, y=None, ws=None):
    """gemv_f32 on h = silu(g) * u (the down projection of a gated MLP); g, u fp32 [B, K]."""
    _need(scales, torch.float32, "scales")
    N, K = _codes_shape(codes, scales.numel())
    g2, u2 = _rows(g, "g"), _rows(u, "u")
    if g2.shape != u2.shape:
        raise ValueError("g and u differ in shape")
    B = g2.shape[0]
    y = torch.empty((B, N), dtype=torch.float32, device=g.device) if y is None else y
    ws = workspace(gemv_f32_workspace_bytes(N, K, B), g.device) if ws is None else ws
    _check(lib().sherry_gemv_swiglu(_ptr(codes), _ptr(scales), _ptr(g2), _ptr(u2), _ptr(y), N, K, B,
                                    _ptr(ws), ws.numel(), _stream(g)), "sherry_gemv_swiglu")
    return y


class GroupedGemvF32:
    """Pre-marshalled grouped GEMV on fp32 activations (sherry_gemv_f32_grouped):
    items are (codes, scales, x fp32 [B, K], u fp32 [B, K] or None, y [B, N])."""

    def __init__(self, items, B, ws=None):
        n = len(items)
        self.descs = (F32Desc * n)()
        total = 0
        for i, (codes, scales, x, u, y) in enumerate(items):
            _need(scales, torch.float32, "scales")
            N, K = _codes_shape(codes, scales.numel())
            _need(x, torch.float32, "x")
            if u is not None:
                _need(u, torch.float32, "u")
            _need(y, torch.float32, "y")
            self.descs[i] = F32Desc(codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
                                    u.data_ptr() if u is not None else None, y.data_ptr(), N, K)
            total += gemv_f32_workspace_bytes(N, K, B)
        self.items = items
        dev = items[0][2].device
        self.ws = torch.empty(max(total, 256), dtype=torch.uint8, device=dev) if ws is None else ws
        self.args = (ctypes.cast(self.descs, ctypes.c_void_p), n, B, _ptr(self.ws),
                     self.ws.numel())
        self.device = dev

    def __call__(self, stream=None):
        s = ctypes.c_void_p(stream if stream is not None
                            else _stream_handle(self.device))
        _check(lib().sherry_gemv_f32_grouped(*self.args, s), "sherry_gemv_f32_grouped")


def gemv_f32_grouped(items, B, ws=None):
    """items: list of (codes, scales, x fp32 [B, K], u fp32 [B, K] or None, y [B, N])."""
    GroupedGemvF32(items, B, ws)()


class GroupedGemv:
    """Pre-marshalled grouped GEMV: descriptors and workspace are built once, and
    each call only passes them to the library (used where per-call Python cost
    matters, e.g. timing a decode step)."""

    def __init__(self, items, B, ws=None):
        n = len(items)
        self.descs = (GemvDesc * n)()
        total = 0
        for i, (codes, scales, x, y) in enumerate(items):
            _need(scales, torch.float32, "scales")
            N, K = _codes_shape(codes, scales.numel())
            _need(x, torch.int8, "x")
            _need(y, torch.float32, "y")
            self.descs[i] = GemvDesc(codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
                                     y.data_ptr(), N, K)
            total += gemv_workspace_bytes(N, K, B)
        self.items = items  # keep the tensors alive
        self.n, self.B = n, B
        dev = items[0][2].device
        self.ws = torch.empty(max(total, 256), dtype=torch.uint8, device=dev) if ws is None else ws
        self.args = (ctypes.cast(self.descs, ctypes.c_void_p), n, B, _ptr(self.ws),
                     self.ws.numel())
        self.device = dev

    def __call__(self, stream=None):
        s = ctypes.c_void_p(stream if stream is not None
                            else _stream_handle(self.device))
        _check(lib().sherry_gemv_grouped(*self.args, s), "sherry_gemv_grouped")

    def prepare(self, stream=None):
        s = ctypes.c_void_p(stream if stream is not None
                            else _stream_handle(self.device))
        _check(lib().sherry_gemv_prepare(*self.args, s), "sherry_gemv_prepare")

    def run(self, stream=None):
        s = ctypes.c_void_p(stream if stream is not None
                            else _stream_handle(self.device))
        _check(lib().sherry_gemv_run(*self.args, s), "sherry_gemv_run")


class GroupedGemvBf16:
    """Pre-marshalled grouped GEMV on bf16 activations (sherry_gemv_bf16_grouped):
    items are (codes, scales, x bf16 [B, K], y [B, N])."""

    def __init__(self, items, B, ws=None):
        n = len(items)
        self.descs = (GemvDesc * n)()  # same field layout as sherry_gemv_bf16_desc
        total = 0
        for i, (codes, scales, x, y) in enumerate(items):
            _need(scales, torch.float32, "scales")
            N, K = _codes_shape(codes, scales.numel())
            _need(x, torch.bfloat16, "x")
            _need(y, torch.float32, "y")
            self.descs[i] = GemvDesc(codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
                                     y.data_ptr(), N, K)
            total += gemv_bf16_workspace_bytes(N, K, B)
        self.items = items
        dev = items[0][2].device
        self.ws = torch.empty(max(total, 256), dtype=torch.uint8, device=dev) if ws is None else ws
        self.args = (ctypes.cast(self.descs, ctypes.c_void_p), n, B, _ptr(self.ws),
                     self.ws.numel())
        self.device = dev

    def __call__(self, stream=None):
        s = ctypes.c_void_p(stream if stream is not None
                            else _stream_handle(self.device))
        _check(lib().sherry_gemv_bf16_grouped(*self.args, s), "sherry_gemv_bf16_grouped")


def gemm(codes, scales, x, y=None):
    """y[M, N] = scales * (x . W^T); x int8 [M, K]."""
    _need(scales, torch.float32, "scales")
    N, K = _codes_shape(codes, scales.numel())
    _need(x, torch.int8, "x")
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().sherry_gemm(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), M, N, K, _stream(x)),
           "sherry_gemm")
    return y


def gemm_acc(codes, x, N, acc=None):
    """Exact int32 accumulators acc[M, N] = x . W^T."""
    N, K = _codes_shape(codes, N)
    _need(x, torch.int8, "x")
    M = x.shape[0]
    if acc is None:
        acc = torch.empty((M, N), dtype=torch.int32, device=x.device)
    _check(lib().sherry_gemm_acc(_ptr(codes), _ptr(x), _ptr(acc), M, N, K, _stream(x)),
           "sherry_gemm_acc")
    return acc


def device_error():
    """Synchronise and return (and clear) the device-side error word (0 = none)."""
    return int(lib().sherry_device_error())


def set_wait_limit(cycles):
    """Limit (SM clock cycles) of the kernels' bounded barrier waits, for
    kernels launched afterwards by this process; 0 restores the default, and with 1
    the attention's waits for pages of few new tokens give up without a look."""
    _check(lib().sherry_set_wait_limit(int(cycles)), "sherry_set_wait_limit")


# ----------------------------------------------------------------------------- comparison formats
CMP_I2 = 1  # 2 bits per weight, aligned
CMP_T3 = 2  # three weights in five bits
_CMP_TILE_WORDS = {CMP_I2: 8, CMP_T3: 5}


def cmp_tiles(fmt, K):
    if fmt == CMP_I2:
        return K // TILE_K
    return 2 * ((K + 191) // 192)


def cmp_transcode(fmt, codes, N):
    """Sherry codes of an N x K matrix -> the same matrix in comparison format
    fmt, int32 [ceil(N/32), tiles, words, 32] holding the uint32 words."""
    N, K = _codes_shape(codes, N)
    shape = ((N + 31) // 32, cmp_tiles(fmt, K), _CMP_TILE_WORDS[fmt], 32)
    out = torch.empty(shape, dtype=torch.int32, device=codes.device)
    assert out.numel() * 4 == lib().sherry_cmp_packed_bytes(fmt, N, K)
    _check(lib().sherry_cmp_transcode(fmt, _ptr(codes), N, K, _ptr(out), _stream(codes)),
           "sherry_cmp_transcode")
    return out


def cmp_gemv_acc(fmt, codes, x, N, K, acc=None):
    """Exact int32 acc[B, N] of a comparison-format matrix against int8 x [B, K]."""
    _need(x, torch.int8, "x")
    x2 = x.view(1, -1) if x.dim() == 1 else x
    B = x2.shape[0]
    if acc is None:
        acc = torch.empty((B, N), dtype=torch.int32, device=x.device)
    nb = lib().sherry_cmp_workspace_bytes(fmt, N, K, B)
    ws = workspace(max(nb, 256), x.device)
    _check(lib().sherry_cmp_gemv_acc(fmt, _ptr(codes), _ptr(x2), _ptr(acc), N, K, B, _ptr(ws),
                                     ws.numel(), _stream(x)), "sherry_cmp_gemv_acc")
    return acc


class GroupedCmpGemv:
    """Pre-marshalled grouped GEMV on comparison-format matrices: items are
    (codes in format fmt, scales, x int8 [B, K], y [B, N], K)."""

    def __init__(self, fmt, items, B):
        n = len(items)
        self.descs = (GemvDesc * n)()
        total = 0
        for i, (codes, scales, x, y, K) in enumerate(items):
            _need(scales, torch.float32, "scales")
            _need(x, torch.int8, "x")
            _need(y, torch.float32, "y")
            N = scales.numel()
            self.descs[i] = GemvDesc(codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
                                     y.data_ptr(), N, K)
            total += lib().sherry_cmp_workspace_bytes(fmt, N, K, B)
        self.items = items
        dev = items[0][2].device
        self.ws = torch.empty(max(total, 256), dtype=torch.uint8, device=dev)
        self.args = (fmt, ctypes.cast(self.descs, ctypes.c_void_p), n, B, _ptr(self.ws),
                     self.ws.numel())
        self.device = dev

    def __call__(self, stream=None):
        s = ctypes.c_void_p(stream if stream is not None
                            else _stream_handle(self.device))
        _check(lib().sherry_cmp_gemv_grouped(*self.args, s), "sherry_cmp_gemv_grouped")


# ----------------------------------------------------------------------------- attention
# The calls of a decode step are small, so the host side counts: descriptors are packed straight into
# bytes, and a tensor's properties are read once each (a call takes 6 to 8 us on the host, about half of
# it the launches; ctypes structures and separate checks took 12 to 22 us).
KV4_PAGE = 64
_TYPES = {torch.float32: 0, torch.bfloat16: 1}
_ROPE = struct.Struct("=QQQQqqqqQQQQqiiiiiiif")   # RopeArgs
_KV4 = struct.Struct("=QqiiQqqQQqq")              # Kv4Args
assert _ROPE.size == ctypes.sizeof(RopeArgs) and _KV4.size == ctypes.sizeof(Kv4Args)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing


def _device(t, name):
    """Index of the CUDA device of a tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    return t.get_device()


def _heads(t, name, dev):
    """(type, rows, heads, D, elements from row to row) of a [T, heads, D] tensor on device `dev` whose
    rows are contiguous; the row stride is free (a slice of a fused product will do)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError("%s must be a tensor on CUDA device %d" % (name, dev))
    ty = _TYPES.get(t.dtype)
    if ty is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if t.dim() != 3:
        raise ValueError("%s must have shape [T, heads, D]" % name)
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError("%s must have contiguous rows (strides %s)" % (name, t.stride()))
    return ty, T, H, D, (st if T > 1 else H * D)


def _index(t, name, dev, dim=1):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.get_device() != dev:
        raise TypeError("%s must be an int32 tensor on CUDA device %d" % (name, dev))
    if t.dim() != dim or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError("%s must have %d dimension(s), the last contiguous" % (name, dim))


def _vector(t, name, dev, n=None):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.get_device() != dev:
        raise TypeError("%s must be a float32 tensor on CUDA device %d" % (name, dev))
    if t.dim() != 1 or (n is not None and t.numel() != n) or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %s elements" % (name, n))


def _bytes(t, name, dev):
    """Size of a scratch buffer given by the caller, which kernels write to."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8 or t.get_device() != dev:
        raise TypeError("%s must be a uint8 tensor on CUDA device %d" % (name, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.numel()


def _call(dev, f, where, *args):
    """f(*args, current stream of device dev), with dev the current device."""
    if _get_device() != dev:
        with torch.cuda.device(dev):
            st = f(*args, _stream_handle(torch.device("cuda", dev)))
    else:
        st = f(*args, _raw_stream(dev) if _raw_stream is not None else _stream_handle(torch.device("cuda", dev)))
    if st:
        _check(st, where)


def _scratch(nbytes, dev):
    """As workspace(); a call under graph capture gets its own buffer from the graph's pool, so that two
    graphs that run at the same time share none."""
    device = torch.device("cuda", dev)
    with torch.cuda.device(dev):
        if _capturing():
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace(nbytes, device)


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-5,
                 interleaved=False, q_out=None, k_out=None, out_dtype=None):
    """Per-head RMS norm (where a weight [D] is given) and rotary positions of q [T, Hq, D] and
    k [T, Hk, D] (fp32 or bf16; either may be None) in one launch.  positions int32 [T], inv_freq
    fp32 [R / 2] (R <= D elements of a head turn).  Pairs are (j, j + R / 2), or (2 j, 2 j + 1) if
    interleaved.  Returns (q_out, k_out) of out_dtype (default bfloat16); q_out may be q itself."""
    if q is None and k is None:
        raise TypeError("q or k must be given")
    dev = _device(q, "q") if q is not None else _device(k, "k")
    qp = kp = qop = kop = qs = ks = qos = kos = Hq = Hk = qw = kw = 0
    shape = None
    if q is not None:
        ty, T, Hq, D, qs = _heads(q, "q", dev)
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=out_dtype or torch.bfloat16, device=q.device)
        oty, oT, oH, oD, qos = _heads(q_out, "q_out", dev)
        if oT != T or oH != Hq or oD != D:
            raise ValueError("q_out has shape %s, expected %s" % ((oT, oH, oD), (T, Hq, D)))
        if q_weight is not None:
            _vector(q_weight, "q_weight", dev, D)
            qw = q_weight.data_ptr()
        qp, qop = q.data_ptr(), q_out.data_ptr()
        shape = (ty, oty, T, D)
    elif q_out is not None or q_weight is not None:
        raise TypeError("q is None but q_out or q_weight is given")
    if k is not None:
        ty, T, Hk, D, ks = _heads(k, "k", dev)
        if k_out is None:
            k_out = torch.empty((T, Hk, D), dtype=out_dtype or torch.bfloat16, device=k.device)
        oty, oT, oH, oD, kos = _heads(k_out, "k_out", dev)
        if oT != T or oH != Hk or oD != D:
            raise ValueError("k_out has shape %s, expected %s" % ((oT, oH, oD), (T, Hk, D)))
        if shape is not None and shape != (ty, oty, T, D):
            raise ValueError("q and k differ in type, tokens or head size")
        if k_weight is not None:
            _vector(k_weight, "k_weight", dev, D)
            kw = k_weight.data_ptr()
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None or k_weight is not None:
        raise TypeError("k is None but k_out or k_weight is given")
    _index(positions, "positions", dev)
    if positions.shape[0] != T:
        raise ValueError("positions has %d entries for %d tokens" % (positions.numel(), T))
    _vector(inv_freq, "inv_freq", dev)
    args = _ROPE.pack(qp, kp, qop, kop, qs, ks, qos, kos, positions.data_ptr(), inv_freq.data_ptr(), qw, kw, T,
                      Hq, Hk, D, 2 * inv_freq.shape[0], ty, oty, 1 if interleaved else 0, eps)
    _call(dev, lib().sherry_qk_norm_rope, "sherry_qk_norm_rope", args)
    return q_out, k_out


def kv4_cache(pages, heads, dim, device):
    """A zeroed 4-bit key/value cache, uint8 [pages, heads, 2, 64 * (dim / 2 + 4)]; dim 64 or 128."""
    nbytes = int(lib().sherry_kv4_bytes(pages, heads, dim))
    if nbytes == 0:
        raise ValueError("no 4-bit cache of %d pages, %d heads of %d" % (pages, heads, dim))
    return torch.zeros((pages, heads, 2, KV4_PAGE * (dim // 2 + 4)), dtype=torch.uint8, device=device)


_BLOCK_DIM = {KV4_PAGE * (d // 2 + 4): d for d in (64, 128)}


def _kv4(cache, page_table, ctx_lens, cu_q, T, dev):
    """(Kv4Args as bytes, heads, D)."""
    if cache.dtype is not torch.uint8:
        raise TypeError("cache must be a uint8 CUDA tensor (kv4_cache)")
    if cache.dim() != 4 or cache.shape[2] != 2 or not cache.is_contiguous():
        raise ValueError("cache must be contiguous, [pages, heads, 2, 64 * (dim / 2 + 4)]")
    pages, H, _, block = cache.shape
    D = _BLOCK_DIM.get(block)
    if D is None:
        raise ValueError("cache blocks of %d bytes are of no head size" % block)
    _index(page_table, "page_table", dev, 2)
    _index(ctx_lens, "ctx_lens", dev)
    B, width = page_table.shape
    if ctx_lens.shape[0] != B:
        raise ValueError("ctx_lens has %d entries, page_table %d rows" % (ctx_lens.numel(), B))
    cu = 0
    if cu_q is not None:
        _index(cu_q, "cu_q", dev)
        if cu_q.shape[0] != B + 1:
            raise ValueError("cu_q has %d entries for %d sequences" % (cu_q.numel(), B))
        cu = cu_q.data_ptr()
    elif T != B:
        raise ValueError("%d rows for %d sequences: give cu_q" % (T, B))
    return _KV4.pack(cache.data_ptr(), pages, H, D, page_table.data_ptr(), width,
                     page_table.stride(0) if B > 1 else width, ctx_lens.data_ptr(), cu, B, T), H, D


def _kv4_rows(f, where, cache, k, v, page_table, ctx_lens, cu_q):
    dev = _device(cache, "cache")
    ty, T, H, D, ks = _heads(k, "k", dev)
    vty, vT, vH, vD, vs = _heads(v, "v", dev)
    if vty != ty or vT != T or vH != H or vD != D:
        raise ValueError("k and v differ in type or shape")
    args, cH, cD = _kv4(cache, page_table, ctx_lens, cu_q, T, dev)
    if H != cH or D != cD:
        raise ValueError("k has %d heads of %d, the cache %d of %d" % (H, D, cH, cD))
    _call(dev, f, where, args, k.data_ptr(), v.data_ptr(), ty, ks, vs)


def kv4_write(cache, k, v, page_table, ctx_lens, cu_q=None):
    """Codes the new tokens' k and v [T, heads, dim] (fp32 or bf16) into the cache.  page_table int32
    [B, width], ctx_lens int32 [B] (the new tokens included); rows cu_q[b] .. cu_q[b + 1] - 1 are the
    last positions of sequence b (cu_q None: one row each)."""
    _kv4_rows(lib().sherry_kv4_write, "sherry_kv4_write", cache, k, v, page_table, ctx_lens, cu_q)


def kv4_read(cache, page_table, ctx_lens, cu_q=None, rows=None, dtype=torch.float32, k=None, v=None):
    """The values that the cache holds for the tokens that kv4_write takes: (k, v) [T, heads, dim].
    Rows without a place in the cache are left as they are (zeros in tensors made here, of `rows`
    rows; needed where cu_q is given)."""
    if (k is None) != (v is None):
        raise TypeError("give both k and v, or neither")
    if k is None:
        if rows is None:
            if cu_q is not None:
                raise TypeError("rows must be given with cu_q")
            rows = ctx_lens.numel()
        dev = _device(cache, "cache")
        _, H, D = _kv4(cache, page_table, ctx_lens, cu_q, rows, dev)
        k = torch.zeros((rows, H, D), dtype=dtype, device=cache.device)
        v = torch.zeros((rows, H, D), dtype=dtype, device=cache.device)
    _kv4_rows(lib().sherry_kv4_read, "sherry_kv4_read", cache, k, v, page_table, ctx_lens, cu_q)
    return k, v


@functools.lru_cache(maxsize=1024)
def attn_kv4_workspace_bytes(T, heads, dim):
    return int(lib().sherry_attn_kv4_workspace_bytes(T, heads, dim))


def attn_kv4(q, cache, page_table, ctx_lens, cu_q=None, max_q=0, scale=None, out=None, ws=None):
    """Causal attention of the new tokens' q bf16 [T, Hq, dim] over the cache (their own keys and values
    written before): out bf16 [T, Hq, dim].  page_table, ctx_lens and cu_q as for kv4_write; scale
    defaults to dim ** -0.5; max_q, the most new tokens of a sequence, helps to pick kernels (0: not
    known); ws, scratch of attn_kv4_workspace_bytes(T, Hq, dim) bytes on the same device.  Rows without a
    position give zeros."""
    dev = _device(cache, "cache")
    ty, T, Hq, D, qs = _heads(q, "q", dev)
    args, H, cD = _kv4(cache, page_table, ctx_lens, cu_q, T, dev)
    if out is None:
        make = torch.empty if cu_q is None else torch.zeros  # rows outside every sequence stay
        out = make((T, Hq, D), dtype=torch.bfloat16, device=q.device)
    oty, oT, oH, oD, os_ = _heads(out, "out", dev)
    if ty != 1 or oty != 1:
        raise TypeError("q and out must be bfloat16")
    if oT != T or oH != Hq or oD != D:
        raise ValueError("out has shape %s, expected %s" % ((oT, oH, oD), (T, Hq, D)))
    if D != cD or Hq % H:
        raise ValueError("q has %d heads of %d, the cache %d of %d" % (Hq, D, H, cD))
    if ws is None:
        need = attn_kv4_workspace_bytes(T, Hq, D)
        if _raw_stream is not None and _get_device() == dev and not _capturing():
            ws = _workspaces.get((dev, _raw_stream(dev)))
        if ws is None or ws.numel() < need:
            ws = _scratch(need, dev)
        nbytes = ws.numel()
    else:
        nbytes = _bytes(ws, "ws", dev)
    _call(dev, lib().sherry_attn_kv4, "sherry_attn_kv4", args, q.data_ptr(), qs, out.data_ptr(), os_, Hq, int(max_q),
          D ** -0.5 if scale is None else scale, ws.data_ptr(), nbytes)
    return out


def probe_mma_i8(iters, stream=None):
    """Launch the tensor-core int8 probe; returns the number of CTAs (one per
    SM).  Each CTA runs iters * 4 MMAs of 128 x 256 x 32."""
    ctas = ctypes.c_int(0)
    s = ctypes.c_void_p(stream if stream is not None else torch.cuda.current_stream().cuda_stream)
    _check(lib().sherry_probe_mma_i8(int(iters), ctypes.byref(ctas), s), "sherry_probe_mma_i8")
    return ctas.value
