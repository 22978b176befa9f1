"""Thin Python binding of libnq.so (include/nq.h) -- argument marshalling only.

Every step of the LRB path runs in the CUDA library; this module checks tensor arguments
(CUDA device, dtype, shape, layout: the C ABI cannot see a tensor's extent), turns them into
device pointers and the current torch stream into a ``cudaStream_t``.  PyTorch provides
device memory and streams, nothing else.  If ``libnq.so`` is missing the import fails: there
is no other implementation to fall back to.

Tensor conventions (device tensors, contiguous):
  packed signs  int32 [rows][ld] (the bits of uint32 words)
  s1, s2        float16 [d_out], [d_in]
  x, y          bfloat16 [M][d_in], [M][d_out]
  latent        float32 [rows][ld_latent]
  adapters      A bfloat16 [n][rank][d_in], B bfloat16 [n][d_out][rank], scale float32 [n]
  row lists     int32 (ids [M], rows [M], offsets [n + 1])
  block norms   y, x, gate bfloat16, the residual stream bfloat16 or float32
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libnq.so is not built (python -m rank_binary_factorized_b200.build): " + LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

NQ_OK = 0
STATUS_NAMES = {0: "NQ_OK", 1: "NQ_ERR_NULL", 2: "NQ_ERR_SHAPE", 3: "NQ_ERR_ALIGN", 4: "NQ_ERR_WORKSPACE",
                5: "NQ_ERR_DEVICE", 6: "NQ_ERR_LAUNCH", 7: "NQ_ERR_TIMEOUT", 8: "NQ_ERR_SCRATCH_LIMIT",
                9: "NQ_ERR_VALUE", 10: "NQ_ERR_INDEX"}
MATVEC_MAX_M = 8

_BF16 = torch.bfloat16
_i64 = ctypes.c_int64
_p = ctypes.c_void_p


class nq_lrb_layer(ctypes.Structure):
    _fields_ = [("d_out", _i64), ("d_in", _i64), ("r", _i64), ("U", _p), ("ldu", _i64), ("V", _p), ("ldv", _i64),
                ("s1", _p), ("s2", _p)]


class nq_adapters(ctypes.Structure):
    _fields_ = [("n", _i64), ("rank", _i64), ("d_in", _i64), ("d_out", _i64), ("A", _p), ("lda", _i64), ("B", _p),
                ("ldb", _i64), ("scale", _p)]


class nq_block_norm(ctypes.Structure):
    _fields_ = [("d", _i64), ("w_pre", _p), ("w_post", _p), ("w_offset", ctypes.c_float), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("post_norm", ctypes.c_int32), ("h_f32", ctypes.c_int32)]


_lib.nq_pack_signs.restype = ctypes.c_int
_lib.nq_pack_signs.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p]
_lib.nq_workspace_bytes.restype = ctypes.c_size_t
_lib.nq_workspace_bytes.argtypes = [ctypes.POINTER(nq_lrb_layer), _i64]
for _name in ("nq_lrb_matvec", "nq_lrb_matmul", "nq_layer_forward"):
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = [ctypes.POINTER(nq_lrb_layer), _p, _p, _i64, _p, ctypes.c_size_t, _p]
_lib.nq_silu_mul.restype = ctypes.c_int
_lib.nq_silu_mul.argtypes = [_p, _p, _p, _i64, _p]
_lib.nq_lrb_transposed.restype = ctypes.c_int
_lib.nq_lrb_transposed.argtypes = [ctypes.POINTER(nq_lrb_layer), _p, _p, _i64, _p, ctypes.c_size_t, _p]
_lib.nq_from_latent_workspace_bytes.restype = ctypes.c_size_t
_lib.nq_from_latent_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64]
_lib.nq_lrb_from_latent.restype = ctypes.c_int
_lib.nq_lrb_from_latent.argtypes = [_p, _i64, _p, _i64, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p,
                                    ctypes.c_size_t, _p]
_lib.nq_mlp_gate_up_workspace_bytes.restype = ctypes.c_size_t
_lib.nq_mlp_gate_up_workspace_bytes.argtypes = [ctypes.POINTER(nq_lrb_layer), ctypes.POINTER(nq_lrb_layer), _i64]
_lib.nq_mlp_gate_up.restype = ctypes.c_int
_lib.nq_mlp_gate_up.argtypes = [ctypes.POINTER(nq_lrb_layer), ctypes.POINTER(nq_lrb_layer), _p, _p, _i64, _p,
                                ctypes.c_size_t, _p]
_lib.nq_group_workspace_bytes.restype = ctypes.c_size_t
_lib.nq_group_workspace_bytes.argtypes = [ctypes.POINTER(ctypes.POINTER(nq_lrb_layer)), ctypes.c_int, _i64]
_lib.nq_layer_forward_group.restype = ctypes.c_int
_lib.nq_layer_forward_group.argtypes = [ctypes.POINTER(ctypes.POINTER(nq_lrb_layer)), ctypes.c_int, _p,
                                        ctypes.POINTER(_p), _i64, _p, ctypes.c_size_t, _p]
_lib.nq_lrb_scale_grads.restype = ctypes.c_int
_lib.nq_lrb_scale_grads.argtypes = [ctypes.POINTER(nq_lrb_layer), _p, _p, _i64, _p, _p, _p, ctypes.c_size_t, _p]
_lib.nq_sync_status.restype = ctypes.c_int
_lib.nq_sign_grads_workspace_bytes.restype = ctypes.c_size_t
_lib.nq_sign_grads_workspace_bytes.argtypes = [ctypes.POINTER(nq_lrb_layer), _i64]
_lib.nq_lrb_sign_grads.restype = ctypes.c_int
_lib.nq_lrb_sign_grads.argtypes = [ctypes.POINTER(nq_lrb_layer), _p, _p, _i64, _p, _i64, _p, _i64, _p, ctypes.c_size_t,
                                   _p]
_lib.nq_selftest_bounded_wait.restype = ctypes.c_int
_lib.nq_selftest_bounded_wait.argtypes = [_i64, _p]
_lib.nq_adapter_rows.restype = ctypes.c_int
_lib.nq_adapter_rows.argtypes = [_p, _i64, _i64, _p, _p, _p]
_lib.nq_adapter_workspace_bytes.restype = ctypes.c_size_t
_lib.nq_adapter_workspace_bytes.argtypes = [ctypes.POINTER(nq_adapters), _i64]
_lib.nq_adapter_forward.restype = ctypes.c_int
_lib.nq_adapter_forward.argtypes = [ctypes.POINTER(nq_adapters), _p, _p, _p, _p, _p, _p, _i64, _p]
_lib.nq_adapter_backward.restype = ctypes.c_int
_lib.nq_adapter_backward.argtypes = [ctypes.POINTER(nq_adapters), _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _p,
                                     ctypes.c_size_t, _p]
_lib.nq_block_norm_forward.restype = ctypes.c_int
_lib.nq_block_norm_forward.argtypes = [ctypes.POINTER(nq_block_norm), _p, _p, _p, _i64, _p, _p, _i64, _p]
_lib.nq_block_norm_workspace_bytes.restype = ctypes.c_size_t
_lib.nq_block_norm_workspace_bytes.argtypes = [ctypes.POINTER(nq_block_norm), _i64]
_lib.nq_block_norm_backward.restype = ctypes.c_int
_lib.nq_block_norm_backward.argtypes = [ctypes.POINTER(nq_block_norm), _p, _p, _p, _i64, _p, _p, _p, _p, _p, _p, _p,
                                        _i64, _p, ctypes.c_size_t, _p]
_lib.nq_sync_status.argtypes = [_p]
_lib.nq_status_string.restype = ctypes.c_char_p
_lib.nq_status_string.argtypes = [ctypes.c_int]
_lib.nq_version.restype = ctypes.c_char_p
_lib.nq_version.argtypes = []


class NQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s: %s" % (fn, _lib.nq_status_string(status).decode()))


def _check(fn: str, status: int) -> None:
    if status != NQ_OK:
        raise NQError(fn, status)


def version() -> str:
    return _lib.nq_version().decode()


def status_string(status: int) -> str:
    return _lib.nq_status_string(status).decode()


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _need(t, name: str, dtype, shape=None, device=None, contiguous: bool = True) -> None:
    """Checks a tensor argument before its address reaches the library, which reads device
    memory only and at the layout nq.h states: a CUDA tensor of the given dtype (and shape and
    device), contiguous unless the call takes a row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %s" % (name, type(t).__name__))
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor, got one on %s" % (name, t.device))
    if t.dtype != dtype:
        raise ValueError("%s: expected dtype %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(int(d) for d in shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if device is not None and t.device != device:
        raise ValueError("%s: on %s, the layer's tensors on %s" % (name, t.device, device))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s: expected a contiguous tensor" % name)


def _need_rows(t, name: str, dtype, rows: int, min_cols: int, device=None) -> None:
    """A 2-D CUDA tensor with `rows` rows of at least `min_cols` columns and unit column stride
    (the call takes its row stride)."""
    _need(t, name, dtype, device=device, contiguous=False)
    if t.dim() != 2 or int(t.shape[0]) != rows or int(t.shape[1]) < min_cols or t.stride(1) != 1:
        raise ValueError("%s: expected [%d][>= %d] with unit column stride, got shape %s strides %s" %
                         (name, rows, min_cols, tuple(t.shape), tuple(t.stride())))


def _need_ws(ws, layer_device) -> None:
    _need(ws, "ws", torch.uint8, device=layer_device)


class Layer:
    """A device-resident LRB layer: packed U, V (int32 words), fp16 s1, s2."""

    def __init__(self, U: torch.Tensor, V: torch.Tensor, s1: torch.Tensor, s2: torch.Tensor, r: int):
        _need(U, "U", torch.int32)
        if U.dim() != 2:
            raise ValueError("U: expected [d_out][ldu] words, got shape %s" % (tuple(U.shape),))
        _need(V, "V", torch.int32, device=U.device)
        if V.dim() != 2:
            raise ValueError("V: expected [d_in][ldv] words, got shape %s" % (tuple(V.shape),))
        _need(s1, "s1", torch.float16, shape=(U.shape[0],), device=U.device)
        _need(s2, "s2", torch.float16, shape=(V.shape[0],), device=U.device)
        self.U, self.V, self.s1, self.s2 = U, V, s1, s2
        self.d_out, self.ldu = int(U.shape[0]), int(U.shape[1])
        self.d_in, self.ldv = int(V.shape[0]), int(V.shape[1])
        self.r = int(r)
        self.struct = nq_lrb_layer(self.d_out, self.d_in, self.r, _ptr(U), self.ldu, _ptr(V), self.ldv, _ptr(s1),
                                   _ptr(s2))
        self._ws = {}

    @classmethod
    def from_host(cls, U, V, s1_bits, s2_bits, r: int, device="cuda", ld_align_words: int = 4) -> "Layer":
        """From numpy arrays: uint32 words and fp16 bit patterns (uint16).  Rows of U and V are
        padded with zero words to a multiple of `ld_align_words` words: at the default 4 (16
        bytes) the tensor-core path loads the packed signs by TMA; any stride works."""
        import numpy as np

        def dev(a, dt):
            return torch.from_numpy(np.ascontiguousarray(a).view(dt)).to(device)

        def words(a):
            a = np.ascontiguousarray(a)
            nw = a.shape[1]
            ld = -(-nw // ld_align_words) * ld_align_words
            if ld != nw:
                b = np.zeros((a.shape[0], ld), dtype=a.dtype)
                b[:, :nw] = a
                a = b
            return dev(a, np.int32)

        return cls(words(U), words(V), dev(s1_bits, np.float16), dev(s2_bits, np.float16), r)

    def workspace_bytes(self, M: int) -> int:
        return int(_lib.nq_workspace_bytes(ctypes.byref(self.struct), M))

    def workspace(self, M: int) -> torch.Tensor:
        """A zero-filled workspace large enough for M rows, cached on the layer and grown on
        demand.  Every call on this layer that passes no ``ws`` uses it, so calls that may run
        at the same time on the GPU (on different streams) must each pass their own ``ws``."""
        need = self.workspace_bytes(M)
        if need == 0:
            raise NQError("nq_workspace_bytes", 2)
        ws = self._ws.get("ws")
        if ws is None or ws.numel() < need:
            ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=self.U.device)
            self._ws["ws"] = ws
        return ws

    @property
    def storage_bytes(self) -> int:
        return 4 * (self.d_out + self.d_in) * self.r // 32 + 2 * (self.d_out + self.d_in)


def pack_signs(latent: torch.Tensor, r: int | None = None, ld_words: int | None = None, out=None,
               stream=None) -> torch.Tensor:
    """sign(latent) >= 0 packed 32 per word along r (bit k%32 of word k/32)."""
    _need(latent, "latent", torch.float32, contiguous=False)
    if latent.dim() != 2 or latent.stride(1) != 1:
        raise ValueError("latent must be a 2-D float32 tensor with unit column stride")
    rows, ld_latent = int(latent.shape[0]), int(latent.stride(0))
    r = int(latent.shape[1]) if r is None else int(r)
    if r > int(latent.shape[1]):
        raise ValueError("r = %d exceeds the latent's %d columns" % (r, int(latent.shape[1])))
    ld_words = r // 32 if ld_words is None else int(ld_words)
    if out is None:
        out = torch.empty((rows, ld_words), dtype=torch.int32, device=latent.device)
    _need(out, "out", torch.int32, shape=(rows, ld_words), device=latent.device)
    _check("nq_pack_signs", _lib.nq_pack_signs(_ptr(latent), rows, r, ld_latent, _ptr(out), ld_words,
                                               _stream_ptr(stream)))
    return out


def _forward(fn_name: str, layer: Layer, x: torch.Tensor, y=None, ws=None, stream=None) -> torch.Tensor:
    dev = layer.U.device
    _need(x, "x", torch.bfloat16, device=dev)
    M = int(x.shape[0])
    _need(x, "x", torch.bfloat16, shape=(M, layer.d_in))
    if y is None:
        y = torch.empty((M, layer.d_out), dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, shape=(M, layer.d_out), device=dev)
    if ws is None:
        ws = layer.workspace(M)
    _need_ws(ws, dev)
    fn = getattr(_lib, fn_name)
    _check(fn_name, fn(ctypes.byref(layer.struct), _ptr(x), _ptr(y), M, _ptr(ws), ws.numel(), _stream_ptr(stream)))
    return y


def lrb_matvec(layer: Layer, x: torch.Tensor, y=None, ws=None, stream=None) -> torch.Tensor:
    return _forward("nq_lrb_matvec", layer, x, y, ws, stream)


def lrb_matmul(layer: Layer, x: torch.Tensor, y=None, ws=None, stream=None) -> torch.Tensor:
    return _forward("nq_lrb_matmul", layer, x, y, ws, stream)


def layer_forward(layer: Layer, x: torch.Tensor, y=None, ws=None, stream=None, adapters=None, groups=None,
                  t=None) -> torch.Tensor:
    """The layer's output; with `adapters` (Adapters of this projection) and `groups` (AdapterRows of
    this batch), each row's low-rank term added to it (adapter_forward, which fills t if given)."""
    if adapters is not None and (adapters.d_in != layer.d_in or adapters.d_out != layer.d_out or groups is None):
        raise ValueError("adapters: of %d x %d with groups %s, the layer is %d x %d" %
                         (adapters.d_out, adapters.d_in, "given" if groups is not None else "missing", layer.d_out,
                          layer.d_in))
    if adapters is not None:
        _check_adapter_call(adapters, groups, x, y, t)
    y = _forward("nq_layer_forward", layer, x, y, ws, stream)
    return y if adapters is None else adapter_forward(adapters, groups, x, y, out=y, t=t, stream=stream)


def lrb_transposed(layer: Layer, ybar: torch.Tensor, xbar=None, ws=None, stream=None) -> torch.Tensor:
    """xbar = the layer's transpose applied to ybar ([M][d_out] bf16 -> [M][d_in] bf16)."""
    dev = layer.U.device
    _need(ybar, "ybar", torch.bfloat16, device=dev)
    M = int(ybar.shape[0])
    _need(ybar, "ybar", torch.bfloat16, shape=(M, layer.d_out))
    if xbar is None:
        xbar = torch.empty((M, layer.d_in), dtype=torch.bfloat16, device=ybar.device)
    _need(xbar, "xbar", torch.bfloat16, shape=(M, layer.d_in), device=dev)
    if ws is None:
        ws = layer.workspace(M)
    _need_ws(ws, dev)
    _check("nq_lrb_transposed", _lib.nq_lrb_transposed(ctypes.byref(layer.struct), _ptr(ybar), _ptr(xbar), M,
                                                       _ptr(ws), ws.numel(), _stream_ptr(stream)))
    return xbar


def lrb_scale_grads(layer: Layer, x: torch.Tensor, ybar: torch.Tensor, ws=None, stream=None):
    """(dL/ds1 [d_out], dL/ds2 [d_in]) fp32 for L = sum <ybar, layer(x)>."""
    dev = layer.U.device
    _need(x, "x", torch.bfloat16, device=dev)
    M = int(x.shape[0])
    _need(x, "x", torch.bfloat16, shape=(M, layer.d_in))
    _need(ybar, "ybar", torch.bfloat16, shape=(M, layer.d_out), device=dev)
    g1 = torch.empty(layer.d_out, dtype=torch.float32, device=x.device)
    g2 = torch.empty(layer.d_in, dtype=torch.float32, device=x.device)
    if ws is None:
        ws = layer.workspace(M)
    _need_ws(ws, dev)
    _check("nq_lrb_scale_grads", _lib.nq_lrb_scale_grads(ctypes.byref(layer.struct), _ptr(x), _ptr(ybar), M,
                                                         _ptr(g1), _ptr(g2), _ptr(ws), ws.numel(),
                                                         _stream_ptr(stream)))
    return g1, g2


def sign_grads_workspace_bytes(layer: Layer, M: int) -> int:
    n = int(_lib.nq_sign_grads_workspace_bytes(ctypes.byref(layer.struct), int(M)))
    if n == 0:
        raise NQError("nq_sign_grads_workspace_bytes", 2)
    return n


def lrb_sign_grads(layer: Layer, x: torch.Tensor, ybar: torch.Tensor, gU=None, gV=None, ws=None, stream=None):
    """(dL/dU [d_out][r], dL/dV [d_in][r]) fp32 for L = sum <ybar, layer(x)>: the gradients the
    identity straight-through estimator passes to the latent factors.  gU, gV may be given
    ([rows][ld] fp32 with ld >= r a multiple of 4); only their first r columns are written."""
    dev = layer.U.device
    _need(x, "x", torch.bfloat16, device=dev)
    M = int(x.shape[0])
    _need(x, "x", torch.bfloat16, shape=(M, layer.d_in))
    _need(ybar, "ybar", torch.bfloat16, shape=(M, layer.d_out), device=dev)
    r = layer.r
    if gU is None:
        gU = torch.empty((layer.d_out, r), dtype=torch.float32, device=x.device)
    if gV is None:
        gV = torch.empty((layer.d_in, r), dtype=torch.float32, device=x.device)
    _need_rows(gU, "gU", torch.float32, layer.d_out, r, device=dev)
    _need_rows(gV, "gV", torch.float32, layer.d_in, r, device=dev)
    if ws is None:
        ws = torch.empty(sign_grads_workspace_bytes(layer, M), dtype=torch.uint8, device=x.device)
    _need_ws(ws, dev)
    _check("nq_lrb_sign_grads", _lib.nq_lrb_sign_grads(ctypes.byref(layer.struct), _ptr(x), _ptr(ybar), M, _ptr(gU),
                                                       gU.stride(0), _ptr(gV), gV.stride(0), _ptr(ws), ws.numel(),
                                                       _stream_ptr(stream)))
    return gU, gV


def lrb_from_latent(Uh: torch.Tensor, Vh: torch.Tensor, r: int | None = None, ld_align_words: int = 4,
                    stream=None):
    """A device Layer from fp32 latent proxies Uh [d_out][r], Vh [d_in][r]: magnitude balancing,
    mean-absolute-value scales, packed signs.  Returns (Layer, eta as a 0-d fp64 tensor)."""
    r = int(Uh.shape[1]) if r is None else int(r)
    _need_rows(Uh, "Uh", torch.float32, int(Uh.shape[0]), r)
    _need_rows(Vh, "Vh", torch.float32, int(Vh.shape[0]), r, device=Uh.device)
    d_out, d_in = int(Uh.shape[0]), int(Vh.shape[0])
    ld = -(-(r // 32) // ld_align_words) * ld_align_words
    dev = Uh.device
    U = torch.empty((d_out, ld), dtype=torch.int32, device=dev)
    V = torch.empty((d_in, ld), dtype=torch.int32, device=dev)
    s1 = torch.empty(d_out, dtype=torch.float16, device=dev)
    s2 = torch.empty(d_in, dtype=torch.float16, device=dev)
    eta = torch.empty((), dtype=torch.float64, device=dev)
    need = int(_lib.nq_from_latent_workspace_bytes(d_out, d_in, r, ld, ld))
    if need == 0:
        raise NQError("nq_from_latent_workspace_bytes", 2)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _check("nq_lrb_from_latent", _lib.nq_lrb_from_latent(_ptr(Uh), int(Uh.stride(0)), _ptr(Vh), int(Vh.stride(0)),
                                                         d_out, d_in, r, _ptr(U), ld, _ptr(V), ld, _ptr(s1),
                                                         _ptr(s2), _ptr(eta), _ptr(ws), need, _stream_ptr(stream)))
    return Layer(U, V, s1, s2, r), eta


def _layer_array(layers):
    arr = (ctypes.POINTER(nq_lrb_layer) * len(layers))()
    for i, L in enumerate(layers):
        arr[i] = ctypes.pointer(L.struct)
    return arr


def group_workspace_bytes(layers, M: int) -> int:
    return int(_lib.nq_group_workspace_bytes(_layer_array(layers), len(layers), M))


def layer_forward_group(layers, x: torch.Tensor, ys=None, ws=None, stream=None):
    """y_l = layers[l](x) for projections sharing x (one decode launch per stage for M <= 8)."""
    if len(layers) == 0:
        raise ValueError("layers: expected at least one layer")
    dev = layers[0].U.device
    _need(x, "x", torch.bfloat16, device=dev)
    M = int(x.shape[0])
    for L in layers:
        if L.U.device != dev:
            raise ValueError("layers: all on one device")
        _need(x, "x", torch.bfloat16, shape=(M, L.d_in))
    if ys is None:
        ys = [torch.empty((M, L.d_out), dtype=torch.bfloat16, device=x.device) for L in layers]
    if len(ys) != len(layers):
        raise ValueError("ys: expected one output per layer")
    for i, (L, y) in enumerate(zip(layers, ys)):
        _need(y, "ys[%d]" % i, torch.bfloat16, shape=(M, L.d_out), device=dev)
    if ws is None:
        need = group_workspace_bytes(layers, M)
        if need == 0:
            raise NQError("nq_group_workspace_bytes", 2)
        ws = torch.zeros(need, dtype=torch.uint8, device=x.device)
    _need_ws(ws, dev)
    yp = (_p * len(ys))(*[_ptr(y) for y in ys])
    _check("nq_layer_forward_group", _lib.nq_layer_forward_group(_layer_array(layers), len(layers), _ptr(x), yp, M,
                                                                 _ptr(ws), ws.numel(), _stream_ptr(stream)))
    return ys


def mlp_gate_up_workspace_bytes(gate: Layer, up: Layer, M: int) -> int:
    return int(_lib.nq_mlp_gate_up_workspace_bytes(ctypes.byref(gate.struct), ctypes.byref(up.struct), M))


def mlp_gate_up(gate: Layer, up: Layer, x: torch.Tensor, h=None, ws=None, stream=None) -> torch.Tensor:
    """h = bf16(silu(bf16(gate x)) * bf16(up x)) ([M][d_out] bf16), SiLU.mul fused into decode."""
    dev = gate.U.device
    if up.U.device != dev:
        raise ValueError("gate, up: expected one device")
    _need(x, "x", torch.bfloat16, device=dev)
    M = int(x.shape[0]) if x.dim() == 2 else -1
    _need(x, "x", torch.bfloat16, shape=(M, gate.d_in), device=dev)
    if h is None:
        h = torch.empty((M, gate.d_out), dtype=torch.bfloat16, device=dev)
    _need(h, "h", torch.bfloat16, shape=(M, gate.d_out), device=dev)
    if ws is None:
        need = mlp_gate_up_workspace_bytes(gate, up, M)
        if need == 0:
            raise NQError("nq_mlp_gate_up_workspace_bytes", 2)
        ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    _need_ws(ws, dev)
    _check("nq_mlp_gate_up", _lib.nq_mlp_gate_up(ctypes.byref(gate.struct), ctypes.byref(up.struct), _ptr(x), _ptr(h),
                                                 M, _ptr(ws), ws.numel(), _stream_ptr(stream)))
    return h


def silu_mul(g: torch.Tensor, u: torch.Tensor, h=None, stream=None) -> torch.Tensor:
    _need(g, "g", torch.bfloat16)
    _need(u, "u", torch.bfloat16, shape=tuple(g.shape), device=g.device)
    if h is None:
        h = torch.empty_like(g)
    _need(h, "h", torch.bfloat16, shape=tuple(g.shape), device=g.device)
    _check("nq_silu_mul", _lib.nq_silu_mul(_ptr(g), _ptr(u), _ptr(h), g.numel(), _stream_ptr(stream)))
    return h


def _on(device):
    """A context in which `device` is the current one (None: whichever is)."""
    if device is None or device.index == torch._C._cuda_getDevice():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _workspace_of(owner, M: int, device, stream) -> torch.Tensor:
    """The workspace of a call that passes none: the owner's cached one or, in a capture, a new one from the
    graph's memory, which no later call can replace or share."""
    with _on(device):
        need = owner.workspace_bytes(M) if torch.cuda.is_current_stream_capturing() else 0
        if need == 0:
            return owner.workspace(M)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    if stream is not None:
        ws.record_stream(stream)
    return ws


class Adapters:
    """The low-rank adapters of one projection: A [n][rank][d_in], B [n][d_out][rank] bf16 (rows may
    be strided), scale [n] fp32 or None (all 1).  Row m with adapter a gets
    scale[a] * B[a] @ (A[a] @ x[m]) added to the projection's output."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor | None = None):
        _need(A, "A", torch.bfloat16, contiguous=False)
        _need(B, "B", torch.bfloat16, device=A.device, contiguous=False)
        if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[1] != B.shape[2]:
            raise ValueError("A, B: expected [n][rank][d_in] and [n][d_out][rank], got shapes %s and %s" %
                             (tuple(A.shape), tuple(B.shape)))
        ld = []
        for t, name in ((A, "A"), (B, "B")):
            n, rows, cols = (int(v) for v in t.shape)
            step = int(t.stride(1)) if rows > 1 else int(t.stride(0)) if n > 1 else cols
            if 0 in (n, rows, cols) or (cols > 1 and t.stride(2) != 1) or step < cols or (n > 1 and
                                                                                     t.stride(0) != rows * step):
                raise ValueError("%s: expected rows of unit stride, evenly spaced over all adapters, got shape %s "
                                 "strides %s" % (name, tuple(t.shape), tuple(t.stride())))
            ld.append(step)
        if scale is not None:
            _need(scale, "scale", torch.float32, shape=(A.shape[0],), device=A.device)
        self.A, self.B, self.scale = A, B, scale
        self.device = A.device
        self.n, self.rank, self.d_in = (int(v) for v in A.shape)
        self.d_out = int(B.shape[1])
        self.struct = nq_adapters(self.n, self.rank, self.d_in, self.d_out, _ptr(A), ld[0], _ptr(B), ld[1],
                                  _ptr(scale))
        self._ref = ctypes.byref(self.struct)
        self._ws = None

    def workspace_bytes(self, M: int) -> int:
        with _on(self.device):  # the size goes by the device's multiprocessors
            return int(_lib.nq_adapter_workspace_bytes(self._ref, int(M)))

    def workspace(self, M: int) -> torch.Tensor:
        """A workspace large enough for M rows, cached here and grown on demand.  Every backward
        call outside a capture that passes no ``ws`` uses it: calls that may run at the same time on
        the GPU must each pass their own.  A captured call that passes none gets one that belongs to
        the graph; one that is passed must outlive the graph (this cache drops the smaller when it grows)."""
        need = self.workspace_bytes(M)
        if need == 0:
            raise NQError("nq_adapter_workspace_bytes", 2)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self._ws


class AdapterRows:
    """The rows of a batch grouped by adapter: rows [M] int32, offsets [n + 1] int32 (see nq.h)."""

    def __init__(self, rows: torch.Tensor, offsets: torch.Tensor):
        _need(rows, "rows", torch.int32)
        _need(offsets, "offsets", torch.int32, device=rows.device)
        if rows.dim() != 1 or offsets.dim() != 1 or offsets.numel() < 2 or rows.numel() < 1:
            raise ValueError("rows, offsets: expected [M] and [n + 1], got shapes %s and %s" %
                             (tuple(rows.shape), tuple(offsets.shape)))
        self.rows, self.offsets = rows, offsets
        self.M, self.n = int(rows.numel()), int(offsets.numel()) - 1
        self._rows_ptr, self._offsets_ptr = _ptr(rows), _ptr(offsets)


def adapter_rows(ids: torch.Tensor, n: int, stream=None) -> AdapterRows:
    """Groups the rows of a batch by adapter: ids [M] int32, values outside 0..n-1 mean none."""
    _need(ids, "ids", torch.int32)
    if ids.dim() != 1:
        raise ValueError("ids: expected [M], got shape %s" % (tuple(ids.shape),))
    rows = torch.empty_like(ids)
    offsets = torch.empty(max(int(n), 1) + 1, dtype=torch.int32, device=ids.device)
    _call("nq_adapter_rows", _lib.nq_adapter_rows, ids.device, stream, ids.data_ptr(), ids.numel(), int(n),
          rows.data_ptr(), offsets.data_ptr())
    return AdapterRows(rows, offsets)


def _call(name: str, fn, device, stream, *args) -> None:
    """Calls the library with the tensors' device current, on `stream` or that device's current one."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream)
    if status != NQ_OK:
        raise NQError(name, status)


def _rows_ptr(t, name: str, dtype, M: int, cols: int, device) -> int:
    """The address of a contiguous [M][cols] tensor on `device`; _need says what is wrong with another."""
    try:
        if t.dtype is dtype and t.get_device() == device.index and t.shape == (M, cols) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtype, shape=(M, cols), device=device)
    return t.data_ptr()


def _array_ptr(t, name: str, dtype, shape, device) -> int:
    """The same for any shape."""
    try:
        if t.dtype is dtype and t.get_device() == device.index and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtype, shape=shape, device=device)
    return t.data_ptr()


def _ws_ptr(ws, device) -> int:
    try:
        if ws.dtype is torch.uint8 and ws.get_device() == device.index and ws.is_contiguous():
            return ws.data_ptr()
    except AttributeError:
        pass
    _need_ws(ws, device)
    return ws.data_ptr()


def _check_groups(ad: Adapters, groups: AdapterRows) -> None:
    if groups.n != ad.n or groups.rows.device != ad.device:
        raise ValueError("groups: for %d adapters on %s, the call has %d on %s" %
                         (groups.n, groups.rows.device, ad.n, ad.device))


def _check_adapter_call(ad: Adapters, groups: AdapterRows, x, y, t) -> None:
    """What adapter_forward would refuse, before the projection in front of it is queued."""
    dev, M = ad.device, groups.M
    _check_groups(ad, groups)
    ptrs = _rows_ptr(x, "x", _BF16, M, ad.d_in, dev) | groups._rows_ptr | groups._offsets_ptr
    if y is not None:
        ptrs |= _rows_ptr(y, "y", _BF16, M, ad.d_out, dev)
    if t is not None:
        ptrs |= _rows_ptr(t, "t", torch.float32, M, ad.rank, dev)
    if ptrs & 15:
        raise NQError("nq_adapter_forward", 3)
    if ad.workspace_bytes(M) == 0:
        raise NQError("nq_adapter_workspace_bytes", 2)


def adapter_forward(ad: Adapters, groups: AdapterRows, x: torch.Tensor, y: torch.Tensor, out=None, t=None,
                    stream=None) -> torch.Tensor:
    """out[m] = y[m] + scale_a B_a A_a x[m] for row m's adapter a (out[m] = y[m] without one).
    x [M][d_in], y [M][d_out] bf16; out may be y.  t [M][rank] fp32, if given, receives
    scale_a A_a x[m] for adapter_backward."""
    dev, M = ad.device, groups.M
    _check_groups(ad, groups)
    px = _rows_ptr(x, "x", _BF16, M, ad.d_in, dev)
    py = _rows_ptr(y, "y", _BF16, M, ad.d_out, dev)
    if out is None:
        out = torch.empty_like(y)
    po = _rows_ptr(out, "out", _BF16, M, ad.d_out, dev)
    pt = 0 if t is None else _rows_ptr(t, "t", torch.float32, M, ad.rank, dev)
    _call("nq_adapter_forward", _lib.nq_adapter_forward, dev, stream, ad._ref, groups._rows_ptr, groups._offsets_ptr, px,
          py, po, pt, M)
    return out


def adapter_backward(ad: Adapters, groups: AdapterRows, x, ybar: torch.Tensor, t, xbar, out=None, gA=None, gB=None,
                     need_x: bool = True, need_weights: bool = True, ws=None, stream=None):
    """(xbar + A_a^T u, gA, gB) with u[m] = scale_a B_a^T ybar[m]: the gradients of the input and of
    the adapters for the output's gradient ybar [M][d_out] bf16.  xbar [M][d_in] bf16 is the shared
    projection's share (lrb_transposed), out may be xbar; t is what adapter_forward wrote.  gA
    [n][rank][d_in], gB [n][d_out][rank] bf16, contiguous.  need_x=False leaves xbar out (xbar may
    be None), need_weights=False leaves gA and gB out (x and t may be None): None in their place."""
    dev, M = ad.device, groups.M
    _check_groups(ad, groups)
    pyb = _rows_ptr(ybar, "ybar", _BF16, M, ad.d_out, dev)
    px = pt = pxb = po = pa = pb = 0
    if need_x:
        pxb = _rows_ptr(xbar, "xbar", _BF16, M, ad.d_in, dev)
        if out is None:
            out = torch.empty_like(xbar)
        po = _rows_ptr(out, "out", _BF16, M, ad.d_in, dev)
    else:
        out = None
    if need_weights:
        px = _rows_ptr(x, "x", _BF16, M, ad.d_in, dev)
        pt = _rows_ptr(t, "t", torch.float32, M, ad.rank, dev)
        if gA is None:
            gA = torch.empty((ad.n, ad.rank, ad.d_in), dtype=_BF16, device=dev)
        if gB is None:
            gB = torch.empty((ad.n, ad.d_out, ad.rank), dtype=_BF16, device=dev)
        pa = _array_ptr(gA, "gA", _BF16, (ad.n, ad.rank, ad.d_in), dev)
        pb = _array_ptr(gB, "gB", _BF16, (ad.n, ad.d_out, ad.rank), dev)
    else:
        gA = gB = None
    if ws is None:
        ws = _workspace_of(ad, M, dev, stream)
    pw = _ws_ptr(ws, dev)
    _call("nq_adapter_backward", _lib.nq_adapter_backward, dev, stream, ad._ref, groups._rows_ptr, groups._offsets_ptr,
          px, pyb, pt, pxb, po, pa, pb, M, pw, ws.numel())
    return out, gA, gB


class BlockNorm:
    """The norms between two blocks (see nq.h): w_pre, w_post [d] bf16 or None (ones); post_norm: the
    block's output is normed before the residual; alpha: residual scale; w_offset is added to the
    weights."""

    def __init__(self, d: int, w_pre=None, w_post=None, post_norm: bool = False, alpha: float = 1.0,
                 eps: float = 1e-5, w_offset: float = 0.0):
        self.d = int(d)
        self.device = None
        for w, name in ((w_pre, "w_pre"), (w_post, "w_post")):
            if w is not None:
                _need(w, name, torch.bfloat16, shape=(self.d,), device=self.device)
                self.device = w.device
        self.w_pre, self.w_post, self.post_norm = w_pre, w_post, bool(post_norm)
        self._structs = {}
        for f32, dtype in ((0, torch.bfloat16), (1, torch.float32)):
            s = nq_block_norm(self.d, _ptr(w_pre), _ptr(w_post), w_offset, alpha, eps, int(self.post_norm), f32)
            self._structs[dtype] = (s, ctypes.byref(s))
        self._ws = {}

    def workspace_bytes(self, M: int, device=None) -> int:
        with _on(torch.device(device) if device is not None else self.device):  # the size goes by the device's multiprocessors
            return int(_lib.nq_block_norm_workspace_bytes(self._structs[torch.float32][1], int(M)))

    def workspace(self, M: int, device=None) -> torch.Tensor:
        """A workspace large enough for M rows, cached here and grown on demand.  Every backward
        call outside a capture that passes no ``ws`` uses it: calls that may run at the same time on
        the GPU must each pass their own.  A captured call that passes none gets one that belongs to
        the graph; one that is passed must outlive the graph (this cache drops the smaller when it grows)."""
        device = torch.device(device if device is not None else self.device if self.device is not None else "cuda")
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        need = self.workspace_bytes(M, device)
        if need == 0:
            raise NQError("nq_block_norm_workspace_bytes", 2)
        ws = self._ws.get(device)
        if ws is None or ws.numel() < need:
            ws = self._ws[device] = torch.empty(need, dtype=torch.uint8, device=device)
        return ws

    def _struct(self, h):
        try:
            return self._structs[h.dtype][1]
        except KeyError:
            raise ValueError("h: expected bfloat16 or float32, got %s" % h.dtype) from None


def _check_h(norm: BlockNorm, h, name: str):
    """(M, device, the parameters for h's type) of a residual tensor."""
    if not isinstance(h, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %s" % (name, type(h).__name__))
    if h.dim() != 2 or h.shape[1] != norm.d:
        raise ValueError("%s: expected [M][%d], got shape %s" % (name, norm.d, tuple(h.shape)))
    params = norm._struct(h)
    if not h.is_cuda or not h.is_contiguous() or (norm.device is not None and norm.device != h.device):
        _need(h, name, h.dtype, device=norm.device)
    return h.shape[0], h.device, params


def _check_gate(norm: BlockNorm, gate, M: int, device):
    """(address, row stride) of a gate [d] (stride 0) or [M][d]."""
    if gate is None:
        return 0, 0
    if isinstance(gate, torch.Tensor) and gate.dim() == 2:
        _need_rows(gate, "gate", _BF16, M, norm.d, device=device)
        if gate.shape[1] != norm.d or gate.stride(0) < norm.d and M > 1:
            raise ValueError("gate: expected [%d] or [%d][%d], got shape %s strides %s" %
                             (norm.d, M, norm.d, tuple(gate.shape), tuple(gate.stride())))
        return gate.data_ptr(), max(int(gate.stride(0)), norm.d)
    return _array_ptr(gate, "gate", _BF16, (norm.d,), device), 0


def block_norm(norm: BlockNorm, y, h: torch.Tensor, gate=None, h_out=None, x=None, stream=None):
    """(h_out, x): h_out = alpha h + gate * z with z the (normed) block output y, x the normed h_out
    for the next block.  y [M][d] bf16 or None, h [M][d] bf16 or fp32, gate [d] or [M][d] bf16 or
    None.  h_out may be h, x may be y."""
    M, dev, params = _check_h(norm, h, "h")
    d = norm.d
    py = 0 if y is None else _rows_ptr(y, "y", _BF16, M, d, dev)
    pg, ldg = _check_gate(norm, gate, M, dev)
    if h_out is None:
        h_out = torch.empty_like(h)
    ph = _rows_ptr(h_out, "h_out", h.dtype, M, d, dev)
    if x is None:
        x = torch.empty((M, d), dtype=_BF16, device=dev)
    px = _rows_ptr(x, "x", _BF16, M, d, dev)
    _call("nq_block_norm_forward", _lib.nq_block_norm_forward, dev, stream, params, py, h.data_ptr(), pg, ldg, ph, px, M)
    return h_out, x


def block_norm_backward(norm: BlockNorm, y, h_out: torch.Tensor, gx, gh_out, gate=None, gh=None, gy=None,
                        g_w_pre=None, g_w_post=None, g_gate=None, need_weights: bool = True, ws=None, stream=None):
    """(gh, gy, g_w_pre, g_w_post, g_gate) for the gradients gx [M][d] bf16 of x and gh_out (h's type)
    of h_out; either may be None (zero).  y, gate: as in the forward call, h_out what it returned.
    gy and g_gate are None without y or gate, g_w_post without post_norm or w_post, g_w_pre without
    w_pre; need_weights=False leaves g_w_pre, g_w_post and a shared gate's g_gate out.  g_w_pre,
    g_w_post and the g_gate of one shared gate are fp32 [d], the g_gate of a gate per row bf16
    [M][d].  gh may be gh_out, gy may be gx."""
    M, dev, params = _check_h(norm, h_out, "h_out")
    d = norm.d
    py = 0 if y is None else _rows_ptr(y, "y", _BF16, M, d, dev)
    pgx = 0 if gx is None else _rows_ptr(gx, "gx", _BF16, M, d, dev)
    pg, ldg = _check_gate(norm, gate, M, dev)
    pgo = 0 if gh_out is None else _rows_ptr(gh_out, "gh_out", h_out.dtype, M, d, dev)

    def vector(v, name, wanted):
        if not wanted:
            return None, 0
        if v is None:
            v = torch.empty(d, dtype=torch.float32, device=dev)
        return v, _array_ptr(v, name, torch.float32, (d,), dev)

    def rows(v, name, dtype):
        if v is None:
            v = torch.empty((M, d), dtype=dtype, device=dev)
        return v, _rows_ptr(v, name, dtype, M, d, dev)

    gh, pgh = rows(gh, "gh", h_out.dtype)
    gy, pgy = (None, 0) if y is None else rows(gy, "gy", _BF16)
    g_w_pre, pwp = vector(g_w_pre, "g_w_pre", need_weights and norm.w_pre is not None)
    g_w_post, pwo = vector(g_w_post, "g_w_post",
                           need_weights and norm.post_norm and norm.w_post is not None and y is not None)
    if gate is None or y is None:
        g_gate, pgg = None, 0
    elif ldg == 0:
        g_gate, pgg = vector(g_gate, "g_gate", need_weights)
    else:
        g_gate, pgg = rows(g_gate, "g_gate", _BF16)
    if ws is None:
        ws = _workspace_of(norm, M, dev, stream)
    pw = _ws_ptr(ws, dev)
    _call("nq_block_norm_backward", _lib.nq_block_norm_backward, dev, stream, params, py, h_out.data_ptr(), pg, ldg, pgx,
          pgo, pgh, pgy, pwp, pwo, pgg, M, pw, ws.numel())
    return gh, gy, g_w_pre, g_w_post, g_gate


def selftest_bounded_wait(limit_us: int = 20000, stream=None) -> None:
    """Launch the diagnostic kernel whose bounded wait runs out (see nq.h); the next
    sync_status raises NQError with NQ_ERR_TIMEOUT."""
    _check("nq_selftest_bounded_wait", _lib.nq_selftest_bounded_wait(int(limit_us), _stream_ptr(stream)))


def sync_status(stream=None) -> None:
    _check("nq_sync_status", _lib.nq_sync_status(_stream_ptr(stream)))


def raw_lib() -> ctypes.CDLL:
    """The loaded libnq.so (for callers that marshal arguments themselves)."""
    return _lib
