"""Python binding of the sm_100a QE linear-layer library (libqe.so, C ABI in include/qe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. PyTorch supplies device memory and the current stream. Importing
works without a GPU (the tests check the exported symbols on CPU). Every
compute call raises QEError when the library is missing or a call fails.
There is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqe.so")

QE_OK, QE_ERR_INVALID_ARG, QE_ERR_UNSUPPORTED, QE_ERR_ALIGNMENT, QE_ERR_WORKSPACE, QE_ERR_CUDA, QE_ERR_TIMEOUT = range(7)
QE_F32, QE_BF16 = 0, 1

# Every symbol include/qe.h declares (the tests check that the library exports them).
EXPORTS = (
    "qe_packed_weight_bytes", "qe_adapter_packed_bytes", "qe_linear_workspace_bytes", "qe_quantize_weights",
    "qe_pack_adapters", "qe_topk_importance", "qe_route", "qe_linear_forward", "qe_status_string",
    "qe_last_cuda_error", "qe_device_error", "qe_unpack_weights", "qe_act_quant", "qe_linear_forward_debug",
    "qe_linear_forward_stages", "qe_linear_kernel_launches", "qe_linear_forward_noalloc",
    "qe_selftest_wait_timeout", "qe_split_channels", "qe_cooccurrence_npmi", "qe_pack_adapters_sparse",
    "qe_linear_plan", "qe_add_rmsnorm_quant", "qe_act_dequant", "qe_mx4_code_bytes", "qe_mx4_scale_bytes",
    "qe_mx4_quantize", "qe_mx4_dequantize", "qe_mx4_product", "qe_mx4_linear_workspace_bytes",
    "qe_mx4_linear_forward", "qe_linear_forward_codes",
)
# fixed scratch of qe_linear_forward_noalloc (bytes), as declared in include/qe.h
NOALLOC_WORKSPACE_BYTES = 32 << 20
QE_STAGE_PROJECT, QE_STAGE_ROUTE, QE_STAGE_QUANT, QE_STAGE_PRODUCT, QE_STAGE_ALL = 1, 2, 4, 8, 15


class QEError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        msg = f"{what} failed: status {status}"
        if _LIB is not None:
            msg += f" ({_LIB.qe_status_string(status).decode()})"
        if detail:
            msg += f": {detail}"
        super().__init__(msg)


class LayerDesc(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("group", ctypes.c_int32),
                ("w_bits", ctypes.c_int32), ("a_bits", ctypes.c_int32), ("rank_shared", ctypes.c_int32),
                ("n_routed", ctypes.c_int32), ("rank_routed", ctypes.c_int32), ("routed_channels", ctypes.c_int32),
                ("w_scale_fp16", ctypes.c_int32)]

    def __repr__(self):
        return "LayerDesc(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class LinearPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("product_tile_tokens", "product_k_splits", "adapter_atoms",
                                              "adapter_gemm_width", "adapter_gemm_tile", "adapter_gemm_splits",
                                              "weight_only")] + [("workspace_bytes", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("decode_product", "decode_ctas", "decode_max_segments")]


class LayerWeights(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("s_inv", ctypes.c_void_p),
                ("adapters", ctypes.c_void_p)]


_LIB: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Loads libqe.so (built by quantized_gemm_moe_b200.build). Raises when it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise QEError(-1, "load", f"{LIB_PATH} is missing; build it with `python -m quantized_gemm_moe_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(LayerDesc)
    sigs = {
        "qe_packed_weight_bytes": ([D], S),
        "qe_adapter_packed_bytes": ([D], S),
        "qe_linear_workspace_bytes": ([D, I], S),
        "qe_quantize_weights": ([D, P, I, P, P, P, P, P, P, P], I),
        "qe_pack_adapters": ([D, P, P, P, P, P, P, P], I),
        "qe_pack_adapters_sparse": ([D, P, P, P, P, P, P, P, P], I),
        "qe_topk_importance": ([P, I, P, I, I, I, P, P, I, P], I),
        "qe_route": ([P, I, P, I, I, I, P, P, P, P, P], I),
        "qe_linear_forward": ([D, ctypes.POINTER(LayerWeights), P, I, I, P, I, P, S, P], I),
        "qe_linear_forward_debug": ([D, ctypes.POINTER(LayerWeights), P, I, I, P, I, P, S, P, P, P, P, P], I),
        "qe_linear_forward_stages": ([D, ctypes.POINTER(LayerWeights), P, I, I, P, I, P, S, I, P], I),
        "qe_linear_kernel_launches": ([D, I, I], I),
        "qe_linear_plan": ([D, I, I, ctypes.POINTER(LinearPlan)], I),
        "qe_linear_forward_noalloc": ([D, ctypes.POINTER(LayerWeights), P, I, I, P, I, P], I),
        "qe_status_string": ([I], ctypes.c_char_p),
        "qe_last_cuda_error": ([], ctypes.c_char_p),
        "qe_device_error": ([P, ctypes.POINTER(I), I], I),
        "qe_unpack_weights": ([D, P, P, P], I),
        "qe_act_quant": ([P, I, P, I, I, I, P, P, P], I),
        "qe_selftest_wait_timeout": ([I, P], I),
        "qe_split_channels": ([P, I, I, I, P, P], I),
        "qe_cooccurrence_npmi": ([P, I, I, P, I, I, P, P, ctypes.c_float, P], I),
        "qe_linear_forward_codes": ([D, ctypes.POINTER(LayerWeights), P, I, P, P, I, P, I, P, S, P], I),
        "qe_add_rmsnorm_quant": ([P, I, P, P, I, ctypes.c_double, I, I, P, I, P, P, P, P, P], I),
        "qe_act_dequant": ([P, P, I, I, P, I, P], I),
        "qe_mx4_code_bytes": ([I, I], S),
        "qe_mx4_scale_bytes": ([I, I], S),
        "qe_mx4_quantize": ([P, I, P, I, I, P, P, P, P], I),
        "qe_mx4_dequantize": ([P, P, I, I, P, I, P], I),
        "qe_mx4_product": ([P, P, P, P, I, I, I, P, I, P], I),
        "qe_mx4_linear_workspace_bytes": ([I, I], S),
        "qe_mx4_linear_forward": ([P, P, P, P, I, I, I, I, P, I, P, S, P], I),
    }
    for name, (args, res) in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _LIB = L
    return L


# ---------------------------------------------------------------- marshalling helpers

def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return QE_F32
    if t.dtype == torch.bfloat16:
        return QE_BF16
    raise QEError(QE_ERR_INVALID_ARG, "dtype", f"unsupported dtype {t.dtype}")


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, what: str):
    if rc != QE_OK:
        detail = load().qe_last_cuda_error().decode() if rc == QE_ERR_CUDA else ""
        raise QEError(rc, what, detail)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise QEError(QE_ERR_INVALID_ARG, "device", "tensors passed to the QE library must be CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise QEError(QE_ERR_INVALID_ARG, "layout", "tensors passed to the QE library must be contiguous")


def make_desc(d_in, d_out, group=128, w_bits=4, a_bits=8, rank_shared=32, n_routed=8, rank_routed=4,
              routed_channels=0, w_scale_fp16=0) -> LayerDesc:
    """routed_channels > 0: cluster-sparse routed experts over that many channels each.
    w_scale_fp16 = 1: the weight group scales are stored as fp16."""
    return LayerDesc(d_in, d_out, group, w_bits, a_bits, rank_shared, n_routed, rank_routed, routed_channels,
                     1 if w_scale_fp16 else 0)


# ---------------------------------------------------------------- the C ABI, one wrapper per entry point

def packed_weight_bytes(desc: LayerDesc) -> int:
    return int(load().qe_packed_weight_bytes(ctypes.byref(desc)))


def adapter_packed_bytes(desc: LayerDesc) -> int:
    return int(load().qe_adapter_packed_bytes(ctypes.byref(desc)))


def linear_workspace_bytes(desc: LayerDesc, T: int) -> int:
    return int(load().qe_linear_workspace_bytes(ctypes.byref(desc), T))


def quantize_weights(desc, W, s, w_packed, w_scale, w_mean=None, w_colmax=None, s_inv=None, stream=None):
    _need_cuda(W, s, w_packed, w_scale, w_mean, w_colmax, s_inv)
    _check(load().qe_quantize_weights(ctypes.byref(desc), _ptr(W), _dtype(W), _ptr(s), _ptr(w_packed),
                                      _ptr(w_scale), _ptr(w_mean), _ptr(w_colmax), _ptr(s_inv), _stream(stream)),
           "qe_quantize_weights")


def pack_adapters(desc, A_s, B_s, A_r, B_r, G, out, stream=None):
    _need_cuda(A_s, B_s, A_r, B_r, G, out)
    _check(load().qe_pack_adapters(ctypes.byref(desc), _ptr(A_s), _ptr(B_s), _ptr(A_r), _ptr(B_r), _ptr(G),
                                   _ptr(out), _stream(stream)), "qe_pack_adapters")


def pack_adapters_sparse(desc, A_s, B_s, channels, A_r, B_r, G, out, stream=None):
    """Cluster-sparse routed experts: channels int32 [N_r][k_c], A_r bf16 [N_r][k_c][r_r]."""
    _need_cuda(A_s, B_s, channels, A_r, B_r, G, out)
    _check(load().qe_pack_adapters_sparse(ctypes.byref(desc), _ptr(A_s), _ptr(B_s), _ptr(channels), _ptr(A_r),
                                          _ptr(B_r), _ptr(G), _ptr(out), _stream(stream)), "qe_pack_adapters_sparse")


def topk_importance(X, w_mean, k, idx, hist=None, accumulate=False, stream=None):
    _need_cuda(X, w_mean, idx, hist)
    T, K = X.shape
    _check(load().qe_topk_importance(_ptr(X), _dtype(X), _ptr(w_mean), T, K, k, _ptr(idx), _ptr(hist),
                                     1 if accumulate else 0, _stream(stream)), "qe_topk_importance")


def split_channels(hist, k, C, channel_pos, stream=None):
    """channel_pos[c] = rank(c) - k for the C channels after the k most frequent ones, else -1."""
    _need_cuda(hist, channel_pos)
    _check(load().qe_split_channels(_ptr(hist), hist.numel(), k, C, _ptr(channel_pos), _stream(stream)),
           "qe_split_channels")


def cooccurrence_npmi(idx, channel_pos, C, O, S=None, threshold=-1.0, stream=None):
    """Counts O[i][j] (int32 [C][C]) and, when S is given, writes their NPMI into S (fp32 [C][C])."""
    _need_cuda(idx, channel_pos, O, S)
    T, k = idx.shape
    _check(load().qe_cooccurrence_npmi(_ptr(idx), T, k, _ptr(channel_pos), channel_pos.numel(), C, _ptr(O), _ptr(S),
                                       float(threshold), _stream(stream)), "qe_cooccurrence_npmi")


def route(X, G, expert, perm, offsets, logits=None, stream=None):
    _need_cuda(X, G, expert, perm, offsets, logits)
    T, K = X.shape
    _check(load().qe_route(_ptr(X), _dtype(X), _ptr(G), T, K, G.shape[1], _ptr(expert), _ptr(perm), _ptr(offsets),
                           _ptr(logits), _stream(stream)), "qe_route")


def linear_forward(desc, weights: LayerWeights, X, Y, workspace, stream=None):
    _need_cuda(X, Y, workspace)
    _check(load().qe_linear_forward(ctypes.byref(desc), ctypes.byref(weights), _ptr(X), _dtype(X), X.shape[0],
                                    _ptr(Y), _dtype(Y), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "qe_linear_forward")


def linear_forward_codes(desc, weights: LayerWeights, X, codes, sa, Y, workspace, stream=None):
    """qe_linear_forward for rows that add_rmsnorm_quant or act_quant quantized (codes int8 [T, d_in], sa [T])."""
    import torch
    T, K = _rows(X, "X")
    _expect(X, X.dtype, (T, desc.d_in), "X")
    _expect(Y, Y.dtype, (T, desc.d_out), "Y")
    _expect(codes, torch.int8, (T, K), "codes")
    _expect(sa, torch.float32, (T,), "sa")
    _launch("qe_linear_forward_codes", stream, ctypes.byref(desc), ctypes.byref(weights), X, _dtype(X), codes, sa, T, Y,
            _dtype(Y), workspace, workspace.numel() * workspace.element_size())


def linear_kernel_launches(desc: LayerDesc, T: int, x_dtype: int = QE_BF16) -> int:
    return int(load().qe_linear_kernel_launches(ctypes.byref(desc), T, x_dtype))


def linear_plan(desc: LayerDesc, T: int, x_dtype: int = QE_BF16) -> dict:
    """How the forward runs this layer for T tokens (tile width, splits, adapter atoms); host only."""
    out = LinearPlan()
    _check(load().qe_linear_plan(ctypes.byref(desc), T, x_dtype, ctypes.byref(out)), "qe_linear_plan")
    return {n: getattr(out, n) for n, _ in LinearPlan._fields_}


def linear_forward_stages(desc, weights: LayerWeights, X, Y, workspace, stages: int, stream=None):
    _need_cuda(X, Y, workspace)
    _check(load().qe_linear_forward_stages(ctypes.byref(desc), ctypes.byref(weights), _ptr(X), _dtype(X), X.shape[0],
                                           _ptr(Y), _dtype(Y), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), stages, _stream(stream)),
           "qe_linear_forward_stages")


def linear_forward_noalloc(desc, weights: LayerWeights, X, Y, stream=None):
    """qe_linear_forward using the library's fixed device scratch instead of a workspace.

    For callers that cannot allocate device memory. The scratch is shared by all
    calls; calls that overlap on the GPU race on it.
    """
    _need_cuda(X, Y)
    _check(load().qe_linear_forward_noalloc(ctypes.byref(desc), ctypes.byref(weights), _ptr(X), _dtype(X),
                                            X.shape[0], _ptr(Y), _dtype(Y), _stream(stream)),
           "qe_linear_forward_noalloc")


def linear_forward_debug(desc, weights, X, Y, workspace, acc=None, expert=None, perm=None, sa=None, stream=None):
    _need_cuda(X, Y, workspace, acc, expert, perm, sa)
    _check(load().qe_linear_forward_debug(ctypes.byref(desc), ctypes.byref(weights), _ptr(X), _dtype(X), X.shape[0],
                                          _ptr(Y), _dtype(Y), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _ptr(acc), _ptr(expert),
                                          _ptr(perm), _ptr(sa), _stream(stream)), "qe_linear_forward_debug")


def unpack_weights(desc, w_packed, codes, stream=None):
    _need_cuda(w_packed, codes)
    _check(load().qe_unpack_weights(ctypes.byref(desc), _ptr(w_packed), _ptr(codes), _stream(stream)),
           "qe_unpack_weights")


def act_quant(X, s_inv, a_bits, codes, sa, stream=None):
    _need_cuda(X, s_inv, codes, sa)
    T, K = X.shape
    _check(load().qe_act_quant(_ptr(X), _dtype(X), _ptr(s_inv), T, K, a_bits, _ptr(codes), _ptr(sa),
                               _stream(stream)), "qe_act_quant")


def _launch(what: str, stream, *args):
    """Calls the entry point on the device of its tensors, with that device's current stream unless one is
    given. Tensors are passed as their pointers, after a check that all are contiguous CUDA tensors of one
    device. (The current stream and device come from torch's raw getters: a decoded token's launch takes
    less time than torch.cuda.current_stream() builds its object in.)"""
    import torch
    dev, raw, Tensor = None, [], torch.Tensor
    for a in args:
        if isinstance(a, Tensor):
            i = a.get_device()
            if i < 0 or not a.is_contiguous():
                _need_cuda(a)
            if dev is None:
                dev = i
            elif i != dev:
                raise QEError(QE_ERR_INVALID_ARG, "device", f"{what}: tensors on devices {dev} and {i}")
            raw.append(a.data_ptr())
        else:
            raw.append(a)
    f = getattr(_LIB or load(), what)
    if stream is not None:
        raw.append(_stream(stream))
    else:
        raw.append(torch._C._cuda_getCurrentRawStream(dev))
    if dev == torch._C._cuda_getDevice():
        rc = f(*raw)
    else:
        with torch.cuda.device(dev):
            rc = f(*raw)
    if rc != QE_OK:
        _check(rc, what)


def _expect(t, dtype, shape, name: str):
    """Checks a tensor's type and shape (an int: its least number of elements) before its pointer is passed on."""
    if t.dtype != dtype or (t.numel() < shape if isinstance(shape, int) else t.shape != shape):
        raise QEError(QE_ERR_INVALID_ARG, name, f"expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")


def _rows(t, name: str):
    if t.dim() != 2:
        raise QEError(QE_ERR_INVALID_ARG, name, f"expected [rows, channels], got {tuple(t.shape)}")
    return t.shape


def _external(handle: int, like):
    import torch
    _need_cuda(like)
    return torch.cuda.ExternalStream(handle, device=like.device)


def _on(stream, like):
    """What is allocated inside belongs to the stream the call runs on (a torch stream, or a raw handle of the
    device of `like`), so the allocator never hands it to another stream, or out of a graph's capture, while it is
    in use."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else _external(int(stream), like))


def _scratch(shape, dtype, like):
    import torch
    return torch.empty(shape, dtype=dtype or torch.uint8, device=like.device)


def _raise(status: int, what: str, detail: str):
    raise QEError(status, what, detail)


@functools.cache
def _native():
    """The extension module of the operators below (csrc/qe_torch.cpp): it checks types, shapes, layout and
    devices and makes the library's call on the tensors' device, with its current stream unless one is given."""
    load()
    import torch  # noqa: F401  (the module's symbols)
    try:
        from . import _qe_torch
    except ImportError as e:
        raise QEError(-1, "load", f"{e}; build it with `python -m quantized_gemm_moe_b200.build`") from e
    _qe_torch.set_raise(_raise)
    return _qe_torch


def add_rmsnorm_quant(X, gamma, eps, a_bits, codes=None, scales=None, residual=None, residual_out=None, Y=None,
                      s_inv=None, stream=None):
    """RMS norm of X + residual, with the normed row in Y and quantized into codes and scales.

    a_bits 8/6: codes int8 [T, d], scales fp32 [T]; 4: MXFP4 codes uint8 [T, d/2] and mx4_scale_bytes(T, d)
    scale bytes; 16: neither.
    """
    _native().add_rmsnorm_quant(X, gamma, eps, a_bits, codes, scales, residual, residual_out, Y, s_inv,
                                None if stream is None else _stream(stream))


def act_dequant(codes, sa, out, stream=None):
    """out = codes * sa per token (fp32 or bf16)."""
    _native().act_dequant(codes, sa, out, None if stream is None else _stream(stream))


def mx4_code_bytes(rows: int, cols: int) -> int:
    return int(load().qe_mx4_code_bytes(rows, cols))


@functools.lru_cache(maxsize=1024)
def mx4_scale_bytes(rows: int, cols: int) -> int:
    return int(load().qe_mx4_scale_bytes(rows, cols))


def mx4_quantize(X, codes, scales, s=None, s_inv=None, stream=None):
    """MXFP4 of fl32(X * s): codes uint8 [rows, cols/2], scales uint8 [mx4_scale_bytes(rows, cols)].
    s_inv (fp32 [cols], with s) receives fl32(1/s)."""
    _native().mx4_quantize(X, codes, scales, s, s_inv, None if stream is None else _stream(stream))


def mx4_dequantize(codes, scales, out, stream=None):
    """The values of MXFP4 codes, in out's type (fp32 or bf16)."""
    _native().mx4_dequantize(codes, scales, out, None if stream is None else _stream(stream))


def mx4_product(x_codes, x_scales, w_codes, w_scales, Y, stream=None):
    """Y [T, d_out] = X . W^T of two MXFP4 matrices."""
    _native().mx4_product(x_codes, x_scales, w_codes, w_scales, Y, None if stream is None else _stream(stream))


@functools.lru_cache(maxsize=1024)
def mx4_linear_workspace_bytes(T: int, d_in: int) -> int:
    return int(load().qe_mx4_linear_workspace_bytes(T, d_in))


def mx4_linear_forward(w_codes, w_scales, X, Y, workspace, s_inv=None, stream=None):
    """Y = MXFP4(X * s_inv) . W^T for an MXFP4 W."""
    _native().mx4_linear_forward(w_codes, w_scales, X, Y, workspace, s_inv, None if stream is None else _stream(stream))


def device_error(clear: bool = True, stream=None) -> int:
    """Synchronizes the stream and returns the device error word (0 = no device wait ran out)."""
    code = ctypes.c_int32(0)
    rc = load().qe_device_error(_stream(stream), ctypes.byref(code), 1 if clear else 0)
    if rc not in (QE_OK, QE_ERR_TIMEOUT):
        _check(rc, "qe_device_error")
    return int(code.value)


def selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Launches one device wait that runs out after limit_us (it records code 0x107)."""
    _check(load().qe_selftest_wait_timeout(int(limit_us), _stream(stream)), "qe_selftest_wait_timeout")


# ---------------------------------------------------------------- a layer object (device buffers via torch)

class QELayer:
    """One QE linear layer resident on the GPU: quantized weights, scales and packed adapters.

    Built from full-precision weights with `from_float`. `forward` runs
    qe_linear_forward on the current stream.
    """

    def __init__(self, desc: LayerDesc, w_packed, w_scale, s_inv, adapters, w_mean=None, w_colmax=None):
        self.desc = desc
        self.w_packed, self.w_scale, self.s_inv, self.adapters = w_packed, w_scale, s_inv, adapters
        self.w_mean, self.w_colmax = w_mean, w_colmax
        self.weights = LayerWeights(w_packed.data_ptr(), w_scale.data_ptr(), s_inv.data_ptr(), adapters.data_ptr())
        self._ws = None

    @classmethod
    def from_float(cls, desc: LayerDesc, W, s, A_s, B_s, A_r, B_r, G, s_inv=None, stream=None,
                   channels=None) -> "QELayer":
        """W [d_out, d_in] (fp32/bf16), s [d_in] fp32, adapters/G bf16 in their natural layouts (CUDA tensors).

        s_inv (fp32 [d_in]) is the stored reciprocal smoothing factor the activations are
        multiplied by. When omitted, the library computes it (qe_quantize_weights writes
        fl32(1/s)). With desc.routed_channels > 0, A_r is bf16 [N_r][k_c][r_r] over `channels`
        (int32 [N_r][k_c]).
        """
        import torch
        dev = W.device
        K, N = desc.d_in, desc.d_out
        w_packed = torch.empty(packed_weight_bytes(desc), dtype=torch.uint8, device=dev)
        w_scale = torch.empty((K // desc.group, N), dtype=torch.float16 if desc.w_scale_fp16 else torch.float32,
                              device=dev)
        w_mean = torch.empty(K, dtype=torch.float32, device=dev)
        w_colmax = torch.empty(K, dtype=torch.float32, device=dev)
        s_inv_out = torch.empty(K, dtype=torch.float32, device=dev) if s_inv is None else None
        quantize_weights(desc, W, s, w_packed, w_scale, w_mean, w_colmax, s_inv_out, stream)
        adapters = torch.empty(adapter_packed_bytes(desc), dtype=torch.uint8, device=dev)
        if desc.routed_channels > 0:
            pack_adapters_sparse(desc, A_s, B_s, channels, A_r, B_r, G, adapters, stream)
        else:
            pack_adapters(desc, A_s, B_s, A_r, B_r, G, adapters, stream)
        if s_inv is None:
            s_inv = s_inv_out
        return cls(desc, w_packed, w_scale, s_inv.contiguous(), adapters, w_mean, w_colmax)

    def workspace(self, T: int):
        import torch
        need = linear_workspace_bytes(self.desc, T)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.w_packed.device)
        return self._ws

    def forward(self, X, out_dtype=None, Y=None, stream=None):
        import torch
        T = X.shape[0]
        if Y is None:
            Y = torch.empty((T, self.desc.d_out), dtype=out_dtype or X.dtype, device=X.device)
        linear_forward(self.desc, self.weights, X, Y, self.workspace(T), stream)
        return Y

    def forward_codes(self, X, codes, sa, out_dtype=None, Y=None, stream=None):
        """forward for rows that are already quantized (add_rmsnorm_quant with this layer's s_inv and a_bits)."""
        T = X.shape[0]
        with _on(stream, X):
            Y = _scratch((T, self.desc.d_out), out_dtype or X.dtype, X) if Y is None else Y
            ws = _scratch((max(256, linear_workspace_bytes(self.desc, T)),), None, X)
            linear_forward_codes(self.desc, self.weights, X, codes, sa, Y, ws, stream)
        return Y


class Mx4Layer:
    """One linear layer with its weights in MXFP4, resident on the GPU.

    Built from full-precision weights with `from_float`. `forward` quantizes its input (times s_inv) and
    multiplies; `forward_codes` takes the MXFP4 activations that add_rmsnorm_quant or mx4_quantize wrote.
    """

    def __init__(self, w_codes, w_scales, s_inv=None):
        self.w_codes, self.w_scales, self.s_inv = w_codes, w_scales, s_inv
        self.d_out, self.d_in = w_codes.shape[0], 2 * w_codes.shape[1]

    @classmethod
    def from_float(cls, W, s=None, stream=None) -> "Mx4Layer":
        """W [d_out, d_in] (fp32/bf16); s (fp32 [d_in]): the smoothing factors W is multiplied by, and the
        input by their reciprocals."""
        import torch
        N, K = _rows(W, "W")
        with _on(stream, W):
            codes = _scratch((N, K // 2), None, W)
            scales = _scratch((mx4_scale_bytes(N, K),), None, W)
            s_inv = None if s is None else _scratch((K,), torch.float32, W)
            mx4_quantize(W, codes, scales, s, s_inv, stream)
        return cls(codes, scales, s_inv)

    def forward(self, X, out_dtype=None, Y=None, stream=None):
        T = _rows(X, "X")[0]
        with _on(stream, X):
            Y = _scratch((T, self.d_out), out_dtype or X.dtype, X) if Y is None else Y
            ws = _scratch((mx4_linear_workspace_bytes(T, self.d_in),), None, X)
            mx4_linear_forward(self.w_codes, self.w_scales, X, Y, ws, self.s_inv, stream)
        return Y

    def forward_codes(self, codes, scales, out_dtype=None, Y=None, stream=None):
        import torch
        with _on(stream, codes):
            if Y is None:
                Y = _scratch((_rows(codes, "codes")[0], self.d_out), out_dtype or torch.bfloat16, codes)
            mx4_product(codes, scales, self.w_codes, self.w_scales, Y, stream)
        return Y
