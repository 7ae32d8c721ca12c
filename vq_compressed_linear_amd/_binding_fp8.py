"""ctypes binding of libhxq's 8-bit path: argument marshalling only, as in
_binding.

8-bit values are torch.float8_e4m3fn tensors whose rows are padded with zeros
to a multiple of 128 columns, their scales torch.float8_e8m0fnu tensors whose
rows are padded with ones to a multiple of 4 (see include/hxq.h).  Every
function checks shapes, types and devices on the host and raises before the
library is reached; nothing is computed here.  All tensors are contiguous, but
for a product's scales: those of a transposed weight, which exchanging two
dimensions gives with other strides, are copied for the call where they are
not (one byte for each 16384 of the weight's).
"""

from __future__ import annotations

import contextlib
import functools

import torch

from . import _binding as B

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu

_DTYPE = {torch.float32: B.HXQ_F32, torch.bfloat16: B.HXQ_BF16, E4M3: B.HXQ_E4M3}
_NO_GUARD = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def fp8_columns(k: int) -> int:
    """Columns of an e4m3 row of k values."""
    return (k + 127) // 128 * 128


def fp8_scale_columns(k: int) -> int:
    """Entries of its row of scales."""
    return (k + 511) // 512 * 4


def _dtype(t, what: str, e4m3: bool = False) -> int:
    d = _DTYPE.get(t.dtype)
    if d is None or (d == B.HXQ_E4M3 and not e4m3):
        raise TypeError("%s must be float32%s or bfloat16, got %s" % (what, ", float8_e4m3fn" if e4m3 else "", t.dtype))
    return d


def _tensor(t, what: str, dtype, shape) -> None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s %s tensor, got %s %s%s" % (
            what, dtype, tuple(shape), t.dtype, tuple(t.shape), "" if t.is_contiguous() else ", not contiguous"))


def _scales(t, what: str, shape) -> None:
    """A product's scales: any strides (_laid_out copies)."""
    if t.dtype is not E8M0 or t.shape != shape:
        raise ValueError("%s must be a %s %s tensor, got %s %s" % (what, E8M0, tuple(shape), t.dtype, tuple(t.shape)))


def _matrix(t, what: str):
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous matrix" % what)
    return t.shape


def _device(*tensors) -> int:
    """Index of the one GPU that every tensor given (None skipped) lives on: the kernels read raw device pointers,
    and a host tensor's would fault them."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("every tensor must be on a GPU; got one on %s" % t.device)
                if dev is not None:
                    raise ValueError("tensors on different devices: cuda:%d and cuda:%d" % (dev, d))
                dev = d
    return dev


def _on(dev: int):
    """Launches go to the tensors' device, whichever is current."""
    return _NO_GUARD if torch.cuda.current_device() == dev else torch.cuda.device(dev)


def _stream(stream, dev: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return B._stream(stream, dev)


def _queue(stream, dev: int):
    """Torch's work for a launch goes to the launch's stream, and its allocations belong there: their memory is not
    handed out again to work that does not wait for the launch."""
    if stream is None:
        return _NO_GUARD  # (the device's current one, and _on has made the device current)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(B._stream(stream), dev)
    return torch.cuda.stream(stream)


def _laid_out(t, dev: int, stream):
    """A product's scales, contiguous; to be kept until the launch is queued."""
    if t is None or t.is_contiguous():
        return t
    with _queue(stream, dev):
        return t.view(torch.uint8).contiguous()


@functools.lru_cache(maxsize=4096)
def _need(dev: int, query: str, *sizes) -> int:
    """A workspace query's answer for the device (it depends on nothing else)."""
    with _on(dev):
        return getattr(B.lib(), query)(*sizes)


def _workspace(workspace, need: int, what: str, dev: int, stream):
    """(pointer, bytes) of the caller's workspace, or of one from torch's caching allocator; the tensor is the
    third, to be kept until the launch is queued."""
    if need < 0:
        raise B.HxqError(need, what)
    if workspace is None:
        if need == 0:
            return None, 0, None
        with _queue(stream, dev):
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    n = workspace.numel() * workspace.element_size()
    return (workspace.data_ptr() if n else None), n, workspace


def hxq_quant_fp8(x, q, scales, stream=None) -> None:
    """q, scales <- the rows of x (float32 or bfloat16 [M, K]) in e4m3 with a power of two for each 128 columns."""
    M, K = _matrix(x, "x")
    dt = _dtype(x, "x")
    _tensor(q, "q", E4M3, (M, fp8_columns(K)))
    _tensor(scales, "scales", E8M0, (M, fp8_scale_columns(K)))
    dev = _device(x, q, scales)
    with _on(dev):
        st = B.lib().hxq_quant_fp8(x.data_ptr(), dt, q.data_ptr(), scales.data_ptr(), M, K, _stream(stream, dev))
    if st != B.HXQ_OK:
        raise B.HxqError(st, "hxq_quant_fp8")


def hxq_quant_fp8_weight(w, q, scales, qt=None, scales_t=None, stream=None) -> None:
    """q, scales <- the weight w (float32 or bfloat16 [N, K], or [E, N, K] for experts) in e4m3 with a power of two
    for each 128 x 128 block; qt, scales_t <- its transposed copy, where given."""
    if w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w must be a contiguous [N, K] or [E, N, K] tensor")
    lead = w.shape[:-2]
    N, K = w.shape[-2:]
    dt = _dtype(w, "w")
    _tensor(q, "q", E4M3, lead + (N, fp8_columns(K)))
    _tensor(scales, "scales", E8M0, lead + ((N + 127) // 128, fp8_scale_columns(K)))
    if (qt is None) != (scales_t is None):
        raise ValueError("qt and scales_t are given both or neither")
    if qt is not None:
        _tensor(qt, "qt", E4M3, lead + (K, fp8_columns(N)))
        _tensor(scales_t, "scales_t", E8M0, lead + ((K + 127) // 128, fp8_scale_columns(N)))
    dev = _device(w, q, scales, qt, scales_t)
    with _on(dev):
        st = B.lib().hxq_quant_fp8_weight(w.data_ptr(), dt, q.data_ptr(), scales.data_ptr(), B._ptr(qt),
                                          B._ptr(scales_t), lead[0] if lead else 1, N, K, _stream(stream, dev))
    if st != B.HXQ_OK:
        raise B.HxqError(st, "hxq_quant_fp8_weight")


def _activations(x, x_scales, Kp):
    """(rows, K, dtype) of a product's input: e4m3 with its scales, or the values themselves."""
    M, cols = _matrix(x, "x")
    dt = _dtype(x, "x", e4m3=True)
    if dt == B.HXQ_E4M3:
        if cols != Kp:
            raise ValueError("x has %d columns, the layer's rows %d" % (cols, Kp))
        if x_scales is None:
            raise ValueError("e4m3 x needs its scales")
        _scales(x_scales, "x_scales", (M, fp8_scale_columns(Kp)))
    else:
        if x_scales is not None:
            raise ValueError("x_scales goes with e4m3 x")
        if fp8_columns(cols) != Kp:
            raise ValueError("x has K=%d, the layer's rows %d columns" % (cols, Kp))
    return M, cols, dt


def hxq_linear_fwd_fp8(x, x_scales, wq, w_scales, bias, y, stream=None, workspace=None) -> None:
    """y <- x W^T + bias for an 8-bit layer wq [N, Kp], w_scales.  x is float32 or bfloat16 [M, K] (x_scales None),
    or e4m3 [M, Kp] with its scales; y float32 or bfloat16 [M, N]; bias float32 [N] or None.  With dy as x and a
    transposed copy as the layer it is the input gradient.  ``workspace``: a device tensor of at least the bytes the
    library asks for; when None, one is taken from torch's caching allocator."""
    if wq.dtype != E4M3 or wq.dim() != 2 or not wq.is_contiguous() or wq.shape[1] % 128:
        raise ValueError("wq must be a contiguous float8_e4m3fn [N, multiple of 128] tensor")
    N, Kp = wq.shape
    M, K, dt = _activations(x, x_scales, Kp)
    _scales(w_scales, "w_scales", ((N + 127) // 128, fp8_scale_columns(Kp)))
    ydt = _dtype(y, "y")
    _tensor(y, "y", y.dtype, (M, N))
    if bias is not None:
        _tensor(bias, "bias", torch.float32, (N,))
    dev = _device(x, x_scales, wq, w_scales, bias, y, workspace)
    lib = B.lib()
    with _on(dev):
        ptr, size, keep = _workspace(workspace, _need(dev, "hxq_linear_fwd_fp8_workspace", dt, M, N, K),
                                     "hxq_linear_fwd_fp8_workspace", dev, stream)
        x_scales, w_scales = _laid_out(x_scales, dev, stream), _laid_out(w_scales, dev, stream)
        st = lib.hxq_linear_fwd_fp8(x.data_ptr(), dt, B._ptr(x_scales), wq.data_ptr(), w_scales.data_ptr(),
                                    B._ptr(bias), y.data_ptr(), ydt, M, N, K, ptr, size, _stream(stream, dev))
    if st != B.HXQ_OK:
        raise B.HxqError(st, "hxq_linear_fwd_fp8")


def hxq_linear_fwd_fp8_experts(x, x_scales, rows, offsets, wq, w_scales, bias, y, stream=None,
                               workspace=None) -> None:
    """y[r] <- W_e x[rows[r]] + bias[e] for the rows r of expert e, offsets[e] <= r < offsets[e + 1], in one launch;
    rows of y past offsets[E] are left as they are.  wq [E, N, Kp] and w_scales hold the experts; rows int32 [M] or
    None (x[r]); offsets int32 [E + 1]; bias float32 [E, N] or None; y [M, N]; the rest as for
    hxq_linear_fwd_fp8."""
    if wq.dtype != E4M3 or wq.dim() != 3 or not wq.is_contiguous() or wq.shape[2] % 128:
        raise ValueError("wq must be a contiguous float8_e4m3fn [E, N, multiple of 128] tensor")
    E, N, Kp = wq.shape
    Mx, K, dt = _activations(x, x_scales, Kp)
    _scales(w_scales, "w_scales", (E, (N + 127) // 128, fp8_scale_columns(Kp)))
    _tensor(offsets, "offsets", torch.int32, (E + 1,))
    M = _matrix(y, "y")[0]
    ydt = _dtype(y, "y")
    _tensor(y, "y", y.dtype, (M, N))
    if rows is not None:
        _tensor(rows, "rows", torch.int32, (M,))
    elif Mx != M:
        raise ValueError("x has %d rows, y %d: without `rows` they are the same" % (Mx, M))
    if bias is not None:
        _tensor(bias, "bias", torch.float32, (E, N))
    dev = _device(x, x_scales, rows, offsets, wq, w_scales, bias, y, workspace)
    lib = B.lib()
    with _on(dev):
        ptr, size, keep = _workspace(workspace, _need(dev, "hxq_linear_fwd_fp8_experts_workspace", dt, Mx, M, E, N, K),
                                     "hxq_linear_fwd_fp8_experts_workspace", dev, stream)
        x_scales, w_scales = _laid_out(x_scales, dev, stream), _laid_out(w_scales, dev, stream)
        st = lib.hxq_linear_fwd_fp8_experts(x.data_ptr(), dt, B._ptr(x_scales), B._ptr(rows), offsets.data_ptr(),
                                            wq.data_ptr(), w_scales.data_ptr(), B._ptr(bias), y.data_ptr(), ydt, Mx,
                                            M, E, N, K, ptr, size, _stream(stream, dev))
    if st != B.HXQ_OK:
        raise B.HxqError(st, "hxq_linear_fwd_fp8_experts")


def hxq_rms_norm(x, weight, eps: float, out, scales=None, residual=None, residual_out=None, rstd=None,
                 stream=None) -> None:
    """out <- h / sqrt(mean h^2 + eps) * weight with h = x + residual, and residual_out <- h (rounded to the
    residual's type; the norm is of the rounded sum).  x and residual float32 or bfloat16 [M, K]; weight float32 [K]
    or None; out float32 or bfloat16 [M, K], or e4m3 [M, fp8_columns(K)] with its scales; rstd float32 [M] or
    None."""
    M, K = _matrix(x, "x")
    dt = _dtype(x, "x")
    odt = _dtype(out, "out", e4m3=True)
    if odt == B.HXQ_E4M3:
        _tensor(out, "out", E4M3, (M, fp8_columns(K)))
        if scales is None:
            raise ValueError("e4m3 out needs scales")
        _tensor(scales, "scales", E8M0, (M, fp8_scale_columns(K)))
    else:
        _tensor(out, "out", out.dtype, (M, K))
        if scales is not None:
            raise ValueError("scales goes with e4m3 out")
    if weight is not None:
        _tensor(weight, "weight", torch.float32, (K,))
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out are given both or neither")
    rdt = 0
    if residual is not None:
        rdt = _dtype(residual, "residual")
        _tensor(residual, "residual", residual.dtype, (M, K))
        _tensor(residual_out, "residual_out", residual.dtype, (M, K))
    if rstd is not None:
        _tensor(rstd, "rstd", torch.float32, (M,))
    dev = _device(x, weight, out, scales, residual, residual_out, rstd)
    with _on(dev):
        st = B.lib().hxq_rms_norm(x.data_ptr(), dt, B._ptr(residual), rdt, B._ptr(weight), eps, B._ptr(residual_out),
                                  out.data_ptr(), odt, B._ptr(scales), B._ptr(rstd), M, K, _stream(stream, dev))
    if st != B.HXQ_OK:
        raise B.HxqError(st, "hxq_rms_norm")


def hxq_rms_norm_bwd(dy, h, weight, rstd, dx, dweight=None, dresidual=None, stream=None, workspace=None) -> None:
    """dx <- the gradient of hxq_rms_norm's x (and residual) for dy, plus dresidual; dweight <- the weight's.  h is
    the forward's residual_out (x without a residual) and rstd what it gave; dx, dresidual float32 [M, K]."""
    M, K = _matrix(dy, "dy")
    dt = _dtype(dy, "dy")
    hdt = _dtype(h, "h")
    _tensor(h, "h", h.dtype, (M, K))
    _tensor(rstd, "rstd", torch.float32, (M,))
    _tensor(dx, "dx", torch.float32, (M, K))
    if weight is not None:
        _tensor(weight, "weight", torch.float32, (K,))
    if dweight is not None:
        _tensor(dweight, "dweight", torch.float32, (K,))
    if dresidual is not None:
        _tensor(dresidual, "dresidual", torch.float32, (M, K))
    dev = _device(dy, h, weight, rstd, dx, dweight, dresidual, workspace)
    lib = B.lib()
    with _on(dev):
        need = 0 if dweight is None else _need(dev, "hxq_rms_norm_bwd_workspace", M, K)
        ptr, size, keep = _workspace(workspace, need, "hxq_rms_norm_bwd_workspace", dev, stream)
        st = lib.hxq_rms_norm_bwd(dy.data_ptr(), dt, h.data_ptr(), hdt, B._ptr(weight), rstd.data_ptr(),
                                  B._ptr(dresidual), dx.data_ptr(), B._ptr(dweight), M, K, ptr, size,
                                  _stream(stream, dev))
    if st != B.HXQ_OK:
        raise B.HxqError(st, "hxq_rms_norm_bwd")
