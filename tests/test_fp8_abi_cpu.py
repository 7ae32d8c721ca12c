"""The 8-bit path's entry points without a GPU: every bad argument is refused
on the host, by the C ABI and by the binding, before anything is launched."""

import pytest
import torch

import vq_compressed_linear_amd as hx
from vq_compressed_linear_amd import _binding as B
from vq_compressed_linear_amd import _binding_fp8 as F

FAKE = 0x100000  # non-null and aligned, never dereferenced
E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def L():
    return B.lib()


def linear(L, x=FAKE, x_dtype=1, xs=None, wq=FAKE, ws=FAKE, bias=None, y=FAKE, y_dtype=0, M=4, N=8, K=256, work=FAKE,
           nbytes=1 << 30):
    return L.hxq_linear_fwd_fp8(x, x_dtype, xs, wq, ws, bias, y, y_dtype, M, N, K, work, nbytes, None)


def experts(L, x=FAKE, x_dtype=1, xs=None, rows=None, offsets=FAKE, wq=FAKE, ws=FAKE, bias=None, y=FAKE, y_dtype=0,
            Mx=4, M=4, E=2, N=8, K=256, work=FAKE, nbytes=1 << 30):
    return L.hxq_linear_fwd_fp8_experts(x, x_dtype, xs, rows, offsets, wq, ws, bias, y, y_dtype, Mx, M, E, N, K, work,
                                        nbytes, None)


def norm(L, x=FAKE, x_dtype=0, res=None, res_dtype=0, w=FAKE, eps=1e-6, res_out=None, out=FAKE, out_dtype=0, scales=None,
         rstd=None, M=4, K=256):
    return L.hxq_rms_norm(x, x_dtype, res, res_dtype, w, eps, res_out, out, out_dtype, scales, rstd, M, K, None)


def norm_bwd(L, dy=FAKE, dy_dtype=0, h=FAKE, h_dtype=0, w=FAKE, rstd=FAKE, dres=None, dx=FAKE, dw=FAKE, M=4, K=256,
             work=FAKE, nbytes=1 << 30):
    return L.hxq_rms_norm_bwd(dy, dy_dtype, h, h_dtype, w, rstd, dres, dx, dw, M, K, work, nbytes, None)


def quant(L, x=FAKE, x_dtype=0, q=FAKE, s=FAKE, M=4, K=256):
    return L.hxq_quant_fp8(x, x_dtype, q, s, M, K, None)


def quant_weight(L, w=FAKE, w_dtype=0, q=FAKE, s=FAKE, qt=None, st=None, E=1, N=8, K=256):
    return L.hxq_quant_fp8_weight(w, w_dtype, q, s, qt, st, E, N, K, None)


SHAPE, NULL, DTYPE, ALIGN, UNSUP = B.HXQ_ERR_SHAPE, B.HXQ_ERR_NULL, B.HXQ_ERR_DTYPE, B.HXQ_ERR_ALIGN, B.HXQ_ERR_UNSUPPORTED
HUGE = 2**31
BAD = [
    (linear, dict(x_dtype=3), DTYPE), (linear, dict(x_dtype=-1), DTYPE), (linear, dict(y_dtype=2), DTYPE),
    (linear, dict(M=-1), SHAPE), (linear, dict(N=-1), SHAPE), (linear, dict(K=-1), SHAPE), (linear, dict(M=HUGE), SHAPE),
    (linear, dict(N=HUGE), SHAPE), (linear, dict(K=HUGE), SHAPE), (linear, dict(nbytes=-1), SHAPE),
    (linear, dict(M=2**30, N=2**30), SHAPE),  # too many tiles
    (linear, dict(x=None), NULL), (linear, dict(wq=None), NULL), (linear, dict(ws=None), NULL), (linear, dict(y=None), NULL),
    (linear, dict(x_dtype=2), NULL),  # e4m3 without scales
    (linear, dict(x=FAKE + 1), ALIGN), (linear, dict(x=FAKE + 2, x_dtype=0), ALIGN), (linear, dict(x=FAKE + 8, x_dtype=2, xs=FAKE), ALIGN),
    (linear, dict(x_dtype=2, xs=FAKE + 1), ALIGN), (linear, dict(wq=FAKE + 8), ALIGN), (linear, dict(ws=FAKE + 2), ALIGN),
    (linear, dict(bias=FAKE + 2), ALIGN), (linear, dict(y=FAKE + 2), ALIGN), (linear, dict(y=FAKE + 1, y_dtype=1), ALIGN),
    (linear, dict(work=FAKE + 8), ALIGN), (linear, dict(M=100, work=None, nbytes=0), UNSUP), (linear, dict(M=100, nbytes=1), UNSUP),
    (experts, dict(E=0), SHAPE), (experts, dict(E=65536), SHAPE), (experts, dict(offsets=None), NULL),
    (experts, dict(Mx=3), SHAPE), (experts, dict(Mx=0, rows=FAKE), SHAPE), (experts, dict(Mx=-1, rows=FAKE), SHAPE),
    (experts, dict(rows=FAKE + 2), ALIGN), (experts, dict(offsets=FAKE + 2), ALIGN), (experts, dict(x=None), NULL),
    (experts, dict(M=100, Mx=100, nbytes=1), UNSUP), (experts, dict(x_dtype=7), DTYPE),
    (norm, dict(x_dtype=2), DTYPE), (norm, dict(out_dtype=3), DTYPE), (norm, dict(res=FAKE, res_dtype=2, res_out=FAKE), DTYPE),
    (norm, dict(M=-1), SHAPE), (norm, dict(K=HUGE), SHAPE), (norm, dict(eps=-1.0), UNSUP), (norm, dict(eps=float("nan")), UNSUP),
    (norm, dict(x=None), NULL), (norm, dict(out=None), NULL), (norm, dict(res=FAKE), NULL), (norm, dict(res_out=FAKE), NULL),
    (norm, dict(out_dtype=2), NULL), (norm, dict(x=FAKE + 2), ALIGN), (norm, dict(w=FAKE + 2), ALIGN), (norm, dict(out=FAKE + 2), ALIGN),
    (norm, dict(out_dtype=2, out=FAKE + 8, scales=FAKE), ALIGN), (norm, dict(out_dtype=2, scales=FAKE + 1), ALIGN),
    (norm, dict(rstd=FAKE + 2), ALIGN), (norm, dict(res=FAKE + 1, res_out=FAKE, res_dtype=1), ALIGN),
    (norm_bwd, dict(dy_dtype=2), DTYPE), (norm_bwd, dict(h_dtype=2), DTYPE), (norm_bwd, dict(M=-1), SHAPE),
    (norm_bwd, dict(dy=None), NULL), (norm_bwd, dict(h=None), NULL), (norm_bwd, dict(rstd=None), NULL), (norm_bwd, dict(dx=None), NULL),
    (norm_bwd, dict(dx=FAKE + 2), ALIGN), (norm_bwd, dict(dres=FAKE + 2), ALIGN), (norm_bwd, dict(dw=FAKE + 2), ALIGN),
    (norm_bwd, dict(nbytes=3), UNSUP), (norm_bwd, dict(work=None), UNSUP), (norm_bwd, dict(nbytes=-1), SHAPE),
    (quant, dict(x_dtype=2), DTYPE), (quant, dict(M=-1), SHAPE), (quant, dict(x=None), NULL), (quant, dict(q=None), NULL),
    (quant, dict(s=None), NULL), (quant, dict(q=FAKE + 8), ALIGN), (quant, dict(s=FAKE + 2), ALIGN), (quant, dict(x=FAKE + 2), ALIGN),
    (quant_weight, dict(w_dtype=2), DTYPE), (quant_weight, dict(E=0), SHAPE), (quant_weight, dict(N=2**20, K=2**20), SHAPE),
    (quant_weight, dict(w=None), NULL), (quant_weight, dict(qt=FAKE), NULL), (quant_weight, dict(st=FAKE), NULL),
    (quant_weight, dict(qt=FAKE + 8, st=FAKE), ALIGN), (quant_weight, dict(s=FAKE + 2), ALIGN),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_bad_arguments_are_refused(L, i):
    fn, args, want = BAD[i]
    assert fn(L, **args) == want, (fn.__name__, args)


@pytest.mark.parametrize("fn,args", [
    (linear, dict(M=0)), (linear, dict(N=0)), (experts, dict(M=0, Mx=0)), (experts, dict(N=0)), (norm, dict(M=0)),
    (norm, dict(K=0)), (norm_bwd, dict(K=0)), (norm_bwd, dict(M=0, dw=None)), (quant, dict(M=0)), (quant, dict(K=0)),
    (quant_weight, dict(N=0)), (quant_weight, dict(K=0))])
def test_empty_calls_do_nothing(L, fn, args):
    assert fn(L, **args) == B.HXQ_OK


def test_workspace_queries(L):
    q = L.hxq_linear_fwd_fp8_workspace
    assert q(1, 0, 8, 8) == 0 and q(1, 8, 0, 8) == 0 and q(2, 100, 20000, 0) == 0
    assert q(3, 1, 1, 1) == DTYPE and q(1, -1, 1, 1) == SHAPE and q(1, 2**30, 2**30, 8) == SHAPE
    for M in (1, 16, 17, 64, 300, 5000):
        for N in (1, 100, 2048, 22016):
            for K in (1, 128, 2048, 11008, 70000):
                rows = M * (-(-K // 128) * 128)
                with_x, without = q(1, M, N, K), q(2, M, N, K)
                # room for the converted rows, unless there are few enough for every workgroup to convert them
                assert q(0, M, N, K) == with_x and (with_x >= rows + without or M * K <= 8 * 11008)
                part = without // (4 * M * N)
                assert without == part * 4 * M * N and part != 1  # whole partial matrices, two or more
    e = L.hxq_linear_fwd_fp8_experts_workspace
    assert e(1, 4, 4, 0, 8, 8) == SHAPE and e(1, 0, 4, 2, 8, 8) == SHAPE and e(1, 0, 0, 2, 8, 8) == 0
    assert e(1, 7, 100, 64, 2048, 2048) >= 7 * 2048
    n = L.hxq_rms_norm_bwd_workspace
    assert n(-1, 8) == SHAPE and n(0, 8) == 0 and n(1, 8) == 32 and n(10**6, 2048) <= 64 << 20


# ------------------------------------------------------------------- the binding

@pytest.fixture
def no_lib(monkeypatch):
    def fail():
        raise AssertionError("the library was reached")

    monkeypatch.setattr(B, "lib", fail)


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=torch.uint8).view(dtype) if dtype in (E4, E8) else torch.zeros(shape, dtype=dtype)


def layer(N=8, K=256, E=None):
    lead = () if E is None else (E,)
    return z(*lead, N, F.fp8_columns(K), dtype=E4), z(*lead, -(-N // 128), F.fp8_scale_columns(K), dtype=E8)


GOOD_CALLS = [
    lambda: F.hxq_quant_fp8(z(4, 200), z(4, 256, dtype=E4), z(4, 4, dtype=E8)),
    lambda: F.hxq_quant_fp8_weight(z(8, 200), *layer(8, 200)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 200), None, *layer(8, 200), None, z(4, 8)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 256, dtype=E4), z(4, 4, dtype=E8), *layer(8, 200), z(8), z(4, 8, dtype=torch.bfloat16)),
    lambda: F.hxq_linear_fwd_fp8_experts(z(4, 200), None, z(9, dtype=torch.int32), z(4, dtype=torch.int32), *layer(8, 200, 3), None, z(9, 8)),
    lambda: F.hxq_rms_norm(z(4, 200), z(200), 1e-6, z(4, 200)),
    lambda: F.hxq_rms_norm_bwd(z(4, 200), z(4, 200), z(200), z(4), z(4, 200)),
]


@pytest.mark.parametrize("i", range(len(GOOD_CALLS)))
def test_host_tensors_are_refused(no_lib, i):
    with pytest.raises(ValueError, match="GPU"):
        GOOD_CALLS[i]()


BAD_CALLS = [
    lambda: F.hxq_quant_fp8(z(4, 200), z(4, 200, dtype=E4), z(4, 4, dtype=E8)),  # unpadded rows
    lambda: F.hxq_quant_fp8(z(4, 200), z(4, 256, dtype=E4), z(4, 2, dtype=E8)),  # unpadded scales
    lambda: F.hxq_quant_fp8(z(4, 200), z(4, 256, dtype=torch.uint8), z(4, 4, dtype=E8)),
    lambda: F.hxq_quant_fp8(z(4, 200, dtype=torch.float16), z(4, 256, dtype=E4), z(4, 4, dtype=E8)),
    lambda: F.hxq_quant_fp8(z(200, 4).t(), z(4, 256, dtype=E4), z(4, 4, dtype=E8)),
    lambda: F.hxq_quant_fp8_weight(z(8, 200), *layer(8, 200), qt=z(200, 128, dtype=E4)),
    lambda: F.hxq_quant_fp8_weight(z(8), *layer(8, 200)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 300), None, *layer(8, 200), None, z(4, 8)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 256, dtype=E4), None, *layer(8, 200), None, z(4, 8)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 200), z(4, 4, dtype=E8), *layer(8, 200), None, z(4, 8)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 200), None, *layer(8, 200), z(4), z(4, 8)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 200), None, *layer(8, 200), None, z(4, 9)),
    lambda: F.hxq_linear_fwd_fp8(z(4, 200), None, *layer(8, 200), None, z(4, 8, dtype=torch.float16)),
    lambda: F.hxq_linear_fwd_fp8(z(2, 2, 200), None, *layer(8, 200), None, z(4, 8)),
    lambda: F.hxq_linear_fwd_fp8_experts(z(4, 200), None, None, z(4, dtype=torch.int32), *layer(8, 200, 3), None, z(9, 8)),
    lambda: F.hxq_linear_fwd_fp8_experts(z(4, 200), None, z(9, dtype=torch.int64), z(4, dtype=torch.int32), *layer(8, 200, 3), None, z(9, 8)),
    lambda: F.hxq_linear_fwd_fp8_experts(z(4, 200), None, z(9, dtype=torch.int32), z(3, dtype=torch.int32), *layer(8, 200, 3), None, z(9, 8)),
    lambda: F.hxq_linear_fwd_fp8_experts(z(4, 200), None, z(9, dtype=torch.int32), z(4, dtype=torch.int32), *layer(8, 200, 3), z(8), z(9, 8)),
    lambda: F.hxq_rms_norm(z(4, 200), z(100), 1e-6, z(4, 200)),
    lambda: F.hxq_rms_norm(z(4, 200), None, 1e-6, z(4, 200), residual=z(4, 200)),
    lambda: F.hxq_rms_norm(z(4, 200), None, 1e-6, z(4, 200), residual=z(4, 200), residual_out=z(4, 200, dtype=torch.bfloat16)),
    lambda: F.hxq_rms_norm(z(4, 200), None, 1e-6, z(4, 256, dtype=E4)),
    lambda: F.hxq_rms_norm(z(4, 200), None, 1e-6, z(4, 200), scales=z(4, 4, dtype=E8)),
    lambda: F.hxq_rms_norm(z(4, 200), None, 1e-6, z(4, 200), rstd=z(5)),
    lambda: F.hxq_rms_norm_bwd(z(4, 200), z(4, 201), None, z(4), z(4, 200)),
    lambda: F.hxq_rms_norm_bwd(z(4, 200), z(4, 200), None, z(4), z(4, 200, dtype=torch.bfloat16)),
    lambda: F.hxq_rms_norm_bwd(z(4, 200), z(4, 200), None, z(4), z(4, 200), dweight=z(4)),
]


@pytest.mark.parametrize("i", range(len(BAD_CALLS)))
def test_binding_refuses(no_lib, i):
    with pytest.raises((ValueError, TypeError)) as e:
        BAD_CALLS[i]()
    assert "GPU" not in str(e.value)  # refused for what is wrong with it, not for being on the host


def permuted(t):
    """The same values in other strides, as exchanging two dimensions of another tensor gives them."""
    u = t.view(torch.uint8).transpose(-1, -2).contiguous().transpose(-1, -2).view(t.dtype)
    assert not u.is_contiguous() and torch.equal(u.view(torch.uint8), t.view(torch.uint8))
    return u


def test_scales_of_any_strides_are_taken(no_lib):
    """Refused for being on the host, the last check, and not for their strides; shapes and types still count."""
    w, s = layer(300, 900)
    xs = permuted(z(4, 8, dtype=E8))
    with pytest.raises(ValueError, match="GPU"):
        F.hxq_linear_fwd_fp8(z(4, 1024, dtype=E4), xs, w, permuted(s), None, z(4, 300))
    we, se = layer(300, 900, 3)
    with pytest.raises(ValueError, match="GPU"):
        F.hxq_linear_fwd_fp8_experts(z(4, 900), None, None, z(4, dtype=torch.int32), we, permuted(se), None, z(4, 300))
    for bad in (permuted(s)[:2], permuted(s)[:, :4], permuted(s).view(torch.uint8)):
        with pytest.raises(ValueError, match="w_scales"):
            F.hxq_linear_fwd_fp8(z(4, 900), None, w, bad, None, z(4, 300))
    with pytest.raises(ValueError, match="contiguous"):  # the values themselves stay as they are laid out
        F.hxq_linear_fwd_fp8(z(4, 900), None, permuted(w), s, None, z(4, 300))


def test_layer_objects_refuse():
    with pytest.raises(ValueError, match="GPU"):
        hx.Fp8Linear(z(8, 200), device="cpu")
    n = hx.RmsNorm(z(200), device="cpu")
    with pytest.raises(ValueError, match="shape"):
        n(z(4, 200), residual=z(3, 200))
    with pytest.raises(ValueError, match="gradient"):
        n(z(4, 200).requires_grad_(), out_dtype=E4)
    with pytest.raises(AttributeError):
        hx.Fp8Nothing
