"""The 8-bit layer objects' own work, without a GPU: shapes, and what the backward pass does with the kernels'
results.  The library's product is replaced by its definition on host tensors, the weight held as it is."""

import pytest
import torch

import vq_compressed_linear_amd as hx
from vq_compressed_linear_amd import _binding_fp8 as F


def product_of_experts(x, x_scales, rows, offsets, w, w_scales, bias, y, stream=None, workspace=None):
    """hxq_linear_fwd_fp8_experts by its definition: indices out of range read the nearest row there is."""
    assert x.dim() == 2 and y.shape[1] == w.shape[1] and (rows is not None or y.shape[0] == x.shape[0])
    off = offsets.tolist()
    for e in range(len(off) - 1):
        for r in range(off[e], off[e + 1]):
            at = r if rows is None else min(max(int(rows[r]), 0), x.shape[0] - 1)
            y[r] = w[e] @ x[at] + (0 if bias is None else bias[e])


@pytest.fixture
def experts(monkeypatch):
    monkeypatch.setattr(F, "hxq_linear_fwd_fp8_experts", product_of_experts)
    layer = hx.Fp8Experts.__new__(hx.Fp8Experts)
    g = torch.Generator().manual_seed(1)
    layer.experts, layer.out_features, layer.in_features = 3, 5, 4
    layer.wq = torch.randn(3, 5, 4, generator=g)
    layer.wt = layer.wq.transpose(1, 2).contiguous()
    layer.w_scales = layer.wt_scales = layer.bias = None
    return layer


def gradient(layer, x, offsets, rows, dy):
    x = x.clone().requires_grad_()
    y = layer(x, offsets, rows)
    y.backward(dy)
    return y.detach(), x.grad


def int32(*v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.mark.parametrize("rows", [None, [5, 0, 3], [1, 2, 5, 0], [0, 1, 2, 3, 4, 5], [4, 4, 4, 1, 4, 2, 0]])
def test_experts_gradient_keeps_the_inputs_shape(experts, rows):
    """x of more than two dimensions: `rows` index its rows as the forward flattens them."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(2, 3, 4, generator=g)
    n = 6 if rows is None else len(rows)
    rows = None if rows is None else int32(*rows)
    offsets = int32(0, n // 2, n // 2, n)
    dy = torch.randn(n, 5, generator=g)
    y, dx = gradient(experts, x, offsets, rows, dy)
    y2, dx2 = gradient(experts, x.reshape(6, 4), offsets, rows, dy)
    assert torch.equal(y, y2) and dx.shape == x.shape and torch.equal(dx.reshape(6, 4), dx2)
    want = torch.zeros(6, 4)
    for r in range(n):
        want[r if rows is None else int(rows[r])] += dy[r] @ experts.wq[0 if r < n // 2 else 2]
    assert torch.allclose(dx2, want, rtol=0, atol=1e-5)


@pytest.mark.parametrize("rows", [[-1, 0, 5, 6], [6, 7, 2**31 - 1, 3], [-(2**31), -7, 1, -6]])
def test_experts_gradient_of_rows_out_of_range(experts, rows):
    """An index out of range reads the nearest row there is, and that row receives its gradient."""
    g = torch.Generator().manual_seed(3)
    x, dy = torch.randn(6, 4, generator=g), torch.randn(4, 5, generator=g)
    offsets = int32(0, 1, 1, 4)
    y, dx = gradient(experts, x, offsets, int32(*rows), dy)
    y2, dx2 = gradient(experts, x, offsets, int32(*[min(max(r, 0), 5) for r in rows]), dy)
    assert torch.equal(y, y2) and torch.equal(dx, dx2)


def test_experts_gradient_leaves_rows_past_the_last_expert_out(experts):
    """Their entries in `rows` and in dy may hold anything."""
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(6, 4, generator=g), torch.randn(5, 5, generator=g)
    dy[3:] = float("nan")
    _, dx = gradient(experts, x, int32(0, 1, 1, 3), int32(2, 2, 0, -9, 2**30), dy)
    want = torch.zeros(6, 4)
    for r, (e, m) in enumerate([(0, 2), (2, 2), (2, 0)]):
        want[m] += dy[r] @ experts.wq[e]
    assert torch.allclose(dx, want, rtol=0, atol=1e-5)
    _, dx = gradient(experts, x, int32(0, 0, 0, 0), int32(2, 2, 0, -9, 2**30), dy)
    assert not dx.any()


def test_experts_gradient_through_rows_is_not_captured(experts, monkeypatch):
    """Its sum goes through a sort whose launches are not known to replay: refused inside a graph, before anything
    of it is queued.  Without `rows` there is no such sum."""
    x, dy = torch.ones(6, 4), torch.ones(6, 5)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="captured"):
        gradient(experts, x, int32(0, 2, 4, 6), int32(0, 1, 2, 3, 4, 5), dy)
    gradient(experts, x, int32(0, 2, 4, 6), None, dy)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    gradient(experts, x, int32(0, 2, 4, 6), int32(0, 1, 2, 3, 4, 5), dy)


def product(x, x_scales, w, w_scales, bias, y, stream=None, workspace=None):
    y.copy_(x @ w.t() + (0 if bias is None else bias))


@pytest.mark.parametrize("N,K", [(5, 0), (0, 4), (0, 0), (5, 4)])
@pytest.mark.parametrize("lead", [(3,), (2, 3), (0,), (2, 0)])
def test_linear_of_no_features(monkeypatch, lead, N, K):
    """Without a sum y is the bias, without outputs it is empty; the gradients likewise."""
    monkeypatch.setattr(F, "hxq_linear_fwd_fp8", product)
    layer = hx.Fp8Linear.__new__(hx.Fp8Linear)
    layer.out_features, layer.in_features, layer.bias = N, K, torch.arange(N).float()
    layer.wq = torch.ones(N, K)
    layer.wt, layer.w_scales, layer.wt_scales = layer.wq.t().contiguous(), None, None
    x = torch.ones(*lead, K, requires_grad=True)
    y = layer(x)
    assert torch.equal(y, (layer.bias + K).expand(*lead, N))
    y.backward(torch.ones_like(y))
    assert torch.equal(x.grad, torch.full((*lead, K), float(N)))


@pytest.mark.parametrize("lead", [(3,), (2, 3), (0,)])
def test_norm_of_no_columns(monkeypatch, lead):
    monkeypatch.setattr(F, "hxq_rms_norm", lambda *a, **k: None)
    monkeypatch.setattr(F, "hxq_rms_norm_bwd", lambda *a, **k: None)
    x, r = torch.ones(*lead, 0, requires_grad=True), torch.ones(*lead, 0, requires_grad=True)
    out, h = hx.RmsNorm(torch.ones(0), device="cpu")(x, r)
    assert out.shape == h.shape == x.shape
    torch.autograd.backward((out, h), (torch.ones_like(out), torch.ones_like(h)))
    assert x.grad.shape == r.grad.shape == x.shape
