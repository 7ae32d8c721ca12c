"""The 8-bit path on the GPU against the oracle in 64 bits.

Tolerances.  Conversion to e4m3 is exact arithmetic (a power of two) and one
rounding, so bytes and scales have to be equal.  Products of e4m3 values are
exact in fp32, their sum is fp32: 1e-5 of |x| |w|^T, the library's bound for
fp32 sums (sqrt(K) 2^-24 at the largest K here is 6e-6); bf16 results add half
a step, 2^-8 of the value, and past 64 rows 2^-10 of |x| |w|^T: there the 8-bit
matrix cores may lose each of a group's 8 products below 2^-13 of the largest.  The norm's statistics are sums of positive terms
in chains of at most K / 64 + 16 additions: each adds 2^-24 relative, half of
it after the square root, and six more roundings follow.
"""

import numpy as np
import pytest
import torch

import vq_compressed_linear_amd as hx
from hxq_synth import gen
from oracle import fp8_oracle as O

from gpu_util import say

pytestmark = pytest.mark.gpu

E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0**-24
HALF = {F32: 0.0, BF16: 2.0**-8}


def up(n, m):
    return -(-n // m) * m


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def make(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(0.7 * torch.randn(shape[-1], generator=g)) * scale
    return x.to(dtype).cuda()


def rows8(x):
    q = torch.full((x.shape[0], up(x.shape[1], 128)), float("nan"), device="cuda").to(E4)
    s = torch.full((x.shape[0], up(-(-x.shape[1] // 128), 4)), 255, dtype=torch.uint8, device="cuda").view(E8)
    hx.hxq_quant_fp8(x, q, s)
    return q, s


def weight8(w, transposed=False):
    lead, (n, k) = w.shape[:-2], w.shape[-2:]

    def new(n, k):
        return (torch.full(lead + (n, up(k, 128)), 0x55, dtype=torch.uint8, device="cuda").view(E4),
                torch.full(lead + (-(-n // 128), up(-(-k // 128), 4)), 255, dtype=torch.uint8, device="cuda").view(E8))

    a = new(n, k)
    b = new(k, n) if transposed else (None, None)
    hx.hxq_quant_fp8_weight(w, *a, *b)
    return (*a, *b) if transposed else a


def near(got, want, bound, what=""):
    got = host(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound, first at %s: %r for %r" % (
        what, bad.sum(), bad.size, np.max(np.abs(got - want) / np.maximum(bound, 1e-300)), np.argwhere(bad)[0],
        got[bad][0], want[bad][0])


# ------------------------------------------------------------------ conversion

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 128), (5, 129), (7, 513), (64, 2048), (33, 2050), (2, 20000)])
def test_rows(M, K, dtype):
    x = make(M * 1000 + K, M, K, dtype=dtype)
    if M > 2:
        x[1] = 0
        x[2, ::3] *= 1e-30
    q, s = rows8(x)
    Q, S = O.quant_rows(host(x))
    assert np.array_equal(raw(q), Q) and np.array_equal(raw(s), S)


def test_rows_of_special_values():
    x = torch.zeros(9, 256)
    x[0, 0], x[0, 5], x[0, 130] = float("inf"), 3.0, -float("inf")
    x[1, 0], x[1, 1] = float("nan"), -1e-3
    x[2] = torch.finfo(F32).max
    x[3] = torch.finfo(F32).tiny / 4  # subnormal
    x[4, :8] = torch.tensor([448.0, 449, 448 * 2.0**-126, 1e-45, -448, 17, 18, 19])
    x[5] = -0.0
    x[6, 7] = 1.75 * 2.0**-118  # 448 2^-126: the smallest scale's largest value
    x[7, 7] = 1.7500001
    x[8] = 1e-45
    q, s = rows8(x.cuda())
    Q, S = O.quant_rows(x.numpy())
    assert np.array_equal(raw(s), S)
    assert np.array_equal(O.E4M3[raw(q)], O.E4M3[Q], equal_nan=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (127, 129), (300, 70), (5, 1000), (2, 130, 250), (3, 128, 64)])
def test_weight_and_its_transpose(shape, dtype):
    w = make(sum(shape), *shape, dtype=dtype, scale=0.02)
    q, s, qt, st = weight8(w, transposed=True)
    q1, s1 = weight8(w)
    assert torch.equal(q.view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s.view(torch.uint8), s1.view(torch.uint8))
    lead = (1,) if w.dim() == 2 else (w.shape[0],)
    flat = [t.reshape(lead + t.shape[-2:]) for t in (w, q, s, qt, st)]
    for e in range(lead[0]):
        W, *got = [t[e] for t in flat]
        Q, S = O.quant_weight(host(W))
        assert np.array_equal(raw(got[0]), Q) and np.array_equal(raw(got[1]), S)
        n, k = W.shape
        T = np.zeros((k, up(n, 128)), dtype=np.uint8)
        T[:, :n] = Q[:, :k].T
        G = np.full((-(-k // 128), up(-(-n // 128), 4)), 127, dtype=np.uint8)
        G[:, : S.shape[0]] = S[:, : -(-k // 128)].T
        assert np.array_equal(raw(got[2]), T) and np.array_equal(raw(got[3]), G)


# -------------------------------------------------------------------- products

def product_bound(Y, B, y_dtype):
    return (1e-5 if y_dtype == F32 else 2.0**-10) * B + (U + HALF[y_dtype]) * np.abs(Y)


def check_linear(M, N, K, x_dtype=BF16, y_dtype=F32, bias=True, seed=0, pair=False):
    say("linear", M, N, K, x_dtype, y_dtype, bias, pair)
    x = make(seed + 1, M, K, dtype=x_dtype)
    q, s = weight8(make(seed + 2, N, K, scale=0.02))
    b = make(seed + 3, N) if bias else None
    y = torch.full((M, N), float("nan"), dtype=y_dtype, device="cuda")
    xq, xs = rows8(x)
    hx.hxq_linear_fwd_fp8(xq if pair else x, xs if pair else None, q, s, b, y)
    Y, B = O.linear(O.wide_rows(raw(xq), raw(xs)), O.wide_weight(raw(q), raw(s)), None if b is None else host(b))
    near(y, Y, product_bound(Y, B, y_dtype), "linear")
    return x, q, s, b, y


@pytest.mark.parametrize("K", [1, 127, 128, 130, 1024, 2048, 4300])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (2, 17), (16, 256), (17, 200), (32, 64), (33, 129), (61, 2048), (64, 96)])
def test_linear_few_rows(M, N, K):
    check_linear(M, N, K, x_dtype=BF16 if K % 2 else F32, bias=bool(N % 2))


@pytest.mark.parametrize("M,N,K", [(65, 130, 256), (128, 128, 128), (200, 257, 384), (255, 512, 130), (256, 256, 2048),
                                   (257, 1000, 640), (500, 300, 1100), (1024, 512, 512), (300, 2048, 4224), (700, 260, 1)])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
def test_linear_many_rows(M, N, K, y_dtype):
    check_linear(M, N, K, y_dtype=y_dtype, bias=bool(M % 2), pair=y_dtype == BF16)


@pytest.mark.parametrize("pair", [True, False])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [
    (2570, 3900, 128), (2700, 3896, 384), (2570, 3900, 1300),  # 256 x 256 tiles, a last one of few rows or a whole one
    (4200, 3901, 250),  # whole rounds of them, and the rows past those in smaller tiles
    (2000, 1300, 600),  # 128 x 128 (float32 y), 64 x 128
    (600, 1100, 3200),  # 64 x 128, the sum split over two workgroups
    (100, 700, 9000),   # 32 x 64, split
])
def test_linear_tiles(M, N, K, y_dtype, pair):
    check_linear(M, N, K, y_dtype=y_dtype, bias=not pair, pair=pair, seed=9)


@pytest.mark.parametrize("M,N,K", [(1, 22016, 2048), (8, 2048, 11008), (61, 2048, 11008), (512, 2048, 2048)])
def test_linear_layer_shapes(M, N, K):
    check_linear(M, N, K, seed=5)


def test_linear_without_a_sum():
    w, s = torch.zeros((5, 0), dtype=torch.uint8, device="cuda").view(E4), torch.zeros((1, 0), dtype=torch.uint8, device="cuda").view(E8)
    b, y = make(1, 5), torch.full((3, 5), float("nan"), device="cuda")
    hx.hxq_linear_fwd_fp8(torch.zeros((3, 0), device="cuda"), None, w, s, b, y)
    assert torch.equal(y, b.expand(3, 5))
    hx.hxq_linear_fwd_fp8(torch.zeros((3, 0), device="cuda"), None, w, s, None, y)
    assert not y.any()
    hx.hxq_linear_fwd_fp8(torch.zeros((0, 0), device="cuda"), None, w, s, None, y[:0])


def test_layers_of_no_features():
    """A sum over nothing is the bias, its gradient has no columns; no outputs: a gradient of zeros."""
    b = make(1, 5)
    layer = hx.Fp8Linear(torch.zeros((5, 0), device="cuda"), b, train=True)
    x = torch.zeros((2, 3, 0), device="cuda", requires_grad=True)
    y = layer(x)
    assert torch.equal(y, b.expand(2, 3, 5))
    y.backward(torch.ones_like(y))
    assert x.grad.shape == x.shape
    none = hx.Fp8Linear(torch.zeros((0, 5), device="cuda"), train=True)
    x = make(2, 3, 5).requires_grad_()
    y = none(x)
    assert y.shape == (3, 0)
    y.backward(torch.ones_like(y))
    assert not x.grad.any()
    z = torch.zeros((2, 3, 0), device="cuda", requires_grad=True)
    out, h = hx.RmsNorm(torch.zeros(0, device="cuda"))(z, z)
    assert out.shape == h.shape == z.shape
    h.sum().backward()
    assert z.grad.shape == z.shape


@pytest.mark.parametrize("M", [1, 20, 60, 300])
def test_linear_with_nan_rows_keeps_them_apart(M):
    """A NaN (or infinity) in x makes its own row of y NaN and no other."""
    x, q, s, b, y = check_linear(M, 200, 300)
    x2 = x.clone()
    x2[M // 2, 7] = float("inf") if M % 2 else float("nan")
    y2 = torch.empty_like(y)
    hx.hxq_linear_fwd_fp8(x2, None, q, s, b, y2)
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(y2[keep], y[keep]) and y2[M // 2].isnan().all()


@pytest.mark.parametrize("M,N,K", [(1, 600, 9000), (48, 130, 5000), (300, 260, 640)])
def test_linear_is_deterministic_and_takes_a_workspace(M, N, K):
    x, q, s, b, y = check_linear(M, N, K)
    need = hx.lib().hxq_linear_fwd_fp8_workspace(hx.HXQ_BF16, M, N, K)
    w = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        y2 = torch.empty_like(y)
        hx.hxq_linear_fwd_fp8(x, None, q, s, b, y2, workspace=w)
        assert torch.equal(y, y2)
        w[:need].random_()
        assert (w[need:] == 255).all()  # nothing past what it asked for
    with pytest.raises(hx.HxqError):
        hx.hxq_linear_fwd_fp8(x, None, q, s, b, y2, workspace=w[: need - 1])
    with pytest.raises(hx.HxqError):
        hx.hxq_linear_fwd_fp8(x, None, q, s, b, y2, workspace=w[:0])


@pytest.mark.parametrize("M,N,K", [(2, 96, 300), (20, 128, 300), (70, 2048, 256), (2000, 1304, 256), (2570, 3904, 256)])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
def test_linear_on_views(M, N, K, y_dtype):
    """x, y and the bias one element into their storage: results as on their own, nothing beside them written."""
    x, q, s, b, y = check_linear(M, N, K, x_dtype=F32, y_dtype=y_dtype)

    def shifted(t):
        store = torch.full((t.numel() + 9,), 7.0, dtype=t.dtype, device="cuda")
        store[1:1 + t.numel()] = t.flatten()
        return store, store[1:1 + t.numel()].view(t.shape)

    store, y2 = shifted(torch.zeros_like(y))
    hx.hxq_linear_fwd_fp8(shifted(x)[1], None, q, s, shifted(b)[1], y2)
    assert torch.equal(y2, y) and store[0] == 7.0 and (store[-8:] == 7.0).all()


def test_norm_on_views():
    for K in (300, 2048, 2052):
        x, r, w = make(1, 5, K), make(2, 5, K, dtype=BF16), make(3, K)
        dy = make(4, 5, K)

        def shifted(t):
            return torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)

        got = []
        for f in (lambda t: t, shifted):
            out, kept, rstd, dx, dw = torch.empty(5, K, device="cuda"), torch.empty_like(r), torch.empty(5, device="cuda"), torch.empty(5, K, device="cuda"), torch.empty(K, device="cuda")
            out, kept, rstd, dx, dw = [f(v) for v in (out, kept, rstd, dx, dw)]
            hx.hxq_rms_norm(f(x), f(w), 1e-6, out, residual=f(r), residual_out=kept, rstd=rstd)
            hx.hxq_rms_norm_bwd(f(dy), kept, f(w), rstd, dx, dweight=dw)
            got.append((out, kept, rstd, dx, dw))
        assert all(torch.equal(a, b) for a, b in zip(*got))


# Shapes that reach every kernel, with more than four 128-blocks of k (so that a word of scales is left behind): few
# rows, 32 x 64 tiles without and with a split sum, 64 x 128 without and with one, 128 x 128 (float32 y), 256 x 256
# with a last one of few rows, and whole rounds of those with the rest in smaller tiles.
EVERY_KERNEL = [(3, 200, 700), (300, 260, 640), (100, 700, 9000), (600, 1100, 3200), (2000, 1300, 600),
                (2570, 3900, 1300), (4200, 3901, 700)]


def whole(seed, K, *rows):
    """e4m3 values that are eighths of whole numbers, 8 to 15 of either sign or zero: (bytes, the whole numbers)."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(8, 16, (*rows, K), generator=g) * (torch.randint(0, 2, (*rows, K), generator=g) * 2 - 1)
    v[torch.rand(*rows, K, generator=g) < 0.1] = 0
    v = torch.nn.functional.pad(v, (0, up(K, 128) - K))
    return (v / 8).to(E4).cuda(), v.double().cuda()


def powers(seed, far, sign, *shape):
    """Exponents [..., blocks of k]: 0 or 1, plus `sign` times a block's own, up to `far` either way."""
    own = torch.randint(-far, far + 1, shape[-1:], generator=torch.Generator().manual_seed(7)) if far else 0
    e = torch.randint(0, 2, shape, generator=torch.Generator().manual_seed(seed)) + sign * own
    pad = torch.nn.functional.pad(e + 127, (0, up(shape[-1], 4) - shape[-1]), value=127)
    return pad.to(torch.uint8).view(E8).cuda(), torch.exp2(e.double()).cuda()


def spread(p, rows):
    """A power for every element, from one for each 128 columns (and, with `rows`, each 128 rows)."""
    p = p.repeat_interleave(128, -1)
    return p if rows is None else p.repeat_interleave(128, -2)[..., :rows, :]


@pytest.mark.parametrize("far", [0, 100])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", EVERY_KERNEL)
def test_linear_of_whole_numbers_is_exact(M, N, K, y_dtype, far):
    """Products of the values are whole multiples of 2^-6 from 64 to 225 or zero, so no group of 8 holds one below
    2^-8 of its largest, and the 8-bit matrix cores keep them whole; powers of two make them 1 to 4 times that,
    their own (2^a for x, 2^-a for w, |a| <= far) cancel, and B, the sum of the magnitudes, stays below 2^24
    of the smallest step: every partial sum is exact in float32, and y is the exact sum, rounded once."""
    say("exact", M, N, K, y_dtype, far)
    G = -(-K // 128)
    (xq, X), (wq, W) = whole(M, K, M), whole(N, K, N)
    (xs, xp), (ws, wp) = powers(1, far, 1, M, G), powers(2, far, -1, -(-N // 128), G)
    b = torch.randint(-999, 999, (N,), generator=torch.Generator().manual_seed(3)).float().cuda() / 64
    X, W = X * spread(xp, None), W * spread(wp, N)
    assert (X.abs() @ W.abs().t()).max() + 999 < 2**24
    want = ((X @ W.t()) / 64 + b).float()
    y = torch.full((M, N), float("nan"), dtype=y_dtype, device="cuda")
    hx.hxq_linear_fwd_fp8(xq, xs, wq, ws, b, y)
    assert torch.equal(y, want.to(y_dtype))


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("counts,Mx,N,K", [([1, 0, 1, 1, 2], 4, 300, 700), ([40] * 20 + [0, 3], 300, 260, 700),
                                           ([300] * 10, 500, 256, 1300), ([5000, 0, 3001, 129, 7000], 4000, 700, 640),
                                           ([5000, 0, 3001, 129, 7000], 4000, 300, 700),
                                           ([3, 0, 2], 4, 48, 9000)])
def test_experts_of_whole_numbers_are_exact(counts, Mx, N, K, y_dtype, gather):
    """The same for rows grouped by expert."""
    say("exact experts", counts[:5], Mx, N, K, y_dtype, gather)
    M, E, G = sum(counts), len(counts), -(-K // 128)
    rows, offsets = routing(M, counts, Mx)
    if not gather:
        rows, Mx = None, M
    (xq, X), (wq, W) = whole(M, K, Mx), whole(N, K, E, N)
    (xs, xp), (ws, wp) = powers(1, 100, 1, Mx, G), powers(2, 100, -1, E, -(-N // 128), G)
    X, W = X * spread(xp, None), W * spread(wp, N)
    want, off = torch.empty((M, N), device="cuda"), offsets.tolist()
    for e in range(E):
        at = slice(off[e], off[e + 1])
        x = X[at] if rows is None else X[rows[at].long()]
        assert not len(x) or (x.abs() @ W[e].abs().t()).max() < 2**24
        want[at] = ((x @ W[e].t()) / 64).float()
    y = torch.full((M, N), float("nan"), dtype=y_dtype, device="cuda")
    hx.hxq_linear_fwd_fp8_experts(xq, xs, rows, offsets, wq, ws, None, y)
    assert torch.equal(y, want.to(y_dtype))


@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", EVERY_KERNEL)
def test_every_kernel_keeps_nan_rows_apart(M, N, K, y_dtype):
    """test_linear_with_nan_rows_keeps_them_apart in every kernel, as an infinity, a NaN and both, in the first, an
    inner and the last row."""
    say("nan", M, N, K, y_dtype)
    x, (q, s) = make(1, M, K, dtype=BF16), weight8(make(2, N, K, scale=0.02))
    y, y2 = [torch.full((M, N), 7.0, dtype=y_dtype, device="cuda") for _ in range(2)]
    hx.hxq_linear_fwd_fp8(x, None, q, s, None, y)
    assert y.isfinite().all()
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    x[0, K - 1], x[M // 2, K // 2], x[M - 1, 0], x[M - 1, 1] = float("inf"), float("nan"), -float("inf"), float("nan")
    bad[[0, M // 2, M - 1]] = True
    hx.hxq_linear_fwd_fp8(x, None, q, s, None, y2)
    assert torch.equal(y2[~bad], y[~bad]) and y2[bad].isnan().all()


@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("counts", [[1, 0, 1, 1], [40] * 20, [300, 0, 290, 310], [5000, 0, 3001, 129, 7000]])
def test_experts_keep_nan_rows_apart(counts, y_dtype):
    """A NaN in a row of x reaches the rows of y that read it and no other; rows past the last expert's stay."""
    Mx, N, K, M = 50, 300, 700, sum(counts)
    say("nan experts", counts[:5], y_dtype)
    rows, offsets = routing(5, counts, Mx, 3)
    rows[0] = 17
    x, (q, s) = make(1, Mx, K), weight8(make(2, len(counts), N, K, scale=0.02))
    y, y2 = [torch.full((M + 3, N), 7.0, dtype=y_dtype, device="cuda") for _ in range(2)]
    hx.hxq_linear_fwd_fp8_experts(x, None, rows, offsets, q, s, None, y)
    x[17, K - 1] = float("nan")
    hx.hxq_linear_fwd_fp8_experts(x, None, rows, offsets, q, s, None, y2)
    bad = rows == 17
    bad[M:] = False
    assert torch.equal(y2[~bad], y[~bad]) and y2[bad].isnan().all() and (y2[M:] == 7.0).all()


@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("M,N", [(2, 40), (40, 200), (300, 260), (2000, 1300), (2570, 3900)])
def test_linear_at_the_ends_of_the_range(M, N, y_dtype):
    """The largest values that e4m3 holds below 2^128 and the smallest that bf16 holds whole, beside weights of
    zero: one product to a sum, so y is that product."""
    K = 300
    x, w = torch.zeros((M, K), device="cuda"), torch.zeros((N, K), device="cuda")
    x[:, 0], w[::2, 0] = 240 * 2.0**120, 1.75 * 2.0**-5
    x[::2, 140], w[1::2, 140] = 1.875 * 2.0**-130, -1.25 * 2.0**120
    y = torch.full((M, N), float("nan"), dtype=y_dtype, device="cuda")
    hx.hxq_linear_fwd_fp8(x, None, *weight8(w), None, y)
    want = torch.zeros((M, N), dtype=torch.float64)
    want[:, ::2] = 240 * 1.75 * 2.0**115
    want[::2, 1::2] = -1.875 * 1.25 * 2.0**-10
    assert torch.equal(y, want.float().to(y_dtype).cuda())


def test_linear_extreme_scales():
    """Weights and rows whose powers of two are far apart."""
    M, N, K = 20, 140, 384
    x = make(1, M, K)
    x[:, :128] *= 1e-12
    x[:, 128:256] *= 1e12
    w = make(2, N, K)
    w[:, :128] *= 1e12
    w[:, 128:256] *= 1e-12
    q, s = weight8(w)
    y = torch.empty((M, N), device="cuda")
    xq, xs = rows8(x)
    hx.hxq_linear_fwd_fp8(x, None, q, s, None, y)
    Y, B = O.linear(O.wide_rows(raw(xq), raw(xs)), O.wide_weight(raw(q), raw(s)))
    near(y, Y, 1e-5 * B)


@pytest.mark.parametrize("M", [3, 40, 700])
@pytest.mark.parametrize("E", [None, 3])
def test_scales_of_any_strides(M, E):
    """Scales of a transposed weight as exchanging two dimensions leaves them, and of rows likewise: the bytes that
    contiguous ones give, on the current stream and on another."""
    N, K = 500, 900  # four blocks of N: nothing is padded, so nothing else would have copied them
    w = make(1, *(() if E is None else (E,)), N, K, scale=0.02)
    _, s, wt, st = weight8(w, transposed=True)
    swapped = s.view(torch.uint8)[..., :8].transpose(-1, -2)  # [blocks of K, blocks of N]
    assert not swapped.is_contiguous() and torch.equal(swapped, st.view(torch.uint8))
    dq, ds = rows8(make(2, M, N))
    loose = ds.view(torch.uint8).t().contiguous().t().view(E8)
    offsets = None if E is None else torch.tensor([0, M // 3, M // 3, M], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def product(xs, ws, stream=None):
        dx = torch.full((M, K), float("nan"), device="cuda")
        torch.cuda.synchronize()
        if E is None:
            hx.hxq_linear_fwd_fp8(dq, xs, wt, ws, None, dx, stream=stream)
        else:
            hx.hxq_linear_fwd_fp8_experts(dq, xs, None, offsets, wt, ws, None, dx, stream=stream)
        torch.cuda.synchronize()
        return dx

    want = product(ds, st)
    assert not want.isnan().any()
    for stream in (None, side, side.cuda_stream):
        assert torch.equal(product(loose, swapped.view(E8), stream), want)


# --------------------------------------------------------------------- experts

def routing(seed, counts, Mx, tail=0):
    rng = np.random.default_rng(seed)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    rows = rng.integers(0, Mx, offsets[-1] + tail)
    return torch.from_numpy(rows).int().cuda(), torch.from_numpy(offsets).int().cuda()


CASES = [
    # counts, rows of x, N, K
    ([1], 1, 40, 128),
    ([0, 0, 3, 0], 5, 100, 200),
    ([1, 1, 1, 1, 1, 1, 1, 1] + [0] * 56, 1, 256, 512),
    ([5, 0, 17, 40, 1, 0, 64, 33], 30, 200, 300),
    ([100, 0, 3, 257, 300, 0], 128, 130, 640),
    ([0] * 130 + [9] + [0] * 5 + [3], 4, 64, 256),
    ([2000, 1, 0, 90], 700, 300, 384),
    ([300] * 10, 500, 256, 256),
    ([0, 0, 0], 3, 64, 128),
    ([5000, 0, 3001, 129, 7000], 4000, 700, 384),  # 256 x 256 tiles, short last ones
    ([700, 300, 0, 129, 1500], 900, 1400, 640),
    ([40] * 40, 300, 260, 700),
]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_experts(i, gather):
    counts, Mx, N, K = CASES[i]
    tail = i % 3 * 5  # rows past the last expert's
    E, M = len(counts), sum(counts) + tail
    say("experts", counts[:10], Mx, N, K, gather, tail)
    y_dtype = BF16 if i % 2 else F32
    rows, offsets = routing(i, counts, Mx, tail)
    rows[M - tail:] = 2**30  # never read
    x = make(i, Mx if gather else M, K, dtype=F32 if i % 2 else BF16)
    q, s = weight8(make(i + 50, E, N, K, scale=0.02))
    b = make(i + 60, E, N) if i % 2 else None
    y = torch.full((M, N), 7.0, dtype=y_dtype, device="cuda")
    hx.hxq_linear_fwd_fp8_experts(x, None, rows if gather else None, offsets, q, s, b, y)
    xq, xs = rows8(x) if M else (None, None)
    n = sum(counts)
    assert (y[n:] == 7.0).all()
    if n:
        Y, B = O.experts(O.wide_rows(raw(xq), raw(xs)), rows.cpu().numpy() if gather else None, offsets.tolist(),
                         [O.wide_weight(raw(q[e]), raw(s[e])) for e in range(E)], None if b is None else host(b))
        near(y[:n], Y, product_bound(Y, B, y_dtype), "experts")


def test_experts_deterministic_with_a_split_sum():
    """Few tiles and a long sum: the parts go through the workspace, rows past the end stay."""
    counts, K, N = [3, 0, 2], 9000, 48
    rows, offsets = routing(3, counts, 4, 2)
    rows[5:] = -5
    x, (q, s), b = make(1, 4, K), weight8(make(2, 3, N, K)), make(3, 3, N)
    out = []
    for _ in range(3):
        y = torch.full((7, N), 7.0, device="cuda")
        hx.hxq_linear_fwd_fp8_experts(x, None, rows, offsets, q, s, b, y)
        out.append(y)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2]) and (out[0][5:] == 7.0).all()
    xq, xs = rows8(x)
    Y, B = O.experts(O.wide_rows(raw(xq), raw(xs)), rows.cpu().numpy(), offsets.tolist(),
                     [O.wide_weight(raw(q[e]), raw(s[e])) for e in range(3)], host(b))
    near(out[0][:5], Y, 1e-5 * B + U * np.abs(Y))


@pytest.mark.parametrize("M", [9, 300, 3000])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
def test_experts_bad_indices_stay_inside(M, y_dtype):
    """Rows out of range and offsets that break their rule: unspecified values, no access outside."""
    x, (q, s) = make(1, 6, 256), weight8(make(2, 4, 256, 256))
    guard = torch.full((20 + M + 20, 256), 7.0, dtype=y_dtype, device="cuda")
    y = guard[20:20 + M]
    rows = torch.arange(M, dtype=torch.int32, device="cuda") % 6
    rows[:8] = torch.tensor([0, -1, 2**31 - 1, -(2**31), 6, 5, 3, 2], dtype=torch.int32, device="cuda")
    for off in ([0, 3, 5, 7, 9], [0, 100, 2**31 - 1, 5, 9], [-5, 4, -(2**31), 9, 9], [9, 7, 5, 3, 0], [3, 3, 3, 3, 3],
                [2**31 - 1, 0, 2**31 - 1, 0, 2**31 - 1]):
        hx.hxq_linear_fwd_fp8_experts(x, None, rows, torch.tensor(off, dtype=torch.int32, device="cuda"), q, s, None, y)
    assert (guard[:20] == 7.0).all() and (guard[20 + M:] == 7.0).all()


# ------------------------------------------------------------------------ norm

def ops(K):
    return K / 64 + 16


@pytest.mark.parametrize("res", [None, F32, BF16])
@pytest.mark.parametrize("out_dtype", [F32, BF16, E4])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 5), (4, 128), (6, 511), (5, 513), (1, 2048), (2100, 1030), (2049, 2048), (7, 2056),
                                 (3, 4097), (2, 11008), (3, 12291), (2, 20001)])
def test_norm(M, K, out_dtype, res):
    x_dtype = BF16 if (M + K) % 2 else F32
    x = make(M + K, M, K, dtype=x_dtype)
    if M > 2:
        x[1] = 0
    r = None if res is None else make(M + K + 1, M, K, dtype=res)
    if r is not None and M > 2:
        r[1] = 0
    w = None if M == 4 else 1 + 0.3 * make(K, K)
    kept = None if r is None else torch.empty_like(r)
    rstd = torch.empty(M, device="cuda")
    out = torch.full((M, up(K, 128) if out_dtype == E4 else K), 1.0, device="cuda").to(out_dtype)
    scales = torch.full((M, up(-(-K // 128), 4)), 255, dtype=torch.uint8, device="cuda").view(E8) if out_dtype == E4 else None
    hx.hxq_rms_norm(x, w, 1e-5, out, scales=scales, residual=r, residual_out=kept, rstd=rstd)
    h = x.cpu().float()
    if r is not None:
        h = (h + r.cpu().float()).to(res)
        assert torch.equal(kept.cpu(), h)
    Y, R = O.rms_norm(host(h), None if w is None else host(w), np.float64(np.float32(1e-5)))
    tol = (ops(K) / 2 + 6) * U
    near(rstd, R, tol * R, "rstd")
    if out_dtype != E4:
        near(out, Y, (tol + HALF[out_dtype]) * np.abs(Y), "norm")
        return
    # e4m3: half a step of 2^-4, or of the smallest value 2^-9; the scale by the rule, from a magnitude
    # within the norm's tolerance
    G = -(-K // 128)
    S = raw(scales)
    assert (S[:, G:] == 127).all()
    top = np.pad(np.abs(Y), ((0, 0), (0, -K % 128))).reshape(M, G, 128).max(2)
    assert ((S[:, :G] == O.scale_byte(top * (1 - tol))) | (S[:, :G] == O.scale_byte(top * (1 + tol)))).all()
    got = O.wide_rows(raw(out), S)
    assert (got[:, K:] == 0).all()
    p = np.repeat(O.power(S[:, :G]), 128, axis=1)[:, :K]
    assert (np.abs(got[:, :K] - Y) <= np.maximum(2.0**-4 * np.abs(Y) * (1 + 2 * tol), 2.0**-10 * p) + tol * np.abs(Y)).all()


def test_norm_in_place_and_special_rows():
    x, r = make(1, 6, 700), make(2, 6, 700, dtype=BF16)
    x[1, 3], x[2, 4], x[3, 5] = float("nan"), float("inf"), 1e30  # (the last one's square overflows)
    want, kept = torch.empty(6, 700, device="cuda"), torch.empty_like(r)
    hx.hxq_rms_norm(x, None, 1e-6, want, residual=r, residual_out=kept)
    r2, out = r.clone(), torch.empty_like(want)
    hx.hxq_rms_norm(x, None, 1e-6, out, residual=r2, residual_out=r2)
    assert torch.equal(r2.view(torch.int16), kept.view(torch.int16)) and torch.equal(out.view(torch.int32), want.view(torch.int32))
    fine = torch.tensor([0, 4, 5])
    Y, _ = O.rms_norm(host(kept)[fine], None, 1e-6)
    near(want[fine], Y, (ops(700) / 2 + 6) * U * np.abs(Y))
    assert want[1].isnan().all() and want[2, 4].isnan() and (want[3] == 0).all()


@pytest.mark.parametrize("dres,dw", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 512), (2100, 513), (4500, 130), (700, 2048), (3, 2056), (1500, 4096), (6, 11008), (5, 20001), (520, 12801)])
def test_norm_gradient(M, K, dres, dw):
    h = make(M + K, M, K, dtype=BF16 if K % 2 else F32)
    dy = make(M + K + 1, M, K, dtype=BF16 if M % 2 else F32)
    w = None if M == 5 else 1 + 0.3 * make(K, K)
    rstd = torch.from_numpy(O.rms_norm(host(h), None, 1e-6)[1]).float().cuda()
    d = make(M + 7, M, K) if dres else None
    dx, dweight = torch.full((M, K), float("nan"), device="cuda"), torch.full((K,), float("nan"), device="cuda") if dw else None
    hx.hxq_rms_norm_bwd(dy, h, w, rstd, dx, dweight=dweight, dresidual=d)
    H, D, W, R = host(h), host(dy), 1 if w is None else host(w), host(rstd)[:, None]
    DX, DW = O.rms_norm_bwd(D, H, None if w is None else W, R[:, 0], None if d is None else host(d))
    g = np.abs(D * W)
    mean = (g * np.abs(H)).mean(1, keepdims=True)
    bound = U * (8 * (R * g + R**3 * np.abs(H) * mean) + (ops(K) + 8) * R**3 * np.abs(H) * mean + 2 * np.abs(DX))
    near(dx, DX, bound, "dx")
    if dw:
        near(dweight, DW, (min(M, 600) + 20) * U * (np.abs(D * H) * R).sum(0), "dweight")
    if d is not None:  # dx over dresidual
        again = torch.empty_like(dweight) if dw else None
        hx.hxq_rms_norm_bwd(dy, h, w, rstd, d, dweight=again, dresidual=d)
        assert torch.equal(d, dx) and (not dw or torch.equal(again, dweight))


def test_norm_gradient_of_no_rows():
    e = torch.empty((0, 9), device="cuda")
    dw = torch.full((9,), 7.0, device="cuda")
    hx.hxq_rms_norm_bwd(e, e, None, torch.empty(0, device="cuda"), e, dweight=dw)
    assert not dw.any()
    hx.hxq_rms_norm(e, None, 1e-6, e)


# ---------------------------------------------------------------- layer objects

def test_norm_under_autograd():
    x, r = make(1, 2, 5, 300).requires_grad_(), make(2, 2, 5, 300, dtype=BF16).requires_grad_()
    norm = hx.RmsNorm(1 + 0.2 * make(3, 300))
    norm.weight.requires_grad_()
    y, h = norm(x, r, out_dtype=F32)
    dy, dh = make(4, 2, 5, 300), make(5, 2, 5, 300, dtype=BF16)
    torch.autograd.backward((y, h), (dy, dh))
    H = host(h).reshape(10, 300)
    Y, R = O.rms_norm(H, host(norm.weight), 1e-6)
    near(y.reshape(10, 300), Y, 20 * U * np.abs(Y))
    DX, DW = O.rms_norm_bwd(host(dy).reshape(10, 300), H, host(norm.weight), R, host(dh).reshape(10, 300))
    near(x.grad.reshape(10, 300), DX, 60 * U * np.abs(DX).max())
    near(r.grad.reshape(10, 300), DX, 60 * U * np.abs(DX).max() + HALF[BF16] * np.abs(DX))
    near(norm.weight.grad, DW, 60 * U * np.abs(DW).max())
    assert x.grad.dtype == F32 and r.grad.dtype == BF16
    # only one of the outputs used; no residual; frozen weight
    x2 = make(1, 5, 300).requires_grad_()
    _, h2 = norm(x2, make(2, 5, 300, dtype=BF16), out_dtype=F32)
    h2.sum().backward()
    assert torch.equal(x2.grad, torch.ones_like(x2))
    x3 = make(1, 5, 300).requires_grad_()
    frozen = hx.RmsNorm(None)
    y3, none = frozen(x3, out_dtype=F32)
    assert none is None
    y3.backward(torch.ones_like(y3))
    DX, _ = O.rms_norm_bwd(np.ones((5, 300)), host(x3), None, O.rms_norm(host(x3), None, 1e-6)[1])
    near(x3.grad, DX, 60 * U * np.abs(DX).max())


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_linear_under_autograd(M, dtype):
    N, K = 300, 200
    w = make(2, N, K, scale=0.02)
    layer = hx.Fp8Linear(w, make(3, N), train=True)
    x = make(1, M, K, dtype=dtype).requires_grad_()
    y = layer(x.reshape(1, M, K))
    assert y.shape == (1, M, N) and y.dtype == F32
    dy = make(4, M, N)
    y.backward(dy[None])
    Q, S = O.quant_weight(host(w))
    W = O.wide_weight(Q, S)
    D = O.wide_rows(*O.quant_rows(host(dy)))[:, :N]
    DX, B = D @ W[:, :K], np.abs(D) @ np.abs(W[:, :K])
    assert x.grad.dtype == dtype
    near(x.grad, DX, 1e-5 * B + HALF[dtype] * np.abs(DX))
    with pytest.raises(RuntimeError, match="train=True"):
        hx.Fp8Linear(w)(x)


def test_experts_under_autograd():
    E, N, K, Mx = 5, 140, 260, 12
    w = make(2, E, N, K, scale=0.02)
    layer = hx.Fp8Experts(w, make(3, E, N), train=True)
    rows, offsets = routing(1, [4, 0, 9, 2, 6], Mx, 3)
    rows[21:] = -3
    x = make(1, Mx, K).requires_grad_()
    y = layer(x, offsets, rows)
    assert (y[21:] == 0).all()
    dy = make(4, 24, N)
    dy[21:] = float("nan")  # gradients of rows that nothing computed
    y.backward(dy)
    D = O.wide_rows(*O.quant_rows(host(dy)[:21]))[:, :N]
    each = [O.wide_weight(*O.quant_weight(host(w[e])))[:, :K] for e in range(E)]
    DX, B = np.zeros((Mx, K)), np.zeros((Mx, K))
    off, r = offsets.tolist(), rows.tolist()
    for e in range(E):
        for i in range(off[e], off[e + 1]):
            DX[r[i]] += D[i] @ each[e]
            B[r[i]] += np.abs(D[i]) @ np.abs(each[e])
    near(x.grad, DX, 1e-5 * B)
    x2 = make(1, 21, K).requires_grad_()
    layer(x2, offsets).backward(dy[:21])
    near(x2.grad[:4], D[:4] @ each[0], 1e-5 * (np.abs(D[:4]) @ np.abs(each[0])))


@pytest.mark.parametrize("fmt", ["u8", "pk12"])
def test_layers_from_compressed_ones(fmt):
    """An 8-bit layer laid out from a compressed one holds its weight to half a step of e4m3."""
    lays = [gen.random_layer(s, 200, 256, fmt, nnz=60, duplicates=True) for s in (1, 2)]
    helix = [hx.HelixLinear.from_layer(l) for l in lays]
    dense = [torch.empty((200, 256), dtype=BF16, device="cuda") for _ in helix]
    for h, d in zip(helix, dense):
        hx.hxq_dequant_bf16(hx.HXQ_FMT_U8 if fmt == "u8" else hx.HXQ_FMT_PK12, h.codebook, h.indices, h.sc_rows, h.sc_cols, h.sc_deltas, d)
    x = make(1, 9, 256)
    X = O.wide_rows(*O.quant_rows(host(x)))
    for h, d in zip(helix, dense):
        layer = hx.Fp8Linear.from_helix(h)
        Y, B = O.linear(X, O.wide_weight(*O.quant_weight(host(d))), None if h.bias is None else host(h.bias))
        near(layer(x), Y, 1e-5 * B + U * np.abs(Y))
        assert layer.compressed_bytes() == 200 * 256 + 2 * 4
    e = hx.Fp8Experts.from_helix(helix)
    y = e(x, torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda"))
    assert torch.equal(y[:4], hx.Fp8Linear.from_helix(helix[0])(x)[:4]) and torch.equal(y[4:], hx.Fp8Linear.from_helix(helix[1])(x)[4:])


# ------------------------------------------------------------- as they are used

def test_a_block_of_experts():
    """norm -> experts -> gate -> experts -> norm, each fed by the one before, against the oracle fed with what
    the GPU's step before it gave."""
    T, K, F, E, top = 37, 256, 200, 6, 2
    x, res = make(1, T, K), make(2, T, K, dtype=BF16)
    norm = hx.RmsNorm(1 + 0.1 * make(3, K))
    up_, down = hx.Fp8Experts(make(4, E, 2 * F, K, scale=0.05)), hx.Fp8Experts(make(5, E, K, F, scale=0.05))
    chosen = torch.rand(T, E, generator=torch.Generator().manual_seed(6)).topk(top).indices.flatten()
    order = chosen.sort(stable=True).indices
    rows = (order // top).int().cuda()
    offsets = torch.nn.functional.pad(torch.bincount(chosen, minlength=E).cumsum(0), (1, 0)).int().cuda()
    (q, s), h = norm(x, res, out_dtype=E4)
    a = up_((q, s), offsets, rows)
    Y, B = O.experts(O.wide_rows(raw(q), raw(s)), rows.cpu().numpy(), offsets.tolist(),
                     [O.wide_weight(raw(up_.wq[e]), raw(up_.w_scales[e])) for e in range(E)])
    near(a, Y, 1e-5 * B)
    g = (torch.nn.functional.silu(a[:, :F]) * a[:, F:]).contiguous()
    d = down(g, offsets)
    Y, B = O.experts(O.wide_rows(*O.quant_rows(host(g))), None, offsets.tolist(),
                     [O.wide_weight(raw(down.wq[e]), raw(down.w_scales[e])) for e in range(E)])
    near(d, Y, 1e-5 * B)
    back = torch.empty(T * top, K, device="cuda")
    back[order.cuda()] = d
    out, h2 = norm(back.view(T, top, K).sum(1), h)
    want = (back.view(T, top, K).sum(1).cpu() + h.cpu().float()).to(BF16)
    assert torch.equal(h2.cpu(), want)
    Y, _ = O.rms_norm(host(want), host(norm.weight), 1e-6)
    near(out, Y, (20 * U + HALF[BF16]) * np.abs(Y))


def test_captured_and_replayed():
    """Norm and products in one graph, inputs changed between replays, eager work in between."""
    T, K, N = 3, 512, 640
    x, res, w = make(1, T, K), make(2, T, K, dtype=BF16), 1 + 0.1 * make(3, K)
    layer = hx.Fp8Linear(make(4, N, K, scale=0.05))
    many = make(8, 300, K, dtype=BF16)
    experts = hx.Fp8Experts(make(5, 4, K, N, scale=0.05))
    offsets = torch.tensor([0, 1, 1, 3, 3], dtype=torch.int32, device="cuda")
    norm = hx.RmsNorm(w)

    def step():
        (q, s), h = norm(x, res, out_dtype=E4)
        y = layer((q, s))
        return y, h, experts(y, offsets), layer(many, out_dtype=BF16)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.copy_(make(10 + i, T, K))
        many.copy_(make(20 + i, 300, K, dtype=BF16))
        offsets.copy_(torch.tensor([0, i % 3, i % 3, 2, 3], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in got]
        for a, b in zip(have, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_scales_of_any_strides_captured():
    """The copy of permuted scales is part of a graph: replays see the scales as they are then."""
    N, K, M = 300, 512, 40  # one row of scales for each 128 of N, four blocks of K: no padding either way
    w, s = weight8(make(1, N, K, scale=0.02))
    loose = s.view(torch.uint8).t().contiguous().t()
    x, y = make(2, M, K), torch.empty((M, N), device="cuda")

    def step(scales, out):
        hx.hxq_linear_fwd_fp8(x, None, w, scales.view(E8), None, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(loose, y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(loose, y)
    for i in range(4):
        loose += i
        graph.replay()
        torch.cuda.synchronize()
        have, want = y.clone(), torch.empty_like(y)
        step(loose.contiguous(), want)
        assert torch.equal(have, want) and not have.isnan().any()
        torch.cuda.synchronize()


def test_gradients_captured_and_replayed():
    """Forward and backward of the layers in one graph, inputs changed between replays, the same work eagerly (on
    leaves of its own) in between."""
    T, K, N, E = 9, 512, 640, 3
    layer = hx.Fp8Linear(make(4, N, K, scale=0.05), train=True)
    experts = hx.Fp8Experts(make(5, E, K, N, scale=0.05), train=True)
    offsets = torch.tensor([0, 4, 4, 7], dtype=torch.int32, device="cuda")
    dy = make(6, T, K)

    def leaves():
        return (make(1, T, K).requires_grad_(), make(2, T, K, dtype=BF16).requires_grad_(),
                hx.RmsNorm((1 + 0.1 * make(3, K)).requires_grad_()))

    def step(x, res, norm):
        y, h = norm(x, res)
        z = experts(layer(y), offsets)
        return (z.detach(), *torch.autograd.grad((z, h), (x, res, norm.weight), (dy, dy.bfloat16())))

    mine, eager = leaves(), leaves()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*mine)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*mine)
    for i in range(4):
        new = make(10 + i, T, K)
        with torch.no_grad():
            mine[0].copy_(new)
            eager[0].copy_(new)
        dy.copy_(make(20 + i, T, K))
        offsets.copy_(torch.tensor([0, i, 5, 5 + i], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in got]
        for a, b in zip(have, step(*eager)):
            assert torch.equal(a, b) and not a.isnan().any()
        torch.cuda.synchronize()


def test_on_another_stream():
    """Calls given a stream run there; two streams at once, each with a workspace of its own."""
    N, K = 2048, 2048
    q, s = weight8(make(1, N, K, scale=0.02))
    xs = [make(i, 40, K, dtype=BF16) for i in range(2)]
    want = [torch.empty((40, N), device="cuda") for _ in xs]
    for x, y in zip(xs, want):
        hx.hxq_linear_fwd_fp8(x, None, q, s, None, y)
    got = [torch.empty_like(y) for y in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for x, y, st in zip(xs, got, streams):
            hx.hxq_linear_fwd_fp8(x, None, q, s, None, y, stream=st)
    for x, y, st in zip(xs, got, streams):
        hx.hxq_linear_fwd_fp8(x, None, q, s, None, y, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("out_dtype,res", [(F32, BF16), (BF16, F32), (E4, BF16), (E4, None)])
def test_norm_of_more_rows_than_a_launch(out_dtype, res):
    """2^22 rows to a launch: the second one's rows are those that a call of their own gives."""
    M, K, cut = 2**22 + 3, 5, 2**22
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda")
    r = None if res is None else torch.randn(M, K, generator=g, device="cuda").to(res)
    w = make(2, K)

    def norm(*at):
        n = len(range(M)[slice(*at)])
        out = torch.full((n, 128 if out_dtype == E4 else K), 3.0, device="cuda").to(out_dtype)
        scales = torch.full((n, 4), 9, dtype=torch.uint8, device="cuda").view(E8) if out_dtype == E4 else None
        kept = None if res is None else torch.full((n, K), 3.0, dtype=res, device="cuda")
        rstd = torch.full((n,), 3.0, device="cuda")
        hx.hxq_rms_norm(x[slice(*at)], w, 1e-6, out, scales=scales, residual=None if r is None else r[slice(*at)],
                        residual_out=kept, rstd=rstd)
        return [t if t.dtype not in (E4, E8) else t.view(torch.uint8) for t in (out, scales, kept, rstd) if t is not None]

    for whole_, first, last in zip(norm(0, M), norm(0, cut), norm(cut, M)):
        assert torch.equal(whole_[:cut], first) and torch.equal(whole_[cut:], last)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_more_groups_than_a_launch(dtype):
    """2^26 groups of a row of scales to a launch, four to a row here."""
    cut = 2**24
    x = torch.randn(cut + 5, 1, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    (q, s), (q1, s1), (q2, s2) = [[t.view(torch.uint8) for t in rows8(v)] for v in (x, x[:cut], x[cut:])]
    assert torch.equal(q[:cut], q1) and torch.equal(s[:cut], s1) and torch.equal(q[cut:], q2) and torch.equal(s[cut:], s2)
    Q, S = O.quant_rows(host(x[cut:]))
    assert np.array_equal(q2.cpu().numpy(), Q) and np.array_equal(s2.cpu().numpy(), S)


def test_rows_past_32_bits():
    """x of more than 2^32 bytes: the last rows are read where they are."""
    M, K, N = 2**21 + 40, 2048, 40
    x = torch.zeros((M, K), dtype=torch.uint8, device="cuda").view(E4)
    s = torch.full((M, 4), 127, dtype=torch.uint8, device="cuda").view(E8)
    last = make(1, 40, K)
    lq, ls = rows8(last)
    x.view(torch.uint8)[-40:] = lq.view(torch.uint8)
    s = torch.full((M, 16), 127, dtype=torch.uint8, device="cuda")
    s[-40:] = ls.view(torch.uint8)
    q, ws = weight8(make(2, N, K, scale=0.02))
    y = torch.empty((M, N), device="cuda")
    hx.hxq_linear_fwd_fp8(x, s.view(E8), q, ws, None, y)
    Y, B = O.linear(O.wide_rows(raw(lq), raw(ls)), O.wide_weight(raw(q), raw(ws)))
    near(y[-40:], Y, 1e-5 * B)
    assert not y[:-40].any()
    rows = torch.arange(M - 40, M, dtype=torch.int32, device="cuda").flip(0).contiguous()
    ye = torch.empty((40, N), device="cuda")
    hx.hxq_linear_fwd_fp8_experts(x, s.view(E8), rows, torch.tensor([0, 40], dtype=torch.int32, device="cuda"), q[None], ws[None], None, ye)
    near(ye.flip(0), Y, 1e-5 * B)
