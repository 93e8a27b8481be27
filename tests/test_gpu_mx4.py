"""MX4 codec, products and linear layer on the GPU against the float64 oracle:
codes bit for bit (every bf16 and fp16 value, fp32 over all exponents), values
exact, products within a bound from the sums' sizes."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from oracle import linear as olin
from oracle import mx4
from tests.gpu_util import DEV, as_f64, assert_close, guarded_like

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _host64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _stored(a):
    return a.codes.cpu().numpy(), a.scales.cpu().numpy()


def _check_codec(x):
    """x [rows, cols] on the device: codes, fill and values against the oracle."""
    rows, cols = x.shape
    slabs = -(-cols // 256)
    gc, codes = guarded_like((rows, 128 * slabs), torch.uint8, 1)
    gs, scales = guarded_like((slabs, rows, 8), torch.uint8, 2)
    a = q.MX4Tensor.quantize(x, out=q.MX4Tensor(codes, scales, rows, cols))
    code, byte = mx4.quantize(_host64(x))
    want_c, want_s = mx4.lay_out(code, byte)
    got_c, got_s = _stored(a)
    np.testing.assert_array_equal(got_s, want_s)
    np.testing.assert_array_equal(got_c, want_c)
    gv, v = guarded_like((rows, cols), BF16, 3)
    a.dequantize(out=v)
    want = mx4.values(code, byte)
    np.testing.assert_array_equal(_host64(v), want)
    assert gc.intact() and gs.intact() and gv.intact()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_codec_every_16_bit_value(dtype):
    g = np.random.default_rng(1)
    bits = np.concatenate([g.permutation(65536), np.arange(65536)]).astype(np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(dtype).reshape(-1, 256)
    finite = torch.where(torch.isfinite(x), x, torch.ones_like(x))
    _check_codec(finite.to(DEV))
    _check_codec(x.to(DEV))            # blocks with NaN and infinities among them


def test_codec_fp32_over_all_exponents():
    g = np.random.default_rng(2)
    bits = g.integers(0, 1 << 32, (512, 256), dtype=np.uint32)
    bits[:, :128] = (bits[:, :128] & 0x807FFFFF) | (g.integers(0, 255, (512, 1)).astype(np.uint32) << 23)   # one exponent a row
    x = torch.from_numpy(bits.view(np.float32))
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    _check_codec(x.to(DEV))
    halfway = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0, 7.999])
    rows = []
    for e in range(-126, 125):
        r = torch.zeros(32)
        r[:11], r[11:22] = halfway, -halfway
        r[22:31] = torch.nextafter(halfway[:9], torch.tensor(9.0))
        r[31] = 7.999
        rows.append(r * 2.0 ** e)
    _check_codec(torch.stack(rows).to(DEV))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 96), (8, 256), (33, 288), (65, 4096), (3, 11008), (2500, 14368)])
def test_codec_shapes(dtype, rows, cols):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g).float())
    x[:, : min(cols, 32)] = 0.0        # a block of zeros
    _check_codec(x.to(dtype).to(DEV))


def test_decode_every_code_under_every_scale():
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8).reshape(256, 1)
    c, s = mx4.lay_out(codes, byte)
    a = q.MX4Tensor(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), 256, 32)
    got = _host64(a.dequantize())
    want = mx4.values(codes, byte)
    want = np.where(np.abs(want) < 2.0 ** 128, want, np.sign(want) * np.inf)   # bytes 252 .. 254 reach past bf16
    np.testing.assert_array_equal(got, want)


def _array(v, seed):
    """An MX4Tensor of host values and the float64 values it holds."""
    code, byte = mx4.quantize(v)
    c, s = mx4.lay_out(code, byte)
    return q.MX4Tensor(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), *v.shape), mx4.values(code, byte)


def _bound(want, size, terms):
    """fp32 sums of `terms` exact products (any order, truncating adders: one
    unit of 2^-23 of the terms' absolute sum an addition), then bf16 (8
    significant bits: half a unit is 2^-8)."""
    d = terms * 2.0 ** -23 * size
    return d + 2.0 ** -8 * (np.abs(want) + d) + 2.0 ** -133


def _product(M, N, K, r, seed, spread=6):
    g = np.random.default_rng(seed)
    x, xv = _array(g.standard_normal((M, K)) * np.exp2(g.integers(-spread, spread, (M, 1))), 0)
    w, wv = _array(g.standard_normal((N, K)) * np.exp2(g.integers(-spread, spread, (N, K // 32))).repeat(32, 1), 1)
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    T = B = None
    if r:
        T = torch.from_numpy(g.standard_normal((M, r)).astype(np.float32)).to(BF16).to(DEV)
        B = torch.from_numpy(g.standard_normal((N, r)).astype(np.float32)).to(BF16).to(DEV)
        t, b = as_f64(T), as_f64(B)
        want, size = want + t @ b.T, size + np.abs(t) @ np.abs(b).T
    gy, Y = guarded_like((M, N), BF16, 5)
    q.mx4_matmul(x, w, T, B, out=Y)
    got = as_f64(Y)
    assert gy.intact()
    bad = ~(np.abs(got - want) <= _bound(want, size, K + r + 1))
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 127, 129, 257])
@pytest.mark.parametrize("N,K,r", [(1, 32, 0), (17, 288, 8), (130, 1056, 64), (264, 512, 128), (203, 256, 33)])
def test_product_small(M, N, K, r):
    _product(M, N, K, r, 100 + M)


@pytest.mark.parametrize("M,N,K,r", [(4097, 4104, 64, 0), (2049, 8200, 288, 65), (4096, 4096, 512, 64),
                                     (300, 5003, 2048, 0), (1, 11008, 4096, 64), (64, 4096, 11008, 64),
                                     (5, 40, 22016, 8), (48, 24, 16384, 16), (100, 2056, 6656, 64),
                                     (200, 1000, 17920, 0), (513, 256, 8192, 1)])
def test_product_large(M, N, K, r):
    _product(M, N, K, r, 200 + M)


def test_product_of_distant_scales():
    """Scales from 2^-60 to 2^60 on both sides in one contraction."""
    _product(40, 72, 1024, 0, 3, spread=60)


@pytest.mark.parametrize("M", [3, 40, 200])
def test_a_nan_block_reaches_the_sums_it_enters_only(M):
    g = np.random.default_rng(8)
    xv, wv = g.standard_normal((M, 544)), g.standard_normal((70, 544))
    xv[1, 100] = np.nan
    wv[5, 543] = np.inf
    x, xq = _array(xv, 0)
    w, wq = _array(wv, 1)
    got = as_f64(q.mx4_matmul(x, w))
    want = xq @ wq.T
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    assert np.isnan(got[1]).all() and np.isnan(got[:, 5]).all() and np.isnan(got).sum() == M + 70 - 1
    ok = ~np.isnan(want)
    size = np.nan_to_num(np.abs(xq)) @ np.nan_to_num(np.abs(wq)).T
    assert (np.abs(got - want)[ok] <= _bound(want, size, 545)[ok]).all()


def _linear_case(M, N, K, r, seed):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(M, K, generator=g).to(BF16)
    W = torch.randn(N, K, generator=g) * 0.02
    A = (torch.randn(r, K, generator=g) * 0.01).to(BF16)
    B = (torch.randn(N, r, generator=g) * 0.01).to(BF16)
    dY = torch.randn(M, N, generator=g).to(BF16)
    return X, W, A, B, dY


@pytest.mark.parametrize("M,N,K,r", [(1, 64, 64, 8), (1, 4096, 4096, 64), (4, 200, 288, 16), (16, 264, 1056, 64), (17, 136, 512, 128),
                                     (64, 1024, 11008, 64), (65, 128, 320, 1), (100, 1000, 544, 33), (300, 512, 768, 64),
                                     (129, 2000, 4096, 0), (7, 77, 96, 0), (33, 129, 2080, 0), (3, 5000, 64, 0)])
def test_linear_forward(M, N, K, r):
    X, W, A, B, _ = _linear_case(M, N, K, max(r, 1), M + N + K)
    w = q.MX4Tensor.quantize(W.to(DEV))
    wv, xv = mx4.quantized(_host64(W)), mx4.quantized(_host64(X))
    gy, Y = guarded_like((M, N), BF16, 6)
    if r == 0:
        _, T = q.mx4_linear_fwd(X.to(DEV), w, out=Y)
        assert T is None
        want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        assert (np.abs(as_f64(Y) - want) <= _bound(want, size, K)).all()
    else:
        scale = 16.0 / r
        gt, T = guarded_like((M, r), BF16, 7)
        q.mx4_linear_fwd(X.to(DEV), w, A.to(DEV), B.to(DEV), scale, T_out=T, out=Y)
        assert gt.intact()
        T64 = scale * _host64(X) @ _host64(A).T
        assert_close(as_f64(T), T64, "T")
        got_t = as_f64(T)
        want = xv @ wv.T + got_t @ _host64(B).T
        size = np.abs(xv) @ np.abs(wv).T + np.abs(got_t) @ np.abs(_host64(B)).T
        assert (np.abs(as_f64(Y) - want) <= _bound(want, size, K + r)).all()
    assert gy.intact()


@pytest.mark.parametrize("M,N,K,r", [(75, 552, 8224, 64), (129, 203, 6656, 0), (70, 1001, 11008, 8), (200, 264, 5632, 100),
                                     (300, 330, 8192, 33), (65, 1, 16384, 1), (128, 136, 22016, 64)])
@pytest.mark.parametrize("keep", [False, True])
def test_linear_forward_of_few_tiles(M, N, K, r, keep):
    """Long contractions of few output tiles, T kept by the caller or not."""
    X, W, A, B, _ = _linear_case(M, N, K, max(r, 1), M + N + K)
    w = q.MX4Tensor.quantize(W.to(DEV))
    wv, xv = mx4.quantized(_host64(W)), mx4.quantized(_host64(X))
    gy, Y = guarded_like((M, N), BF16, 8)
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    if r:
        T = torch.empty(M, r, dtype=BF16, device=DEV) if keep else None
        _, T = q.mx4_linear_fwd(X.to(DEV), w, A.to(DEV), B.to(DEV), 0.5, T_out=T, out=Y)
        assert_close(as_f64(T), 0.5 * _host64(X) @ _host64(A).T, "T")
        want, size = want + as_f64(T) @ _host64(B).T, size + np.abs(as_f64(T)) @ np.abs(_host64(B)).T
    else:
        q.mx4_linear_fwd(X.to(DEV), w, out=Y)
    assert (np.abs(as_f64(Y) - want) <= _bound(want, size, K + r)).all()
    assert gy.intact()
    first = Y.clone()
    q.mx4_linear_fwd(X.to(DEV), w, *((A.to(DEV), B.to(DEV), 0.5) if r else ()), out=Y)
    assert torch.equal(first, Y)


@pytest.mark.parametrize("M,N,K,r", [(2047, 72, 1056, 64), (2048, 136, 288, 64), (2050, 64, 1056, 5), (2081, 128, 320, 33),
                                     (100, 264, 512, 100), (2100, 24, 96, 128), (65, 4104, 96, 0), (130, 33000, 64, 0),
                                     (100, 66000, 32, 8)])
def test_linear_forward_of_many_tokens(M, N, K, r):
    """X rounded and multiplied by the adapter in one pass or by parts; large and small tiles."""
    X, W, A, B, _ = _linear_case(M, N, K, max(r, 1), M + N + K)
    w = q.MX4Tensor.quantize(W.to(DEV))
    wv, xv = mx4.quantized(_host64(W)), mx4.quantized(_host64(X))
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    if r:
        Y, T = q.mx4_linear_fwd(X.to(DEV), w, A.to(DEV), B.to(DEV), 0.25)
        assert_close(as_f64(T), 0.25 * _host64(X) @ _host64(A).T, "T")
        want, size = want + as_f64(T) @ _host64(B).T, size + np.abs(as_f64(T)) @ np.abs(_host64(B)).T
    else:
        Y, _ = q.mx4_linear_fwd(X.to(DEV), w)
    assert (np.abs(as_f64(Y) - want) <= _bound(want, size, K + r)).all()


@pytest.mark.parametrize("M,N,K,r", [(1, 64, 64, 8), (40, 128, 320, 16), (300, 512, 768, 64), (129, 192, 4096, 33)])
def test_linear_backward(M, N, K, r):
    X, W, A, B, dY = _linear_case(M, N, K, r, M + N)
    w = q.MX4Tensor.quantize(W.to(DEV))
    scale = 8.0 / r
    Xd, Ad, Bd, dYd = (t.to(DEV) for t in (X, A, B, dY))
    _, T = q.mx4_linear_fwd(Xd, w, Ad, Bd, scale)
    want = olin.linear_bwd(*(t.contiguous().view(torch.int16).numpy().view(np.uint16) for t in (dY, X)),
                           mx4.quantized(_host64(W)), *(t.contiguous().view(torch.int16).numpy().view(np.uint16) for t in (A, B)),
                           scale)
    got = q.mx4_linear_bwd(dYd, Xd, T, w, Ad, Bd, scale)
    for name, a, b in zip(("dX", "dA", "dB"), got, want):
        assert_close(as_f64(a), b, name)
    again = q.mx4_linear_bwd(dYd, Xd, None, w, Ad, Bd, scale)      # T recomputed, its sums in another order
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert_close(as_f64(again[2]), want[2], "dB, T recomputed")
    only = q.mx4_linear_bwd(dYd, Xd, T, w, Ad, Bd, scale, need_dX=False, need_dB=False)
    assert only[0] is None and only[2] is None
    assert_close(as_f64(only[1]), want[1], "dA alone")


@pytest.mark.parametrize("M,N,K,r", [(69, 2240, 2560, 64), (75, 576, 1344, 33), (200, 1024, 192, 100), (1, 4096, 64, 8),
                                     (513, 1344, 704, 64), (33, 22016, 128, 1), (128, 512, 320, 128), (65, 8192, 64, 64),
                                     (1100, 256, 4096, 64), (700, 320, 2048, 16)])
def test_linear_backward_of_few_tiles(M, N, K, r):
    X, W, A, B, dY = _linear_case(M, N, K, r, M + N)
    w = q.MX4Tensor.quantize(W.to(DEV))
    scale = 8.0 / r
    Xd, Ad, Bd, dYd = (t.to(DEV) for t in (X, A, B, dY))
    want = olin.linear_bwd(*(t.contiguous().view(torch.int16).numpy().view(np.uint16) for t in (dY, X)),
                           mx4.quantized(_host64(W)), *(t.contiguous().view(torch.int16).numpy().view(np.uint16) for t in (A, B)),
                           scale)
    gx, dX = guarded_like((M, K), BF16, 9)
    got = q.mx4_linear_bwd(dYd, Xd, None, w, Ad, Bd, scale, dX_out=dX)
    for name, a, b in zip(("dX", "dA", "dB"), got, want):
        assert_close(as_f64(a), b, name)
    assert gx.intact()
    only = q.mx4_linear_bwd(dYd, Xd, None, w, Ad, Bd, scale, need_dA=False, need_dB=False)
    assert torch.equal(only[0], got[0])


def test_pair_gradients_against_differences():
    """Y is linear in A and in B, the codes of X fixed: central differences of
    sum(dY * Y), in float64 on the oracle's values, are exact up to rounding."""
    M, N, K, r = 5, 64, 64, 4
    X, W, A, B, dY = _linear_case(M, N, K, r, 77)
    w = q.MX4Tensor.quantize(W.to(DEV))
    lin = q.MX4Linear(W.to(DEV), r, 8.0, A.to(DEV), B.to(DEV))
    Xd = X.to(DEV).requires_grad_()
    y = lin(Xd)
    y.backward(dY.to(DEV))
    wv, x, a, b, g = mx4.quantized(_host64(W)), _host64(X), _host64(A), _host64(B), _host64(dY)

    def loss(a, b):
        return (g * (mx4.quantized(x) @ wv.T + 2.0 * (x @ a.T) @ b.T)).sum()

    for got, at, which in ((lin.lora_A.grad, a, 0), (lin.lora_B.grad, b, 1)):
        d = np.zeros_like(at)
        for i in np.ndindex(at.shape):
            hi, lo = at.copy(), at.copy()
            hi[i] += 0.5
            lo[i] -= 0.5
            d[i] = loss(*((hi, b) if which == 0 else (a, hi))) - loss(*((lo, b) if which == 0 else (a, lo)))
        assert_close(as_f64(got), d, "AB"[which])
    assert_close(as_f64(Xd.grad), g @ wv + 2.0 * (g @ b) @ a, "dX, straight through")


def test_no_tokens_and_another_stream():
    X, W, A, B, dY = _linear_case(37, 128, 320, 8, 5)
    w = q.MX4Tensor.quantize(W.to(DEV))
    Ad, Bd = A.to(DEV), B.to(DEV)
    Y, T = q.mx4_linear_fwd(torch.empty(0, 320, dtype=BF16, device=DEV), w, Ad, Bd, 1.0)
    assert Y.shape == (0, 128) and T.shape == (0, 8)
    assert q.MX4Tensor.quantize(torch.empty(0, 64, device=DEV)).dequantize().shape == (0, 64)
    Xd, dYd = X.to(DEV), dY.to(DEV)
    Y0, T0 = q.mx4_linear_fwd(Xd, w, Ad, Bd, 1.0)
    d0 = q.mx4_linear_bwd(dYd, Xd, T0, w, Ad, Bd, 1.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        w1 = q.MX4Tensor.quantize(W.to(DEV))
        Y1, T1 = q.mx4_linear_fwd(Xd, w1, Ad, Bd, 1.0)
        d1 = q.mx4_linear_bwd(dYd, Xd, T1, w1, Ad, Bd, 1.0)
    s.synchronize()
    assert torch.equal(Y0, Y1) and torch.equal(T0, T1) and all(torch.equal(a, b) for a, b in zip(d0, d1))


def test_graph_replays_equal_eager():
    """Forward at a decode and a tile size, captured and replayed on new inputs."""
    for M in (4, 200):
        X, W, A, B, _ = _linear_case(M, 256, 512, 16, 9)
        w = q.MX4Tensor.quantize(W.to(DEV))
        Ad, Bd, Xd = A.to(DEV), B.to(DEV), X.to(DEV)
        Y = torch.empty(M, 256, dtype=BF16, device=DEV)
        T = torch.empty(M, 16, dtype=BF16, device=DEV)
        ws = torch.empty(max(16, q.lib().qlora_mx4_linear_workspace_bytes(M, 256, 512, 16, 0)), dtype=torch.uint8, device=DEV)
        q.mx4_linear_fwd(Xd, w, Ad, Bd, 1.0, T_out=T, out=Y, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q.mx4_linear_fwd(Xd, w, Ad, Bd, 1.0, T_out=T, out=Y, workspace=ws)
        for k in range(4):
            Xd.copy_(X.roll(k, 1).to(DEV))
            graph.replay()
            torch.cuda.synchronize()
            want, wt = q.mx4_linear_fwd(Xd, w, Ad, Bd, 1.0)
            torch.cuda.synchronize()
            assert torch.equal(Y, want) and torch.equal(T, wt), (M, k)


def test_refusals():
    X = torch.zeros(4, 64, dtype=BF16, device=DEV)
    w = q.MX4Tensor.quantize(torch.zeros(8, 64, device=DEV))
    A, B = torch.zeros(8, 64, dtype=BF16, device=DEV), torch.zeros(8, 8, dtype=BF16, device=DEV)
    with pytest.raises(q.QLoRAError):
        q.MX4Tensor.quantize(torch.zeros(4, 48, device=DEV))              # cols % 32
    with pytest.raises(TypeError):
        q.MX4Tensor.quantize(torch.zeros(4, 64, dtype=torch.float64, device=DEV))
    with pytest.raises(ValueError):
        q.MX4Tensor.quantize(torch.zeros(4, 128, device=DEV)[:, :64])     # not contiguous
    with pytest.raises(ValueError):
        q.mx4_linear_fwd(X, w, A)                                         # half a pair
    with pytest.raises(ValueError):
        q.mx4_linear_fwd(torch.zeros(4, 32, dtype=BF16, device=DEV), w)
    with pytest.raises(TypeError):
        q.mx4_linear_fwd(X.float(), w)
    with pytest.raises(ValueError):
        q.mx4_linear_fwd(X, w, A, B, 1.0, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(q.QLoRAError):
        q.mx4_linear_fwd(X, w, A, B, float("nan"))
    with pytest.raises(q.QLoRAError):                                      # dX wants N % 64 == 0
        q.mx4_linear_bwd(torch.zeros(4, 8, dtype=BF16, device=DEV), X, None, w, A, B, 1.0,
                         workspace=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        q.MX4Tensor(w.codes, w.scales, 8, 512).dequantize()               # storage of another shape
    with pytest.raises(q.QLoRAError):
        q.mx4_matmul(q.MX4Tensor.quantize(X), q.MX4Tensor.quantize(torch.zeros(8, 96, device=DEV)))
