"""The norm of many tensors and clipping by it on the GPU against float64.

Bounds: squares are exact to 2^-53 and summed in 64 bits, so the norm is off by its
one rounding to fp32, 2^-24 (2^-23 allowed), a clipped value by the factor's rounding
(2^-24), the product's (2^-24) and the result's to its type."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from oracle import adapters as oad
from tests.gpu_util import DEV, Guarded

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
SMALL = {BF16: 2.0 ** -126, FP16: 2.0 ** -25, FP32: 2.0 ** -126}


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _grads(shapes, dtypes, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(*s, generator=g) * size).to(dtypes[k % len(dtypes)]).to(DEV) for k, s in enumerate(shapes)]


def _check(grads, max_norm, groups=1):
    want_n, want = oad.clip([_f64(t) for t in grads], max_norm, groups)
    before = [t.clone() for t in grads]
    n = q.grad_norm(grads, groups)
    assert n.shape == (groups,) and n.dtype == FP32
    np.testing.assert_allclose(_f64(n), want_n, rtol=2.0 ** -23)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    outs = [torch.full_like(t, float("nan")) for t in grads]
    n2 = q.clip_grad_norm(grads, max_norm, groups, out=outs)
    assert torch.equal(n, n2) and all(torch.equal(a, b) for a, b in zip(grads, before))
    n3 = q.clip_grad_norm(grads, max_norm, groups)
    assert torch.equal(n, n3)
    for a, b, w in zip(grads, outs, want):
        assert torch.equal(a, b)
        np.testing.assert_allclose(_f64(a), w, rtol=UNIT[a.dtype] + 3 * 2.0 ** -24, atol=SMALL[a.dtype])
    return n


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("count", [1, 7, 8, 4095, 4096, 4097, 100003, 2500000])
def test_one_tensor(count, dtype):
    _check(_grads([(count,)], [dtype], count), 0.5)


@pytest.mark.parametrize("max_norm", [0.0, 0.3, 1e9, float("inf")])
@pytest.mark.parametrize("groups", [1, 3])
def test_many_tensors_of_mixed_types_and_sizes(groups, max_norm):
    shapes = [(groups * r, c) for r, c in ((1, 1), (8, 513), (2, 4096), (3, 0), (1, 7), (64, 100), (5, 3333))] * 45
    _check(_grads(shapes, [BF16, FP32, FP16, BF16], 1, size=0.1), max_norm, groups)


def test_a_tensor_past_32_bits():
    """More than 2^32 elements, whole numbers in a few places."""
    n = 2 ** 32 + 4099
    x = torch.zeros(n, dtype=BF16, device=DEV)
    at = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, n - 1], device=DEV)
    x[at] = torch.tensor([1, 2, 3, 4, 5, 3], dtype=BF16, device=DEV)
    assert q.clip_grad_norm([x], 4.0).item() == 8.0
    assert x[at].tolist() == [0.5, 1.0, 1.5, 2.0, 2.5, 1.5] and int(x.count_nonzero()) == 6


def test_groups_are_clipped_each_by_its_own_norm():
    n = 16
    a, b = _grads([(n, 8, 320), (n, 264, 8)], [BF16], 2)
    size = torch.logspace(-3, 1, n).to(DEV)
    a, b = (a * size.view(n, 1, 1)).to(BF16), (b * size.view(n, 1, 1)).to(BF16)
    norms = _check([a, b], 2.0, n)
    assert (norms < 2).any() and (norms > 2).any()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_any_element_alignment(dtype):
    flat = torch.randn(30000, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    for a, b in ((1, 3), (3, 4), (0, 5), (5, 5), (7, 0)):
        x = flat[a:a + 9001]
        y = torch.empty(9100, dtype=dtype, device=DEV)[b:b + 9001]
        want_n, want = oad.clip([_f64(x)], 1.0)
        n = q.clip_grad_norm([x], 1.0, out=[y])
        np.testing.assert_allclose(_f64(n), want_n, rtol=2.0 ** -23)
        np.testing.assert_allclose(_f64(y), want[0], rtol=UNIT[dtype] + 3 * 2.0 ** -24, atol=SMALL[dtype])


def test_sizes_that_squares_in_32_bits_do_not_hold():
    big = torch.full((5000,), 3e38, dtype=FP32, device=DEV)
    assert torch.isinf(q.clip_grad_norm([big], 1.0)).all()     # above fp32 itself ...
    np.testing.assert_allclose(_f64(big), 5000 ** -0.5, rtol=1e-6)   # ... but clipped all the same
    x = torch.full((100,), 1e30, dtype=FP32, device=DEV)
    np.testing.assert_allclose(_f64(q.grad_norm([x])), float(x[0]) * 10, rtol=1e-6)
    x = torch.full((100,), 1e-30, dtype=FP32, device=DEV)
    np.testing.assert_allclose(_f64(q.grad_norm([x])), float(x[0]) * 10, rtol=1e-6)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_a_number_stays_in_its_group(bad):
    n = 4
    grads = _grads([(n, 300), (n, 5000)], [BF16, FP32], 5)
    ref = [t.clone() for t in grads]
    norms = q.clip_grad_norm(ref, 1.0, n)
    grads[1][2, 77] = bad
    got = q.clip_grad_norm(grads, 1.0, n)
    ok = torch.tensor([0, 1, 3], device=DEV)
    assert torch.equal(got[ok], norms[ok]) and not torch.isfinite(got[2])
    for a, b in zip(grads, ref):
        assert torch.equal(a[ok], b[ok])
    assert torch.isnan(grads[1][2, 77])
    if bad != bad:
        assert torch.isnan(grads[0][2]).all()
    else:
        assert not grads[0][2].any()


def test_empty_tensors_alone():
    e = torch.empty(0, 5, device=DEV)
    assert q.grad_norm([e, e]).tolist() == [0.0]
    assert q.clip_grad_norm([e], 1.0, groups=3).tolist() == [0.0] * 3


def test_nothing_outside_is_written():
    b = [Guarded(4 * 5001, 1), Guarded(2 * 4099, 2)]
    xs = [b[0].tensor((5001,), FP32), b[1].tensor((4099,), BF16)]
    for k, x in enumerate(xs):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)))
    ws = Guarded(1 << 12, 3)
    q.clip_grad_norm(xs, 0.1, workspace=ws.payload)
    assert all(g.intact() for g in b + [ws])


def test_captured_and_replayed():
    grads = _grads([(33, 77), (5000,), (3, 2)], [BF16, FP32], 7)
    outs = [torch.empty_like(t) for t in grads]
    ws = torch.empty(1 << 14, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q.clip_grad_norm(grads, 0.5, out=outs, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = q.clip_grad_norm(grads, 0.5, out=outs, workspace=ws)
    for k in range(3):
        for t in grads:
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(k)) * 10.0 ** -k)
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(t) for t in grads]
        assert torch.equal(norm, q.clip_grad_norm(grads, 0.5, out=want))
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_another_stream():
    grads = _grads([(700, 300)], [BF16], 7)
    want = [torch.empty_like(grads[0])]
    n = q.clip_grad_norm(grads, 0.5, out=want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [torch.empty_like(grads[0])]
        n2 = q.clip_grad_norm(grads, 0.5, out=got)
    s.synchronize()
    assert torch.equal(n, n2) and torch.equal(got[0], want[0])


def test_refusals():
    x, y = _grads([(6, 10), (6, 4)], [FP32], 1)
    for bad, err in (((["x"], 1.0), TypeError), (([x.double()], 1.0), TypeError), (([x.t()], 1.0), ValueError), (([x, y.cpu()], 1.0), ValueError),
                     (([], 1.0), ValueError), (([x], -1.0), ValueError), (([x], float("nan")), ValueError), (([x], 1.0, 4), ValueError),
                     (([x], 1.0, 0), ValueError), (([x], 1.0, 1, [x, y]), ValueError), (([x, y], 1.0, 1, [x, x]), ValueError),
                     (([x, x], 1.0), ValueError), (([x], 1.0, 1, [x.bfloat16()]), ValueError)):
        with pytest.raises(err):
            q.clip_grad_norm(*bad)
    with pytest.raises(ValueError):
        q.grad_norm([x], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
