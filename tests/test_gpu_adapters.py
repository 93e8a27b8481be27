"""The linear layer with many adapters on the GPU against the float64 oracle.

Bounds, elementwise.  Products of bf16 values are exact in fp32; a sum of n terms
of sizes t_i in fp32, in any order, is off by at most n 2^-24 sum t_i (2^-23
here, for the scale's and the constants' roundings).  T and G are rounded to
bf16 once, at most 2^-8 of their value, and so are the outputs.  Up to 64 tokens the weight
is bf16(level) times the block's constant, above it is their product rounded to
bf16; the oracle is given the one that applies, so no term for it is needed."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from oracle import adapters as oad
from oracle import bf16 as obf16
from oracle import nf4
from tests.gpu_util import DEV, Guarded, guarded_like

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
R = 2.0 ** -8      # a rounding to bf16
S = 2.0 ** -23     # a term of an fp32 sum


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _close(got, want, tol, name):
    got = _f64(got)
    bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (name, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


def _weights(w, small):
    """The weight that the kernels multiply, float64."""
    p, c8, c2, mean = (t.cpu().numpy() for t in (w.packed, w.code8, w.c2, w.mean))
    if not small:
        return _f64(w.dequantize())
    level = obf16.bf16_bits_to_fp64(obf16.round_fp32_to_bf16_bits(nf4.q4_levels(w.qtype)))
    codes = nf4.unpack_nibbles(p, w.rows * w.cols)
    chat = np.asarray(nf4.decode_constants(c8, c2, np.float32(mean[0])), np.float64)
    return (level[codes].reshape(-1, 64) * chat[:, None]).reshape(w.rows, w.cols)


def _case(M, N, K, n, r, seed, qtype="nf4"):
    g = torch.Generator().manual_seed(seed)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(BF16).to(DEV)

    w = q.NF4Weight.quantize((torch.randn(N, K, generator=g) * 0.02).to(DEV), qtype)
    scale = (torch.rand(n, generator=g) * 2 - 0.5).to(DEV)
    return dict(X=normal(M, K), w=w, A=normal(n, r, K, std=0.05), B=normal(n, N, r, std=0.05), scale=scale), normal(M, N)


def _index(kind, M, n, seed):
    g = np.random.default_rng(seed)
    if kind == "mixed":
        i = g.integers(-1, n + 1, M)                    # -1 and n: no adapter
    elif kind == "runs":
        i = np.sort(g.integers(0, n, M))[::-1].copy()
    elif kind == "one":
        i = np.full(M, n - 1)
    else:
        i = np.full(M, -100)
    return torch.from_numpy(i.astype(np.int64)).to(DEV)


def _sizes(c, dY, idx):
    """Sums of the sizes of the terms of each output."""
    X, A, B, s = (np.abs(_f64(c[k])) for k in ("X", "A", "B", "scale"))
    W, dY = np.abs(_weights(c["w"], False)), np.abs(_f64(dY))
    i = idx.cpu().numpy()
    return oad.forward(X, W, A, B, s, i), oad.backward(dY, X, W, A, B, s, i)


def _check(c, dY, idx, grown=0):
    """grown: the calls get that many adapters, of which the first and the last are c's two and the others zeros."""
    own, oidx = c, idx
    if grown:
        own = dict(c, scale=torch.ones(grown, device=DEV))
        for k in ("A", "B"):
            own[k] = torch.zeros(grown, *c[k].shape[1:], dtype=BF16, device=DEV)
        for k in ("A", "B", "scale"):
            own[k][0], own[k][-1] = c[k][0], c[k][1]
        oidx = torch.where(idx == 1, grown - 1, idx)
    M, K = c["X"].shape
    n, N, r = c["B"].shape
    small = M <= 64
    host = {k: _f64(c[k]) for k in ("X", "A", "B", "scale")}
    i = idx.cpu().numpy()
    (sY, sT), (sdX, sdA, sdB) = _sizes(c, dY, idx)
    Y, T = oad.forward(host["X"], _weights(c["w"], small), host["A"], host["B"], host["scale"], i)
    gY, gT = q.adapter_linear_fwd(index=oidx, **own)
    _close(gT, T, R * np.abs(T) + K * S * sT * (1 + R) + 1e-37, "T")
    # T's error goes through B: at most (R + K S) of sum |T| |B|, itself at most sY
    lora = oad.forward(np.abs(host["X"]), np.zeros((N, K)), np.abs(host["A"]), np.abs(host["B"]), np.abs(host["scale"]), i)[0]
    viaT = np.zeros((M, N))
    for m, a in enumerate(i):
        if 0 <= a < n:
            viaT[m] = np.abs(host["B"][a]) @ np.abs(T[m])
    eY = R * viaT + K * S * lora + (K + r) * S * sY
    _close(gY, Y, R * (np.abs(Y) + eY) + eY, "Y")
    if dY is None:
        return gY, gT
    dYh = _f64(dY)
    dX, dA, dB = oad.backward(dYh, host["X"], _weights(c["w"], False), host["A"], host["B"], host["scale"], i)
    gdX, gdA, gdB = q.adapter_linear_bwd(dY, own["X"], gT, own["w"], own["A"], own["B"], own["scale"], oidx)
    if grown:
        assert not gdA[1:-1].any() and not gdB[1:-1].any()
        gdA, gdB = gdA[::grown - 1], gdB[::grown - 1]
    G = np.zeros((M, r))
    for m, a in enumerate(i):
        if 0 <= a < n:
            G[m] = np.abs(host["scale"][a] * (dYh[m] @ host["B"][a]))
    viaG, eA, eB = np.zeros((M, K)), np.zeros(dA.shape), np.zeros(dB.shape)
    aT = np.abs(T)
    for m, a in enumerate(i):
        if 0 <= a < n:
            viaG[m] = G[m] @ np.abs(host["A"][a])
            eA[a] += np.outer(G[m], np.abs(host["X"][m]))
            eB[a] += np.outer(np.abs(dYh[m]), aT[m])
    e = R * viaG + (2 * N + r) * S * sdX
    _close(gdX, dX, R * (np.abs(dX) + e) + e, "dX")
    e = R * eA + (N + M) * S * sdA
    _close(gdA, dA, R * (np.abs(dA) + e) + e, "dA")
    e = R * eB + (K + M) * S * sdB
    _close(gdB, dB, R * (np.abs(dB) + e) + e, "dB")
    return gY, gT


SHAPES = [
    (1, 8, 64, 1, 8), (1, 520, 320, 3, 24), (5, 72, 1088, 7, 16), (17, 264, 128, 20, 8), (33, 48, 2048, 5, 40), (64, 136, 704, 64, 128),
    (65, 8, 64, 2, 8), (66, 264, 192, 1, 128), (130, 520, 320, 9, 24), (257, 72, 1088, 300, 16), (300, 320, 64, 3, 72),
    (513, 256, 256, 1023, 8), (100, 1160, 128, 3, 16), (70, 136, 2112, 2, 32),
]


@pytest.mark.parametrize("kind", ["mixed", "runs", "one", "none"])
@pytest.mark.parametrize("M,N,K,n,r", SHAPES)
def test_layer(M, N, K, n, r, kind):
    c, dY = _case(M, N, K, n, r, seed=M + N + K)
    _check(c, dY, _index(kind, M, n, seed=n + r))


@pytest.mark.parametrize("M,N,K,n,r", [(2304, 4096, 256, 2, 16), (2304, 256, 4096, 4, 24)])
def test_tiles_of_256(M, N, K, n, r):
    """Enough tiles for the large ones, forward or backward, and long runs of an adapter."""
    c, dY = _case(M, N, K, n, r, seed=9)
    _check(c, dY, _index("mixed", M, n, seed=2))


@pytest.mark.parametrize("M", [20, 70])
@pytest.mark.parametrize("N,K", [(72, 16448), (16456, 64)])
def test_adapters_past_32_bits(M, N, K):
    """1023 adapters of rank 128 whose A or B has more than 2^31 elements."""
    c, dY = _case(M, N, K, 2, 128, seed=3)
    _check(c, dY, _index("mixed", M, 2, seed=4) % 2, grown=1023)


@pytest.mark.parametrize("qtype", ["fp4", "int4"])
@pytest.mark.parametrize("M", [3, 70])
def test_other_level_tables(M, qtype):
    c, dY = _case(M, 72, 128, 4, 16, seed=M, qtype=qtype)
    _check(c, dY, _index("mixed", M, 4, seed=M))


@pytest.mark.parametrize("M", [4, 40, 100, 300])
def test_one_adapter_agrees_with_the_plain_layer(M):
    """All tokens on one adapter: the layer with a single pair, to within T's order of sums."""
    c, dY = _case(M, 264, 320, 2, 16, seed=M)
    idx = torch.ones(M, dtype=torch.int64, device=DEV)
    Y, T = q.adapter_linear_fwd(index=idx, **c)
    A, B, s = c["A"][1].contiguous(), c["B"][1].contiguous(), float(c["scale"][1])
    Y1, T1 = q.linear_fwd(c["X"], c["w"], A, B, s)
    np.testing.assert_allclose(_f64(T), _f64(T1), rtol=2 * R, atol=1e-4)
    np.testing.assert_allclose(_f64(Y), _f64(Y1), rtol=2 * R, atol=4 * R * float(Y1.abs().max()))


@pytest.mark.parametrize("M", [6, 40, 65, 300])
def test_nan_and_infinity_stay_with_their_adapter_and_token(M):
    n, N, K, r = 5, 136, 192, 16
    c, dY = _case(M, N, K, n, r, seed=M)
    idx = _index("mixed", M, n, seed=M + 1)
    idx[:2] = torch.tensor([0, 1])
    idx[M // 2] = -1
    ok = q.adapter_linear_fwd(index=idx, **c)
    okb = q.adapter_linear_bwd(dY, c["X"], ok[1], c["w"], c["A"], c["B"], c["scale"], idx)
    bad = dict(c)
    bad["A"], bad["B"], bad["X"] = c["A"].clone(), c["B"].clone(), c["X"].clone()
    bad["A"][0] = float("nan")
    bad["B"][0, :, 3] = float("inf")
    bad["X"][M // 2] = float("nan")              # a token on the bare base
    dYb = dY.clone()
    dYb[M // 2] = float("inf")
    Y, T = q.adapter_linear_fwd(index=idx, **bad)
    dX, dA, dB = q.adapter_linear_bwd(dYb, bad["X"], T, bad["w"], bad["A"], bad["B"], bad["scale"], idx)
    clean = idx != 0
    clean[M // 2] = False
    for got, want in ((Y, ok[0]), (T, ok[1]), (dX, okb[0])):
        assert torch.equal(got[clean], want[clean])
    assert torch.equal(dA[1:], okb[1][1:]) and torch.equal(dB[1:], okb[2][1:])
    assert torch.isnan(Y[0]).all() and torch.isnan(Y[M // 2]).all()


@pytest.mark.parametrize("M", [1, 30, 64, 65, 200])
def test_repeats_and_the_first_request_beside_others(M):
    """Two calls give the same bits, and so does the first token's request alone among bare tokens."""
    c, dY = _case(M, 72, 320, 6, 24, seed=M)
    idx = _index("mixed", M, 6, seed=3)
    Y, T = q.adapter_linear_fwd(index=idx, **c)
    again = q.adapter_linear_fwd(index=idx, **c)
    assert torch.equal(Y, again[0]) and torch.equal(T, again[1])
    other = idx.clone()
    other[1:] = -1
    Y1, T1 = q.adapter_linear_fwd(index=other, **c)
    assert torch.equal(T1[:1], T[:1]) and torch.equal(Y1[:1], Y[:1])


@pytest.mark.parametrize("M", [9, 64, 100, 257])
def test_nothing_outside_the_outputs_is_written(M):
    N, K, n, r = 72, 128, 3, 8
    c, dY = _case(M, N, K, n, r, seed=M)
    idx = _index("mixed", M, n, seed=1)
    L = q.lib()
    gs = [guarded_like(s, seed=k) for k, s in enumerate(((M, N), (M, r), (M, K), (n, r, K), (n, N, r)))]
    fb, bb = (L.qlora_adapter_linear_workspace_bytes(M, N, K, n, r, k) for k in (0, 1))
    wf, wb = Guarded(fb, 7), Guarded(bb, 8)
    Y, T = q.adapter_linear_fwd(index=idx, T_out=gs[1][1], out=gs[0][1], workspace=wf.payload, **c)
    q.adapter_linear_bwd(dY, c["X"], T, c["w"], c["A"], c["B"], c["scale"], idx, workspace=wb.payload, dX_out=gs[2][1],
                         dA_out=gs[3][1], dB_out=gs[4][1])
    assert all(g.intact() for g, _ in gs) and wf.intact() and wb.intact()
    for g, t in gs:
        assert torch.isfinite(t).all()


def test_subsets_of_the_gradients_and_a_recomputed_T():
    c, dY = _case(150, 72, 192, 4, 24, seed=2)
    idx = _index("mixed", 150, 4, seed=5)
    T = q.adapter_linear_fwd(index=idx, **c)[1]
    args = (c["w"], c["A"], c["B"], c["scale"], idx)
    want = q.adapter_linear_bwd(dY, c["X"], T, *args)
    for mask in range(1, 8):
        need = [bool(mask & b) for b in (1, 2, 4)]
        for t in (T, None):
            got = q.adapter_linear_bwd(dY, c["X"], t, *args, need_dX=need[0], need_dA=need[1], need_dB=need[2])
            for k in range(3):
                assert (got[k] is not None) == need[k]
                if need[k]:
                    assert torch.equal(got[k], want[k])


def test_no_tokens():
    c, dY = _case(0, 72, 192, 4, 24, seed=2)
    idx = torch.empty(0, dtype=torch.int64, device=DEV)
    Y, T = q.adapter_linear_fwd(index=idx, **c)
    assert Y.shape == (0, 72) and T.shape == (0, 24)
    dX, dA, dB = q.adapter_linear_bwd(dY, c["X"], T, c["w"], c["A"], c["B"], c["scale"], idx)
    assert dX.shape == (0, 192) and not dA.any() and not dB.any()


@pytest.mark.parametrize("M", [7, 90])
def test_module_gradients_against_differences(M):
    n, N, K, r = 3, 64, 128, 8
    c, dY = _case(M, N, K, n, r, seed=M)
    lin = q.AdapterLinear(c["w"], n, r, [8.0, 4.0, 2.0], c["A"].clone(), c["B"].clone())
    idx = _index("mixed", M, n, seed=4)
    x = c["X"].clone().requires_grad_()
    lin(x, idx).backward(dY)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(lin(x, idx).sum(), x, create_graph=True)[0].sum().backward()
    W, s, i = _weights(c["w"], False), _f64(lin.scale), idx.cpu().numpy()
    X, A, B, d = (_f64(t) for t in (x, lin.lora_A, lin.lora_B, dY))

    def f(X, A, B):
        return (oad.forward(X, W, A, B, s, i)[0] * d).sum()

    g = np.random.default_rng(0)
    for k, grad in enumerate((x.grad, lin.lora_A.grad, lin.lora_B.grad)):
        v = g.standard_normal(grad.shape)
        args = [X, A, B]
        h = 1e-4
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + h * v, args[k] - h * v
        want = (f(*up) - f(*down)) / (2 * h)
        got = (_f64(grad) * v).sum()
        # each gradient within 3 roundings of its terms, which add up like their root mean square
        assert abs(got - want) <= 6 * R * np.sqrt((_f64(grad) ** 2 * v ** 2).sum()) + 1e-6 * abs(want)


@pytest.mark.parametrize("M", [16, 200])
def test_captured_and_replayed(M):
    N, K, n, r = 72, 320, 6, 16
    c, dY = _case(M, N, K, n, r, seed=M)
    idx = _index("mixed", M, n, seed=4)
    outs = [torch.empty(s, dtype=BF16, device=DEV) for s in ((M, N), (M, r), (M, K), (n, r, K), (n, N, r))]
    L = q.lib()
    ws = [torch.empty(L.qlora_adapter_linear_workspace_bytes(M, N, K, n, r, k), dtype=torch.uint8, device=DEV) for k in (0, 1)]

    def step():
        q.adapter_linear_fwd(index=idx, out=outs[0], T_out=outs[1], workspace=ws[0], **c)
        q.adapter_linear_bwd(dY, c["X"], outs[1], c["w"], c["A"], c["B"], c["scale"], idx, workspace=ws[1], dX_out=outs[2],
                             dA_out=outs[3], dB_out=outs[4])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(9)
    for k in range(3):
        c["X"].copy_(torch.randn(M, K, generator=g))
        dY.copy_(torch.randn(M, N, generator=g))
        idx.copy_(_index("mixed" if k else "runs", M, n, seed=k))
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        Y, T = q.adapter_linear_fwd(index=idx, **c)
        want = (Y, T) + q.adapter_linear_bwd(dY, c["X"], T, c["w"], c["A"], c["B"], c["scale"], idx)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    c, dY = _case(70, 72, 192, 4, 24, seed=2)
    idx = _index("mixed", 70, 4, seed=5)

    def call(**k):
        return q.adapter_linear_fwd(**{**c, "index": idx, **k})

    for bad, err in (({"index": idx.int()}, TypeError), ({"index": idx[:-1]}, ValueError), ({"scale": c["scale"].double()}, TypeError),
                     ({"scale": c["scale"][:3]}, ValueError), ({"A": c["A"][0]}, ValueError), ({"A": c["A"][:3]}, ValueError),
                     ({"B": c["B"].float()}, TypeError), ({"B": c["B"].transpose(0, 1).contiguous()}, ValueError),
                     ({"X": c["X"][:, :128].contiguous()}, ValueError), ({"X": c["X"].cpu()}, ValueError),
                     ({"A": c["A"][:, :20].contiguous(), "B": c["B"][:, :, :20].contiguous()}, q.QLoRAError),
                     ({"workspace": torch.empty(64, dtype=torch.uint8, device=DEV)}, ValueError)):
        with pytest.raises(err):
            call(**bad)
    with pytest.raises(ValueError):
        q.adapter_linear_bwd(dY[:-1], c["X"], None, c["w"], c["A"], c["B"], c["scale"], idx)
