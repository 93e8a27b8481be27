"""Token log probabilities and top-logit distillation on the GPU against the
float64 oracle.

Bounds.  A row's sum of e_j = 2^((z_j - a) c) has at most about 80 fp32
additions on the way from an element to its slice's sum (72 in a thread, 8
in the trees), each 2^-24, and each e_j an error of 2^-22 + |t_j| 2^-23 with
the p-weighted |t_j| at most log2(V) <= 17: below 1e-5 relative in all.  So
log probabilities are held to 1e-5 plus their own rounding, entropies to 1e-5
(1 + H), and gradients to 3e-5 of their terms' sizes plus one rounding to the
logits' type."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from oracle import vocab
from tests.gpu_util import DEV, Guarded

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
SMALL = {BF16: 2.0 ** -126, FP16: 2.0 ** -25, FP32: 2.0 ** -126}   # below the normal range


def _host64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _rows(z, dtype, pitch, shift=0):
    """z (host) as a [M, V] view of a device buffer of that row pitch that
    starts `shift` elements in; the rest is NaN, so a read past a row shows."""
    M, V = z.shape
    buf = torch.full((M * pitch + shift + 8,), float("nan"), dtype=dtype, device=DEV)
    v = torch.as_strided(buf, (M, V), (pitch, 1), shift)
    v.copy_(torch.as_tensor(z).to(dtype))
    return v


def _logits(M, V, seed, masked=True):
    g = np.random.default_rng(seed)
    z = g.standard_normal((M, V)) * 2
    z[np.arange(M), g.integers(0, V, M)] += 9
    if masked and V > 3:
        z[:, 1::5] = -np.inf
        if M > 2:
            z[2] = -np.inf                       # nothing left
        if M > 4:
            z[4, :] = -np.inf
            z[4, V // 2] = 0.5                   # one word left
    return z


def _close(got, want, tol, name):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= tol)
    assert ok.all(), (name, np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5])


def _check_logprobs(z, target, top):
    r = q.token_logprobs(z, target, top)
    z64, t = _host64(z), target.cpu().numpy()
    lp, h, tl, ti = vocab.logprobs(z64, t, top)
    fin = np.nan_to_num(np.abs(lp), posinf=0, neginf=0)
    _close(_host64(r.logprob), lp, 1e-5 + 2.0 ** -23 * fin, "logprob")
    _close(_host64(r.entropy), h, 1e-5 * (1 + h), "entropy")
    if top:
        np.testing.assert_array_equal(r.top_index.cpu().numpy(), ti)
        _close(_host64(r.top_logprob), tl, 1e-5 + 2.0 ** -23 * np.nan_to_num(np.abs(tl), posinf=0, neginf=0), "top")
    return r


def _check_logprobs_grad(z, target, r, seed):
    M, V = z.shape
    g = np.random.default_rng(seed)
    gl, gh = g.standard_normal(M).astype(np.float32), g.standard_normal(M).astype(np.float32)
    d = q.token_logprobs_bwd(z, target, r.lse, r.entropy, torch.from_numpy(gl).to(DEV), torch.from_numpy(gh).to(DEV))
    z64, t = _host64(z), target.cpu().numpy()
    want = vocab.logprobs_grad(z64, t, gl, gh)
    lp = vocab.log_softmax(z64)
    p = np.exp(lp)
    h = -np.where(p > 0, p * np.where(p > 0, lp, 0), 0).sum(1, keepdims=True)
    size = p * (np.abs(gl[:, None]) + np.abs(gh[:, None]) * (np.where(p > 0, np.abs(lp), 0) + h))
    _close(_host64(d), want, 3e-5 * size + UNIT[z.dtype] * (np.abs(want) + 3e-5 * size) + SMALL[z.dtype], "dz")
    return d


def _teacher(z64, K, seed):
    g = np.random.default_rng(seed)
    M, V = z64.shape
    idx = np.stack([g.permutation(V)[:K] if V >= K else np.resize(g.permutation(V), K) for _ in range(M)]).astype(np.int64)
    val = g.standard_normal((M, K)).astype(np.float32) * 3
    if K > 2:
        idx[0, K // 2:] = -1                     # a short list
        idx[-1, 1] = idx[-1, 0]                  # a word listed twice
        val[0, 0] = -np.inf                      # listed, but impossible for the teacher
    if M > 3:
        idx[3] = V + 5                           # no entry at all
    return idx, val


def _check_distill(z, idx, val, temperature, seed):
    M, V = z.shape
    w = np.random.default_rng(seed).standard_normal(M).astype(np.float32)
    ti, tv, tw = (torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in (idx, val, w))
    z64 = _host64(z)
    want_l, want_d = vocab.distill(z64, idx, val, temperature, w)
    p = np.exp(vocab.log_softmax(z64 / temperature))
    size = (p + np.abs(vocab.distill(z64, idx, val, 1.0 * temperature, np.full(M, temperature))[1])) * np.abs(w[:, None]) / temperature
    tol = 3e-5 * size + UNIT[z.dtype] * (np.abs(want_d) + 3e-5 * size) + SMALL[z.dtype]
    loss, d = q.distill_topk(z, ti, tv, temperature, weight=tw)
    # sum q |log p| <= loss + entropy of q; log p within 1e-5 + 2^-23 |log p|
    ltol = 1e-5 + 2.0 ** -22 * (1 + np.nan_to_num(np.abs(want_l), posinf=0) + 10)
    _close(_host64(loss), want_l, ltol, "loss")
    _close(_host64(d), want_d, tol, "dz")
    loss2, lse = q.distill_topk_fwd(z, ti, tv, temperature)
    _close(_host64(loss2), want_l, ltol, "loss alone")
    d2 = q.distill_topk_bwd(z, ti, tv, temperature, lse, weight=tw)
    _close(_host64(d2), want_d, tol, "dz alone")
    return loss, d


SHAPES = [(1, 1, 1, 0), (3, 2, 2, 1), (5, 7, 9, 3), (5, 64, 64, 0), (6, 100, 101, 5), (5, 1000, 1000, 1), (5, 2047, 2050, 0),
          (7, 4099, 4099, 0), (5, 32000, 32000, 0), (5, 50001, 50048, 2), (2, 131072, 131072, 0), (1, 140001, 140003, 1),
          (1300, 1025, 1028, 0), (600, 16384, 16384, 0), (520, 16390, 16395, 0)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,V,pitch,shift", SHAPES)
def test_logprobs(dtype, M, V, pitch, shift):
    z = _rows(_logits(M, V, M + V), dtype, pitch, shift)
    g = np.random.default_rng(V)
    t = g.integers(0, V, M)
    t[M // 2] = -100 if M % 2 else V
    target = torch.from_numpy(t).to(DEV)
    r = None
    for top in sorted({0, 1, min(5, V), min(64, V)}):
        r = _check_logprobs(z, target, top)
    _check_logprobs_grad(z, target, r, 9)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,V,pitch,shift", SHAPES)
def test_distill(dtype, M, V, pitch, shift):
    z = _rows(_logits(M, V, 3 * M + V, masked=False), dtype, pitch, shift)
    z64 = _host64(z)
    for K, temperature in ((1, 1.0), (min(64, V), 2.0), (256, 0.7)):
        idx, val = _teacher(z64, K, K)
        _check_distill(z, idx, val, temperature, 4)


@pytest.mark.parametrize("dtype,M,V", [(FP32, 12, 37902), (BF16, 300, 50001), (BF16, 9, 70000), (FP16, 5, 131073)])
def test_alternatives_wherever_they_lie(dtype, M, V):
    """The best words in one slice, in few, at the end, at equal steps, or too few."""
    g = np.random.default_rng(V)
    z = g.standard_normal((M, V))
    ramp = np.linspace(-8.0, 8.0, V)
    z[0] = ramp
    z[1] = -ramp
    z[2, V // 2 : V // 2 + 64] += 20.0
    z[3, V - 70 :] += 20.0
    z[4] = -np.inf
    z[4, V - 30 :] = ramp[:30]                   # the others follow in the order of their indices
    if M > 8:
        z[5, :: V // 64] += 20.0
        z[6, :300] += 15.0
        z[6, V // 3 : V // 3 + 300] += 15.0
        z[7, g.permutation(V)[:40]] += 30.0
        z[8] = 1.0
    v = _rows(z, dtype, V + 3, 1)
    t = torch.from_numpy(g.integers(0, V, M)).to(DEV)
    for top in (1, 5, 64):
        _check_logprobs(v, t, top)


@pytest.mark.parametrize("M", [1, 40, 700])
def test_equal_words_and_flat_rows(M):
    """Few distinct logits: the lower index first, over slices and threads."""
    g = np.random.default_rng(M)
    z = g.integers(0, 3, (M, 20000)).astype(np.float64)
    z[0] = 0.0
    if M > 1:
        z[1] = np.where(np.arange(20000) % 2 == 0, 0.0, -0.0)
        z[2] = -np.inf
        z[2, 19990:] = 1.0
        z[3, :] = np.arange(20000) // 6000
        z[4, :] = -np.arange(20000) // 6000
    for dtype in (BF16, FP32):
        target = torch.zeros(M, dtype=torch.int64, device=DEV)
        _check_logprobs(_rows(z, dtype, 20000), target, 64)
        _check_logprobs(_rows(z, dtype, 20001), target, 3)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_rows_of_the_lowest_value(dtype):
    """Masks of the type's lowest value: over a whole row, the words are equally likely."""
    low = torch.finfo(dtype).min
    z = _logits(4, 3001, 5, masked=False)
    z[0] = low
    z[1, 7:] = low
    z[2] = np.where(np.arange(3001) < 10, low, -np.inf)
    zd = _rows(z, dtype, 3001)
    target = torch.tensor([5, 9, 4, 2], device=DEV)
    r = _check_logprobs(zd, target, 4)
    assert abs(r.logprob[0].item() + np.log(3001)) < 1e-5 and abs(r.entropy[2].item() - np.log(10)) < 1e-5
    _check_logprobs_grad(zd, target, r, 1)
    idx, val = _teacher(_host64(zd), 8, 3)
    _check_distill(zd, idx[:4] % 7, val, 1.0, 2)


def test_masked_students():
    """All words masked: no gradient, an infinite loss where the teacher has words."""
    z = _logits(6, 500, 8)
    zd = _rows(z, FP32, 500)
    idx, val = _teacher(z, 9, 2)
    _check_distill(zd, idx, val, 1.5, 3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_nan_and_infinity_stay_in_their_rows(dtype):
    z = _logits(5, 9000, 6, masked=False)
    z[1, 4000], z[3, 8999] = np.nan, np.inf
    zd = _rows(z, dtype, 9000)
    target = torch.arange(5, device=DEV)
    r = q.token_logprobs(zd, target, 8)
    for v in (r.logprob, r.entropy, r.top_logprob[:, 0]):
        assert torch.isnan(v).tolist() == [False, True, False, True, False]
    assert (r.top_index >= 0).all() and (r.top_index < 9000).all()
    one = torch.ones(5, device=DEV)
    d = q.token_logprobs_bwd(zd, target, r.lse, r.entropy, one, one)
    assert torch.isnan(d).any(1).tolist() == [False, True, False, True, False]
    keep = [0, 2, 4]
    rk = q.token_logprobs(zd[keep].contiguous(), target[keep], 8)
    assert torch.equal(rk.logprob, r.logprob[keep]) and torch.equal(rk.top_index, r.top_index[keep])
    idx = torch.arange(10, device=DEV).repeat(5, 1)
    loss, dd = q.distill_topk(zd, idx, torch.zeros(5, 10, device=DEV))
    assert torch.isnan(loss).tolist() == [False, True, False, True, False]
    assert torch.isnan(dd).any(1).tolist() == [False, True, False, True, False]


@pytest.mark.parametrize("dtype,V,pitch", [(BF16, 40000, 40000), (FP32, 1001, 1003), (FP16, 70001, 70001)])
def test_gradients_in_place_and_guarded(dtype, V, pitch):
    M = 9
    z = _rows(_logits(M, V, 2), dtype, pitch)
    target = torch.arange(M, device=DEV) * 3
    r = q.token_logprobs(z, target)
    g = torch.linspace(-1, 1, M, device=DEV)
    want = q.token_logprobs_bwd(z, target, r.lse, r.entropy, g, g)
    gb = Guarded(M * V * z.element_size())
    out = gb.tensor((M, V), dtype)
    assert torch.equal(q.token_logprobs_bwd(z, target, r.lse, r.entropy, g, g, out=out), want) and gb.intact()
    idx = torch.stack([torch.randperm(V)[:20] for _ in range(M)]).to(DEV)
    val = torch.randn(M, 20, device=DEV)
    loss, dd = q.distill_topk(z, idx, val, 1.0, weight=g)
    gb2 = Guarded(M * V * z.element_size())
    out = gb2.tensor((M, V), dtype)
    loss2, _ = q.distill_topk(z, idx, val, 1.0, weight=g, out=out)
    assert torch.equal(out, dd) and torch.equal(loss, loss2) and gb2.intact()
    z2, z3 = (torch.as_strided(z._base.clone() if z._base is not None else z.clone(), z.shape, z.stride(), z.storage_offset())
              for _ in range(2))
    q.token_logprobs_bwd(z2, target, r.lse, r.entropy, g, g, out=z2)
    assert torch.equal(z2, want)
    loss3, _ = q.distill_topk(z3, idx, val, 1.0, weight=g, out=z3)
    assert torch.equal(z3, dd) and torch.equal(loss3, loss)


def test_autograd_and_streams():
    M, V = 12, 3000
    z = _rows(_logits(M, V, 1, masked=False), FP32, V).clone().requires_grad_()
    target = torch.arange(M, device=DEV)
    lp, h = q.TokenLogprobsFn.apply(z, target)
    (lp.sum() + 0.3 * h.sum()).backward()
    z64 = z.detach().double().cpu().requires_grad_()
    l64 = torch.log_softmax(z64, 1)
    (l64[torch.arange(M), torch.arange(M)].sum() - 0.3 * (l64.exp() * l64).sum()).backward()
    _close(_host64(z.grad), z64.grad.numpy(), 3e-5, "autograd")
    zb = z.detach().clone().requires_grad_()
    idx = torch.stack([torch.randperm(V)[:30] for _ in range(M)]).to(DEV)
    val = torch.randn(M, 30, device=DEV)
    q.DistillTopKFn.apply(zb, idx, val, 2.0).mean().backward()
    want = vocab.distill(_host64(zb), idx.cpu().numpy(), _host64(val), 2.0, np.full(M, 1 / M))[1]
    _close(_host64(zb.grad), want, 1e-5, "distill autograd")
    base = q.token_logprobs(z.detach(), target, 10)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = q.token_logprobs(z.detach(), target, 10)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(base, other))


def test_same_bits_twice_and_in_graph_replays():
    M, V = 33, 40000
    z = _rows(_logits(M, V, 4), BF16, V)
    target = torch.arange(M, device=DEV)
    idx = torch.stack([torch.randperm(V)[:64] for _ in range(M)]).to(DEV)
    val = torch.randn(M, 64, device=DEV)

    def both():
        return (*q.token_logprobs(z, target, 20), *q.distill_topk(z, idx, val, 2.0))

    a, b = both(), both()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for k in range(3):
        z.copy_(z.roll(1, 1))
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(held, want)), k


def test_no_rows():
    z = torch.empty(0, 50, dtype=BF16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    r = q.token_logprobs(z, none, 3)
    assert r.logprob.shape == (0,) and r.top_index.shape == (0, 3)
    assert q.token_logprobs_bwd(z, none, r.lse, r.entropy).shape == (0, 50)
    loss, d = q.distill_topk(z, torch.empty(0, 4, dtype=torch.int64, device=DEV), torch.empty(0, 4, device=DEV))
    assert loss.shape == (0,) and d.shape == (0, 50)


def test_refusals():
    z = torch.zeros(4, 50, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    idx, val = torch.zeros(4, 3, dtype=torch.int64, device=DEV), torch.zeros(4, 3, device=DEV)
    for bad in (z.double(), z.cpu(), z[0]):
        with pytest.raises((TypeError, ValueError)):
            q.token_logprobs(bad, t)
    with pytest.raises(ValueError):
        q.token_logprobs(z.t(), torch.zeros(50, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        q.token_logprobs(z[:1].expand(4, 50), t)                  # overlapping rows
    with pytest.raises(TypeError):
        q.token_logprobs(z, t.int())
    with pytest.raises(ValueError):
        q.token_logprobs(z, t[:3])
    for top in (51, 65, -1):
        with pytest.raises(ValueError):
            q.token_logprobs(z, t, top)
    with pytest.raises(ValueError):
        q.token_logprobs(torch.zeros(4, 200000, device=DEV), t, workspace=torch.empty(4, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        q.token_logprobs_bwd(z, t, torch.zeros(4, device=DEV), torch.zeros(4, device=DEV))
    with pytest.raises(ValueError):
        q.distill_topk(z, torch.zeros(4, 257, dtype=torch.int64, device=DEV), torch.zeros(4, 257, device=DEV))
    for temperature in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        with pytest.raises(q.QLoRAError):
            q.distill_topk(z, idx, val, temperature)
    with pytest.raises(ValueError):
        q.distill_topk(z, idx, val[:, :2])
    with pytest.raises(ValueError):
        q.distill_topk(z, idx, val, out=torch.empty(4, 49, device=DEV))
