"""Measured cases of the microscaled 4-bit (MX4) linear layer and of the
losses over the vocabulary.

Four operators that meet at the output head of a model tuned through LoRA
pairs:

  codec     an array to MX4 and back: blocks of 32 along a row share a
            power-of-two scale 2^s (s in [-127, 125], held as the byte
            s + 127), elements are E2M1 floats (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
            their negatives).  s = floor(log2(max |x|)) - 2; elements are
            x / 2^s rounded to nearest, ties to the even code, clipped to 6.
  linear    Y = Q(X) deq(W)^T + T B^T with T = scale X A^T, W held in MX4 and
            X rounded to MX4 on the way in; the training step adds
            dX = dY deq(W) + G A, dA = G^T X, dB = dY^T T with G = scale dY B
            (the rounding of X passes gradients straight through).
  logprobs  of given tokens under softmax(logits), with the entropy and the
            most likely alternatives, and the gradient of the first two.
  distill   KL(teacher || student) at a temperature, the teacher known by its
            top logits alone, with the gradient of the student's logits.

`run` computes them in elementary torch operations in 32 bits, or (`own`)
through bit_nf4_quantized_absmax_amd.
"""

import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORED = -100   # a target position without a token (padding, prompt)


# ---- cases ----------------------------------------------------------------------

def listed():
    return [
        # activations of a decoding batch on their way into a 4-bit product
        {"name": "codec 16 x 4096 bf16", "op": "codec", "rows": 16, "cols": 4096, "dtype": "bf16"},
        # the largest projection of a LLaMA-65B-shaped layer, loaded into 4 bits
        {"name": "codec 22016 x 8192 fp32", "op": "codec", "rows": 22016, "cols": 8192, "dtype": "fp32"},
        # one token through the 7B-shaped gate projection: the weight's bytes count
        {"name": "linear 1 x 11008 x 4096 r64", "op": "linear", "M": 1, "N": 11008, "K": 4096, "r": 64, "train": False},
        # a batch of 64 tokens through the 7B-shaped down projection
        {"name": "linear 64 x 4096 x 11008 r64", "op": "linear", "M": 64, "N": 4096, "K": 11008, "r": 64, "train": False},
        # odd token and feature counts, a row that ends inside a 256-wide slab, no adapter
        {"name": "linear 777 x 5003 x 1056", "op": "linear", "M": 777, "N": 5003, "K": 1056, "r": 0, "train": False},
        # 16 x 512 tokens through the 7B-shaped up projection
        {"name": "linear 8192 x 11008 x 4096 r64", "op": "linear", "M": 8192, "N": 11008, "K": 4096, "r": 64, "train": False},
        # the training step (forward and backward) of a 7B-shaped attention projection
        {"name": "linear step 8192 x 4096 x 4096 r64", "op": "linear", "M": 8192, "N": 4096, "K": 4096, "r": 64, "train": True},
        # one decoded token with 20 alternatives
        {"name": "logprobs 1 x 32000 top 20", "op": "logprobs", "M": 1, "V": 32000, "ld": 32000, "dtype": "bf16", "top": 20, "grad": False},
        # scoring with masked words, padded rows, many alternatives, an odd vocabulary
        {"name": "logprobs 300 x 50001 fp32 top 64", "op": "logprobs", "M": 300, "V": 50001, "ld": 50048, "dtype": "fp32", "top": 64, "grad": False},
        # a policy-gradient step with an entropy term over a large vocabulary
        {"name": "logprobs step 4096 x 131072", "op": "logprobs", "M": 4096, "V": 131072, "ld": 131072, "dtype": "bf16", "top": 0, "grad": True},
        # a short sequence against 16 teacher logits a token
        {"name": "distill 128 x 32000 fp16 top 16", "op": "distill", "M": 128, "V": 32000, "ld": 32000, "dtype": "fp16", "K": 16, "temperature": 1.0},
        # 16 x 512 tokens against 64 teacher logits a token
        {"name": "distill 8192 x 32000 bf16 top 64", "op": "distill", "M": 8192, "V": 32000, "ld": 32000, "dtype": "bf16", "K": 64, "temperature": 2.0},
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("codec", "linear", "linear", "logprobs", "distill"))
    if op == "codec":
        cols = 32 * spread(4, 688)
        return {"op": op, "rows": spread(1, min(60000, 22016 * 8192 // cols)), "cols": cols,
                "dtype": rng.choice(("bf16", "fp16", "fp32"))}
    if op == "linear":
        train = rng.random() < 0.3
        if train:   # the backward pass wants N, K in multiples of 64
            N, K = 64 * spread(4, 64), 64 * spread(4, 64)
            return {"op": op, "M": spread(65, 8192), "N": N, "K": K, "r": rng.choice((8, 16, 64)), "train": True}
        M = rng.choice((spread(1, 16), spread(17, 128), spread(129, 8192)))
        K = 32 * spread(8, 344)
        N = min(spread(256, 22016), 11008 * 4096 // K)
        r = rng.choice((0, 8, 64))
        return {"op": op, "M": M, "N": N - N % 8 if r else N, "K": K, "r": r, "train": False}
    V = spread(1000, 131072)
    M = min(spread(1, 8192), 4096 * 131072 // V)
    ld = V + rng.choice((0, 0, 7, -V % 64))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "logprobs":
        return {"op": op, "M": min(M, max(1, 4096 * 65536 // V)) if dtype == "fp32" else M, "V": V, "ld": ld, "dtype": dtype,
                "top": rng.choice((0, 1, 5, 20, 64)), "grad": rng.random() < 0.5}
    M = min(M, 8192 * 32000 // V if dtype != "fp32" else 8192 * 16000 // V)
    return {"op": op, "M": max(1, M), "V": V, "ld": ld, "dtype": dtype, "K": spread(1, 128),
            "temperature": rng.choice((0.5, 1.0, 2.0, 4.0))}


def work(case):
    if case["op"] == "codec":
        n = case["rows"] * case["cols"]
        held = n * (0.5 + 1 / 32)          # codes and scales, written once and read once
        return {"bytes": n * (DTYPES[case["dtype"]].itemsize + 2) + 2 * held, "flops": 2 * n}
    if case["op"] == "linear":
        M, N, K, r = case["M"], case["N"], case["K"], case["r"]
        b = 2 * M * K + N * K * (0.5 + 1 / 32) + 2 * r * (N + K) + 2 * M * N + 2 * M * r
        f = 2 * M * N * K + 2 * M * r * (N + K)
        if case["train"]:
            b += 2 * M * N + 2 * M * K + 2 * r * (N + K)
            f += 2 * M * N * K + 4 * M * r * (N + K)
        return {"bytes": b, "flops": f}
    M, V, e = case["M"], case["V"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "logprobs":
        return {"bytes": M * V * e * (3 if case["grad"] else 1) + M * (8 + 12 + 12 * case["top"] + (8 if case["grad"] else 0)),
                "flops": M * V * (12 if case["grad"] else 6)}
    return {"bytes": 2 * M * V * e + M * (8 + 12 * case["K"]), "flops": 8 * M * V}


# ---- inputs ---------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "codec":
        x = _randn(g, case["rows"], case["cols"], std=0.02 if case["dtype"] == "fp32" else 1.0)
        if case["dtype"] != "fp32":        # activations have a few large channels
            x[:, :: 97] *= 30.0
        st["x"] = x.to(DTYPES[case["dtype"]])
        return st
    if case["op"] == "linear":
        M, N, K, r = case["M"], case["N"], case["K"], case["r"]
        st["x"] = _randn(g, M, K).to(torch.bfloat16)
        st["codes"], st["scales"] = _lay_out(*_quantize(_randn(g, N, K, std=0.02)))
        st["scale"] = 0.25
        if r:
            st["A"] = _randn(g, r, K, std=0.01).to(torch.bfloat16)
            st["B"] = _randn(g, N, r, std=0.01).to(torch.bfloat16)
        if case["train"]:
            st["dy"] = _randn(g, M, N).to(torch.bfloat16)
        return st
    M, V, ld, dtype = case["M"], case["V"], case["ld"], DTYPES[case["dtype"]]
    # a language model's logits: a broad bulk and some dozens of likely words
    z = torch.empty(M, ld, dtype=dtype, device=DEV)
    z.copy_(_randn(g, M, ld, std=2.0))
    z = z[:, :V]
    band = V // 24                      # one likely word in each of 24 bands: no word twice
    likely = (torch.rand(M, 24, generator=g, device=DEV) * band).long().clamp_(max=band - 1)
    likely += band * torch.arange(24, device=DEV)
    z.scatter_(1, likely, _randn(g, M, 24, std=3.0).add_(8.0).to(dtype))
    st["z"] = z
    if case["op"] == "logprobs":
        t = torch.randint(V, (M,), generator=g, device=DEV)
        if M > 1:
            t = torch.where(torch.rand(M, generator=g, device=DEV) < 0.5, likely[:, 0], t)
            if case["dtype"] == "fp32":    # constrained decoding: words that are not allowed
                z[:, 5 :: 7] = -math.inf
            if M > 64:
                t[:: 13] = IGNORED
        st["t"] = t
        if case["grad"]:
            st["g_logprob"] = _randn(g, M, std=1.0 / M)
            st["g_entropy"] = _randn(g, M, std=0.01 / M)
        return st
    K = case["K"]
    idx = torch.cat((likely, torch.randint(V, (M, max(0, 2 * K)), generator=g, device=DEV)), 1)
    # every index once in a row, as a teacher's top list has it
    idx, _ = idx.sort(1)
    first = torch.ones_like(idx, dtype=torch.bool)
    first[:, 1:] = idx[:, 1:] != idx[:, :-1]
    score = z.gather(1, idx).float() + _randn(g, M, idx.shape[1])
    score, at = score.masked_fill(~first, -math.inf).sort(1, descending=True)
    idx = idx.gather(1, at)[:, :K].contiguous()
    score = score[:, :K].contiguous()
    idx = torch.where(score > -math.inf, idx, torch.full_like(idx, -1))   # short lists are filled up with -1
    st["idx"], st["val"] = idx, score
    st["weight"] = torch.full((M,), 1.0 / M, device=DEV)
    if M > 64:
        st["weight"][:: 17] = 0.0          # padding
    return st


# ---- the plain forms --------------------------------------------------------------

def _quantize(x):
    """Element values (signed E2M1, fp32) [rows, nb, 32] and scale exponents [rows, nb] of x [rows, cols], cols % 32 == 0."""
    b = x.float().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(top)
    s = torch.where((top == 0) | bad, torch.full_like(top, -127.0), torch.frexp(top)[1].float() - 3.0).clamp(min=-127.0)
    a = b * torch.exp2(-s).unsqueeze(2)
    m = a.abs()
    step = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0))
    v = (torch.round(m / step) * step).clamp(max=6.0)
    v = torch.where(bad.unsqueeze(2), torch.zeros_like(v), v)
    return torch.copysign(v, a), torch.where(bad, torch.full_like(s, 128.0), s)


def _values(v, s):
    """What the held values stand for: v 2^s; a scale of 2^128 (the byte 255) marks a block with a NaN or an infinity."""
    f = torch.where(s > 127.0, torch.full_like(s, math.nan), torch.exp2(s))
    return (v * f.unsqueeze(2)).reshape(v.shape[0], -1)


def _lay_out(v, s):
    """Codes [rows, Kp / 2] (element 2 j in the low half of byte j) and scales
    [Kp / 256, rows, 8], both with the row filled up to Kp, a multiple of 256,
    with zeros."""
    rows, nb = s.shape
    m = v.abs()
    code = sum((m >= e).to(torch.uint8) for e in (0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0))
    code = code + 8 * torch.signbit(v).to(torch.uint8)
    fill = -nb % 8
    code = torch.nn.functional.pad(code, (0, 0, 0, fill)).reshape(rows, -1, 2)
    byte = torch.nn.functional.pad((s + 127.0).to(torch.uint8), (0, fill))
    return code[:, :, 0] + 16 * code[:, :, 1], byte.reshape(rows, -1, 8).permute(1, 0, 2).contiguous()


def _held(codes, scales, cols):
    """The fp32 values [rows, cols] of codes and scales as _lay_out gives them."""
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    rows = codes.shape[0]
    v = level[torch.stack((codes & 15, codes >> 4), 2).reshape(rows, -1)[:, :cols].long()].reshape(rows, -1, 32)
    s = scales.permute(1, 0, 2).reshape(rows, -1)[:, : cols // 32].float() - 127.0
    return _values(v, s)


def _plain_linear(st):
    c = st["case"]
    x, w = st["x"].float(), _held(st["codes"], st["scales"], c["K"])
    y = _values(*_quantize(st["x"])) @ w.t()
    if not c["r"]:
        return {"Y": y.to(torch.bfloat16)}
    A, B = st["A"].float(), st["B"].float()
    T = st["scale"] * (x @ A.t())
    out = {"Y": (y + T @ B.t()).to(torch.bfloat16), "T": T.to(torch.bfloat16)}
    if c["train"]:
        dy = st["dy"].float()
        G = st["scale"] * (dy @ B)
        out.update(dX=(dy @ w + G @ A).to(torch.bfloat16), dA=(G.t() @ x).to(torch.bfloat16), dB=(dy.t() @ T).to(torch.bfloat16))
    return out


def _log_softmax(z):
    """(log p, p, log of the sum of exponentials); a row that is all -inf has p = 0 and log p = -inf."""
    top = z.amax(1, keepdim=True)
    lse = torch.where(top == -math.inf, top, top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))
    logp = torch.where(lse == -math.inf, lse, z - lse)
    return logp, torch.exp(logp), lse


def _plain_logprobs(st):
    c, z, t = st["case"], st["z"].float(), st["t"]
    logp, p, lse = _log_softmax(z)
    real = (t >= 0) & (t < c["V"])
    at = torch.where(real, t, torch.zeros_like(t)).unsqueeze(1)
    picked = torch.where(real, logp.gather(1, at).squeeze(1), torch.zeros_like(logp[:, 0]))
    h = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    out = {"logprob": picked, "entropy": h}
    if c["top"]:
        order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, : c["top"]]
        out.update(top_logprob=logp.gather(1, order), top_index=order)
    if c["grad"]:
        alive = lse.squeeze(1) > -math.inf   # a row that is all -inf has no gradient
        gl = torch.where(real & alive, st["g_logprob"], torch.zeros_like(h)).unsqueeze(1)
        gh = st["g_entropy"].unsqueeze(1)
        d = torch.where(p > 0, -p * (gl + gh * (logp + h.unsqueeze(1))), torch.zeros_like(p))
        d.scatter_add_(1, at, gl)
        out["dlogits"] = d.to(st["z"].dtype)
    return out


def _plain_distill(st):
    c, z = st["case"], st["z"].float() / st["case"]["temperature"]
    logp, p, lse = _log_softmax(z)
    real = (st["idx"] >= 0) & (st["idx"] < c["V"])
    at = torch.where(real, st["idx"], torch.zeros_like(st["idx"]))
    logq, q, _ = _log_softmax(torch.where(real, st["val"].float() / c["temperature"], torch.full_like(st["val"], -math.inf)))
    loss = torch.where(q > 0, q * (logq - logp.gather(1, at)), torch.zeros_like(q)).sum(1)
    d = p * (q.sum(1, keepdim=True) > 0)
    d.scatter_add_(1, at, -q)
    d *= torch.where(lse > -math.inf, (st["weight"] / c["temperature"]).unsqueeze(1), torch.zeros_like(lse))
    return {"loss": loss, "dlogits": d.to(st["z"].dtype)}


# ---- one pass -----------------------------------------------------------------------

def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "codec":
            return _values(*_quantize(st["x"])).to(torch.bfloat16)
        return {"linear": _plain_linear, "logprobs": _plain_logprobs, "distill": _plain_distill}[c["op"]](st)
    import bit_nf4_quantized_absmax_amd as q
    if c["op"] == "codec":
        return q.MX4Tensor.quantize(st["x"]).dequantize()
    if c["op"] == "linear":
        w = q.MX4Tensor(st["codes"], st["scales"], c["N"], c["K"])
        if not c["r"]:
            return {"Y": q.mx4_linear_fwd(st["x"], w)[0]}
        Y, T = q.mx4_linear_fwd(st["x"], w, st["A"], st["B"], st["scale"])
        out = {"Y": Y, "T": T}
        if c["train"]:
            out["dX"], out["dA"], out["dB"] = q.mx4_linear_bwd(st["dy"], st["x"], T, w, st["A"], st["B"], st["scale"])
        return out
    if c["op"] == "logprobs":
        r = q.token_logprobs(st["z"], st["t"], top=c["top"])
        out = {"logprob": r.logprob, "entropy": r.entropy}
        if c["top"]:
            out.update(top_logprob=r.top_logprob, top_index=r.top_index)
        if c["grad"]:
            out["dlogits"] = q.token_logprobs_bwd(st["z"], st["t"], r.lse, r.entropy, st["g_logprob"], st["g_entropy"])
        return out
    loss, d = q.distill_topk(st["z"], st["idx"], st["val"], c["temperature"], weight=st["weight"])
    return {"loss": loss, "dlogits": d}


# ---- the definitions in 64 bits -------------------------------------------------------

def _mx4_64(x):
    """The nearest-level definition, by distance to every level (float64)."""
    x = x.double()
    out = torch.empty_like(x)
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    edge = (level[1:] + level[:-1]) / 2
    for r0 in range(0, x.shape[0], 4096):
        b = x[r0 : r0 + 4096].reshape(-1, 32)
        big = b.abs().max(1, keepdim=True)[0]
        e = torch.floor(torch.log2(torch.where(big > 0, big, torch.ones_like(big))))
        e = torch.where(torch.exp2(e) > big, e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= big, e + 1, e)
        f = torch.exp2((e - 2).clamp(min=-127))
        m = (b / f).abs()
        k = torch.bucketize(m, edge)                      # lower code on a tie ...
        tie = (k < 7) & (m == edge[k.clamp(max=6)]) & (k % 2 == 1)
        k = k + tie.long()                                # ... unless the upper one is even
        out[r0 : r0 + 4096] = (torch.sign(b) * level[k] * f).reshape(-1, x.shape[1])
    return out


def _weight_64(codes, scales, cols):
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.long, device=codes.device)
    c[:, 0::2], c[:, 1::2] = lo, hi
    mag, sign = c & 7, 1.0 - 2.0 * (c >> 3).double()
    val = torch.where(mag < 2, mag.double() / 2, (2 + (mag & 1)).double() * torch.exp2((mag >> 1).double() - 2))
    byte = torch.cat(list(scales), 1).double()
    return (sign * val * torch.exp2(byte - 127).repeat_interleave(32, 1))[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "codec":
        return _mx4_64(st["x"])
    if case["op"] == "linear":
        x, w = st["x"].double(), _weight_64(st["codes"], st["scales"], case["K"])
        Y = _mx4_64(st["x"]) @ w.t()
        if not case["r"]:
            return {"Y": Y}
        A, B, s = st["A"].double(), st["B"].double(), st["scale"]
        T = s * x @ A.t()
        out = {"Y": Y + T @ B.t(), "T": T}
        if case["train"]:
            dy = st["dy"].double()
            out.update(dX=dy @ w + s * (dy @ B) @ A, dA=s * (dy @ B).t() @ x, dB=dy.t() @ T)
        return out
    z = st["z"].double()
    if case["op"] == "logprobs":
        lse = torch.logsumexp(z, 1)
        t = st["t"]
        on = (t >= 0).double()
        tt = t.clamp(min=0).unsqueeze(1)
        p = torch.exp(z - lse.unsqueeze(1))
        h = lse - (p * torch.where(p > 0, z, torch.zeros_like(z))).sum(1)
        out = {"logprob": (z.gather(1, tt).squeeze(1) - lse) * on, "entropy": h}
        if case["top"]:
            out["top_logprob"] = torch.topk(z, case["top"], dim=1)[0] - lse.unsqueeze(1)
            out["top_index"] = None
        if case["grad"]:
            gl, gh = (st["g_logprob"].double() * on), st["g_entropy"].double()
            # d logprob / dz = e_t - p,  d entropy / dz_j = -p_j (log p_j + H)
            d = -p * (gl + gh * (h - lse)).unsqueeze(1)
            d -= torch.where(p > 0, p * z, torch.zeros_like(z)) * gh.unsqueeze(1)
            d[torch.arange(t.numel(), device=DEV), tt.squeeze(1)] += gl
            out["dlogits"] = d
        return out
    tau = case["temperature"]
    z = z / tau
    lse = torch.logsumexp(z, 1, keepdim=True)
    idx, val = st["idx"], st["val"].double() / tau
    on = (idx >= 0).double()
    val = torch.where(idx >= 0, val, torch.full_like(val, -math.inf))
    q = torch.softmax(val, 1) * on
    logq = val - torch.logsumexp(val, 1, keepdim=True)
    diff = torch.where(q > 0, logq - (z.gather(1, idx.clamp(min=0)) - lse), torch.zeros_like(q))
    d = torch.exp(z - lse)
    rows = torch.arange(z.shape[0], device=DEV).unsqueeze(1).expand_as(idx)
    d.index_put_((rows.reshape(-1), idx.clamp(min=0).reshape(-1)), -q.reshape(-1), accumulate=True)
    return {"loss": (q * diff).sum(1), "dlogits": d * (st["weight"].double() / tau).unsqueeze(1)}
