"""Measured cases of the operators that tune and serve many LoRA adapters over
one frozen base.

  adapters  Y_m = X_m deq(W)^T + T_m B_a^T, T_m = s_a X_m A_a^T, where a =
            index[m] names the adapter of token m's request among the n that
            are held, A [n, r, K], B [n, N, r], s [n]; an index outside [0, n)
            has none.  W [N, K] is in NF4.  The training step adds, with
            G_m = s_a dY_m B_a,  dX_m = dY_m deq(W) + G_m A_a,
            dA_a = sum of G_m^T X_m and dB_a = sum of dY_m^T T_m over the
            tokens m of adapter a.
  head      softmax cross entropy through a frozen output head without the
            logits: z = X W^T, loss_m = log sum_j e^z_mj - z_m,target; a target
            outside [0, V) (prompt, padding) has loss and gradient 0.  The
            training step adds dX = dz W, dz = weight (softmax(z) - [target]),
            and where the head is tuned as well dW = dz^T X.
  clip      the global norm of a model's gradients and the gradients times
            min(1, max_norm / (norm + 1e-6)); with groups > 1 every tensor holds
            that many adapters along its first axis, each with a norm of its own.

`run` computes them in elementary torch operations in 32 bits, or (`own`)
through bit_nf4_quantized_absmax_amd.
"""

import math
from statistics import NormalDist

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORED = -100


# ---- cases ----------------------------------------------------------------------

def listed():
    return [
        # one token of one request through the 7B-shaped attention projection, 64 adapters held
        {"name": "adapters 1 x 4096 x 4096 r64", "op": "adapters", "M": 1, "N": 4096, "K": 4096, "r": 64, "n": 64, "used": 1,
         "bare": False, "train": False},
        # a decoding batch, every token of another tenant, 7B-shaped gate projection
        {"name": "adapters 64 x 11008 x 4096 r16 of 64", "op": "adapters", "M": 64, "N": 11008, "K": 4096, "r": 16, "n": 64,
         "used": 64, "bare": False, "train": False},
        # some short prompts at once, odd sizes, one request on the bare model
        {"name": "adapters 777 x 5000 x 1088 r8 of 21", "op": "adapters", "M": 777, "N": 5000, "K": 1088, "r": 8, "n": 33,
         "used": 21, "bare": True, "train": False},
        # prompts of eight tenants, 16 x 512 tokens, 7B-shaped down projection
        {"name": "adapters 8192 x 4096 x 11008 r64 of 8", "op": "adapters", "M": 8192, "N": 4096, "K": 11008, "r": 64, "n": 16,
         "used": 8, "bare": False, "train": False},
        # the training step of 32 small adapters that share a batch and an attention projection
        {"name": "adapters step 8192 x 4096 x 4096 r16", "op": "adapters", "M": 8192, "N": 4096, "K": 4096, "r": 16, "n": 32,
         "used": 32, "bare": False, "train": True},
        # the loss of one position (scoring an answer token by token)
        {"name": "head 1 x 32000 x 4096", "op": "head", "M": 1, "V": 32000, "K": 4096, "prompt": 0, "train": "no"},
        # a short training batch, an odd vocabulary
        {"name": "head step 300 x 50001 x 1088", "op": "head", "M": 300, "V": 50001, "K": 1088, "prompt": 1, "train": "X"},
        # 16 x 512 tokens into the head of a 7B-shaped model, a quarter of each sequence its prompt
        {"name": "head step 8192 x 32000 x 4096", "op": "head", "M": 8192, "V": 32000, "K": 4096, "prompt": 1, "train": "X"},
        # a large vocabulary whose head is tuned as well
        {"name": "head step 2048 x 131072 x 4096 and W", "op": "head", "M": 2048, "V": 131072, "K": 4096, "prompt": 0, "train": "XW"},
        # one layer's seven LoRA pairs
        {"name": "clip 1 layer r8 bf16", "op": "clip", "layers": 1, "hidden": 4096, "inner": 11008, "r": 8, "dtype": "bf16",
         "groups": 1, "extra": 0},
        # every pair of a 7B-shaped model
        {"name": "clip 32 layers r64 bf16", "op": "clip", "layers": 32, "hidden": 4096, "inner": 11008, "r": 64, "dtype": "bf16",
         "groups": 1, "extra": 0},
        # 16 adapters trained at once, each clipped by itself; beside them odd fp32 vectors
        {"name": "clip 4 layers r16 fp32 of 16", "op": "clip", "layers": 4, "hidden": 1000, "inner": 2751, "r": 16, "dtype": "fp32",
         "groups": 16, "extra": 5},
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("adapters", "adapters", "head", "head", "clip"))
    if op == "adapters":
        M = rng.choice((spread(1, 16), spread(5, 64), spread(65, 1024), spread(65, 8192)))
        K = 64 * spread(4, 172)
        N = 8 * max(16, min(spread(32, 1376), 4096 * 11008 // K // 8))
        n = spread(1, 64)
        used = min(M, spread(1, n))
        train = M > 64 and rng.random() < 0.35
        return {"op": op, "M": M, "N": min(N, 4096) if train else N, "K": min(K, 4096) if train else K,
                "r": rng.choice((8, 16, 16, 32)) if train else rng.choice((8, 16, 24, 64)), "n": n, "used": used,
                "bare": used > 1 and rng.random() < 0.4, "train": train}
    if op == "head":
        V = spread(1000, 131072)
        K = 64 * spread(4, 64)
        M = min(rng.choice((spread(1, 64), spread(65, 8192))), max(1, 8192 * 32000 * 4096 // V // K))
        train = rng.choice(("no", "X", "X", "XW"))
        if train == "XW":
            M = max(1, min(M, 2048 * 131072 // V))
        return {"op": op, "M": M, "V": V, "K": K, "prompt": rng.choice((0, 1)) if M > 64 else 0, "train": train}
    layers, groups = spread(1, 32), rng.choice((1, 1, spread(2, 32)))
    hidden = spread(256, 4096)
    r = rng.choice((8, 16, 64))
    layers = max(1, min(layers, 32 * 4096 * 64 // (hidden * r * groups)))
    return {"op": op, "layers": layers, "hidden": hidden, "inner": hidden * 11 // 4 + 1, "r": r,
            "dtype": rng.choice(("bf16", "fp16", "fp32")) if layers <= 16 else "bf16", "groups": groups, "extra": rng.choice((0, 3, 9))}


def work(case):
    if case["op"] == "adapters":
        M, N, K, r = case["M"], case["N"], case["K"], case["r"]
        used = case["used"] - (1 if case["bare"] else 0)
        b = 2 * M * (K + N + r) + N * K * (0.5 + 1 / 64) + 2 * used * r * (N + K) + 8 * M
        f = 2 * M * N * K + 2 * M * r * (N + K)
        if case["train"]:
            b += 2 * M * (K + N) + 2 * case["n"] * r * (N + K)
            f += 2 * M * N * K + 4 * M * r * (N + K)
        return {"bytes": b, "flops": f}
    if case["op"] == "head":
        V, K = case["V"], case["K"]
        M = sum(_answered(m, case["prompt"]) for m in range(case["M"]))
        products = {"no": 1, "X": 2, "XW": 3}[case["train"]]
        return {"bytes": 2 * V * K + 2 * M * K + 12 * case["M"] + (0 if products == 1 else 2 * case["M"] * K) +
                (2 * V * K if products == 3 else 0), "flops": 2 * M * V * K * products}
    n = sum(math.prod(s) for s in _shapes(case))
    x = sum(math.prod(s) for s in _extra_shapes(case))
    return {"bytes": 2 * (n * DTYPES[case["dtype"]].itemsize + 4 * x), "flops": 3 * (n + x)}


# ---- inputs ---------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def _answered(m, prompt):
    """Whether position m has a target: with prompt, the first 128 of every 512 have none."""
    return not prompt or m % 512 >= 128


def _shapes(case):
    """The pairs' gradients, A [groups * r, in] and B [groups, out, r], of the seven linears of each layer."""
    h, i, r, n = case["hidden"], case["inner"], case["r"], case["groups"]
    layer = []
    for out, inp in ((h, h),) * 4 + ((i, h),) * 2 + ((h, i),):
        layer += [(n * r, inp), (n, out, r)]
    return layer * case["layers"]


def _extra_shapes(case):
    return [(case["groups"], (1, 4097, 63)[k % 3] + k) for k in range(case["extra"])]


def _nf4_levels():
    p = 1 - (1 / 30 + 1 / 32) / 2
    q = NormalDist().inv_cdf
    up = [q(p + (0.5 - p) * k / 8) for k in range(8)]
    down = [-q(p + (0.5 - p) * k / 7) for k in range(7)]
    return [v / up[0] for v in sorted(down + [0.0] + up)]


def _t8_levels():
    """The 256 levels of a block constant's code: a float of 4 exponent and 3 fraction bits over its largest, 480, in rising order."""
    mag = [((k & 7) / 512 if k < 8 else (1 + (k & 7) / 8) * 2.0 ** ((k >> 3) - 7)) / 480 for k in range(128)]
    return [-m for m in reversed(mag)] + mag


def _nearest(x, levels):
    edge = torch.tensor([(a + b) / 2 for a, b in zip(levels, levels[1:])], device=DEV)
    return torch.bucketize(x, edge)


def _pack_nf4(w):
    """A Gaussian weight as a 4-bit checkpoint holds it: codes of blocks of 64,
    8-bit constants in groups of 256 about their mean."""
    b = w.reshape(-1, 64)
    top = b.abs().amax(1)
    mean = top.mean().reshape(1)
    d = top - mean
    d = torch.nn.functional.pad(d, (0, -d.numel() % 256)).reshape(-1, 256)
    c2 = d.abs().amax(1)
    code8 = _nearest(d / c2.clamp(min=1e-30).unsqueeze(1), _t8_levels()).reshape(-1)[: top.numel()]
    code = _nearest(b / top.unsqueeze(1), _nf4_levels()).reshape(-1, 2).to(torch.uint8)
    return code[:, 0] + 16 * code[:, 1], code8.to(torch.uint8), c2, mean


def _requests(case, g):
    """Index [M] of the adapter of every token: `used` requests of different
    adapters, one token each in turn while decoding, runs of ragged length in a prompt."""
    M, n, used = case["M"], case["n"], case["used"]
    who = torch.randperm(n, generator=g, device=DEV)[:used]
    if case["bare"]:
        who[used - 1] = -1
    if M <= 64:
        return who[torch.arange(M, device=DEV) % used]
    cuts = torch.randperm(M - 1, generator=g, device=DEV)[: used - 1] + 1
    return who[torch.bucketize(torch.arange(M, device=DEV), cuts.sort()[0], right=True)]


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    bf = torch.bfloat16
    if case["op"] == "adapters":
        M, N, K, r, n = case["M"], case["N"], case["K"], case["r"], case["n"]
        st["packed"], st["code8"], st["c2"], st["mean"] = _pack_nf4(_randn(g, N, K, std=0.02))
        st["x"] = _randn(g, M, K).to(bf)
        st["A"], st["B"] = _randn(g, n, r, K, std=0.01).to(bf), _randn(g, n, N, r, std=0.01).to(bf)
        st["scale"] = torch.tensor([0.25, 0.5, 1.0, 2.0], device=DEV)[torch.arange(n, device=DEV) % 4]
        st["index"] = _requests(case, g)
        if case["train"]:
            st["dy"] = _randn(g, M, N).to(bf)
        return st
    if case["op"] == "head":
        M, V, K = case["M"], case["V"], case["K"]
        W = _randn(g, V, K, std=2 * K ** -0.5).to(bf)
        t = torch.randint(V, (M,), generator=g, device=DEV)
        # a hidden state leans towards the word that follows, more or less surely
        lean = torch.rand(M, 1, generator=g, device=DEV).mul_(3.0)
        st["W"], st["x"] = W, (_randn(g, M, K) + lean * W[t].float()).to(bf)
        m = torch.arange(M, device=DEV)
        if case["prompt"]:
            t = torch.where(m % 512 < 128, torch.full_like(t, IGNORED), t)
        st["t"], st["weight"] = t, torch.full((M,), 1.0 / M, device=DEV)
        return st
    dtype, n = DTYPES[case["dtype"]], case["groups"]
    # adapters differ in how far they have come, and so in their gradients' sizes
    size = torch.exp(_randn(g, n, 1, std=0.7))
    grads = [(_randn(g, n, math.prod(s) // n, std=1e-2) * size).to(dtype).reshape(s) for s in _shapes(case)]
    extra = [(_randn(g, n, s[1], std=1e-1) * size) for s in _extra_shapes(case)]
    count = sum(x.numel() for x in grads) + sum(x.numel() for x in extra)
    st["max_norm"] = 0.5 * 1e-2 * (count / n) ** 0.5    # most are clipped
    st["grads"] = grads + extra
    # what the optimizer reads: one flat buffer a type
    for name, parts in (("flat", grads), ("flat_extra", extra)):
        if parts:
            st[name] = torch.empty(sum(x.numel() for x in parts), dtype=parts[0].dtype, device=DEV)
    st["outs"] = [v.view_as(x) for name, parts in (("flat", grads), ("flat_extra", extra)) if parts
                  for v, x in zip(st[name].split([x.numel() for x in parts]), parts)]
    return st


# ---- the plain forms --------------------------------------------------------------

def _weight(st, N, K):
    """The values of the NF4 weight, level times block constant, in fp32."""
    level = torch.tensor(_nf4_levels(), device=DEV)
    t8 = torch.tensor(_t8_levels(), device=DEV)
    scale = t8[st["code8"].long()] * st["c2"].repeat_interleave(256)[: N * K // 64] + st["mean"]
    p = st["packed"]
    codes = torch.stack((p & 15, p >> 4), 1).reshape(-1, 64).long()
    return (level[codes] * scale.unsqueeze(1)).reshape(N, K)


def _plain_adapters(st):
    """All adapters side by side as one of n * r rows, of which a token keeps its own r."""
    c = st["case"]
    M, N, K, r, n = c["M"], c["N"], c["K"], c["r"], c["n"]
    x, w = st["x"].float(), _weight(st, N, K)
    A, B = st["A"].float().reshape(n * r, K), st["B"].float().permute(1, 0, 2).reshape(N, n * r)
    mine = (torch.arange(n, device=DEV) == st["index"].unsqueeze(1)).unsqueeze(2)
    scale = torch.where(mine, st["scale"].reshape(1, n, 1), torch.zeros((), device=DEV))

    def keep(t):
        return (t.reshape(M, n, r) * scale).reshape(M, n * r)

    T = keep(x @ A.t())
    out = {"Y": (x @ w.t() + T @ B.t()).to(torch.bfloat16), "T": T.reshape(M, n, r).sum(1).to(torch.bfloat16)}
    if c["train"]:
        dy = st["dy"].float()
        G = keep(dy @ B)
        out.update(dX=(dy @ w + G @ A).to(torch.bfloat16), dA=(G.t() @ x).reshape(n, r, K).to(torch.bfloat16),
                   dB=(dy.t() @ T).reshape(N, n, r).permute(1, 0, 2).contiguous().to(torch.bfloat16))
    return out


def _plain_head(st):
    c, x, w, t = st["case"], st["x"].float(), st["W"].float(), st["t"]
    z = x @ w.t()
    real = (t >= 0) & (t < c["V"])
    at = torch.where(real, t, torch.zeros_like(t)).unsqueeze(1)
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, at) - top
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    loss = (torch.log(total.double()) - picked.double()).squeeze(1).float()
    out = {"loss": torch.where(real, loss, torch.zeros_like(loss))}
    if c["train"] != "no":
        d = e / total
        d.scatter_add_(1, at, torch.full_like(picked, -1.0))
        d *= torch.where(real, st["weight"], torch.zeros_like(st["weight"])).unsqueeze(1)
        out["dX"] = (d @ w).to(torch.bfloat16)
        if c["train"] == "XW":
            out["dW"] = (d.t() @ x).to(torch.bfloat16)
    return out


def _plain_clip(st):
    n = st["case"]["groups"]
    square = sum([g.double().square().reshape(n, -1).sum(1) for g in st["grads"]])
    norm = torch.sqrt(square).float()
    coef = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).unsqueeze(1)
    done = [(g.float().reshape(n, -1) * coef).to(g.dtype).reshape(-1) for g in st["grads"]]
    k = len(done) - st["case"]["extra"]
    out = {"norm": norm, "flat": torch.cat(done[:k])}
    if k < len(done):
        out["flat_extra"] = torch.cat(done[k:])
    return out


# ---- one pass -----------------------------------------------------------------------

def run(st):
    c = st["case"]
    if not own:
        return {"adapters": _plain_adapters, "head": _plain_head, "clip": _plain_clip}[c["op"]](st)
    import bit_nf4_quantized_absmax_amd as q
    if c["op"] == "adapters":
        w = q.NF4Weight(st["packed"], st["code8"], st["c2"], st["mean"], c["N"], c["K"])
        Y, T = q.adapter_linear_fwd(st["x"], w, st["A"], st["B"], st["scale"], st["index"])
        out = {"Y": Y, "T": T}
        if c["train"]:
            out["dX"], out["dA"], out["dB"] = q.adapter_linear_bwd(st["dy"], st["x"], T, w, st["A"], st["B"], st["scale"], st["index"])
        return out
    if c["op"] == "head":
        if c["train"] == "no":
            return {"loss": q.head_cross_entropy_fwd(st["x"], st["W"], st["t"])[0]}
        loss, lse, dX = q.head_cross_entropy(st["x"], st["W"], st["t"], weight=st["weight"])
        out = {"loss": loss, "dX": dX}
        if c["train"] == "XW":
            out["dW"] = q.head_cross_entropy_dW(st["x"], st["W"], st["t"], lse, weight=st["weight"])
        return out
    out = {"norm": q.clip_grad_norm(st["grads"], st["max_norm"], groups=c["groups"], out=st["outs"]), "flat": st["flat"]}
    if c["extra"]:
        out["flat_extra"] = st["flat_extra"]
    return out


# ---- the definitions in 64 bits -------------------------------------------------------

def _weight_64(st, N, K):
    code = torch.empty(N * K, dtype=torch.long, device=DEV)
    code[0::2], code[1::2] = (st["packed"] & 15).long(), (st["packed"] >> 4).long()
    level = torch.tensor(_nf4_levels(), dtype=torch.float32, device=DEV).double()
    held = torch.tensor(_t8_levels(), dtype=torch.float32, device=DEV).double()[st["code8"].long()]
    block = torch.arange(N * K // 64, device=DEV)
    held = held * st["c2"].double()[block // 256] + st["mean"].double()
    return (level[code] * held.repeat_interleave(64)).reshape(N, K)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adapters":
        M, N, K, r, n = (case[k] for k in ("M", "N", "K", "r", "n"))
        x, w = st["x"].double(), _weight_64(st, N, K)
        out = {"Y": x @ w.t(), "T": torch.zeros(M, r, dtype=torch.float64, device=DEV)}
        if case["train"]:
            dy = st["dy"].double()
            out.update(dX=dy @ w, dA=torch.zeros(n, r, K, dtype=torch.float64, device=DEV),
                       dB=torch.zeros(n, N, r, dtype=torch.float64, device=DEV))
        for a in range(n):
            m = (st["index"] == a).nonzero().squeeze(1)
            if not m.numel():
                continue
            A, B, s = st["A"][a].double(), st["B"][a].double(), st["scale"][a].double()
            T = s * (x[m] @ A.t())
            out["T"][m] = T
            out["Y"][m] += T @ B.t()
            if case["train"]:
                G = s * (dy[m] @ B)
                out["dX"][m] += G @ A
                out["dA"][a], out["dB"][a] = G.t() @ x[m], dy[m].t() @ T
        return out
    if case["op"] == "head":
        x, w, t = st["x"].double(), st["W"].double(), st["t"]
        m = (t >= 0).nonzero().squeeze(1)
        z = x[m] @ w.t()
        logp = torch.log_softmax(z, 1)
        out = {"loss": torch.zeros(case["M"], dtype=torch.float64, device=DEV)}
        out["loss"][m] = -logp.gather(1, t[m].unsqueeze(1)).squeeze(1)
        if case["train"] != "no":
            d = torch.exp(logp)
            d[torch.arange(m.numel(), device=DEV), t[m]] = torch.expm1(-out["loss"][m])
            d *= st["weight"][m].double().unsqueeze(1)
            out["dX"] = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
            out["dX"][m] = d @ w
            if case["train"] == "XW":
                out["dW"] = d.t() @ x[m]
        return out
    n = case["groups"]
    norm = torch.zeros(n, dtype=torch.float64, device=DEV)
    for g in st["grads"]:
        norm += torch.linalg.vector_norm(g.double().reshape(n, -1), dim=1).square()
    norm = norm.sqrt()
    coef = torch.minimum(st["max_norm"] / (norm + 1e-6), torch.ones_like(norm))
    done = [(g.double().reshape(n, -1) * coef.unsqueeze(1)).reshape(-1) for g in st["grads"]]
    k = len(done) - case["extra"]
    out = {"norm": norm, "flat": torch.cat(done[:k])}
    if case["extra"]:
        out["flat_extra"] = torch.cat(done[k:])
    return out
