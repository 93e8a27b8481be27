"""Tunes several tenants' LoRA adapters over one frozen base in one batch, then decodes for all of them.

The base is a hidden linear in NF4 and a frozen output head.  Every sequence of a
batch belongs to one tenant; a step is the linear with each token's own adapter,
the head's cross entropy without its logits, the backward pass into all
adapters, each adapter's gradients clipped by its own norm, and a step of
Adam.  Then one token of every tenant goes through the same linear in one call.

    python examples/tune_adapters.py --tenants 8 --tokens 512 --hidden 1024 --words 32000
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_nf4_quantized_absmax_amd as q


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tenants", 8), ("tokens", 512), ("prompt", 64), ("hidden", 1024), ("words", 32000), ("rank", 16), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--lr", type=float, default=2e-3)
    o = p.parse_args(argv)
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(1)
    D, V, n = o.hidden, o.words, o.tenants

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(torch.bfloat16)

    A = normal(n, o.rank, D, scale=D ** -0.5)
    layer = q.AdapterLinear(normal(D, D, scale=D ** -0.5).float(), n, o.rank, 2.0 * o.rank, lora_A=A)
    head = normal(V, D, scale=4.0 * D ** -0.5)
    x = normal(n, o.tokens, D)
    tenant = torch.arange(n, device=dev)[:, None].expand(n, o.tokens)
    # every tenant's own rule: its next words are those that a low-rank change of the base would say
    change = normal(n, D, 4, scale=D ** -0.5) @ normal(n, 4, D, scale=2.0)
    said = torch.stack([(x[i] @ (layer.w.dequantize() + change[i]).t()) @ head.t() for i in range(n)])
    target = said.argmax(2)
    target[:, :o.prompt] = -100
    real = (target >= 0).sum()
    pairs = [layer.lora_A, layer.lora_B]
    opt = torch.optim.Adam(pairs, lr=o.lr)
    losses = []
    for step in range(o.steps):
        opt.zero_grad(set_to_none=True)
        loss = q.HeadCrossEntropyFn.apply(layer(x, tenant).reshape(-1, D), head, target.reshape(-1)).sum() / real
        loss.backward()
        norm = q.clip_grad_norm([t.grad for t in pairs], 1.0, groups=n)
        opt.step()
        losses.append(loss.item())
        if step % 5 == 0 or step == o.steps - 1:
            print("step %3d  loss %.4f  largest norm %.3f" % (step, losses[-1], norm.max().item()), flush=True)
    # one token of every tenant at once, and of a request without an adapter (index -1)
    last = torch.cat([x[:, -1], x[:1, -1]])
    who = torch.cat([torch.arange(n, device=dev), torch.full((1,), -1, device=dev)])
    with torch.no_grad():
        words = (layer(last, who) @ head.t()).argmax(1)
    print("next words of %d tenants and of the base: %s" % (n, words.tolist()))
    return losses, pairs, words


if __name__ == "__main__":
    main()
