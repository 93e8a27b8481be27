"""Distils a teacher into a student whose frozen weights are in MX4.

The student is a hidden linear and an output head, both MX4Linear: 4-bit
frozen weights, activations rounded to 4 bits for them, a LoRA pair each.  The
teacher has the same weights before rounding, moved by a low-rank change, and is
known by its top logits only.  A step is forward, KL divergence to those logits,
backward into the pairs.  Held-out tokens of the teacher are then scored by
their log probabilities under the student, before and after.

    python examples/distill_mx4.py --tokens 8192 --hidden 512 --words 32000
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_nf4_quantized_absmax_amd as q


class Student(torch.nn.Module):
    def __init__(self, hidden, head, r, gen):
        super().__init__()

        def layer(w):
            a = torch.randn(r, w.shape[1], generator=gen, device=w.device) * w.shape[1] ** -0.5
            return q.MX4Linear(w, r, 2.0 * r, lora_A=a.to(torch.bfloat16))

        self.hidden, self.head = layer(hidden), layer(head)

    def forward(self, x):
        return self.head(torch.tanh(self.hidden(x)))


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 8192), ("hidden", 512), ("words", 32000), ("rank", 16), ("entries", 64), ("steps", 40)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--temperature", type=float, default=2.0)
    p.add_argument("--lr", type=float, default=4e-3)
    o = p.parse_args(argv)
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(1)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * scale

    D, V = o.hidden, o.words
    w1, w2 = normal(D, D, scale=D ** -0.5), normal(V, D, scale=4.0 * D ** -0.5)
    student = Student(w1, w2, o.rank, gen)
    w2 = w2 + normal(V, 4, scale=2.0 * D ** -0.5) @ normal(4, D)      # what the student has to learn
    inputs, held = normal(o.tokens, D), normal(o.tokens // 4 + 1, D)

    def teacher(x):
        return torch.tanh(x @ w1.t()) @ w2.t()

    logit, index = teacher(inputs).topk(o.entries, dim=1)
    truth = teacher(held).argmax(1)
    inputs, held = inputs.to(torch.bfloat16), held.to(torch.bfloat16)

    @torch.no_grad()
    def score():
        r = q.token_logprobs(student(held), truth, top=5)
        hits = (r.top_index == truth[:, None]).any(1).float().mean().item()
        return r.logprob.mean().item(), r.entropy.mean().item(), hits

    before = score()
    opt = torch.optim.Adam(student.parameters(), lr=o.lr)
    losses = []
    for step in range(o.steps):
        loss = q.DistillTopKFn.apply(student(inputs), index, logit, o.temperature).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if step % 10 == 0 or step == o.steps - 1:
            print("step %3d  loss %.4f" % (step, losses[-1].item()), flush=True)
    after = score()
    for name, (lp, h, hits) in (("before", before), ("after", after)):
        print("%-6s  log probability %.3f  entropy %.3f  among the 5 most likely %.3f" % (name, lp, h, hits), flush=True)
    return [v.item() for v in losses], before, after


if __name__ == "__main__":
    main()
