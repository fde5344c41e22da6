"""One training step of the adapters of a mixture of experts, every heavy part through the library.

A norm, a frozen router that sends each token to two experts, the experts'
adapted up and down projections with a gate between them, and a residual; the
frozen weights in NF4, the adapters trained by AdamW with its moments in 8 bits
and the gradients held to a norm.  The router's result stays on the device: the
experts' rows are found from offsets there.

    python examples/experts_step.py [steps]

needs one MI355X; data and weights are synthetic.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_fine_qlora_amd as Q  # noqa: E402

TOKENS, WIDTH, INNER, EXPERTS, CHOSEN, RANK, SCALE = 200, 256, 512, 6, 2, 16, 1.0
LR, MAX_NORM, SEED = 2e-3, 0.5, 0  # SEED: of the second moments' codes, a step at a time


class Trained:
    """fp32 weights of all experts, AdamW moments in 8 bits and the bf16 copy that the kernels read."""

    def __init__(self, value: torch.Tensor):
        self.master = value.float().contiguous()
        self.copy = self.master.to(torch.bfloat16)
        self.grad = torch.empty_like(self.copy)
        self.m = Q.alloc_moment8(value.numel(), True)
        self.v = Q.alloc_moment8(value.numel(), False)

    def entry(self):
        return self.master, self.copy, self.grad, self.m, self.v


def make_model(gen):
    def normal(*shape, std):
        return std * torch.randn(*shape, generator=gen, device="cuda")

    def adapted(m, n):
        return {"q": Q.quantize_nf4_dq(normal(EXPERTS * m, n, std=n ** -0.5)),
                "A": Trained(normal(EXPERTS, RANK, n, std=1 / 16)),
                "B": Trained(torch.zeros(EXPERTS, m, RANK, device="cuda"))}

    model = {"norm": torch.ones(WIDTH, device="cuda"), "router": normal(WIDTH, EXPERTS, std=WIDTH ** -0.5),
             "up": adapted(INNER, WIDTH), "down": adapted(WIDTH, INNER)}
    model["trained"] = [model[p][k] for p in ("up", "down") for k in ("A", "B")]
    model["optimizer"] = Q.AdamWStep([t.entry() for t in model["trained"]])
    return model


def route(model, y):
    """For each of the rows that the experts see, in order of their expert: its token and its weight; the rows of each
    token, and the experts' offsets."""
    weight, expert = torch.softmax(y.float() @ model["router"], 1).topk(CHOSEN, 1)
    expert = expert.reshape(-1)
    order = torch.argsort(expert, stable=True)
    count = (expert[:, None] == torch.arange(EXPERTS, device="cuda")).sum(0)
    offsets = torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    return order // CHOSEN, weight.reshape(-1)[order], place.view(-1, CHOSEN), offsets


def forward(model, x):
    """The block's output, and what the backward pass keeps."""
    y, _, _ = Q.norm_fwd(x, model["norm"])
    token, weight, place, offsets = route(model, y)
    up, down = model["up"], model["down"]
    rows = y[token]
    h, u1 = Q.experts_fwd(rows, offsets, up["q"], up["A"].copy, up["B"].copy, SCALE)
    a = torch.nn.functional.silu(h)
    o, u2 = Q.experts_fwd(a, offsets, down["q"], down["A"].copy, down["B"].copy, SCALE)
    out = x.float() + (weight[:, None] * o.float())[place].sum(1)  # no atomics: the same bits each time
    return out, {"rows": rows, "h": h, "a": a, "u1": u1, "u2": u2, "token": token, "weight": weight, "offsets": offsets}


def backward(model, kept, grad_out):
    """Fills the adapters' gradients; the block's input and its router are frozen."""
    up, down, offsets = model["up"], model["down"], kept["offsets"]
    g = (kept["weight"][:, None] * grad_out[kept["token"]]).to(torch.bfloat16)
    ga = torch.empty_like(kept["a"])
    Q.experts_bwd(kept["a"], g, offsets, down["q"], down["A"].copy, down["B"].copy, SCALE, u=kept["u2"],
                  out=(ga, down["A"].grad, down["B"].grad))
    h = kept["h"].float()
    s = torch.sigmoid(h)
    gh = (ga.float() * s * (1 + h * (1 - s))).to(torch.bfloat16)
    Q.experts_bwd(kept["rows"], gh, offsets, up["q"], up["A"].copy, up["B"].copy, SCALE, u=kept["u1"],
                  out=(None, up["A"].grad, up["B"].grad))


def loss_of(out, target):
    """Mean squared distance and its gradient."""
    d = out - target
    return d.square().mean(), d * (2.0 / d.numel())


def train_step(model, x, target, step):
    """(loss before the step, gradient norm)."""
    out, kept = forward(model, x)
    loss, grad = loss_of(out, target)
    backward(model, kept, grad)
    clip = model["optimizer"].clip(MAX_NORM)
    model["optimizer"].run(LR, weight_decay=0.01, step=step, clip=clip, seed=SEED)
    return loss, clip[0]


def train(steps: int = 20, seed: int = 0, say=print):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    model = make_model(gen)
    x = torch.randn(TOKENS, WIDTH, generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.randn(TOKENS, WIDTH, generator=gen, device="cuda")
    seen = []
    for step in range(1, steps + 1):
        loss, norm = train_step(model, x, target, step)
        seen.append((loss, norm))
        if step == 1:
            state = sum(t.m.nbytes() + t.v.nbytes() for t in model["trained"])
            say(f"optimizer moments: {state} bytes ({sum(8 * t.master.numel() for t in model['trained'])} in fp32)")
        if step == 1 or step % 10 == 0:
            say(f"step {step:3d}  loss {loss.item():.4f}  gradient norm {norm.item():.4f}")
    return [(a.item(), b.item()) for a, b in seen]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
