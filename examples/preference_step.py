"""Preference tuning of a small adapted block, every step through the library.

A frozen embedding, a norm, an adapted linear layer with a residual, a second
norm and an adapted vocabulary projection; the frozen weights in NF4, the
adapters and the norms' weights trained by Adam on pairs of answers.  What the
backward pass needs of the activations is kept in 8 bits: the norms write the
checkpoints of the layers' inputs while they make them, and the residual
stream is packed once for the norms' own backward.

    python examples/preference_step.py [steps]

needs one MI355X; data and weights are synthetic.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_fine_qlora_amd as Q  # noqa: E402

WIDTH, VOCAB, RANK, SCALE = 512, 1024, 16, 2.0
PAIRS, LENGTH, PROMPT = 8, 24, 8
BETA, LR = 0.1, 2e-3


class Trained:
    """fp32 weights, Adam moments and the bf16 copy that the kernels read."""

    def __init__(self, value: torch.Tensor):
        self.master = value.float().contiguous()
        self.copy = self.master.to(torch.bfloat16)
        self.m = torch.zeros_like(self.master)
        self.v = torch.zeros_like(self.master)


def make_model(gen):
    def normal(*shape, std):
        return std * torch.randn(*shape, generator=gen, device="cuda")

    def adapted(m, n):
        return {"q": Q.quantize_nf4_dq(normal(m, n, std=n ** -0.5)), "A": Trained(normal(RANK, n, std=1 / 16)),
                "B": Trained(torch.zeros(m, RANK, device="cuda"))}

    return {"embed": normal(VOCAB, WIDTH, std=1.0).to(torch.bfloat16),
            "norm1": Trained(torch.ones(WIDTH, device="cuda")), "inner": adapted(WIDTH, WIDTH),
            "norm2": Trained(torch.ones(WIDTH, device="cuda")), "head": adapted(VOCAB, WIDTH)}


def make_pairs(gen):
    """Prompts that both answers share; preferred answers follow a rule, the others do not."""
    seqs = []
    for _ in range(PAIRS):
        prompt = torch.randint(0, VOCAB, (PROMPT,), generator=gen, device="cuda")
        good = [int(prompt[-1])]
        while len(good) <= LENGTH - PROMPT:
            good.append((5 * good[-1] + 3) % VOCAB)
        good = torch.tensor(good[1:], device="cuda")
        bad = torch.randint(0, VOCAB, (LENGTH - PROMPT,), generator=gen, device="cuda")
        seqs += [torch.cat([prompt, good]), torch.cat([prompt, bad])]
    tokens = torch.cat([s[:-1] for s in seqs])
    labels = torch.cat([torch.cat([torch.full((PROMPT - 1,), -100, device="cuda"), s[PROMPT:]]) for s in seqs])
    offsets = torch.arange(0, 2 * PAIRS + 1, dtype=torch.int32, device="cuda") * (LENGTH - 1)
    return tokens, labels, offsets


def forward(model, tokens):
    """Logits, and what the backward pass keeps."""
    x0 = model["embed"][tokens]
    y, _, rstd1, y8 = Q.norm_fwd(x0, model["norm1"].copy, checkpoint=True)
    inner = model["inner"]
    h, u1 = Q.linear_fwd(y, inner["q"], inner["A"].copy, inner["B"].copy, SCALE)
    x1 = x0 + h
    z, _, rstd2, z8 = Q.norm_fwd(x1, model["norm2"].copy, checkpoint=True)
    head = model["head"]
    logits, u2 = Q.linear_fwd(z, head["q"], head["A"].copy, head["B"].copy, SCALE)
    kept = {"x0": Q.checkpoint_pack(x0), "x1": Q.checkpoint_pack(x1), "y": y8, "z": z8, "u1": u1, "u2": u2,
            "rstd1": rstd1, "rstd2": rstd2}
    return logits, kept


def backward(model, kept, grad_logits):
    """(weights, gradient) pairs."""
    inner, head = model["inner"], model["head"]
    gz, gA2, gB2 = Q.linear_bwd(kept["z"], grad_logits, head["q"], head["A"].copy, head["B"].copy, SCALE, u=kept["u2"])
    gx1, gw2, _ = Q.norm_bwd(kept["x1"], gz, model["norm2"].copy, kept["rstd2"], kind=Q.NORM_RMS)
    gy, gA1, gB1 = Q.linear_bwd(kept["y"], gx1, inner["q"], inner["A"].copy, inner["B"].copy, SCALE, u=kept["u1"])
    _, gw1, _ = Q.norm_bwd(kept["x0"], gy, model["norm1"].copy, kept["rstd1"], kind=Q.NORM_RMS)
    return [(inner["A"], gA1), (inner["B"], gB1), (head["A"], gA2), (head["B"], gB2), (model["norm1"], gw1),
            (model["norm2"], gw2)]


def train(steps: int = 30, seed: int = 0, say=print):
    """The loss before each step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    model = make_model(gen)
    tokens, labels, offsets = make_pairs(gen)
    reference = Q.sequence_logps(forward(model, tokens)[0], labels, offsets)
    losses = []
    for step in range(1, steps + 1):
        logits, kept = forward(model, tokens)
        result = Q.preference_fwd(logits, labels, offsets, reference, beta=BETA)
        grads = backward(model, kept, Q.preference_bwd(logits, labels, result, out=logits))
        Q.adam_step([(w.master, w.copy, g, w.m, w.v) for w, g in grads], LR, 0.9, 0.999, 1e-8, 0.0, step)
        losses.append(result.loss)
        if step == 1:
            packed = sum(kept[k].nbytes() for k in ("x0", "x1", "y", "z"))
            plain = sum(2 * kept[k].codes.numel() for k in ("x0", "x1", "y", "z"))
            say(f"activations kept for the backward pass: {packed} bytes ({plain} in bf16)")
        if step == 1 or step % 10 == 0:
            say(f"step {step:3d}  loss {result.loss.item():.4f}")
    return [v.item() for v in losses]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
