"""The operators together: examples/preference_step.py, its gradients against
float64 autograd of the same model, and its training."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import qlora_oracle as O
from parity_utils import f64, host_bits

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    spec = importlib.util.spec_from_file_location("preference_step", os.path.join(ROOT, "examples", "preference_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def values(t):
    return torch.from_numpy(f64(host_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64))


def dense(q):
    bits = O.dequant_nf4_dq(q.codes.cpu().numpy(), q.absmax8.cpu().numpy(), q.c2.cpu().numpy(), q.m * q.n)
    return torch.from_numpy(f64(bits).reshape(q.m, q.n))


def test_one_step_against_autograd(example):
    """Each stage of the library rounds to bf16 (2^-8) and the saved inputs to 8 bits (under 1 % of a block's
    size): the common tolerance of the float outputs, 1e-2 in the 2-norm, is widened by that to 3e-2."""
    print("[case] one training step", flush=True)
    Q = example.Q
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    model = example.make_model(gen)
    for name in ("inner", "head"):  # a trained adapter: B is not zero
        b = model[name]["B"]
        b.master.copy_(0.05 * torch.randn(b.master.shape, generator=gen, device="cuda"))
        b.copy.copy_(b.master)
    tokens, labels, offsets = example.make_pairs(gen)
    logits, kept = example.forward(model, tokens)
    reference = Q.sequence_logps(logits, labels, offsets) + 3.0 * torch.randn(len(offsets) - 1, generator=gen, device="cuda")
    result = Q.preference_fwd(logits, labels, offsets, reference, beta=example.BETA)
    grads = example.backward(model, kept, Q.preference_bwd(logits, labels, result))

    leaf = {id(w): values(w.copy).requires_grad_(True) for w, _ in grads}
    norm = lambda x, w: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * w  # noqa: E731
    lin = lambda x, L: x @ dense(L["q"]).T + example.SCALE * (x @ leaf[id(L["A"])].T) @ leaf[id(L["B"])].T  # noqa: E731
    x0 = values(model["embed"])[tokens.cpu()]
    x1 = x0 + lin(norm(x0, leaf[id(model["norm1"])]), model["inner"])
    lp = torch.log_softmax(lin(norm(x1, leaf[id(model["norm2"])]), model["head"]), 1)
    lab = labels.cpu()
    lp = torch.where(lab >= 0, lp.gather(1, lab.clamp(min=0)[:, None])[:, 0], 0.0)
    cut = offsets.tolist()
    seq = torch.stack([lp[a:b].sum() for a, b in zip(cut, cut[1:])]) - values(reference)
    z = example.BETA * (seq[0::2] - seq[1::2])
    loss = -torch.nn.functional.logsigmoid(z).mean()
    loss.backward()
    assert abs(result.loss.item() - loss.item()) <= 3e-2 * loss.item()
    for w, g in grads:
        want = leaf[id(w)].grad.numpy()
        got = values(g).numpy()
        assert got.shape == want.shape
        assert np.linalg.norm(got - want) <= 3e-2 * np.linalg.norm(want)


def test_training_lowers_the_loss(example):
    print("[case] training", flush=True)
    losses = example.train(30, seed=1, say=lambda *_: None)
    assert abs(losses[0] - np.log(2.0)) < 1e-6  # the policy starts as the reference
    assert losses[-1] < 0.5 * losses[0]
    assert losses == example.train(30, seed=1, say=lambda *_: None)  # bit for bit


def test_captured_graph_replays(example):
    """A captured chain of the new operators gives its eager bits on every replay, with other work between."""
    print("[case] graph replays", flush=True)
    Q = example.Q
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    model = example.make_model(gen)
    tokens, labels, offsets = example.make_pairs(gen)
    head = model["head"]
    x = torch.empty((tokens.numel(), example.WIDTH), dtype=torch.bfloat16, device="cuda")

    def chain():
        z, _, rstd, z8 = Q.norm_fwd(x, model["norm2"].copy, checkpoint=True)
        logits, u = Q.linear_fwd(z, head["q"], head["A"].copy, head["B"].copy, example.SCALE)
        r = Q.preference_fwd(logits, labels, offsets, beta=example.BETA)
        g = Q.preference_bwd(logits, labels, r)
        gz, gA, gB = Q.linear_bwd(z8, g, head["q"], head["A"].copy, head["B"].copy, example.SCALE, u=u)
        gx, gw, _ = Q.norm_bwd(Q.checkpoint_pack(x), gz, model["norm2"].copy, rstd)
        return r.loss, r.logps, g, gA, gB, gx, gw

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x.normal_(generator=gen)
        chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain()
    for seed in range(4):
        gen.manual_seed(seed)
        x.normal_(generator=gen)
        eager = [t.clone() for t in chain()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)
