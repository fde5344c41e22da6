"""The experts' operators together: examples/experts_step.py, its gradients against float64 autograd of the same
model, one optimizer step from them against the oracle, and the chain captured into a graph."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import experts_oracle as X
from oracle import qlora_oracle as O
from parity_utils import f64, host_bits

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    spec = importlib.util.spec_from_file_location("experts_step", os.path.join(ROOT, "examples", "experts_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def values(t):
    return torch.from_numpy(f64(host_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64))


def dense(q, E):
    bits = O.dequant_nf4_dq(q.codes.cpu().numpy(), q.absmax8.cpu().numpy(), q.c2.cpu().numpy(), q.m * q.n)
    return torch.from_numpy(f64(bits).reshape(E, q.m // E, q.n))


def trained_model(example, gen):
    model = example.make_model(gen)
    for p in ("up", "down"):  # a trained adapter: B is not zero
        b = model[p]["B"]
        b.master.copy_(0.05 * torch.randn(b.master.shape, generator=gen, device="cuda"))
        b.copy.copy_(b.master)
    return model


def test_one_step_against_autograd(example):
    """Each stage of the library rounds to bf16 (2^-8); the common tolerance of the float outputs, 1e-2 in the 2-norm,
    is widened by the chain's five roundings to 3e-2."""
    print("[case] one training step of experts", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    model = trained_model(example, gen)
    x = torch.randn(example.TOKENS, example.WIDTH, generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.randn(example.TOKENS, example.WIDTH, generator=gen, device="cuda")
    out, kept = example.forward(model, x)
    loss, grad = example.loss_of(out, target)
    example.backward(model, kept, grad)

    leaf = {id(t): values(t.copy).requires_grad_(True) for t in model["trained"]}
    token, weight, cut = kept["token"].cpu(), values(kept["weight"]), kept["offsets"].tolist()
    assert cut[-1] == example.TOKENS * example.CHOSEN and sorted(token.tolist()) == sorted(list(range(example.TOKENS)) * 2)

    def layer(rows, p):
        W, A, B = dense(p["q"], example.EXPERTS), leaf[id(p["A"])], leaf[id(p["B"])]
        return torch.cat([rows[a:b] @ W[e].T + example.SCALE * (rows[a:b] @ A[e].T) @ B[e].T
                          for e, (a, b) in enumerate(zip(cut, cut[1:]))])

    x64 = values(x)
    y = x64 * torch.rsqrt(x64.square().mean(1, keepdim=True) + 1e-5)
    o = layer(torch.nn.functional.silu(layer(y[token], model["up"])), model["down"])
    want = (x64.index_add(0, token, weight[:, None] * o) - values(target)).square().mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 3e-2 * want.item()
    for t in model["trained"]:
        g, ref = values(t.grad).numpy(), leaf[id(t)].grad.numpy()
        assert np.linalg.norm(g - ref) <= 3e-2 * np.linalg.norm(ref)

    # the optimizer's step from these gradients
    grads = [values(t.grad).numpy().ravel() for t in model["trained"]]
    before = [values(t.master).numpy().ravel() for t in model["trained"]]
    clip = model["optimizer"].clip(example.MAX_NORM)
    model["optimizer"].run(example.LR, weight_decay=0.01, step=1, clip=clip)
    norm, factor = X.grad_clip(grads, example.MAX_NORM)
    assert abs(clip[0].item() - norm) <= 2.0 ** -23 * norm and abs(clip[1].item() - factor) <= 2.0 ** -23 * factor
    for t, p, g in zip(model["trained"], before, grads):
        z = np.zeros_like(p)
        ref, m, v = X.adamw_step(p, g, z, z, 1, example.LR, 0.9, 0.999, 1e-8, 0.01, factor=clip[1].item())
        got = values(t.master).numpy().ravel()
        # the step itself is at most LR (m / sqrt(v) = g / |g| in the first), 20 roundings of 2^-24 of it and 4 of p
        assert np.all(np.abs(got - ref) <= 2.0 ** -24 * (20 * example.LR + 4 * np.abs(p)))
        for mom, exact in ((t.m, m), (t.v, v)):
            codes, steps = X.moment8_pack(exact, mom.signed)
            near = np.abs(mom.codes.cpu().numpy().astype(int) - codes.astype(int)) <= 1  # a border, or the step's last bit
            assert near.all() and (mom.codes.cpu().numpy() == codes).mean() > 0.999
            assert np.all(np.abs(mom.steps.cpu().numpy() - steps) <= 2.0 ** -23 * steps)


def test_runs_and_repeats(example):
    print("[case] training", flush=True)
    first = example.train(12, seed=1, say=lambda *_: None)
    assert np.isfinite(first).all()
    assert first == example.train(12, seed=1, say=lambda *_: None)  # bit for bit


def test_captured_chain_replays(example):
    """The experts' layers, their backward, the clip and the step in one graph: each replay is the eager chain."""
    print("[case] graph of the experts' chain", flush=True)
    Q = example.Q
    gen = torch.Generator(device="cuda")
    models = []
    for _ in range(2):
        gen.manual_seed(7)
        models.append(trained_model(example, gen))
    M = example.TOKENS * example.CHOSEN
    rows = torch.empty((M, example.WIDTH), dtype=torch.bfloat16, device="cuda")
    g = torch.empty((M, example.WIDTH), dtype=torch.bfloat16, device="cuda")
    offsets = torch.zeros(example.EXPERTS + 1, dtype=torch.int32, device="cuda")

    def chain(model):
        up, down = model["up"], model["down"]
        h, u1 = Q.experts_fwd(rows, offsets, up["q"], up["A"].copy, up["B"].copy, example.SCALE)
        o, u2 = Q.experts_fwd(h, offsets, down["q"], down["A"].copy, down["B"].copy, example.SCALE)
        gh, gA, gB = Q.experts_bwd(h, g, offsets, down["q"], down["A"].copy, down["B"].copy, example.SCALE, u=u2)
        down["A"].grad.copy_(gA)
        down["B"].grad.copy_(gB)
        Q.experts_bwd(rows, gh, offsets, up["q"], up["A"].copy, up["B"].copy, example.SCALE, u=u1,
                      out=(None, up["A"].grad, up["B"].grad))
        clip = model["optimizer"].clip(example.MAX_NORM)
        model["optimizer"].run(example.LR, step=2, clip=clip)
        return o, clip

    def fill(seed):
        gen.manual_seed(seed)
        rows.normal_(generator=gen)
        g.normal_(generator=gen)
        cut = torch.randint(0, M + 1, (example.EXPERTS - 1,), generator=gen, device="cuda").sort()[0]
        offsets[1:-1] = cut.int()
        offsets[-1] = M

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for model in models:
            chain(model)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain(models[1])
    for seed in range(1, 5):
        fill(seed)
        eager = chain(models[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)
        for s, t in zip(models[0]["trained"], models[1]["trained"]):
            for a, b in ((s.master, t.master), (s.copy, t.copy), (s.grad, t.grad), (s.m.codes, t.m.codes),
                         (s.m.steps, t.m.steps), (s.v.codes, t.v.codes), (s.v.steps, t.v.steps)):
                assert torch.equal(a, b)
