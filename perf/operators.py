"""Cases of the training operators around the adapted linear layer, and their plain forms.

Four kinds of case, by `op`:

  norm_fwd    y = (x - mean) rstd w + b over the last axis (kind "layer"), or y = x rstd w (kind "rms", no mean);
              with `checkpoint`, also y kept in 8 bits and restored as the backward pass reads it.
  norm_bwd    its gradients with respect to x, w and b; with `checkpoint`, x is read from its 8-bit checkpoint.
  linear_bwd  the adapted linear layer's backward pass whose saved input is an 8-bit checkpoint:
              v = g B, grad_x = g W' + s v A, grad_A = s v^T x8, grad_B = s g^T u.
  preference  the paired log-ratio loss of packed sequences from their logits, and the gradient of the logits:
              z = beta ((lp_c - ref_c) - (lp_r - ref_r)), loss = mean of -(1 - e) log sigma(z) - e log sigma(-z).

The 8-bit checkpoint of a bf16 tensor keeps, for each 32 consecutive values of a row, 8-bit integers k and one byte c:
value = k 2^(c - 127), where c = max(E, 7) - 6 with E the exponent field of the block's largest magnitude (c = 255 marks a
block that is not finite).  A row of scale bytes is padded with zeros to a multiple of 4.
"""
import math
import statistics

import torch

own = False

BLOCK = 32

# The 16 levels of the frozen weight's 4-bit codes (normal quantiles at the middles of 16 buckets over the largest), ascending.
_Q = [statistics.NormalDist().inv_cdf((i - 0.5) / 16) for i in range(1, 17)]
LEVELS = [q / _Q[-1] for q in _Q]


def listed():
    return [
        # the norm in front of a block's projections, at the training step's batch and width, its output checkpointed for their backward pass
        {"name": "norm_fwd rms 8192x8192 ckpt", "op": "norm_fwd", "kind": "rms", "M": 8192, "n": 8192, "dtype": "bf16", "bias": False, "checkpoint": True},
        # a small batch's norm: latency
        {"name": "norm_fwd layer 16x4096", "op": "norm_fwd", "kind": "layer", "M": 16, "n": 4096, "dtype": "bf16", "bias": True, "checkpoint": False},
        # the backward pass of the first, from the checkpoint of the residual stream
        {"name": "norm_bwd rms 8192x8192 ckpt", "op": "norm_bwd", "kind": "rms", "M": 8192, "n": 8192, "dtype": "bf16", "bias": False, "checkpoint": True},
        # an odd width and token count in fp32, both weight gradients
        {"name": "norm_bwd layer 2049x5001 fp32", "op": "norm_bwd", "kind": "layer", "M": 2049, "n": 5001, "dtype": "fp32", "bias": True, "checkpoint": False},
        # the input of the widest down projection, kept over the forward pass and restored
        {"name": "checkpoint 8192x28672", "op": "checkpoint", "M": 8192, "n": 28672},
        # a ragged few rows: latency
        {"name": "checkpoint 33x1000", "op": "checkpoint", "M": 33, "n": 1000},
        # the gate projection of the bench's 4096-token workload, all three gradients
        {"name": "linear_bwd 14336x4096 M4096", "op": "linear_bwd", "M": 4096, "n": 4096, "m": 14336, "r": 16, "grad_x": True},
        # the widest down projection of the bench's block where nothing below it trains: the adapters' gradients alone
        {"name": "linear_bwd 8192x28672 ab", "op": "linear_bwd", "M": 8192, "n": 28672, "m": 8192, "r": 64, "grad_x": False},
        # the smallest layer of the tests: latency
        {"name": "linear_bwd 256x256 M32", "op": "linear_bwd", "M": 32, "n": 256, "m": 256, "r": 8, "grad_x": True},
        # eight pairs of long answers over a large vocabulary
        {"name": "preference 8 pairs V131072", "op": "preference", "pairs": 8, "T": 6144, "V": 131072, "dtype": "bf16"},
        # one pair of short answers over a small one: latency
        {"name": "preference 1 pair V32000", "op": "preference", "pairs": 1, "T": 24, "V": 32000, "dtype": "bf16"},
        # an odd vocabulary, fp32 logits
        {"name": "preference 5 pairs V50021 fp32", "op": "preference", "pairs": 5, "T": 1501, "V": 50021, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "checkpoint", "linear_bwd", "preference"])
    if op == "preference":
        V = _log(rng, 1000, 131072)
        pairs = rng.randint(1, 16)
        T = _log(rng, 2 * pairs, max(2 * pairs, min(16384, 6144 * 131072 // V)))
        dtype = rng.choice(["bf16", "fp32"]) if T * V <= 6144 * 65536 else "bf16"
        return {"op": op, "pairs": pairs, "T": T, "V": V, "dtype": dtype}
    if op == "linear_bwd":
        n, m = 64 * _log(rng, 4, 448), 64 * _log(rng, 4, 448) + rng.choice([0, 0, 0, 8, 3])
        M = _log(rng, 1, max(1, min(8192, 4096 * 14336 * 4096 // (n * m))))
        return {"op": op, "M": M, "n": n, "m": m, "r": rng.choice([4, 8, 16, 24, 32, 64, 128]), "grad_x": rng.random() < 0.7}
    n = _log(rng, 64, 16384)
    M = _log(rng, 1, min(16384, 8192 * 8192 // n))
    if op == "checkpoint":
        return {"op": op, "M": M, "n": n}
    ckpt = rng.random() < 0.5
    kind = rng.choice(["rms", "layer"])
    return {"op": op, "kind": kind, "M": M, "n": n, "dtype": "bf16" if ckpt else rng.choice(["bf16", "fp32"]), "bias": kind == "layer", "checkpoint": ckpt}


def _lengths(case):
    """Tokens of each packed sequence (2 for each pair), and of its prompt, whose tokens are not scored."""
    count = 2 * case["pairs"]
    weight = [2 + (3 * i) % 5 for i in range(count)]
    cut = [case["T"] * sum(weight[:i]) // sum(weight) for i in range(count + 1)]
    lens = [b - a for a, b in zip(cut, cut[1:])]
    return lens, [2 * n // 5 for n in lens]


def _size(case):
    return 4 if case.get("dtype") == "fp32" else 2


def work(case):
    op = case["op"]
    if op == "preference":
        lens, prompts = _lengths(case)
        live = sum(lens) - sum(prompts)
        cells = live * case["V"]
        # the scored rows are read once, every row of the gradient is written once (an unscored one with zeros)
        return {"bytes": (cells + case["T"] * case["V"]) * _size(case) + 8 * case["T"], "flops": 8 * cells}
    M, n = case["M"], case["n"]
    cell, packed = M * n, M * n + M * (-(-n // BLOCK))
    if op == "checkpoint":
        return {"bytes": 4 * cell + 2 * packed, "flops": 4 * cell}
    if op == "linear_bwd":
        m, r = case["m"], case["r"]
        flops = 2 * M * m * r + 2 * M * r * (m + n)
        nbytes = packed + 2 * M * m + 4 * M * r + 2 * 2 * r * (n + m) - (0 if case["grad_x"] else 2 * r * n)
        if case["grad_x"]:
            flops += 2 * M * m * n + 2 * M * n * r
            nbytes += 2 * cell + m * n // 2 + m * n // 64 + 4 * (-(-m * n // 16384))
        return {"bytes": nbytes, "flops": flops}
    e = _size(case)
    if op == "norm_fwd":
        return {"bytes": 2 * e * cell + (2 * packed + 2 * cell if case["checkpoint"] else 0) + 8 * M + 8 * n, "flops": 8 * cell}
    return {"bytes": (packed if case["checkpoint"] else e * cell) + 2 * e * cell + 8 * M + 16 * n, "flops": 14 * cell}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------


def _pack(x):
    """(codes int8 [M, n], scales uint8 [M, 4 ceil(n / 128)]) of a bf16 tensor."""
    M, n = x.shape
    nb = -(-n // BLOCK)
    xf = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - n)).view(M, nb, BLOCK)
    field = (xf.abs().amax(-1).view(torch.int32) >> 23) & 255
    field = torch.where(torch.isnan(xf).any(-1), torch.full_like(field, 255), field)
    c = torch.where(field == 255, field, field.clamp(min=7) - 6)
    k = torch.round(xf * ((254 - c).clamp(min=0) << 23).view(torch.float32)[..., None]).clamp(-127, 127)
    k = torch.where((c == 255)[..., None], torch.zeros_like(k), k)
    scales = torch.nn.functional.pad(c.to(torch.uint8), (0, -nb % 4))
    return k.view(M, nb * BLOCK)[:, :n].to(torch.int8).contiguous(), scales.contiguous()


def _unpack(codes, scales):
    """The values a checkpoint stands for."""
    n = codes.shape[1]
    step = (scales.to(torch.int32) << 23).view(torch.float32)  # 2^(c - 127) by its bits; infinite at c = 255, where k = 0
    return codes.float() * step.repeat_interleave(BLOCK, 1)[:, :n]


def _activations(M, n, gen, dtype):
    """Normal values over channels of unequal size, a few of them far larger than the rest."""
    dev = gen.device
    width = torch.exp(0.5 * torch.randn(n, generator=gen, device=dev))
    width = width * torch.where(torch.rand(n, generator=gen, device=dev) < 0.004, 12.0, 1.0)
    shift = 0.1 * torch.randn(n, generator=gen, device=dev)
    return (torch.randn(M, n, generator=gen, device=dev) * width + shift).to(dtype)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    op = case["op"]
    st = {"case": case}
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    if op == "preference":
        T, V = case["T"], case["V"]
        lens, prompts = _lengths(case)
        # answers that the model finds likely: about one nat a token
        labels = torch.randint(0, V, (T,), generator=gen, device=dev)
        logits = torch.empty(T, V, device=dev, dtype=dtype)
        lse = torch.empty(T, device=dev)
        for a in range(0, T, 1024):
            part = 2.0 * torch.randn(min(1024, T - a), V, generator=gen, device=dev)
            own_logit = math.log(V) + 2.0 + torch.randn(part.shape[0], 1, generator=gen, device=dev)
            part.scatter_(1, labels[a:a + 1024, None], own_logit)
            logits[a:a + 1024] = part
            lse[a:a + 1024] = torch.logsumexp(logits[a:a + 1024].float(), 1)
        lp = logits.gather(1, labels[:, None])[:, 0].float() - lse
        cut = [0]
        for n in lens:
            cut.append(cut[-1] + n)
        scored = torch.zeros(T, dtype=torch.bool)
        for a, n, p in zip(cut, lens, prompts):
            scored[a + p:a + n] = True
        scored = scored.to(dev)
        labels = torch.where(scored, labels, torch.full_like(labels, -100))
        lp = torch.where(scored, lp, torch.zeros_like(lp))
        offsets = torch.tensor(cut, dtype=torch.int32, device=dev)
        # the reference model that training started from: near the policy
        logps = torch.stack([lp[a:b].sum() for a, b in zip(cut, cut[1:])])
        ref = logps + 4.0 * torch.randn(len(lens), generator=gen, device=dev)
        st.update(logits=logits, labels=labels, offsets=offsets, ref=ref, beta=0.1, smoothing=0.05)
        return st
    M, n = case["M"], case["n"]
    x = _activations(M, n, gen, dtype)
    if op == "checkpoint":
        return {**st, "x": x}
    if op == "linear_bwd":
        m, r = case["m"], case["r"]
        A, B = normal(r, n, scale=1 / 16), normal(m, r, scale=0.01)
        codes8, scales8 = _pack(x)
        st.update(x8=(codes8, scales8), u=x.float() @ A.float().t(), A=A, B=B, s=0.25, g=normal(M, m))
        # a normal weight's codes are equally likely and its block maxima near 2.4 deviations
        st.update(codes=torch.randint(0, 256, (m * n // 2,), generator=gen, device=dev, dtype=torch.uint8),
                  absmax8=torch.randint(0x2e, 0x39, (m * n // 64,), generator=gen, device=dev, dtype=torch.uint8),
                  c2=0.06 + 0.01 * torch.rand(-(-m * n // 16384), generator=gen, device=dev))
        return st
    w = 1.0 + normal(n, scale=0.1, dtype=torch.float32)
    st.update(w=w.to(dtype), b=normal(n, scale=0.1, dtype=dtype) if case["bias"] else None, eps=1e-5)
    if op == "norm_fwd":
        return {**st, "x": x}
    xf = x.float()
    mean = xf.mean(1) if case["kind"] == "layer" else None
    var = xf.square().mean(1) if mean is None else (xf - mean[:, None]).square().mean(1)
    st.update(mean=mean, rstd=torch.rsqrt(var + st["eps"]), g=normal(M, n, scale=0.1, dtype=dtype))
    if case["checkpoint"]:
        return {**st, "x8": _pack(x)}
    return {**st, "x": x}


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------


def _dequantized(st, dtype=torch.float32):
    """The frozen weight's bf16 values: 4-bit sign-magnitude codes, 8 to a word, over doubly quantized block scales."""
    case = st["case"]
    m, n = case["m"], case["n"]
    by = st["codes"].view(-1, 4)
    code = torch.cat([by & 15, by >> 4], 1).view(-1).to(torch.int64)  # byte j: weight j, weight j + 4
    upper = torch.tensor(LEVELS[8:], dtype=torch.float32, device=by.device)
    table = torch.cat([upper, -upper])
    a = st["absmax8"].view(torch.float8_e4m3fn).float()
    scale = a * st["c2"].repeat_interleave(256)[:a.numel()]
    w = (table[code].view(-1, 64) * scale[:, None]).to(torch.bfloat16)
    return w.view(m, n).to(dtype)


def _plain_norm_fwd(st):
    x = st["x"].float()
    layer = st["case"]["kind"] == "layer"
    mean = x.mean(1) if layer else None
    d = x - mean[:, None] if layer else x
    rstd = torch.rsqrt(d.square().mean(1) + st["eps"])
    y = d * rstd[:, None] * st["w"].float()
    if st["b"] is not None:
        y = y + st["b"].float()
    y = y.to(st["x"].dtype)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if st["case"]["checkpoint"]:
        out["kept"] = _unpack(*_pack(y)).to(torch.bfloat16)
    return out


def _plain_norm_bwd(st):
    x = _unpack(*st["x8"]) if st["case"]["checkpoint"] else st["x"].float()
    layer = st["case"]["kind"] == "layer"
    g, w, rstd = st["g"].float(), st["w"].float(), st["rstd"][:, None]
    xhat = (x - st["mean"][:, None] if layer else x) * rstd
    gw = g * w
    gx = gw - xhat * (gw * xhat).mean(1, keepdim=True)
    if layer:
        gx = gx - gw.mean(1, keepdim=True)
    gx = (gx * rstd).to(st["g"].dtype)
    out = {"grad_x": gx, "grad_w": (g * xhat).sum(0).to(st["w"].dtype)}
    if st["b"] is not None:
        out["grad_b"] = g.sum(0).to(st["w"].dtype)
    return out


def _plain_linear_bwd(st):
    x, g, A, B, s = _unpack(*st["x8"]), st["g"].float(), st["A"].float(), st["B"].float(), st["s"]
    v = g @ B
    out = {"grad_A": (s * (v.t() @ x)).to(torch.bfloat16), "grad_B": (s * (g.t() @ st["u"])).to(torch.bfloat16)}
    if st["case"]["grad_x"]:
        out["grad_x"] = (g @ _dequantized(st) + s * (v @ A)).to(torch.bfloat16)
    return out


def _plain_preference(st):
    logits, labels, offsets = st["logits"].float(), st["labels"], st["offsets"].long()
    scored = labels >= 0
    at = labels.clamp(min=0)[:, None]
    top = logits.amax(1, keepdim=True)
    lse = top + (logits - top).exp().sum(1, keepdim=True).log()
    lp = torch.where(scored, (logits.gather(1, at) - lse)[:, 0], torch.zeros_like(lse[:, 0]))
    t = torch.arange(labels.numel(), device=labels.device)
    member = ((t >= offsets[:-1, None]) & (t < offsets[1:, None])).float()
    logps = (member * lp).sum(1)
    ratio = (logps - st["ref"]).view(-1, 2)
    z = st["beta"] * (ratio[:, 0] - ratio[:, 1])
    e = st["smoothing"]
    soft = lambda v: torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))  # noqa: E731  (log(1 + e^v))
    loss = ((1 - e) * soft(-z) + e * soft(z)).mean()
    dz = (e * torch.sigmoid(z) - (1 - e) * torch.sigmoid(-z)) * (st["beta"] / z.numel())
    coef = torch.where(scored, (torch.stack([dz, -dz], 1).view(-1, 1) * member).sum(0), torch.zeros_like(lp))
    grad = (logits - lse).exp_().mul_(-coef[:, None])
    grad.scatter_add_(1, at, coef[:, None])
    return {"loss": loss, "logps": logps, "grad_logits": grad.to(st["logits"].dtype)}


def run(st):
    op = st["case"]["op"]
    if not own:
        if op == "checkpoint":
            return {"kept": _unpack(*_pack(st["x"])).to(torch.bfloat16)}
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "linear_bwd": _plain_linear_bwd,
                "preference": _plain_preference}[op](st)
    import bit_quantized_fine_qlora_amd as Q
    case = st["case"]
    if op == "checkpoint":
        return {"kept": Q.checkpoint_unpack(Q.checkpoint_pack(st["x"]))}
    if op == "norm_fwd":
        kind = Q.NORM_LAYER if case["kind"] == "layer" else Q.NORM_RMS
        if not case["checkpoint"]:
            y, mean, rstd = Q.norm_fwd(st["x"], st["w"], st["b"], kind=kind, eps=st["eps"])
            return {"y": y, "mean": mean, "rstd": rstd}
        y, mean, rstd, y8 = Q.norm_fwd(st["x"], st["w"], st["b"], kind=kind, eps=st["eps"], checkpoint=True)
        return {"y": y, "mean": mean, "rstd": rstd, "kept": Q.checkpoint_unpack(y8)}
    if op == "norm_bwd":
        x = Q.Checkpoint8(*st["x8"]) if case["checkpoint"] else st["x"]
        gx, gw, gb = Q.norm_bwd(x, st["g"], st["w"], st["rstd"], st["mean"], bias=case["bias"])
        out = {"grad_x": gx, "grad_w": gw}
        return {**out, "grad_b": gb} if case["bias"] else out
    if op == "linear_bwd":
        q = Q.QuantizedWeight(st["codes"], st["absmax8"], st["c2"], case["m"], case["n"])
        gx, gA, gB = Q.linear_bwd(Q.Checkpoint8(*st["x8"]), st["g"], q, st["A"], st["B"], st["s"], u=st["u"],
                                  need_grad_x=case["grad_x"])
        out = {"grad_A": gA, "grad_B": gB}
        return {**out, "grad_x": gx} if case["grad_x"] else out
    saved = Q.preference_fwd(st["logits"], st["labels"], st["offsets"], st["ref"], beta=st["beta"],
                             label_smoothing=st["smoothing"])
    grad = Q.preference_bwd(st["logits"], st["labels"], saved)
    return {"loss": saved.loss, "logps": saved.logps, "grad_logits": grad}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------


def _exact_checkpoint(x):
    """Each 32 values over the power of two that puts the largest of them into [64, 128), rounded half to even."""
    d = x.double()
    M, n = d.shape
    pad = torch.zeros(M, -n % BLOCK, dtype=d.dtype, device=d.device)
    d = torch.cat([d, pad], 1).reshape(-1, BLOCK)
    _, e = torch.frexp(d.abs().max(1).values)  # largest = f 2^e, 1/2 <= f < 1
    step = torch.exp2((e - 7).clamp(min=-126).double())[:, None]
    return (torch.clamp(torch.round(d / step), -127, 127) * step).reshape(M, -1)[:, :n]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return {"kept": _exact_checkpoint(st["x"])}
    if op == "norm_fwd":
        x = st["x"].double()
        mu = x.sum(1) / case["n"] if case["kind"] == "layer" else torch.zeros(case["M"], dtype=torch.float64, device=x.device)
        x = x - mu[:, None]
        r = (x.pow(2).sum(1) / case["n"] + st["eps"]) ** -0.5
        y = torch.einsum("mn,m,n->mn", x, r, st["w"].double()) + (0.0 if st["b"] is None else st["b"].double())
        out = {"y": y, "mean": mu if case["kind"] == "layer" else None, "rstd": r}
        return {**out, "kept": _exact_checkpoint(y.to(torch.bfloat16))} if case["checkpoint"] else out
    if op == "norm_bwd":
        if case["checkpoint"]:
            k, c = (t.double() for t in st["x8"])
            x = k * torch.exp2(c - 127).repeat_interleave(BLOCK, 1)[:, :case["n"]]
        else:
            x = st["x"].double()
        g, w, r = st["g"].double(), st["w"].double(), st["rstd"].double()
        h = (x if st["mean"] is None else x - st["mean"].double()[:, None]) * r[:, None]
        p = (g * h) @ w / case["n"]
        q = g @ w / case["n"] if case["kind"] == "layer" else torch.zeros_like(p)
        gx = r[:, None] * (g * w - q[:, None] - h * p[:, None])
        out = {"grad_x": gx, "grad_w": torch.einsum("mn,mn->n", g, h)}
        return {**out, "grad_b": g.sum(0)} if case["bias"] else out
    if op == "linear_bwd":
        k, c = (t.double() for t in st["x8"])
        x = k * torch.exp2(c - 127).repeat_interleave(BLOCK, 1)[:, :case["n"]]
        g, A, B, s = st["g"].double(), st["A"].double(), st["B"].double(), st["s"]
        out = {"grad_A": s * (g @ B).t() @ x, "grad_B": s * g.t() @ st["u"].double()}
        if case["grad_x"]:
            # W': bit 3 of a code is its sign, bits 0-2 the rank of its magnitude among the 8 upper levels
            word = st["codes"].view(-1, 4).long()
            code = torch.stack([word & 15, word >> 4], 1).reshape(-1)
            mag = torch.tensor(LEVELS[8:], dtype=torch.float64, device=word.device).float()[code & 7]
            e, f = (st["absmax8"].long() >> 3) - 7, (st["absmax8"].long() & 7).double() / 8
            blk = (torch.exp2(e.double()) * (1 + f)).float() * st["c2"].repeat_interleave(256)[:e.numel()]
            w = (mag.view(-1, 64) * blk[:, None]).to(torch.bfloat16).double().reshape(-1)
            w = torch.where(code >= 8, -w, w).view(case["m"], case["n"])
            out["grad_x"] = g @ w + s * (g @ B) @ A
        return out
    labels, dev = st["labels"], st["labels"].device
    T, V, beta, e = case["T"], case["V"], st["beta"], st["smoothing"]
    lp, lses = torch.zeros(T, dtype=torch.float64, device=dev), torch.zeros(T, dtype=torch.float64, device=dev)
    for a in range(0, T, 512):
        part = st["logits"][a:a + 512].double()
        lses[a:a + 512] = torch.logsumexp(part, 1)
        lp[a:a + 512] = part[torch.arange(part.shape[0], device=dev), labels[a:a + 512].clamp(min=0)] - lses[a:a + 512]
    lp[labels < 0] = 0.0
    cut = st["offsets"].tolist()
    logps = torch.stack([lp[a:b].sum() for a, b in zip(cut, cut[1:])])
    pairs = case["pairs"]
    z = beta * ((logps[0::2] - st["ref"][0::2].double()) - (logps[1::2] - st["ref"][1::2].double()))
    loss = -((1 - e) * torch.nn.functional.logsigmoid(z) + e * torch.nn.functional.logsigmoid(-z)).sum() / pairs
    slope = beta / pairs * (torch.sigmoid(z) - 1 + e)
    grad = torch.zeros(T, V, dtype=torch.float64, device=dev)
    for i, (a, b) in enumerate(zip(cut, cut[1:])):
        for c in range(a, b, 512):
            rows = torch.arange(c, min(c + 512, b), device=dev)
            rows = rows[labels[rows] >= 0]
            f = slope[i // 2] * (1 if i % 2 == 0 else -1)
            grad[rows] = -f * torch.exp(st["logits"][rows].double() - lses[rows, None])
            grad[rows, labels[rows]] += f
    return {"loss": loss, "logps": logps, "grad_logits": grad}
