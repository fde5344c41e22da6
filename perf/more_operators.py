"""Cases of the adapted experts' products and of the optimizer step over their adapters, and their plain forms.

Three kinds of case, by `op`:

  experts_fwd  the adapted layer of E experts, rows in order of their expert: for the rows offsets[e] .. offsets[e + 1] - 1
               u = x A_e^T, h = x W'_e^T + s u B_e^T, with W'_e rows e m .. (e + 1) m - 1 of one stacked 4-bit weight.
  experts_bwd  its gradients: v = g B_e, grad_x = g W'_e + s v A_e, grad_A_e = s v^T x, grad_B_e = s g^T u, the last two over
               the expert's rows (zeros where it has none).
  adamw        Adam with decoupled weight decay over many tensors at once, moments in 32 bits or in 8, the gradients held to
               a norm first where `clip` says so.

A moment in 8 bits: blocks of 128 consecutive values share one fp32 step d.  The first moment keeps a sign and k in 0 .. 127
and stands for +-k^2 d with d = max / 127^2; of the second its root is kept, k in 0 .. 255, root = k^2 d with d = max root /
255^2, value = root^2, and no value but zero takes k = 0.  Each value takes the nearest k (the lower of two as near).
"""
import math
import statistics

import torch

own = False

# The 16 levels of the frozen weight's 4-bit codes (normal quantiles at the middles of 16 buckets over the largest), ascending.
_Q = [statistics.NormalDist().inv_cdf((i - 0.5) / 16) for i in range(1, 17)]
LEVELS = [q / _Q[-1] for q in _Q]

BLOCK = 128


def listed():
    return [
        # a feed-forward projection of eight experts, each as wide as the 8B gate projection, two experts for each of 4096 tokens
        {"name": "experts_fwd 8x14336x4096 M8192", "op": "experts_fwd", "E": 8, "idle": 0, "M": 8192, "n": 4096, "m": 14336, "r": 16},
        # the same layer where eight tokens are being generated: latency, bound by the weights
        {"name": "experts_fwd 8x14336x4096 M16", "op": "experts_fwd", "E": 8, "idle": 0, "M": 16, "n": 4096, "m": 14336, "r": 16},
        # many narrow experts, some of them without a row, about a hundred rows each
        {"name": "experts_fwd 64x1024x2048 M6000", "op": "experts_fwd", "E": 64, "idle": 5, "M": 6000, "n": 2048, "m": 1024, "r": 8},
        # the backward pass of the first, all three gradients
        {"name": "experts_bwd 8x14336x4096 M8192", "op": "experts_bwd", "E": 8, "idle": 0, "M": 8192, "n": 4096, "m": 14336, "r": 16, "grad_x": True},
        # the widest down projection where nothing below it trains: the adapters' gradients alone
        {"name": "experts_bwd 4x8192x28672 M4096 ab", "op": "experts_bwd", "E": 4, "idle": 0, "M": 4096, "n": 28672, "m": 8192, "r": 64, "grad_x": False},
        # odd sizes, experts without rows: latency
        {"name": "experts_bwd 6x259x320 M203", "op": "experts_bwd", "E": 6, "idle": 2, "M": 203, "n": 320, "m": 259, "r": 12, "grad_x": True},
        # all adapters of a 32-layer 8B-shaped model at 16 ranks, 448 tensors
        {"name": "adamw 8 bits, 448 tensors", "op": "adamw", "state": 8, "layers": 32, "experts": 0, "r": 16, "grad": "bf16", "clip": True},
        # the adapters of eight experts in 12 layers of that shape, 576 tensors
        {"name": "adamw 8 bits, experts", "op": "adamw", "state": 8, "layers": 12, "experts": 8, "r": 16, "grad": "bf16", "clip": False},
        # one layer's worth of a small adapter: latency
        {"name": "adamw 8 bits, 3 small tensors", "op": "adamw", "state": 8, "tensors": 3, "size": 16384, "grad": "bf16", "clip": True},
        # tensors of odd sizes, gradients summed in fp32, moments in 32 bits
        {"name": "adamw 32 bits, odd sizes", "op": "adamw", "state": 32, "tensors": 97, "size": 100003, "grad": "fp32", "clip": True},
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts_fwd", "experts_bwd", "adamw"])
    if op == "adamw":
        tensors = _log(rng, 1, 600)
        return {"op": op, "state": rng.choice([8, 8, 32]), "tensors": tensors, "size": _log(rng, 100, 40_000_000 // tensors),
                "grad": rng.choice(["bf16", "fp32"]), "clip": rng.random() < 0.5}
    n, m = 64 * _log(rng, 2, 224), 64 * _log(rng, 2, 224) + rng.choice([0, 0, 0, 8, 3])
    E = _log(rng, 1, max(1, min(64, 8 * 14336 * 4096 // (n * m))))
    M = _log(rng, 1, max(1, min(16384, 8192 * 14336 * 4096 // (n * m))))
    case = {"op": op, "E": E, "idle": rng.randint(0, E - 1) // 2, "M": M, "n": n, "m": m, "r": rng.choice([4, 8, 16, 20, 32, 64, 128])}
    return {**case, "grad_x": rng.random() < 0.7} if op == "experts_bwd" else case


def _cuts(case):
    """First row of each expert, and the end: unequal shares of the rows, none for the idle experts."""
    E, M = case["E"], case["M"]
    idle = set(sorted(range(E), key=lambda e: (37 * e + 11) % 101)[:case["idle"]])
    weight = [0 if e in idle else 2 + (3 * e) % 5 for e in range(E)]
    return [M * sum(weight[:e]) // sum(weight) for e in range(E + 1)]


def _sizes(case):
    """Number of values of each trained tensor."""
    if "tensors" in case:
        return [max(1, case["size"] - (case["size"] * ((7 * i) % 10)) // 12 + i % 3) for i in range(case["tensors"])]
    hidden, kv, ffn, r = 4096, 1024, 14336, case["r"]
    feed = [(ffn, hidden), (ffn, hidden), (hidden, ffn)]
    layer = feed * case["experts"] if case["experts"] else [(hidden, hidden), (kv, hidden), (kv, hidden), (hidden, hidden)] + feed
    return [size for _ in range(case["layers"]) for m, n in layer for size in (r * n, m * r)]


def work(case):
    if case["op"] == "adamw":
        sizes = _sizes(case)
        total, blocks = sum(sizes), sum(-(-n // BLOCK) for n in sizes)
        # weight read and written, its bf16 copy written, gradient and both moments read, moments written (as codes and as values)
        cell = 8 + 2 + (2 if case["grad"] == "bf16" else 4) + (4 + 8 if case["state"] == 8 else 16)
        return {"bytes": total * cell + (16 * blocks if case["state"] == 8 else 0), "flops": 16 * total}
    cut = _cuts(case)
    live = sum(b > a for a, b in zip(cut, cut[1:]))
    M, n, m, r, E = case["M"], case["n"], case["m"], case["r"], case["E"]
    weight = live * (m * n // 2 + m * n // 64 + m * n // 4096)
    if case["op"] == "experts_fwd":
        return {"bytes": weight + 2 * M * (n + m) + 4 * M * r + 2 * live * r * (n + m), "flops": 2 * M * n * m + 2 * M * r * (n + m)}
    nbytes = 2 * M * (n + m) + 4 * M * r + 2 * live * r * m + 2 * E * r * (n + m)
    flops = 2 * M * m * r + 2 * M * r * (n + m)
    if case["grad_x"]:
        nbytes += weight + 2 * M * n + 2 * live * r * n
        flops += 2 * M * n * m + 2 * M * n * r
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------


def _root_code(x, most):
    """The k of 0 .. most whose square is nearest to x (float64, >= 0)."""
    k = x.sqrt().floor()
    return torch.where(x > k * k + k + 0.5, k + 1, k).clamp(max=most)


def _pack(m, v):
    """(codes, steps) of the two moments' 8-bit form; m, v float64, a whole number of blocks each."""
    m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
    tiny = 2.0 ** -126
    dm = (m.abs().amax(1) / 127 ** 2).float()
    dm = torch.where(dm < tiny, torch.zeros_like(dm), dm)
    dv = (v.amax(1).sqrt() / 255 ** 2).float()
    dv = torch.where(dv < tiny, torch.zeros_like(dv), dv)
    one = torch.ones((), dtype=torch.float64, device=m.device)
    k = _root_code(m.abs() / torch.where(dm > 0, dm.double(), one)[:, None], 127)
    k = torch.where((dm > 0)[:, None], k, torch.zeros_like(k))
    km = torch.where((m < 0) & (k > 0), k + 128, k).to(torch.uint8)
    k = _root_code(v.sqrt() / torch.where(dv > 0, dv.double(), one)[:, None], 255)
    k = torch.where(v > 0, k.clamp(min=1), k)
    kv = torch.where((dv > 0)[:, None], k, torch.zeros_like(k)).to(torch.uint8)
    return (km.view(-1), dm), (kv.view(-1), dv)


def _values(codes, steps, signed):
    """The moment that its 8-bit form stands for, in 64 bits."""
    c = codes.view(-1, BLOCK).double()
    d = steps.double()[:, None]
    if not signed:
        return (c * c * d).square().view(-1)
    k = torch.where(c >= 128, c - 128, c)
    return (torch.where(c >= 128, -k, k) * k * d).view(-1)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    st = {"case": case}
    if case["op"] == "adamw":
        # all tensors in one flat storage, each from a block's border on, zeros between them
        sizes = _sizes(case)
        room = [-(-n // BLOCK) * BLOCK for n in sizes]
        total = sum(room)
        # each value lies inside its tensor; the gradients' magnitudes differ from tensor to tensor
        inside = torch.arange(total, device=dev)
        start = torch.tensor(room, device=dev).cumsum(0) - torch.tensor(room, device=dev)
        which = torch.repeat_interleave(torch.arange(len(sizes), device=dev), torch.tensor(room, device=dev))
        inside = inside - start[which] < torch.tensor(sizes, device=dev)[which]
        scale = (10.0 ** (2 * torch.rand(len(sizes), generator=gen, device=dev)))[which] * inside
        scale *= 0.6 / (scale.double().square().sum().sqrt().float() * 1.3)  # gradients of norm 0.6 or so
        del which
        g = scale * torch.randn(total, generator=gen, device=dev) * torch.exp(0.5 * torch.randn(total, generator=gen, device=dev))
        m = 0.3 * scale * torch.randn(total, generator=gen, device=dev)
        v = (scale * (0.1 + torch.rand(total, generator=gen, device=dev))).square()
        p = 0.02 * torch.randn(total, generator=gen, device=dev) * inside
        del inside, scale
        st.update(p=p, p16=p.to(torch.bfloat16), g=g.to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32),
                  hyper=dict(lr=2e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=12), max_norm=0.3)
        if case["state"] == 8:
            st["m"], st["v"] = _pack(m.double(), v.double())
        else:
            st["m"], st["v"] = m, v
        if own:  # the prepared list of tensors, which a program keeps over its steps
            import bit_quantized_fine_qlora_amd as Q
            cut, tensors = 0, []
            for n, w in zip(sizes, room):
                def part(t):
                    return t[cut:cut + n]
                if case["state"] == 8:
                    blocks = slice(cut // BLOCK, (cut + w) // BLOCK)
                    mv = [Q.Moment8(part(c), d[blocks], signed) for (c, d), signed in ((st["m"], True), (st["v"], False))]
                else:
                    mv = [part(st["m"]), part(st["v"])]
                tensors.append((part(p), part(st["p16"]), part(st["g"]), *mv))
                cut += w
            st["step"] = Q.AdamWStep(tensors)
        return st
    M, n, m, r, E = case["M"], case["n"], case["m"], case["r"], case["E"]
    cut = _cuts(case)
    # a normal weight's codes are equally likely and its block maxima near 2.4 deviations
    st.update(cut=cut, offsets=torch.tensor(cut, dtype=torch.int32, device=dev), s=0.25,
              x=normal(M, n) * torch.exp(0.5 * normal(n)), A=normal(E, r, n, scale=1 / 16), B=normal(E, m, r, scale=0.01),
              codes=torch.randint(0, 256, (E * m * n // 2,), generator=gen, device=dev, dtype=torch.uint8),
              absmax8=torch.randint(0x2e, 0x39, (E * m * n // 64,), generator=gen, device=dev, dtype=torch.uint8),
              c2=0.06 + 0.01 * torch.rand(-(-E * m * n // 16384), generator=gen, device=dev))
    if case["op"] == "experts_bwd":
        u = torch.cat([st["x"][a:b].float() @ st["A"][e].float().t() for e, (a, b) in enumerate(zip(cut, cut[1:]))])
        st.update(g=normal(M, m), u=u)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------


def _weight(st, e):
    """Expert e's frozen weight: 4-bit sign-magnitude codes, 8 to a word, over doubly quantized block scales, rounded to bf16."""
    case = st["case"]
    m, n = case["m"], case["n"]
    blocks = m * n // 64
    by = st["codes"][e * m * n // 2:(e + 1) * m * n // 2].view(-1, 4)
    code = torch.cat([by & 15, by >> 4], 1).view(-1).to(torch.int32)  # byte j: weight j, weight j + 4
    upper = torch.tensor(LEVELS[8:], dtype=torch.float32, device=by.device)
    block = torch.arange(e * blocks, (e + 1) * blocks, device=by.device)
    scale = st["absmax8"][e * blocks:(e + 1) * blocks].view(torch.float8_e4m3fn).float() * st["c2"][block >> 8]
    w = torch.cat([upper, -upper])[code].view(-1, 64) * scale[:, None]
    return w.to(torch.bfloat16).float().view(m, n)


def _plain_experts_fwd(st):
    x, s, h, u = st["x"].float(), st["s"], [], []
    for e, (a, b) in enumerate(zip(st["cut"], st["cut"][1:])):
        if b > a:
            u.append(x[a:b] @ st["A"][e].float().t())
            h.append((x[a:b] @ _weight(st, e).t() + s * (u[-1] @ st["B"][e].float().t())).to(torch.bfloat16))
    return {"h": torch.cat(h), "u": torch.cat(u)}


def _plain_experts_bwd(st):
    case, x, g, u, s = st["case"], st["x"].float(), st["g"].float(), st["u"], st["s"]
    gA, gB, gx = torch.zeros_like(st["A"]), torch.zeros_like(st["B"]), []
    for e, (a, b) in enumerate(zip(st["cut"], st["cut"][1:])):
        if b > a:
            v = g[a:b] @ st["B"][e].float()
            gA[e] = (s * (v.t() @ x[a:b])).to(torch.bfloat16)
            gB[e] = (s * (g[a:b].t() @ u[a:b])).to(torch.bfloat16)
            if case["grad_x"]:
                gx.append((g[a:b] @ _weight(st, e) + s * (v @ st["A"][e].float())).to(torch.bfloat16))
    out = {"grad_A": gA, "grad_B": gB}
    return {**out, "grad_x": torch.cat(gx)} if case["grad_x"] else out


def _plain_adamw(st):
    hp, eight = st["hyper"], st["case"]["state"] == 8
    out = {}
    g = st["g"].double()  # the 8-bit codes go by which of two values is nearer: everything they depend on in 64 bits
    if st["case"]["clip"]:
        norm = g.square().sum().sqrt()
        factor = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        g = g * factor.double()
        out.update(norm=norm.float(), factor=factor)
    b1, b2 = hp["beta1"], hp["beta2"]
    m = _values(*st["m"], True) if eight else st["m"]
    v = _values(*st["v"], False) if eight else st["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g.square()
    if eight:
        (cm, dm), (cv, dv) = _pack(m, v)
        for (code, step), new in ((st["m"], (cm, dm)), (st["v"], (cv, dv))):
            code.copy_(new[0])
            step.copy_(new[1])
        out.update(m=_values(cm, dm, True).float(), v=_values(cv, dv, False).float())
    else:
        out.update(m=st["m"].copy_(m), v=st["v"].copy_(v))
    c1, c2 = 1 - b1 ** hp["step"], 1 - b2 ** hp["step"]
    p = st["p"] * (1 - hp["lr"] * hp["weight_decay"]) - ((hp["lr"] / c1) * (m / ((v / c2).sqrt() + hp["eps"]))).float()
    return {**out, "p": st["p"].copy_(p), "p16": st["p16"].copy_(p)}


def run(st):
    case = st["case"]
    if not own:
        return {"experts_fwd": _plain_experts_fwd, "experts_bwd": _plain_experts_bwd, "adamw": _plain_adamw}[case["op"]](st)
    import bit_quantized_fine_qlora_amd as Q
    if case["op"] == "adamw":
        out, clip = {}, None
        if case["clip"]:
            clip = st["step"].clip(st["max_norm"])
            out.update(norm=clip[0], factor=clip[1])
        st["step"].run(**st["hyper"], clip=clip)
        out.update(m=st["m"], v=st["v"], p=st["p"], p16=st["p16"])
        if case["state"] == 8:
            out.update(m=Q.moment8_values(Q.Moment8(*st["m"], True)), v=Q.moment8_values(Q.Moment8(*st["v"], False)))
        return out
    q = Q.QuantizedWeight(st["codes"], st["absmax8"], st["c2"], case["E"] * case["m"], case["n"])
    if case["op"] == "experts_fwd":
        h, u = Q.experts_fwd(st["x"], st["offsets"], q, st["A"], st["B"], st["s"])
        return {"h": h, "u": u}
    gx, gA, gB = Q.experts_bwd(st["x"], st["g"], st["offsets"], q, st["A"], st["B"], st["s"], u=st["u"], need_grad_x=case["grad_x"])
    out = {"grad_A": gA, "grad_B": gB}
    return {**out, "grad_x": gx} if case["grad_x"] else out


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------


def _exact_moment(x, most):
    """The k of each of x (float64, >= 0; one block a row) as the nearest k^2 d, and the blocks' d."""
    d = (x.max(1).values / most ** 2).to(torch.float32).double()[:, None]
    k = torch.arange(most, dtype=torch.float64, device=x.device)
    border = k * k + k + 0.5  # between k^2 and (k + 1)^2; a value on it stays below
    code = torch.bucketize(x / torch.where(d > 0, d, torch.ones_like(d)), border)
    return code.double(), d


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        hp, out = st["hyper"], {}
        g = st["g"].double()
        if case["clip"]:
            norm = torch.linalg.vector_norm(g)
            factor = min(1.0, st["max_norm"] / (float(norm) + 1e-6))
            factor = torch.tensor(factor, dtype=torch.float32).item()  # what the step reads is an fp32 number
            g = g * factor
            out = {"norm": norm, "factor": factor}
        if case["state"] == 8:
            (cm, dm), (cv, dv) = st["m"], st["v"]
            m = (cm.view(-1, BLOCK) & 127).double() ** 2 * torch.where(cm.view(-1, BLOCK) > 127, -1.0, 1.0) * dm.double()[:, None]
            v = (cv.view(-1, BLOCK).double() ** 2 * dv.double()[:, None]) ** 2
            m, v = m.view(-1), v.view(-1)
        else:
            m, v = st["m"].double(), st["v"].double()
        m = torch.lerp(g, m, hp["beta1"])
        v = torch.lerp(g * g, v, hp["beta2"])
        mhat, vhat = m / (1 - hp["beta1"] ** hp["step"]), v / (1 - hp["beta2"] ** hp["step"])
        p = st["p"].double()
        p = p - hp["lr"] * hp["weight_decay"] * p - hp["lr"] * mhat / (torch.sqrt(vhat) + hp["eps"])
        if case["state"] == 8:
            k, d = _exact_moment(m.abs().view(-1, BLOCK), 127)
            m = (torch.sign(m.view(-1, BLOCK)) * k * k * d).view(-1)
            k, d = _exact_moment(v.sqrt().view(-1, BLOCK), 255)
            k = torch.where((k == 0) & (v.view(-1, BLOCK) > 0), torch.ones_like(k), k)
            v = ((k * k * d) ** 2).view(-1)
        return {**out, "m": m, "v": v, "p": p, "p16": p}
    cut, s, n, m = st["cut"], st["s"], case["n"], case["m"]
    cells = m * n
    mag = torch.tensor(LEVELS[8:], dtype=torch.float64, device="cuda").float()

    def weight(e):
        # bit 3 of a code is its sign, bits 0-2 the rank of its magnitude among the 8 upper levels
        word = st["codes"][e * cells // 2:(e + 1) * cells // 2].view(-1, 4).long()
        code = torch.stack([word & 15, word >> 4], 1).reshape(-1)
        a = st["absmax8"].long()
        a = (torch.exp2(((a >> 3) - 7).double()) * (1 + (a & 7).double() / 8)).float()
        blk = (a * st["c2"].repeat_interleave(256)[:a.numel()])[e * cells // 64:(e + 1) * cells // 64]
        w = (mag[code & 7].view(-1, 64) * blk[:, None]).to(torch.bfloat16).double().reshape(-1)
        return torch.where(code >= 8, -w, w).view(m, n)

    spans = [(e, slice(cut[e], cut[e + 1])) for e in range(case["E"]) if cut[e + 1] > cut[e]]
    x = st["x"].double()
    if case["op"] == "experts_fwd":
        u = torch.cat([x[t] @ st["A"][e].double().t() for e, t in spans])
        h = torch.cat([torch.cat([x[t], s * u[t]], 1) @ torch.cat([weight(e), st["B"][e].double()], 1).t() for e, t in spans])
        return {"h": h, "u": u}
    g, u = st["g"].double(), st["u"].double()
    gA = torch.zeros(st["A"].shape, dtype=torch.float64, device=x.device)
    gB = torch.zeros(st["B"].shape, dtype=torch.float64, device=x.device)
    for e, t in spans:
        gA[e] = s * st["B"][e].double().t() @ g[t].t() @ x[t]
        gB[e] = s * (g[t].t() @ u[t])
    out = {"grad_A": gA, "grad_B": gB}
    if case["grad_x"]:
        out["grad_x"] = torch.cat([g[t] @ (weight(e) + s * st["B"][e].double() @ st["A"][e].double()) for e, t in spans])
    return out
