"""What is measured of the causal operators: the selective scan and its short convolution
(prompts, single tokens, training), and clipping by the gradients' common norm.

Every case names an operator (``op``), its sizes and its element type.  ``run`` computes
it in plain torch operations (``own`` false) or through vision_mamba_selective_b200.vimscan
(``own`` true); ``exact`` computes it once more in 64 bits, token by token.
"""
import math

import torch

own = False

EPS = 1e-6   # added to the norm before the division, so that a zero norm divides by something


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def listed():
    bf, f32 = "bf16", "f32"
    return [
        # one token of one sequence, the smallest serving call: all latency
        dict(name="conv_step_1x2048_bf16", op="conv_step", batch=1, d=2048, width=4, slots=8, dtype=bf),
        # a mixed batch of prompts, packed, x being half of a wider projection; states kept by slot
        dict(name="conv_prompt_8192x2048_bf16_ragged", op="conv_prompt", nseq=11, L=8192, d=2048, width=4, dtype=bf),
        # training at the 1024 px sequence length of the repository's workloads: forward and gradients
        dict(name="conv_train_8x4097x384_bf16", op="conv_train", batch=8, nseq=0, L=4097, d=384, width=4, dtype=bf),
        # one token of one sequence through the scan: all latency
        dict(name="scan_step_1x2048_bf16", op="scan_step", batch=1, d=2048, N=16, slots=8, dtype=bf),
        # one token of each of 256 sequences: the state cache's traffic
        dict(name="scan_step_256x4096_bf16", op="scan_step", batch=256, d=4096, N=16, slots=300, dtype=bf),
        # the repository's 224 px sequence in fp32: a short sequence, one wave of little work
        dict(name="scan_prompt_1x197x384_f32", op="scan_prompt", batch=1, nseq=0, L=197, d=384, N=16, gate=True, dtype=f32),
        # the repository's longest workload (2048 px), few channels and many tokens
        dict(name="scan_prompt_4x16385x384_bf16", op="scan_prompt", batch=4, nseq=0, L=16385, d=384, N=16, gate=True,
             dtype=bf),
        # a mixed batch of prompts, packed: some continue from a kept state, some are fresh
        dict(name="scan_prompt_8192x2048_bf16_ragged", op="scan_prompt", batch=1, nseq=11, L=8192, d=2048, N=16,
             gate=True, dtype=bf),
        # a short training step in fp32
        dict(name="scan_train_2x197x384_f32", op="scan_train", batch=2, nseq=0, L=197, d=384, N=16, gate=True, dtype=f32),
        # training at the repository's 1024 px workload: forward and all gradients
        dict(name="scan_train_8x4097x384_bf16", op="scan_train", batch=8, nseq=0, L=4097, d=384, N=16, gate=True,
             dtype=bf),
        # gradients of a few small blocks in fp32: many tensors, little data
        dict(name="clip_6x192_f32", op="clip", layers=6, model=192, inner=384, N=16, vocab=0, max_norm=1.0, dtype=f32),
        # gradients of a large stack, weights in bf16 and the scan's parameters in fp32
        dict(name="clip_10x2048_bf16", op="clip", layers=10, model=2048, inner=4096, N=16, vocab=32000, max_norm=1.0,
             dtype=bf),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_prompt", "conv_train", "scan_step", "scan_prompt", "scan_prompt", "scan_train",
                     "scan_train", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    # channel counts: mostly whole vectors, some odd
    d = _log(rng, 24, 4096)
    d = d if rng.random() < 0.3 else max(8, d // 8 * 8)
    N = rng.choice([16, 16, 16, 8, 4, 2])
    if op in ("conv_step", "scan_step"):
        batch = _log(rng, 1, 256)
        case = dict(op=op, batch=batch, d=d, slots=batch + rng.randrange(1, 40), dtype=dtype)
        case.update(dict(width=rng.choice([2, 3, 4])) if op == "conv_step" else dict(N=N))
        return case
    if op == "clip":
        model = _log(rng, 64, 2048)
        return dict(op=op, layers=rng.randrange(1, 11), model=model, inner=2 * model + rng.randrange(0, 3), N=N,
                    vocab=rng.choice([0, _log(rng, 100, 32000)]), max_norm=rng.choice([0.1, 1.0, 1e6]), dtype=dtype)
    # tokens: what the channels leave of the largest listed case's token-channels
    most = {"conv_prompt": 16e6, "conv_train": 12e6, "scan_prompt": 16e6, "scan_train": 6e6}[op]
    L = _log(rng, 1, max(2, min(12000, most / d)))
    packed = rng.random() < 0.5
    batch = 1 if packed or L * d * 2 > most else rng.randrange(1, max(2, min(16, int(most / (L * d)))))
    case = dict(op=op, batch=batch, nseq=rng.randrange(1, 24) if packed else 0, L=L, d=d, dtype=dtype)
    if op == "conv_prompt":
        case["nseq"] = max(1, case["nseq"])
        case.pop("batch")
    if op.startswith("conv"):
        case["width"] = rng.choice([2, 3, 4])
    else:
        case.update(N=N, gate=rng.random() < 0.8)
    return case


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _cu_seqlens(total, nseq, seed):
    """Ragged lengths that sum to ``total``: spread over a wide range, one of length one and
    one empty among them where there are enough."""
    g = torch.Generator().manual_seed(seed)
    share = torch.exp(torch.randn(nseq, generator=g, dtype=torch.float64))
    if nseq > 4:
        share[1] = 0.0
    edges = torch.round(torch.cumsum(share, 0) / share.sum() * total).to(torch.int64)
    if nseq > 4 and total > 8:
        edges[3] = min(int(edges[2]) + 1, total)
    edges = torch.cummax(edges, 0).values
    edges[-1] = total
    return torch.cat([torch.zeros(1, dtype=torch.int64), edges]).to(torch.int32)


def _gradient_shapes(case):
    """A stack's gradients as a mixer block has them: two projections and the scan's
    parameters per layer, and the embedding."""
    m, i, n = case["model"], case["inner"], case["N"]
    shapes = []
    for _ in range(case["layers"]):
        shapes += [((2 * i, m), True), ((i, 4), False), ((i, 2 * n + 1), True), ((i, n), False), ((i,), False),
                   ((m, i), True)]
    if case["vocab"]:
        shapes.append(((case["vocab"], m), True))
    return shapes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    io = _type(case)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=io):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = dict(case=case)
    if op == "clip":
        s["grads"] = [normal(*shape, std=0.01, dtype=io if wide else torch.float32)
                      for shape, wide in _gradient_shapes(case)]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        return s
    d = case["d"]
    single = op.endswith("step")
    packed = not single and case["nseq"] > 0
    rows = (case["batch"],) if single else (case["L"],) if packed else (case["batch"], case["L"])
    # x (or u's neighbour) and the gate z are halves of one projection: rows 2 d apart
    xz = normal(*rows, 2 * d)
    s["z"] = xz[..., d:]
    f32 = torch.float32
    if packed:
        s["cu"] = _cu_seqlens(case["L"], case["nseq"], seed).cuda()
    if single:
        # distinct slots of a larger cache, in no order
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:case["batch"]].to(torch.int32)
    elif packed:
        s["slots"] = torch.randperm(case["nseq"] + 3, generator=g, device="cuda")[:case["nseq"]].to(torch.int32)
        s["fresh"] = uniform(case["nseq"]) < 0.5
    cache = case["slots"] if single else case["nseq"] + 3 if packed else 0
    if op.startswith("conv"):
        w = case["width"]
        s["x"] = xz[..., :d]
        s["w"] = (uniform(d, w) * 2 - 1) / math.sqrt(w)
        s["b"] = (uniform(d) * 2 - 1) / math.sqrt(w)
        if op != "conv_train":
            s["state"] = normal(cache, w - 1, d)
            s["state_out"] = torch.zeros_like(s["state"])
        else:
            s["dout"] = normal(*rows, d)
        return s
    N = case["N"]
    s["u"] = normal(*rows, d)
    s["delta"] = normal(*rows, d, std=0.5)
    # B and C are columns of one projection, behind the columns that give delta
    r = max(8, d // 16 // 8 * 8)
    proj = normal(*rows, r + 2 * N)
    s["B"], s["C"] = proj[..., r:r + N], proj[..., r + N:]
    if not case.get("gate", True):
        s["z"] = None
    # trained-like decays around -(n + 1); softplus(bias) log-uniform in [1e-3, 1e-1]
    s["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=f32) * torch.exp(normal(d, N, std=0.2, dtype=f32)))
    s["D"] = 1 + normal(d, std=0.1, dtype=f32)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * uniform(d).double())
    s["bias"] = torch.log(torch.expm1(step)).float()
    if op == "scan_train":
        s["dout"] = normal(*rows, d)
        s.pop("fresh", None), s.pop("slots", None)
    elif cache:
        s["state"] = normal(cache, d, N, std=0.3, dtype=f32)
        s["state_out"] = torch.zeros_like(s["state"])
    return s


# --------------------------------------------------------------------------------------
# plain forms: 32 bits, whole tensors at a time
# --------------------------------------------------------------------------------------
def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def _prefix(a, b):
    """h_t = a_t h_(t-1) + b_t for all t of dimension 1 of [rows, t, d, N], by doubling.
    Both arguments are overwritten; returns h."""
    k, L = 1, a.shape[1]
    while k < L:
        b[:, k:] += a[:, k:] * b[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return b


def _starts(s, rows, L):
    """Per token of [rows, L]: whether a sequence starts there, and which sequence it is in."""
    if "cu" not in s:
        first = torch.zeros(rows, L, dtype=torch.bool, device="cuda")
        first[:, :1] = True
        return first, None
    t = torch.arange(L, device="cuda")
    cu = s["cu"].long()
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return (t == cu[seq])[None], seq


def _plain_scan(s, gradients):
    u, delta, B, C = (s[k].float() for k in ("u", "delta", "B", "C"))
    z = None if s["z"] is None else s["z"].float()
    if u.dim() == 2:
        u, delta, B, C = u[None], delta[None], B[None], C[None]
        z = None if z is None else z[None]
    A, D, bias = s["A"], s["D"], s["bias"]
    rows, L = u.shape[:2]
    first, seq = _starts(s, rows, L)
    raw = delta + bias
    step = _softplus(raw)
    a = torch.exp(step[..., None] * A)
    a[first] = 0.0
    b = (step * u)[..., None] * B[:, :, None, :]
    slots, state_out = s.get("slots"), s.get("state_out")
    if slots is not None:
        start = s["state"][slots.long()]
        start = torch.where(s["fresh"][:, None, None], torch.zeros_like(start), start)
        cu = s["cu"].long()
        some = cu[1:] > cu[:-1]
        at = cu[:-1][some]
        b[0, at] += torch.exp(step[0, at][..., None] * A) * start[some]
    h = _prefix(a.clone() if gradients else a, b)
    y = (C[:, :, None, :] * h).sum(-1) + D * u
    gated = y if z is None else y * (z / (1 + torch.exp(-z)))
    io = s["u"].dtype
    out = dict(y=gated.to(io).reshape(s["u"].shape))
    if slots is not None:
        last = torch.where(some[:, None, None], h[0, torch.clamp(cu[1:] - 1, min=0)], start)
        state_out[slots.long()] = last
        out["state"] = state_out
    if not gradients:
        return out
    dout = s["dout"].float().reshape(u.shape)
    dy = dout
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        dy = dout * z * sg
        out["dz"] = (dout * y * sg * (1 + z * (1 - sg))).to(io).reshape(s["u"].shape)
    # adjoint: g_t = C_t dy_t + a_(t+1) g_(t+1)
    back = torch.zeros_like(a)
    back[:, 1:] = a[:, 1:].flip(1)
    g = _prefix(back, (C[:, :, None, :] * dy[..., None]).flip(1)).flip(1)
    out["dC"] = (dy[..., None] * h).sum(2).reshape(s["B"].shape)
    out["dB"] = ((step * u)[..., None] * g).sum(2).reshape(s["B"].shape)
    gB = (g * B[:, :, None, :]).sum(-1)
    out["du"] = (step * gB + D * dy).to(io).reshape(s["u"].shape)
    # what the decay passes on: a_t h_(t-1)
    kept = torch.zeros_like(h)
    kept[:, 1:] = a[:, 1:] * h[:, :-1]
    g *= kept
    dstep = (g * A).sum(-1) + u * gB
    dlt = dstep / (1 + torch.exp(-raw))
    out["ddelta"] = dlt.to(io).reshape(s["u"].shape)
    out["dA"] = (g * step[..., None]).sum((0, 1), dtype=torch.float64).float()
    out["dD"] = (dy * u).sum((0, 1), dtype=torch.float64).float()
    out["ddelta_bias"] = dlt.sum((0, 1), dtype=torch.float64).float()
    return out


def _plain_scan_step(s):
    u, delta, z, B, C = (s[k].float() for k in ("u", "delta", "z", "B", "C"))
    step = _softplus(delta + s["bias"])
    at = s["slots"].long()
    h = torch.exp(step[..., None] * s["A"]) * s["state"][at] + (step * u)[..., None] * B[:, None, :]
    s["state_out"][at] = h
    y = (C[:, None, :] * h).sum(-1) + s["D"] * u
    return dict(y=(y * (z / (1 + torch.exp(-z)))).to(s["u"].dtype), state=s["state_out"])


def _silu(v):
    return v / (1 + torch.exp(-v))


def _taps(s):
    """x k tokens back, per tap of the convolution and token, zero (or a state row) before
    the sequence: [width, rows, L, d] in 32 bits, the newest tap last."""
    x = s["x"].float()
    x = x[None] if x.dim() == 2 else x
    rows, L = x.shape[:2]
    W = s["w"].shape[1]
    t = torch.arange(L, device="cuda")
    if "cu" in s:
        _, seq = _starts(s, rows, L)
        since = t - s["cu"].long()[seq]
    else:
        since = t
    back = torch.arange(W - 1, -1, -1, device="cuda")[:, None]
    inside = since[None] >= back
    taps = x[:, torch.clamp(t[None] - back, min=0)].permute(1, 0, 2, 3) * inside[:, None, :, None]
    if "slots" in s and "fresh" in s:
        start = s["state"].float()[s["slots"].long()] * (~s["fresh"])[:, None, None]
        row = torch.clamp(W - 1 - back + since[None], max=W - 2)
        taps[:, 0] += start[seq[None].expand_as(row), row] * ~inside[..., None]
    return taps


def _plain_conv_prompt(s):
    taps = _taps(s)
    w = s["w"]
    y = _silu((taps * w.t()[:, None, None, :]).sum(0) + s["b"])
    # the last width - 1 inputs of each sequence, older state rows where it is shorter
    W = w.shape[1]
    cu = s["cu"].long()
    at = s["slots"].long()
    n = (cu[1:] - cu[:-1])[:, None]
    old = s["state"][at] * (~s["fresh"])[:, None, None]
    row = n + torch.arange(W - 1, device="cuda")[None]      # position in [state rows, sequence]
    held = torch.gather(old, 1, torch.clamp(row, max=W - 2)[..., None].expand(-1, -1, old.shape[2]))
    new = s["x"][torch.clamp(cu[:-1, None] + row - (W - 1), 0, s["x"].shape[0] - 1)]
    s["state_out"][at] = torch.where((row < W - 1)[..., None], held, new)
    return dict(y=y[0].to(s["x"].dtype), state=s["state_out"])


def _plain_conv_train(s):
    taps = _taps(s)
    w = s["w"]
    W = w.shape[1]
    pre = (taps * w.t()[:, None, None, :]).sum(0) + s["b"]
    sg = 1 / (1 + torch.exp(-pre))
    io, shape = s["x"].dtype, s["x"].shape
    dpre = s["dout"].float().reshape(pre.shape) * sg * (1 + pre * (1 - sg))
    L = pre.shape[1]
    # the tap of age k reads x_(t-k): x_t gets it from token t + k of the same sequence
    t = torch.arange(L, device="cuda")
    end = s["cu"].long()[1:][_starts(s, 1, L)[1]] if "cu" in s else torch.full_like(t, L)
    ahead = torch.arange(W - 1, -1, -1, device="cuda")[:, None]
    inside = t[None] + ahead < end[None]
    fed = dpre[:, torch.clamp(t[None] + ahead, max=L - 1)].permute(1, 0, 2, 3) * inside[:, None, :, None]
    dx = (fed * w.t()[:, None, None, :]).sum(0)
    dw = (taps * dpre).sum((1, 2), dtype=torch.float64).t().float().contiguous()
    return dict(y=(pre * sg).to(io).reshape(shape), dx=dx.to(io).reshape(shape), dw=dw,
                db=dpre.sum((0, 1), dtype=torch.float64).float())


def _plain_conv_step(s):
    at = s["slots"].long()
    past = torch.cat([s["state"][at], s["x"][:, None]], 1)
    y = _silu((past.float() * s["w"].t()[None]).sum(1) + s["b"])
    s["state_out"][at] = past[:, 1:]
    return dict(y=y.to(s["x"].dtype), state=s["state_out"])


def _plain_clip(s):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = total.sqrt()
    factor = torch.clamp(s["case"]["max_norm"] / (norm + EPS), max=1.0).float()
    out = [(t.float() * factor).to(t.dtype) for t in s["grads"]]
    return dict(norm=norm.float().reshape(1), out=out)


# --------------------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------------------
def _own(s):
    from vision_mamba_selective_b200 import vimscan as vs

    op = s["case"]["op"]
    if op == "clip":
        norm = vs.clip_grad_norm(s["grads"], s["case"]["max_norm"], out=s["out"])
        return dict(norm=norm, out=s["out"])
    if op == "conv_step":
        y = vs.causal_conv_step(s["x"], s["w"], s["b"], s["state"], state_out=s["state_out"], slots=s["slots"])
        return dict(y=y, state=s["state_out"])
    if op == "conv_prompt":
        y = vs.causal_conv(s["x"], s["w"], s["b"], cu_seqlens=s["cu"], state=s["state"], state_out=s["state_out"],
                           slots=s["slots"], fresh=s["fresh"])
        return dict(y=y, state=s["state_out"])
    if op == "conv_train":
        y = vs.causal_conv(s["x"], s["w"], s["b"], cu_seqlens=s.get("cu"))
        g = vs.causal_conv_bwd(s["x"], s["w"], s["b"], s["dout"], cu_seqlens=s.get("cu"))
        return dict(y=y, dx=g["dx"], dw=g["dw"], db=g["db"])
    args = [s[k] for k in ("u", "delta", "z", "B", "C", "A", "D", "bias")]
    if op == "scan_step":
        y = vs.causal_scan_step(*args, s["state"], state_out=s["state_out"], slots=s["slots"])
        return dict(y=y, state=s["state_out"])
    if op == "scan_prompt":
        if "state" not in s:
            return dict(y=vs.causal_scan(*args))
        y = vs.causal_scan(*args, cu_seqlens=s["cu"], state=s["state"], state_out=s["state_out"], slots=s["slots"],
                           fresh=s["fresh"])
        return dict(y=y, state=s["state_out"])
    rows = s["u"].shape[:-1]
    ckpt = torch.empty(vs.causal_ckpt_shape(1 if len(rows) == 1 else rows[0], rows[-1], s["u"].shape[-1],
                                            s["B"].shape[-1]), device="cuda")
    y = vs.causal_scan(*args, cu_seqlens=s.get("cu"), ckpt=ckpt)
    g = vs.causal_scan_bwd(*args, s["dout"], cu_seqlens=s.get("cu"), ckpt=ckpt)
    out = {k: g[k] for k in ("du", "ddelta", "dB", "dC", "dA", "dD", "ddelta_bias")}
    out["y"] = y
    if s["z"] is not None:
        out["dz"] = g["dz"]
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "clip":
        return _plain_clip(state)
    if op == "conv_step":
        return _plain_conv_step(state)
    if op == "conv_prompt":
        return _plain_conv_prompt(state)
    if op == "conv_train":
        return _plain_conv_train(state)
    if op == "scan_step":
        return _plain_scan_step(state)
    return _plain_scan(state, op == "scan_train")


# --------------------------------------------------------------------------------------
# work
# --------------------------------------------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "clip":
        count = [(math.prod(shape), e if wide else 4) for shape, wide in _gradient_shapes(case)]
        return dict(bytes=sum(2 * n * b for n, b in count), flops=sum(3 * n for n, _ in count))
    d = case["d"]
    if op == "conv_step":
        w, n = case["width"], case["batch"] * d
        return dict(bytes=n * e * (2 + 2 * (w - 1)) + d * (w + 1) * 4, flops=n * (2 * w + 4))
    if op == "scan_step":
        N, n = case["N"], case["batch"] * d
        return dict(bytes=n * (4 * e + 8 * N) + case["batch"] * 2 * N * e + d * (N + 2) * 4, flops=n * (7 * N + 12))
    tokens = case.get("batch", 1) * case["L"]
    n = tokens * d
    kept = 2 * case["nseq"] * d
    if op.startswith("conv"):
        w = case["width"]
        params = d * (w + 1) * 4
        if op == "conv_prompt":
            return dict(bytes=n * 2 * e + kept * (w - 1) * e + params, flops=n * (2 * w + 4))
        # forward: x, y; gradients: x, dout, dx
        return dict(bytes=n * 5 * e + 3 * params, flops=n * (8 * w + 14))
    N = case["N"]
    gate = 1 if case["gate"] else 0
    params = d * (N + 2) * 4
    if op == "scan_prompt":
        return dict(bytes=n * e * (3 + gate) + tokens * 2 * N * e + kept * N * 4 + params, flops=n * (7 * N + 12))
    # forward: u, delta, z, y; gradients: u, delta, z, dout and du, ddelta, dz
    return dict(bytes=n * e * (3 + gate + 5 + 2 * gate) + tokens * 2 * N * (2 * e + 4) + 3 * params,
                flops=n * (7 * N + 12 + 22 * N + 30))


# --------------------------------------------------------------------------------------
# the definitions in 64 bits, token by token
# --------------------------------------------------------------------------------------
def _exact_scan(s, gradients):
    f = lambda k: None if s.get(k) is None else s[k].double()
    leaf = {k: f(k) for k in ("u", "delta", "z", "B", "C", "A", "D", "bias")}
    if gradients:
        leaf = {k: None if v is None else v.clone().requires_grad_() for k, v in leaf.items()}
    u, delta, z, B, C, A, D, bias = (leaf[k] for k in ("u", "delta", "z", "B", "C", "A", "D", "bias"))
    if u.dim() == 2:
        cu = s["cu"].tolist()
        bounds = list(zip(cu[:-1], cu[1:]))
    else:
        bounds = [(0, u.shape[1])]
    step = torch.nn.functional.softplus(delta + bias, threshold=700)
    pieces, last = [], []
    for q, (t0, t1) in enumerate(bounds):
        h = torch.zeros(u.shape[:-2] + A.shape, dtype=torch.float64, device="cuda")
        if "state" in s and not bool(s["fresh"][q]):
            h = s["state"][int(s["slots"][q])].double()
        for t in range(t0, t1):
            st = step[..., t, :, None]
            h = torch.exp(st * A) * h + st * u[..., t, :, None] * B[..., t, None, :]
            pieces.append((h * C[..., t, None, :]).sum(-1))
        last.append(h)
    y = torch.stack(pieces, -2) + D * u
    if z is not None:
        y = y * torch.nn.functional.silu(z)
    out = dict(y=y.detach())
    if "state" in s:
        kept = torch.zeros_like(s["state"], dtype=torch.float64)
        kept[s["slots"].long()] = torch.stack(last)
        out["state"] = kept
    if gradients:
        named = {k: v for k, v in leaf.items() if v is not None}
        got = torch.autograd.grad(y, list(named.values()), s["dout"].double())
        out.update({{"bias": "ddelta_bias"}.get(k, "d" + k): v for k, v in zip(named, got)})
    return out


def _exact_conv(s, gradients):
    x, w, b = (s[k].double() for k in ("x", "w", "b"))
    if gradients:
        x, w, b = (t.clone().requires_grad_() for t in (x, w, b))
    W = w.shape[1]
    if x.dim() == 2:
        cu = s["cu"].tolist()
        parts = [x[t0:t1] for t0, t1 in zip(cu[:-1], cu[1:])]
    else:
        parts = list(x)
    ys, last = [], []
    for q, part in enumerate(parts):
        before = torch.zeros(W - 1, x.shape[-1], dtype=torch.float64, device="cuda")
        if "state" in s and not bool(s["fresh"][q]):
            before = s["state"][int(s["slots"][q])].double()
        ext = torch.cat([before, part], 0)
        pre = sum(ext[k:k + part.shape[0]] * w[:, k] for k in range(W)) + b
        ys.append(torch.nn.functional.silu(pre))
        last.append(ext[ext.shape[0] - (W - 1):])
    y = torch.cat(ys, 0) if x.dim() == 2 else torch.stack(ys)
    out = dict(y=y.detach())
    if "state" in s:
        kept = torch.zeros_like(s["state"], dtype=torch.float64)
        kept[s["slots"].long()] = torch.stack(last)
        out["state"] = kept
    if gradients:
        out["dx"], out["dw"], out["db"] = torch.autograd.grad(y, [x, w, b], s["dout"].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        grads = [t.double() for t in s["grads"]]
        norm = math.sqrt(math.fsum(float(torch.dot(t.reshape(-1), t.reshape(-1))) for t in grads))
        factor = min(1.0, case["max_norm"] / (norm + EPS))
        return dict(norm=torch.tensor([norm], dtype=torch.float64), out=[t * factor for t in grads])
    if op.endswith("step"):
        # one token is a prompt of length one for each row's slot
        n = case["batch"]
        s["cu"] = torch.arange(n + 1, dtype=torch.int32)
        s["fresh"] = torch.zeros(n, dtype=torch.bool)
    if op.startswith("conv"):
        return _exact_conv(s, op == "conv_train")
    return _exact_scan(s, op == "scan_train")
