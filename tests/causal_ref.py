"""The causal operators' definitions in plain Python loops over tokens, in fp64 on the CPU,
for the tests: no vectorised recurrence and no code in common with the library."""
import torch

F64 = torch.float64


def softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def bounds(x, cu):
    """(batch row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    return [(None, cu[s], cu[s + 1]) for s in range(len(cu) - 1)]


def scan(u, delta, z, B, C, A, D, bias, cu=None, starts=None):
    """(y, final states): y zero where no sequence is; ``starts`` [n_seqs, d, N] or None.
    Differentiable in every tensor argument."""
    u, delta, B, C, A, D, bias = (t.to(F64) for t in (u, delta, B, C, A, D, bias))
    z = None if z is None else z.to(F64)
    rows, last = {}, []
    for s, (b, t0, t1) in enumerate(bounds(u, cu)):
        h = torch.zeros_like(A) if starts is None else starts[s].to(F64)
        for t in range(t0, t1):
            at = t if b is None else (b, t)
            dt = softplus(delta[at] + bias)
            h = torch.exp(dt[:, None] * A) * h + (dt * u[at])[:, None] * B[at]
            y = (h * C[at]).sum(-1) + D * u[at]
            if z is not None:
                y = y * z[at] / (1 + torch.exp(-z[at]))
            rows[at] = y
        last.append(h)
    zero = torch.zeros(u.shape[-1], dtype=F64)
    if cu is None:
        y = torch.stack([torch.stack([rows[b, t] for t in range(u.shape[1])]) if u.shape[1] else
                         torch.zeros(u.shape[1:], dtype=F64) for b in range(u.shape[0])])
    else:
        y = torch.stack([rows.get(t, zero) for t in range(u.shape[0])]) if u.shape[0] else torch.zeros(u.shape, dtype=F64)
    return y, (torch.stack(last) if last else torch.zeros((0,) + A.shape, dtype=F64))


def conv(x, w, b, silu=True, cu=None, starts=None):
    """(y, final states [n_seqs, W - 1, channels]); differentiable."""
    x, w = x.to(F64), w.to(F64)
    W = w.shape[1]
    out, last = torch.zeros_like(x), []
    rows = {}
    for s, (row, t0, t1) in enumerate(bounds(x, cu)):
        seq = x[t0:t1] if row is None else x[row, t0:t1]
        before = torch.zeros((W - 1, x.shape[-1]), dtype=F64) if starts is None else starts[s].to(F64)
        ext = torch.cat([before, seq], 0)
        for t in range(t1 - t0):
            pre = (ext[t:t + W] * w.t()).sum(0)
            if b is not None:
                pre = pre + b.to(F64)
            rows[(t0 + t) if row is None else (row, t0 + t)] = pre / (1 + torch.exp(-pre)) if silu else pre
        last.append(ext[ext.shape[0] - (W - 1):])
    zero = torch.zeros(x.shape[-1], dtype=F64)
    if cu is None:
        y = torch.stack([torch.stack([rows[r, t] for t in range(x.shape[1])]) for r in range(x.shape[0])]) if rows else out
    else:
        y = torch.stack([rows.get(t, zero) for t in range(x.shape[0])]) if x.shape[0] else out
    return y, (torch.stack(last) if last else torch.zeros((0, W - 1, x.shape[-1]), dtype=F64))
