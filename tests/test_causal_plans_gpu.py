"""The causal operators at sizes whose cut is that of large calls: a warp of causal_scan_step that
takes its channels through several groups of sequences, CTAs of the derivative that take several
blocks of channels, threads of the convolution whose runs are several turns long; with outputs in
the place of inputs where that is allowed.  References in fp64 on the GPU.  And the roundings that
the decays and softplus are built to avoid.

Tolerances are those that test_causal_scan_gpu.py, test_causal_scan_bwd_gpu.py and
test_causal_conv_gpu.py derive.  One token alone carries one decay (1.5e-7 of the exp2 unit and
6e-8 of its argument's rounding, times |Delta A| log2 e < 3), Delta and Delta u (3e-7) and a
multiply-add (6e-8): below 1e-6 of the largest state.  The gradients' sums are over 64 tokens in
a chunk and 16 chunk sums a thread and 16 threads: 96 roundings in a row, 6e-6 of a partial sum,
with 4e-5 of the states and adjoints still within the derivative's 5e-5.  The convolution's are
over 64 tokens, 4 runs, 10 groups and 16 threads: 94 roundings, within its 2e-5.
"""
import pytest
import torch

from test_causal_conv_gpu import SUM_TOL, close as conv_close, cuda as move, inputs as conv_inputs
from test_causal_scan_bwd_gpu import check
from test_causal_scan_gpu import BF, F32, STATE_TOL, Y_TOL, close, cuda, inputs, vs  # noqa: F401

pytestmark = pytest.mark.gpu
ONE_TOKEN = 1e-6


def params(g, d, N):
    A = -(torch.arange(1, N + 1, dtype=F32) * torch.exp(0.2 * torch.randn((d, N), generator=g)))
    step = torch.exp(torch.rand(d, generator=g) * 4.6 - 6.9)      # 1e-3 .. 1e-1
    return A.contiguous().cuda(), torch.randn(d, generator=g).cuda(), torch.log(torch.expm1(step)).cuda()


# batch, d, N, dtype: 16 sequences a warp in groups of 4 (131 leaves a group of 3), 4 in groups of 1
# and of 2, 32 in groups of 4; channels that end inside a CTA
STEPS = [(131, 2050, 16, BF), (131, 2048, 16, F32), (130, 2048, 2, BF), (127, 3001, 8, F32), (1030, 600, 16, BF),
         (260, 2500, 4, F32)]


@pytest.mark.parametrize("batch,d,N,dtype", STEPS)
@pytest.mark.parametrize("over", [None, 0, 1, 2], ids=["own_output", "over_u", "over_delta", "over_z"])
def test_step_in_groups(vs, batch, d, N, dtype, over):
    """Padding rows all over the batch; states in place and to another cache; y in the place of an
    input, its padding rows left as they were."""
    g = torch.Generator().manual_seed(batch + d)
    r = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()
    wide = r(batch, 2 * d + 2)
    u, delta, z, B, C = r(batch, d), r(batch, d), wide[:, d + 2:], r(batch, N), r(batch, N)
    A, D, bias = params(g, d, N)
    slots = torch.randperm(batch + 7, generator=g)[:batch].to(torch.int32)
    skipped = torch.rand(batch, generator=g) < 0.15
    slots[skipped] = torch.where(torch.rand(int(skipped.sum()), generator=g) < 0.5, -1, batch + 7).to(torch.int32)
    cache = torch.randn((batch + 7, d, N), generator=g).cuda()
    use, rows = (~skipped).cuda(), slots[~skipped].long().cuda()
    rest = torch.ones(batch + 7, dtype=torch.bool, device="cuda")
    rest[rows] = False

    dt = torch.nn.functional.softplus(delta[use].double() + bias.double(), threshold=700)
    h = torch.exp(dt[..., None] * A.double()) * cache[rows].double() + (dt * u[use].double())[..., None] * B[use].double()[:, None]
    zs = z[use].double()
    want = ((h * C[use].double()[:, None]).sum(-1) + D.double() * u[use].double()) * zs * torch.sigmoid(zs)

    for in_place in (True, False):
        io = [u.clone(), delta.clone(), wide.clone()[:, d + 2:]]
        y = torch.full_like(u, 3.0) if over is None else io[over]
        before = y.clone()
        state = cache.clone()
        out = state if in_place else torch.full_like(state, 7.0)
        got = vs.causal_scan_step(*io, B, C, A, D, bias, state, state_out=None if in_place else out,
                                  slots=slots.cuda(), y=y)
        assert got is y
        close(y[use], want.cpu(), Y_TOL[dtype], "y")
        assert torch.equal(y[~use], before[~use])
        close(out[rows], h.cpu(), ONE_TOKEN, "state")
        assert torch.equal(out[rest], cache[rest] if in_place else torch.full_like(cache[rest], 7.0))
        if not in_place:
            assert torch.equal(state, cache)


@pytest.mark.parametrize("d,W,dtype", [(2048, 4, BF), (1030, 4, F32), (512, 3, BF), (77, 2, F32)])
def test_conv_step_in_place(vs, d, W, dtype):
    """States in place (also with y in the place of x) give the bits of separate buffers."""
    g = torch.Generator().manual_seed(d)
    batch = 190
    x = torch.randn((batch, d), generator=g).to(dtype).cuda()
    w, b = torch.randn((d, W), generator=g).cuda(), torch.randn(d, generator=g).cuda()
    cache = torch.randn((batch + 3, W - 1, d), generator=g).to(dtype).cuda()
    slots = torch.randperm(batch + 3, generator=g)[:batch].to(torch.int32).cuda()
    out = cache.clone()
    y = vs.causal_conv_step(x, w, b, cache, state_out=out, slots=slots)
    assert torch.equal(out[slots.long(), -1], x)
    state, io = cache.clone(), x.clone()
    assert torch.equal(vs.causal_conv_step(io, w, b, state, slots=slots, y=io), y)
    assert torch.equal(state, out)


def scan_reference(p, bounds, dout):
    """(y, final states, gradients) in fp64, all sequences of ``bounds`` (None or a batch row, first
    token, end) side by side, padded at their ends with steps of 0."""
    lens = [t1 - t0 for _, t0, t1 in bounds]
    L, n = max(lens), len(bounds)
    leaf = {k: v.cuda().double().requires_grad_() for k, v in p.items()}
    at = lambda t, b, t0, t1: t[t0:t1] if b is None else t[b, t0:t1]
    pad = lambda t: torch.stack([torch.nn.functional.pad(at(t, *s), (0, 0, 0, L - m)) for s, m in zip(bounds, lens)])
    inside = torch.stack([torch.arange(L, device="cuda") < m for m in lens])[..., None]
    u, z, B, C = (pad(leaf[k]) for k in ("u", "z", "B", "C"))
    dt = torch.nn.functional.softplus(pad(leaf["delta"]) + leaf["bias"], threshold=700) * inside
    h = torch.zeros((n, *leaf["A"].shape), dtype=torch.float64, device="cuda")
    ys = []
    for t in range(L):
        h = torch.exp(dt[:, t, :, None] * leaf["A"]) * h + (dt[:, t] * u[:, t])[..., None] * B[:, t, None]
        ys.append((h * C[:, t, None]).sum(-1))
    y = (torch.stack(ys, 1) + leaf["D"] * u) * z * torch.sigmoid(z) * inside
    names = list(leaf)
    grads = torch.autograd.grad(y, [leaf[k] for k in names], pad(dout.cuda().double()) * inside)
    whole = torch.zeros(p["u"].shape, dtype=torch.float64)
    for i, (b, t0, t1) in enumerate(bounds):
        (whole if b is None else whole[b])[t0:t1] = y[i, :t1 - t0].detach().cpu()
    return whole, h.detach().cpu(), {"d" + {"bias": "delta_bias"}.get(k, k): g.cpu() for k, g in zip(names, grads)}


def slices_of(vs, batch, L, d, N):
    """Channel slices of a derivative's call, from what it needs besides: carries, chunk sums, and
    2 N sums a token and slice."""
    up = lambda floats: (4 * floats + 255) // 256 * 256
    chunks = batch * ((L + 63) // 64)
    rest = vs.causal_bwd_workspace_bytes(batch, L, d, N, True) - 2 * up(chunks * d * N) - up(2 * chunks * d)
    return rest // (2 * batch * L * N * 4)


LENS = [2000, 1999, 0, 1, 1700, 2048, 640, 64, 1987, 1500, 1801, 2300]


@pytest.mark.parametrize("batch,L,d,N,dtype,blocks", [(8, 2000, 200, 16, F32, 7), (8, 1941, 205, 16, BF, 7),
                                                      (None, None, 200, 16, F32, 7), (None, None, 232, 16, BF, 8),
                                                      (6, 2301, 460, 8, F32, 8), (None, None, 700, 2, F32, 6)])
def test_channel_blocks_of_the_derivative(vs, batch, L, d, N, dtype, blocks):
    """Long rows with few channels: a CTA of the derivative goes through several blocks of channels
    and adds up its dB and dC over them; eight warps a CTA in the scans."""
    if batch is None:
        cu = [5]
        for n in LENS:
            cu.append(cu[-1] + n)
        rows, bounds = (cu[-1] + 2,), [(None, t0, t1) for t0, t1 in zip(cu[:-1], cu[1:])]
        off, inside = torch.tensor(cu, dtype=torch.int32, device="cuda"), slice(cu[0], cu[-1])
        size = (1, rows[0])
    else:
        rows, bounds, off, inside = (batch, L), [(b, 0, L) for b in range(batch)], None, slice(None)
        size = rows
    assert 1 <= slices_of(vs, *size, d, N) < blocks
    p = inputs(rows, d, N, dtype, seed=d + N)
    dout = torch.randn((*rows, d), generator=torch.Generator().manual_seed(d)).to(dtype)
    y0, last, want = scan_reference(p, bounds, dout)
    args = cuda(p)
    ck = torch.full(vs.causal_ckpt_shape(*size, d, N), float("nan"), device="cuda")
    state = torch.empty((len(bounds), d, N), device="cuda")
    y = vs.causal_scan(*args, cu_seqlens=off, ckpt=ck, state_out=state)
    close(y[inside], y0[inside], Y_TOL[dtype], "y")
    close(state, last, STATE_TOL, "state")
    for kept in (None, ck):
        got = vs.causal_scan_bwd(*args, dout.cuda(), cu_seqlens=off, ckpt=kept)
        check(got, want, dtype, inside if batch is None else None)
        again = vs.causal_scan_bwd(*args, dout.cuda(), cu_seqlens=off, ckpt=kept)
        assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("rows,d,W,dtype,run", [((40000,), 512, 4, BF, 64), ((30000,), 300, 3, F32, 32),
                                                ((20011,), 507, 4, F32, 40), ((6, 5003), 512, 4, BF, 56),
                                                ((5, 8001), 128, 2, F32, 16)])
def test_long_runs_of_the_convolution(vs, rows, d, W, dtype, run):
    """Runs of several turns of tokens loaded ahead: sequences that start, end and lie inside a run
    and a turn, and span many runs; prompts with their final states, and the derivative.

    Outputs are compared each by itself, as millions of them include sums that nearly cancel.  With
    P = |b| + sum |w x| over the taps, pre is off by at most 5 roundings of 2^-24, 3e-7 P; its
    sigmoid by 3e-7 of itself (exp2 and reciprocal).  silu has slope at most 1.1: y is off by at
    most 3.3e-7 P + 3e-7 |pre| + 6e-8 |y| < 1e-6 P.  silu' = s + v s - (v s) s moves with the error
    of s by at most 3e-7 (1 + |v|), with that of v by half of it, and by 4 roundings of at most
    1 + |v|: below 7e-7 (1 + P).  dx adds W products and their sum, at most 5 roundings, 3e-7: off
    by at most 1e-6 of the sum of |w dout| (1 + P) over its taps.  bf16 adds half a step, 2^-8 of
    the value."""
    x, w, b = conv_inputs(rows, d, W, dtype, seed=d, strided=True)
    packed, size = len(rows) == 1, rows if len(rows) == 2 else (1, rows[0])
    groups = vs.causal_conv_bwd_workspace_bytes(*size, d, W) // (d * (W + 1) * 4)
    assert (size[0] * -(-size[1] // run) + 3) // 4 == groups           # 32 strips a CTA, 4 runs
    cu = [0]
    if packed:
        cu = [3, 4, 11, 19, 67, 71, 71, 130, 131, 133, 198, 1003, 1011, 1013, 9000, 9000 + run, 17001, rows[0] - 70,
              rows[0] - 65, rows[0] - 2]
    bounds = [(None, t0, t1) for t0, t1 in zip(cu[:-1], cu[1:])] if packed else [(i, 0, rows[1]) for i in range(rows[0])]
    dout = torch.randn((*rows, d), generator=torch.Generator().manual_seed(1)).to(dtype)
    start = torch.randn((len(bounds), W - 1, d), generator=torch.Generator().manual_seed(2)).to(dtype)

    def reference(states):
        xd, wd, bd = (t.cuda().double().requires_grad_() for t in (x, w, b))
        y, last = torch.zeros((*rows, d), dtype=torch.float64, device="cuda"), []
        for i, (r, t0, t1) in enumerate(bounds):
            ext = torch.cat([states[i].cuda().double(), xd[t0:t1] if r is None else xd[r, t0:t1]])
            pre = sum(ext[k:k + t1 - t0] * wd[:, k] for k in range(W)) + bd
            (y if r is None else y[r])[t0:t1] = pre * torch.sigmoid(pre)
            last.append(ext[ext.shape[0] - (W - 1):].detach())
            with torch.no_grad():
                P = sum((ext[k:k + t1 - t0] * wd[:, k]).abs() for k in range(W)) + bd.abs()
                at = (lambda t: t[t0:t1]) if r is None else (lambda t: t[r, t0:t1])
                at(size_y)[:] = P
                reach = torch.nn.functional.pad(at(dout.cuda().double()).abs() * (1 + P), (0, 0, 0, W - 1))
                at(size_dx)[:] = sum(reach[k:k + t1 - t0] * wd[:, W - 1 - k].abs() for k in range(W))
        return y, torch.stack(last), (xd, wd, bd)

    def each(got, want, size):
        got, want, size = got[inside].double(), want.detach()[inside], size[inside]
        bound = 1e-6 * size + (2.0 ** -8 * want.abs() if dtype == BF else 0)
        assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound).max().item()

    size_y, size_dx = (torch.zeros((*rows, d), dtype=torch.float64, device="cuda") for _ in range(2))

    inside = slice(cu[0], cu[-1]) if packed else slice(None)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    want, last, _ = reference(start)
    state = start.cuda()
    y = vs.causal_conv(move(x), w.cuda(), b.cuda(), cu_seqlens=off, state=state)
    each(y, want, size_y)
    assert torch.equal(state.double(), last)
    want, last, leaf = reference(torch.zeros_like(start))
    grads = torch.autograd.grad(want, leaf, dout.cuda().double())
    got = vs.causal_conv_bwd(move(x), w.cuda(), b.cuda(), dout.cuda(), cu_seqlens=off)
    each(got["dx"], grads[0], size_dx)
    conv_close(got["dw"], grads[1].cpu(), SUM_TOL)
    conv_close(got["db"], grads[2].cpu(), SUM_TOL)
    if packed:
        assert (got["dx"][:cu[0]] == 0).all() and (got["dx"][cu[-1]:] == 0).all()


def test_decays_are_centred(vs):
    """One token with u = 0 leaves the decay in a state of 1.  For decays from 0.75 to 0.995 its mean
    error is at most 1.5e-8 of it: low by 1.6e-8 or more it would be with the exp2 unit alone.
    (Roundings are of either sign; over 2 million arguments their mean is below 1e-10.)"""
    d, batch = 4096, 32
    g = torch.Generator().manual_seed(1)
    step = 21 + 10 * torch.rand(d, generator=g)                 # above 20 softplus is its argument
    decay = 0.75 + 0.245 * torch.rand((d, 16), generator=g, dtype=torch.float64)
    A = (decay.log() / step.double()[:, None]).float()
    zero = torch.zeros((1, d), device="cuda")
    state = torch.ones((1, d, 16), device="cuda")
    mean = []
    for k in range(batch):
        bias = step * (1 + k * 2.0 ** -12)
        state.fill_(1.0)
        vs.causal_scan_step(zero, zero, None, *torch.ones((2, 1, 16), device="cuda"), A.cuda(), zero[0], bias.cuda(), state)
        want = torch.exp(A.double() * bias.double()[:, None])
        mean.append(((state[0].cpu().double() - want) / want).mean())
    assert abs(torch.stack(mean).mean().item()) <= 1.5e-8


def test_softplus_keeps_its_arguments_rounding(vs):
    """One token with A = 0, u = B = 1 leaves Delta in a state of 0.  Its error for raw steps from
    -11 to -5.6 (x log2 e from 8 to 16) is at most 1.1e-7 rms: the exponential's, at most 1.5e-7 and
    so 8.7e-8 rms, and three roundings of at most 6e-8, 3.5e-8 rms each.  The rounding of x log2 e
    alone would add 3.3e-7, 1.9e-7 rms."""
    d = 1 << 17
    x = -11 + 5.4 * torch.rand(d, generator=torch.Generator().manual_seed(1))
    zero, one = torch.zeros((1, d), device="cuda"), torch.ones((1, d), device="cuda")
    state = torch.zeros((1, d, 2), device="cuda")
    vs.causal_scan_step(one, zero, None, *torch.ones((2, 1, 2), device="cuda"), torch.zeros((d, 2), device="cuda"), zero[0],
                        x.cuda(), state)
    want = torch.nn.functional.softplus(x.double())
    err = (state[0, :, 0].cpu().double() - want) / want
    assert err.square().mean().sqrt().item() <= 1.1e-7
