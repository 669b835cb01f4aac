"""causal_conv, causal_conv_step and causal_conv_bwd against the definition in fp64.

Tolerances.  An output is a sum of at most 4 products and the bias in fp32 (5 roundings of
2^-24 of the largest partial sum) through SiLU, whose sigmoid comes from the exp2 and
reciprocal units (3e-7 relative together): 1e-6 normwise.  bf16 outputs are rounded once,
half a step: 2^-8 of the value.  dw and db sum over at most 2000 tokens here, in runs of at
most 64 and then by 16 partial sums: fewer than 300 roundings in a row of 2^-24 of a partial
sum that is at most sqrt-like of the total's terms, 2e-5 with a factor of safety of one.
"""
import pytest
import torch

import causal_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 1e-6, BF: 2.0 ** -8 + 1e-6}
SUM_TOL = 2e-5


@pytest.fixture(scope="module")
def vs():
    from vision_mamba_selective_b200 import vimscan

    return vimscan


def inputs(rows, d, W, dtype, seed, strided=False, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((*rows, 2 * d + 3 if strided else d), generator=g).to(dtype)
    x = x[..., :d] if strided else x
    w = (torch.rand((d, W), generator=g) * 2 - 1) / W ** 0.5
    b = (torch.rand(d, generator=g) * 2 - 1) / W ** 0.5 if bias else None
    return x, w.contiguous(), b


def cuda(t):
    if t is None:
        return None
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)


def close(got, want, tol):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    if got.numel():
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= tol * torch.maximum(want.abs(), want.abs().max() * 0.1)).all(), \
            ((got - want).abs().max() / want.abs().max()).item()


BATCH = [
    # batch, L, d, W, dtype, silu, strided, bias
    (1, 1, 16, 4, BF, True, False, True),
    (2, 3, 33, 4, F32, True, False, True),
    (3, 17, 40, 3, BF, False, False, False),
    (2, 64, 8, 2, F32, True, True, True),
    (1, 200, 72, 4, BF, True, True, False),
    (4, 129, 1, 4, F32, False, False, True),
    (2, 9, 2048, 4, BF, True, False, True),
    (1, 700, 12, 3, BF, True, True, True),       # whole vectors of 4, not of 8
]


@pytest.mark.parametrize("case", BATCH, ids=lambda c: "_".join(str(v).replace("torch.", "") for v in c))
def test_batch_and_gradients(vs, case):
    batch, L, d, W, dtype, silu, strided, bias = case
    x, w, b = inputs((batch, L), d, W, dtype, seed=L + d, strided=strided, bias=bias)
    state = torch.full((batch, W - 1, d), float("nan"), dtype=dtype, device="cuda")
    y = vs.causal_conv(cuda(x), cuda(w), cuda(b), silu=silu, state_out=state)
    leaf = [t.double().requires_grad_() for t in (x, w)] + ([b.double().requires_grad_()] if bias else [])
    want, last = causal_ref.conv(leaf[0], leaf[1], leaf[2] if bias else None, silu)
    close(y, want.detach(), TOL[dtype])
    assert torch.equal(state.cpu().double(), last.detach())
    dout = torch.randn((batch, L, d), generator=torch.Generator().manual_seed(1)).to(dtype)
    grads = torch.autograd.grad(want, leaf, dout.double())
    got = vs.causal_conv_bwd(cuda(x), cuda(w), cuda(b), dout.cuda(), silu=silu)
    close(got["dx"], grads[0], TOL[dtype])
    close(got["dw"], grads[1], SUM_TOL)
    if bias:
        close(got["db"], grads[2], SUM_TOL)
    else:
        assert got["db"] is None


PACKED = [
    # lengths, d, W, dtype, tokens before the first sequence, tokens after the last
    ([1], 16, 4, BF, 0, 0),
    ([5, 0, 1, 40, 2, 1, 1, 64, 3], 40, 4, F32, 0, 0),
    ([3, 33, 0, 0, 7], 24, 3, BF, 4, 9),
    ([100, 29, 2], 9, 4, F32, 1, 0),
    ([0, 0], 16, 2, F32, 0, 3),
    ([1] * 20, 64, 4, BF, 0, 1),
    ([300, 2, 170], 64, 4, BF, 5, 0),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"n{len(c[0])}_d{c[1]}_W{c[2]}_{str(c[3])[6:]}_{c[4]}_{c[5]}")
def test_packed(vs, case):
    lens, d, W, dtype, lead, tail = case
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    T, n = cu[-1] + tail, len(lens)
    x, w, b = inputs((T,), d, W, dtype, seed=T + d, strided=True)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(n + 3, generator=g)[:n]
    cache = torch.randn((n + 3, W - 1, d), generator=g).to(dtype)
    fresh = torch.rand(n, generator=g) < 0.4
    starts = torch.where(fresh[:, None, None], torch.zeros((), dtype=dtype), cache[slots])
    want, last = causal_ref.conv(x, w, b, True, cu, starts)
    inside = slice(cu[0], cu[-1])
    leaf = [t.double().requires_grad_() for t in (x, w, b)]
    zero_start, _ = causal_ref.conv(*leaf, True, cu)
    dout = torch.randn((T, d), generator=g).to(dtype)
    grads = torch.autograd.grad(zero_start, leaf, dout.double()) if cu[-1] > cu[0] else [torch.zeros_like(t) for t in leaf]
    for t in (x, dout):   # tokens of no sequence
        t[:lead] = float("nan")
        t[cu[-1]:] = float("inf")
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for in_place in (False, True):
        state = cache.cuda()
        out = state if in_place else torch.full_like(state, 7.0)
        y = torch.full((T, d), 3.0, dtype=dtype, device="cuda")
        vs.causal_conv(cuda(x), cuda(w), cuda(b), cu_seqlens=off, state=state, state_out=None if in_place else out,
                       slots=slots.to(torch.int32).cuda(), fresh=fresh.cuda(), y=y)
        close(y[inside], want[inside], TOL[dtype])
        assert (y[:cu[0]] == 3.0).all() and (y[cu[-1]:] == 3.0).all()
        assert torch.equal(out[slots.cuda()].cpu().double(), last)
        others = [i for i in range(n + 3) if i not in slots.tolist()]
        assert torch.equal(out[others].cpu(), cache[others] if in_place else torch.full_like(cache[others], 7.0))
    got = vs.causal_conv_bwd(cuda(x), cuda(w), cuda(b), dout.cuda(), cu_seqlens=off)
    assert (got["dx"][:lead] == 0).all() and (got["dx"][cu[-1]:] == 0).all()
    close(got["dx"][inside], grads[0][inside], TOL[dtype])
    close(got["dw"], grads[1], SUM_TOL)
    close(got["db"], grads[2], SUM_TOL)


def test_sequences_across_runs(vs):
    """Many short runs: 40000 tokens of 64 channels, so that a thread's run is longest, and the
    same with few tokens; dw and db against the fp64 sums of the whole."""
    for T, cu in ((40000, [0, 1, 64, 65, 127, 129, 20000, 39999, 40000]), (130, [0, 7, 8, 9, 63, 64, 130])):
        x, w, b = inputs((T,), 64, 4, BF, seed=T)
        dout = torch.randn((T, 64), generator=torch.Generator().manual_seed(1)).to(BF)
        off = torch.tensor(cu, dtype=torch.int32, device="cuda")
        y = vs.causal_conv(cuda(x), cuda(w), cuda(b), cu_seqlens=off)
        got = vs.causal_conv_bwd(cuda(x), cuda(w), cuda(b), dout.cuda(), cu_seqlens=off)
        xd, wd, bd = x.double(), w.double(), b.double()
        pre, dx, dw = torch.zeros_like(xd), torch.zeros_like(xd), torch.zeros_like(wd)
        for t0, t1 in zip(cu[:-1], cu[1:]):
            ext = torch.cat([torch.zeros(3, 64, dtype=torch.float64), xd[t0:t1]])
            pre[t0:t1] = sum(ext[k:k + t1 - t0] * wd[:, k] for k in range(4)) + bd
        sg = torch.sigmoid(pre)
        dpre = dout.double() * sg * (1 + pre * (1 - sg))
        for t0, t1 in zip(cu[:-1], cu[1:]):
            ext = torch.cat([torch.zeros(3, 64, dtype=torch.float64), xd[t0:t1]])
            for k in range(4):
                dw[:, k] += (dpre[t0:t1] * ext[k:k + t1 - t0]).sum(0)
                n = t1 - t0 - (3 - k)
                if n > 0:
                    dx[t0:t0 + n] += dpre[t1 - n:t1] * wd[:, k]
        close(y, pre * sg, TOL[BF])
        close(got["dx"], dx, TOL[BF])
        close(got["dw"], dw, SUM_TOL)
        close(got["db"], dpre.sum(0), SUM_TOL)


@pytest.mark.parametrize("d,W,dtype", [(32, 4, BF), (33, 4, F32), (12, 3, BF), (64, 2, F32), (1, 4, BF)])
@pytest.mark.parametrize("batch", [1, 9])
def test_step_follows_the_prompt(vs, batch, d, W, dtype):
    L = 7
    x, w, b = inputs((batch, L), d, W, dtype, seed=d + batch, strided=True)
    want, last = causal_ref.conv(x, w, b)
    slots = torch.randperm(batch + 4, generator=torch.Generator().manual_seed(1))[:batch].to(torch.int32)
    if batch > 2:
        slots[1] = batch + 4
    state = torch.zeros((batch + 4, W - 1, d), dtype=dtype, device="cuda")
    xs, ws, bs, dev = cuda(x), cuda(w), cuda(b), slots.cuda()
    y = torch.full((L, batch, d), 3.0, dtype=dtype, device="cuda")
    for t in range(L):
        vs.causal_conv_step(xs[:, t], ws, bs, state, slots=dev, y=y[t])
    use = [i for i in range(batch) if slots[i] < batch + 4]
    close(y.permute(1, 0, 2)[use], want[use], TOL[dtype])
    assert torch.equal(state[slots[use].long().cuda()].cpu().double(), last[use])
    if batch > 2:
        assert (y[:, 1] == 3.0).all()
    before, new = state.clone(), torch.full_like(state, 5.0)
    vs.causal_conv_step(xs[:, 0], ws, bs, state, slots=dev, state_out=new)
    assert torch.equal(state, before)
    rest = [i for i in range(batch + 4) if i not in slots.tolist()]
    assert (new[rest] == 5.0).all()


def test_prompt_in_parts(vs):
    """Parts shorter than the window keep the older inputs."""
    x, w, b = inputs((2, 23), 24, 4, F32, 3)
    want, last = causal_ref.conv(x, w, b)
    state = torch.zeros((2, 3, 24), device="cuda")
    got, at = [], 0
    for n in (1, 2, 1, 9, 3, 7):
        got.append(vs.causal_conv(cuda(x)[:, at:at + n], cuda(w), cuda(b), state=state))
        at += n
    close(torch.cat(got, 1), want, TOL[F32])
    assert torch.equal(state.cpu().double(), last)


def test_gradient_against_differences(vs):
    x, w, b = (t.double() for t in inputs((1, 12), 3, 4, F32, 8))
    dout = torch.randn((1, 12, 3), generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    got = vs.causal_conv_bwd(x.float().cuda(), w.float().cuda(), b.float().cuda(), dout.float().cuda())
    loss = lambda x, w, b: (causal_ref.conv(x, w, b)[0] * dout).sum().item()
    for i, key in enumerate(("dx", "dw", "db")):
        args = [x, w, b]
        way = torch.randn(args[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-5 * way, args[i] - 1e-5 * way
        slope = (loss(*hi) - loss(*lo)) / 2e-5
        mine = got[key].cpu().double() * way
        assert abs(mine.sum().item() - slope) <= 1e-4 * mine.abs().sum().item(), key


def test_stream_graph_and_repeats(vs):
    x, w, b = (cuda(t) for t in inputs((2, 300), 64, 4, BF, 4))
    dout = torch.randn_like(x)
    y, g = vs.causal_conv(x, w, b), vs.causal_conv_bwd(x, w, b, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, g2 = vs.causal_conv(x, w, b, stream=side), vs.causal_conv_bwd(x, w, b, dout, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)
    ws = torch.empty(vs.causal_conv_bwd_workspace_bytes(2, 300, 64, 4), dtype=torch.uint8, device="cuda")
    y3, g3 = torch.zeros_like(y), {k: torch.zeros_like(v) for k, v in g.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vs.causal_conv(x, w, b, y=y3)
        vs.causal_conv_bwd(x, w, b, dout, workspace=ws, out=g3)
    for _ in range(2):
        y3.zero_()
        graph.replay()
        assert torch.equal(y, y3) and all(torch.equal(g[k], g3[k]) for k in g)


def test_time_major_and_far_rows(vs):
    """[L, batch, channels] in memory; rows 2^27 elements apart (element offsets to 2^32)."""
    x, w, b = inputs((3, 40), 24, 4, F32, 6)
    want, _ = causal_ref.conv(x, w, b)
    y = vs.causal_conv(x.transpose(0, 1).contiguous().cuda().transpose(0, 1), cuda(w), cuda(b))
    close(y, want, TOL[F32])
    L, d = 34, 16
    x, w, b = inputs((1, L), d, 4, BF, 7)
    base = torch.empty((L, 1 << 27), dtype=BF, device="cuda")
    far = base[:, :d]
    far.copy_(x[0].cuda())
    y = base[:, 64:64 + d][None]
    vs.causal_conv(far[None], cuda(w), cuda(b), y=y)
    want, _ = causal_ref.conv(x, w, b)
    close(y, want, TOL[BF])


def test_overlapping_rows(vs):
    """Rows that are windows over one signal, one element apart."""
    d, L = 16, 21
    _, w, b = inputs((1, 1), d, 4, F32, 8)
    signal = torch.randn(L + d, generator=torch.Generator().manual_seed(8))
    x = signal.as_strided((2, L, d), (0, 1, 1))
    dev = signal.cuda().as_strided((2, L, d), (0, 1, 1))
    y = vs.causal_conv(dev, cuda(w), cuda(b))
    close(y, causal_ref.conv(x, w, b)[0], TOL[F32])
    got = vs.causal_conv_bwd(dev, cuda(w), cuda(b), torch.ones_like(y))
    dense = vs.causal_conv_bwd(dev.contiguous(), cuda(w), cuda(b), torch.ones_like(y))
    close(got["dx"], dense["dx"].cpu(), TOL[F32])
    close(got["dw"], dense["dw"].cpu(), SUM_TOL)
    close(got["db"], dense["db"].cpu(), SUM_TOL)


def test_refusals(vs):
    x, w, b = (cuda(t) for t in inputs((2, 10), 32, 4, F32, 1))
    state = torch.zeros((2, 3, 32), device="cuda")
    dout = torch.zeros_like(x)
    bad = [
        (TypeError, lambda: vs.causal_conv(x.cpu(), w, b)),
        (TypeError, lambda: vs.causal_conv(x.half(), w, b)),
        (TypeError, lambda: vs.causal_conv(x, w.bfloat16(), b)),
        (ValueError, lambda: vs.causal_conv(x, w[:31], b)),
        (ValueError, lambda: vs.causal_conv(x, w, b[:31])),
        (ValueError, lambda: vs.causal_conv(x, w, b, state=state[:, :2])),
        (ValueError, lambda: vs.causal_conv(x, w, b, state=state[:1])),
        (TypeError, lambda: vs.causal_conv(x, w, b, state=state.bfloat16())),
        (ValueError, lambda: vs.causal_conv(x[0], w, b)),
        (vs.VimScanError, lambda: vs.causal_conv(x, torch.zeros((32, 5), device="cuda"), b)),
        (vs.VimScanError, lambda: vs.causal_conv(x, torch.zeros((32, 1), device="cuda"), b)),
        (vs.VimScanError, lambda: vs.causal_conv(x, w, b, y=x)),                          # in place
        (ValueError, lambda: vs.causal_conv_step(x, w, b, state)),
        (ValueError, lambda: vs.causal_conv_step(x[:, 0], w, b, None)),
        (ValueError, lambda: vs.causal_conv_bwd(x, w, b, dout[:, :9])),
        (ValueError, lambda: vs.causal_conv_bwd(x, w, None, dout, out=vs.causal_conv_bwd(x, w, b, dout))),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            raise AssertionError(f"call {i} was not refused")
    assert vs.causal_conv(x[:, :0], w, b, state=state).shape == (2, 0, 32)
    g = vs.causal_conv_bwd(x[:, :0], w, b, dout[:, :0])
    assert (g["dw"] == 0).all() and (g["db"] == 0).all()
