"""The causal operators at sizes whose cut is that of large calls: a warp of causal_scan_step that
takes its channels through several groups of sequences, CTAs of the derivative that take several
blocks of channels, threads of the convolution whose runs are several turns long; with outputs in
the place of inputs where that is allowed.  References in fp64 on the GPU.

Tolerances are those that test_causal_scan_gpu.py, test_causal_scan_bwd_gpu.py and
test_causal_conv_gpu.py derive.  One token alone carries one decay (1.5e-7 of the exp2 unit and
6e-8 of its argument's rounding, times |Delta A| log2 e < 3), Delta and Delta u (3e-7) and a
multiply-add (6e-8): below 1e-6 of the largest state.
"""
import pytest
import torch

from test_causal_scan_gpu import BF, F32, Y_TOL, close, vs  # noqa: F401

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
