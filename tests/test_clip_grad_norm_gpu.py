"""clip_grad_norm against fp64.

Tolerances: squares are summed in fp32 over at most 8 elements (8 roundings of 2^-24 each
relative to a sum of positive terms, 5e-7 at most, halved by the square root) and in fp64
after that; the norm is rounded once more: 4e-7 relative.  A scaled fp32 value carries the
factor's and its own rounding besides: 6e-7; a bf16 one half a step, 2^-8, more.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NORM_TOL = 4e-7


@pytest.fixture(scope="module")
def vs():
    from vision_mamba_selective_b200 import vimscan

    return vimscan


def grads(shapes, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * std).to(t) for s, t in shapes]


def true_norm(ts):
    return math.sqrt(math.fsum((t.double() ** 2).sum().item() for t in ts))


SETS = {
    "one": [((1,), F32)],
    "mixed": [((100, 33), F32), ((7,), BF), ((0,), F32), ((8192,), BF), ((8193,), F32), ((3, 5, 7), BF), ((), F32)],
    "many": [((i % 50 + 1,), BF if i % 3 else F32) for i in range(401)],     # several launches
    "large": [((3000, 1001), BF), ((2000, 999), F32)],
    "empty": [((0,), F32), ((0, 4), BF)],
}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("how", ["in place", "out", "dict"])
def test_against_fp64(vs, name, how):
    src = grads(SETS[name], seed=len(name))
    norm = true_norm(src)
    for max_norm in (0.0, 0.37 * norm, 2 * norm + 1, math.inf):
        dev = [t.cuda() for t in src]
        out = [torch.full_like(t, 7.0) for t in dev] if how == "out" else dev
        if how == "dict":
            got = vs.clip_grad_norm({i: t for i, t in enumerate(dev)} | {"none": None}, max_norm)
        else:
            got = vs.clip_grad_norm(dev, max_norm, out=out if how == "out" else None)
        assert got.shape == (1,) and got.dtype == F32
        assert abs(got.item() - norm) <= NORM_TOL * norm
        factor = min(1.0, max_norm / (norm + 1e-6))
        for t, o in zip(src, out):
            want = t.double() * factor
            tol = 0.0 if factor == 1.0 else 6e-7 + (2.0 ** -8 if t.dtype == BF else 0.0)
            assert ((o.cpu().double() - want).abs() <= tol * want.abs() + (1e-40 if tol else 0)).all()
        if how == "out":
            assert all(torch.equal(t.cpu(), s) for t, s in zip(dev, src))


def test_large_small_and_nonfinite_values(vs):
    """Squares that overflow or vanish in fp32; NaN and infinity scale nothing."""
    for scale in (1e25, 1e-25):
        src = [torch.full((1000,), scale), torch.full((9,), 3 * scale)]
        dev = [t.cuda() for t in src]
        got = vs.clip_grad_norm(dev, math.inf).item()
        assert abs(got - true_norm(src)) <= NORM_TOL * true_norm(src)
    big = [torch.full((16,), 2e38, device="cuda"), torch.zeros(5, device="cuda")]
    assert vs.clip_grad_norm(big, 1.0).item() == math.inf     # the norm itself is past fp32
    for bad in (math.nan, math.inf):
        src = grads([((50,), F32), ((20,), BF)], 1)
        src[1][3] = bad
        dev = [t.cuda() for t in src]
        got = vs.clip_grad_norm(dev, 0.1).item()
        assert math.isnan(got) if math.isnan(bad) else got == math.inf
        assert torch.equal(dev[0].cpu(), src[0]) and torch.equal(dev[1].cpu().view(torch.int16), src[1].view(torch.int16))
        out = [torch.zeros_like(t) for t in dev]
        vs.clip_grad_norm(dev, 0.1, out=out)
        assert torch.equal(out[0], dev[0])


def test_views_and_alignment(vs):
    """Tensors that start anywhere in their storage; the neighbours stay."""
    base = torch.randn(5000, generator=torch.Generator().manual_seed(1))
    for t in (base.cuda(), base.to(BF).cuda()):
        before = t.clone()
        parts = [t[1:1000], t[1003:1004], t[1007:4999]]
        norm = true_norm([p.cpu() for p in parts])
        got = vs.clip_grad_norm(parts, 1.0)
        assert abs(got.item() - norm) <= NORM_TOL * norm
        keep = [0, *range(1000, 1003), *range(1004, 1007), 4999]
        assert torch.equal(t[keep], before[keep])
        want = before.cpu().double() / (norm + 1e-6)
        tol = 6e-7 + (2.0 ** -8 if t.dtype == BF else 0.0)
        assert ((t[1:1000].cpu().double() - want[1:1000]).abs() <= tol * want[1:1000].abs()).all()


def test_repeats_stream_and_graph(vs):
    src = [t.cuda() for t in grads(SETS["many"] + SETS["large"], 3)]
    out = [torch.empty_like(t) for t in src]
    norm = vs.clip_grad_norm(src, 1.0, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = [torch.empty_like(t) for t in src]
    norm2 = vs.clip_grad_norm(src, 1.0, out=out2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(out, out2))
    ws = torch.empty(vs.clip_grad_norm_workspace_bytes(len(src)), dtype=torch.uint8, device="cuda")
    norm3, out3 = torch.zeros(1, device="cuda"), [torch.zeros_like(t) for t in src]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vs.clip_grad_norm(src, 1.0, out=out3, norm=norm3, workspace=ws)
    for _ in range(2):
        norm3.zero_()
        g.replay()
        assert torch.equal(norm, norm3) and all(torch.equal(a, b) for a, b in zip(out, out3))


def test_refusals(vs):
    t = torch.ones(64, device="cuda")
    h = torch.ones((8, 8), device="cuda")
    bad = [
        (TypeError, lambda: vs.clip_grad_norm([t.cpu()], 1.0)),
        (TypeError, lambda: vs.clip_grad_norm([t.half()], 1.0)),
        (ValueError, lambda: vs.clip_grad_norm([h.t()], 1.0)),
        (ValueError, lambda: vs.clip_grad_norm([t], -1.0)),
        (ValueError, lambda: vs.clip_grad_norm([t], math.nan)),
        (ValueError, lambda: vs.clip_grad_norm([t], 1.0, out=[])),
        (ValueError, lambda: vs.clip_grad_norm([t], 1.0, out=[t.bfloat16()])),
        (ValueError, lambda: vs.clip_grad_norm([t], 1.0, norm=torch.zeros(2, device="cuda"))),
        (vs.VimScanError, lambda: vs.clip_grad_norm([t, t], 1.0)),                      # the same tensor twice
        (vs.VimScanError, lambda: vs.clip_grad_norm([t[:40], t[39:]], 1.0)),
        (vs.VimScanError, lambda: vs.clip_grad_norm([t[:40]], 1.0, out=[t[1:41]])),
        (vs.VimScanError, lambda: vs.clip_grad_norm([t, h], 1.0, out=[torch.empty_like(t), t.view(8, 8)])),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            raise AssertionError(f"call {i} was not refused")
    assert (t == 1).all() and (h == 1).all()
    assert vs.clip_grad_norm([], 1.0).item() == 0.0
    same = vs.clip_grad_norm([t, t], 1.0, out=[torch.empty_like(t), torch.empty_like(t)])   # read twice, counted twice
    assert abs(same.item() - math.sqrt(128)) < 1e-5
