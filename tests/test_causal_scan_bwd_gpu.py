"""causal_scan_bwd against the definition's gradients in fp64 (automatic differentiation of the
token loop), and against differences of the forward operator's definition.

Tolerances: the kernels' states and adjoints each carry at most the 2e-5 that the forward
tests derive for a state; every gradient is a sum of products of one of each, so 4e-5, and
fp32 rounding of the sums another 1e-6 at these lengths: 5e-5 normwise.  bf16 gradients
(du, ddelta, dz) are rounded once, half a step 2^-8 of the value, besides.
"""
import pytest
import torch

import causal_ref
from test_causal_scan_gpu import BF, F32, cuda, inputs, packed_case

pytestmark = pytest.mark.gpu
TOL = 5e-5
IO_TOL = {F32: TOL, BF: 2.0 ** -8 + TOL}
KEYS = ("du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddelta_bias")


@pytest.fixture(scope="module")
def vs():
    from vision_mamba_selective_b200 import vimscan

    return vimscan


def want_grads(p, dout, cu=None):
    leaf = {k: (None if v is None else v.double().requires_grad_()) for k, v in p.items()}
    y, _ = causal_ref.scan(leaf["u"], leaf["delta"], leaf["z"], leaf["B"], leaf["C"], leaf["A"], leaf["D"], leaf["bias"], cu)
    names = [k for k, v in leaf.items() if v is not None]
    got = torch.autograd.grad(y, [leaf[k] for k in names], dout.double())
    rename = {"bias": "ddelta_bias"}
    return {rename.get(k, "d" + k): g for k, g in zip(names, got)}


def check(got, want, dtype, inside=None):
    for k in KEYS:
        if k not in want:
            assert got[k] is None, k
            continue
        g, w = got[k].detach().cpu().double(), want[k]
        if inside is not None and k in ("du", "ddelta", "dz", "dB", "dC"):
            g, w = g[inside], w[inside]
        tol = IO_TOL[dtype] if k in ("du", "ddelta", "dz") else TOL
        assert g.shape == w.shape, k
        if not w.numel():
            continue
        assert torch.isfinite(g).all(), k
        err = (g - w).abs().max().item() / max(w.abs().max().item(), 1e-30)
        assert err <= tol, (k, err)
        if k not in ("dD", "ddelta_bias"):   # and row by row, floored at the rms row
            rows = w.norm(dim=-1)
            floor = rows.square().mean().sqrt()
            worst = ((g - w).norm(dim=-1) / torch.maximum(rows, floor).clamp_min(1e-30)).max().item()
            assert worst <= tol, (k, worst)


CASES = [
    # batch, L, d, N, dtype, gate, strided
    (1, 1, 8, 16, F32, True, False),
    (2, 7, 33, 16, F32, True, False),
    (1, 64, 32, 16, BF, True, False),
    (2, 65, 40, 16, F32, False, True),
    (3, 63, 24, 8, F32, True, True),
    (1, 130, 8, 4, BF, True, False),
    (2, 71, 130, 2, F32, True, False),
    (1, 200, 72, 16, F32, True, True),
    (1, 150, 1, 16, F32, True, False),
    (2, 40, 300, 8, BF, False, False),
    (1, 129, 200, 4, F32, True, True),
    (3, 90, 264, 16, F32, True, True),         # segments of 16, 4 lanes a channel
    (1, 150, 700, 16, BF, True, False),
    (2, 145, 600, 16, F32, True, False),       # segments of 8
    (2, 21, 4100, 16, F32, True, False),       # 8200 channels: eight states a lane
    (1, 70, 8200, 16, BF, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{c[0]}_L{c[1]}_d{c[2]}_N{c[3]}_{str(c[4])[6:]}"
                         f"{'' if c[5] else '_nogate'}{'_strided' if c[6] else ''}")
@pytest.mark.parametrize("kept", [False, True])
def test_batch(vs, case, kept):
    batch, L, d, N, dtype, gate, strided = case
    p = inputs((batch, L), d, N, dtype, seed=L + d, gate=gate, strided=strided)
    dout = torch.randn((batch, L, d), generator=torch.Generator().manual_seed(L)).to(dtype)
    args = cuda(p)
    ck = None
    if kept:
        ck = torch.full(vs.causal_ckpt_shape(batch, L, d, N), float("nan"), device="cuda")
        vs.causal_scan(*args, ckpt=ck)
    got = vs.causal_scan_bwd(*args, dout.cuda(), ckpt=ck)
    check(got, want_grads(p, dout), dtype)


PACKED = [
    # lengths, d, N, dtype, tokens before the first sequence, tokens after the last
    ([1], 32, 16, F32, 0, 0),
    ([5, 0, 1, 40, 31, 1, 1, 64], 40, 16, F32, 0, 0),
    ([3, 33, 0, 0, 7], 24, 8, BF, 4, 9),
    ([100, 29, 2], 9, 16, F32, 1, 0),
    ([64, 64], 16, 16, F32, 0, 70),
    ([60, 8, 90], 16, 4, F32, 68, 3),
    ([17] * 12, 64, 2, BF, 0, 1),
    ([9, 0, 20, 3], 4100, 16, F32, 0, 2),            # enough channels for eight states a lane
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"n{len(c[0])}_d{c[1]}_N{c[2]}_{str(c[3])[6:]}_{c[4]}_{c[5]}")
@pytest.mark.parametrize("kept", [False, True])
def test_packed(vs, case, kept):
    """Tokens of no sequence hold NaN in every input and keep what the outputs held."""
    lens, d, N, dtype, lead, tail = case
    p, cu = packed_case(lens, d, N, dtype, seed=sum(lens) + d, lead=lead, tail=tail)
    T = p["u"].shape[0]
    dout = torch.randn((T, d), generator=torch.Generator().manual_seed(7)).to(dtype)
    want = want_grads(p, dout, cu)
    inside = slice(cu[0], cu[-1])
    for t in [p[k] for k in ("u", "delta", "z", "B", "C")] + [dout]:
        t[:lead] = float("nan")
        t[cu[-1]:] = float("nan")
    args = cuda(p)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ck = None
    if kept:
        ck = torch.full(vs.causal_ckpt_shape(1, T, d, N), float("nan"), device="cuda")
        vs.causal_scan(*args, cu_seqlens=off, ckpt=ck)
    out = vs.causal_scan_bwd(*args, dout.cuda(), cu_seqlens=off, ckpt=ck)
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        assert (out[k][:lead] == 0).all() and (out[k][cu[-1]:] == 0).all(), k
    check(out, want, dtype, inside)
    for t in out.values():
        t.fill_(3.0)
    vs.causal_scan_bwd(*args, dout.cuda(), cu_seqlens=off, ckpt=ck, out=out)
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        assert (out[k][:lead] == 3).all() and (out[k][cu[-1]:] == 3).all(), k
    check(out, want, dtype, inside)


def test_against_differences(vs):
    """Central differences of the fp64 definition along random directions."""
    p = inputs((1, 20), 6, 4, F32, 17)
    p = {k: v.double() for k, v in p.items()}
    dout = torch.randn((1, 20, 6), generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    got = vs.causal_scan_bwd(*cuda({k: v.float() for k, v in p.items()}), dout.float().cuda())
    names = dict(u="du", delta="ddelta", z="dz", B="dB", C="dC", A="dA", D="dD", bias="ddelta_bias")
    def loss(q):
        y, _ = causal_ref.scan(q["u"], q["delta"], q["z"], q["B"], q["C"], q["A"], q["D"], q["bias"])
        return (y * dout).sum().item()
    eps = 1e-5
    for i, (k, g) in enumerate(names.items()):
        way = torch.randn(p[k].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        slope = (loss({**p, k: p[k] + eps * way}) - loss({**p, k: p[k] - eps * way})) / (2 * eps)
        mine = (got[g].cpu().double() * way).sum().item()
        scale = (got[g].cpu().double() * way).abs().sum().item()
        assert abs(mine - slope) <= 1e-4 * scale, (k, mine, slope)


def test_repeats_and_graph(vs):
    """Bit for bit the same, on another stream, and replayed from a graph with its own
    workspace while eager calls run between the replays."""
    p = inputs((2, 200), 64, 16, BF, 5)
    dout = torch.randn((2, 200, 64), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    args = cuda(p)
    first = vs.causal_scan_bwd(*args, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = vs.causal_scan_bwd(*args, dout, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in KEYS:
        assert torch.equal(first[k], other[k]), k
    ws = torch.empty(vs.causal_bwd_workspace_bytes(2, 200, 64, 16, False), dtype=torch.uint8, device="cuda")
    out = {k: torch.zeros_like(v) for k, v in first.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vs.causal_scan_bwd(*args, dout, workspace=ws, out=out)
    for _ in range(2):
        for v in out.values():
            v.zero_()
        g.replay()
        again = vs.causal_scan_bwd(*args, dout)
        for k in KEYS:
            assert torch.equal(out[k], first[k]) and torch.equal(again[k], first[k]), k


def test_many_slices_and_chunks(vs):
    """A single chunk with many channels (several slices of channels) and many chunks with few
    (one slice), against each other's halves and the definition's dD."""
    p = inputs((1, 50), 1000, 16, F32, 9)
    dout = torch.randn((1, 50, 1000), generator=torch.Generator().manual_seed(2)).cuda()
    args = cuda(p)
    whole = vs.causal_scan_bwd(*args, dout)
    parts = []
    for c in (slice(0, 500), slice(500, 1000)):
        parts.append(vs.causal_scan_bwd(args[0][..., c], args[1][..., c], args[2][..., c], args[3], args[4],
                                        args[5][c], args[6][c], args[7][c], dout[..., c]))
    for k in ("dB", "dC"):
        s = parts[0][k] + parts[1][k]
        assert ((whole[k] - s).abs().max() / s.abs().max()) <= 2e-6, k   # a few fp32 steps of reordering
    for k in ("du", "ddelta", "dz"):
        assert torch.equal(whole[k], torch.cat([q[k] for q in parts], -1)), k


def test_strided_outputs(vs):
    p = inputs((2, 30), 32, 16, F32, 6, strided=True)
    dout = torch.randn((2, 30, 32), generator=torch.Generator().manual_seed(1))
    args = cuda(p)
    plain = vs.causal_scan_bwd(*args, dout.cuda())
    wide = torch.full((2, 30, 64 + 5), 3.0, device="cuda")
    out = dict(plain, du=wide[..., :32], dz=wide[..., 37:], ddelta=torch.empty((2, 30, 32), device="cuda"))
    vs.causal_scan_bwd(*args, dout.cuda(), out=out)
    want = want_grads(p, dout)
    check(out, want, F32)
    assert (wide[..., 32:37] == 3).all()


def test_refusals_and_empty(vs):
    p = inputs((2, 10), 32, 16, F32, 1)
    a = cuda(p)
    dout = torch.randn((2, 10, 32), device="cuda")
    good = vs.causal_scan_bwd(*a, dout)
    for kind, call in [
        (ValueError, lambda: vs.causal_scan_bwd(*a, dout[:, :9])),
        (TypeError, lambda: vs.causal_scan_bwd(*a, dout.bfloat16())),
        (ValueError, lambda: vs.causal_scan_bwd(*a, dout, ckpt=torch.zeros((2, 1, 32, 16), device="cuda"))),
        (ValueError, lambda: vs.causal_scan_bwd(*a, dout, out=dict(good, dz=None))),
        (ValueError, lambda: vs.causal_scan_bwd(*a, dout, out=dict(good, dA=good["dA"][:, :8]))),
        (ValueError, lambda: vs.causal_scan_bwd(*a, dout, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (vs.VimScanError, lambda: vs.causal_scan_bwd(*a, dout, out=dict(good, du=good["du"][:1].expand(2, 10, 32)))),
    ]:
        with pytest.raises(kind):
            call()
    p = inputs((2, 0), 32, 16, F32, 1)
    g = vs.causal_scan_bwd(*cuda(p), torch.zeros((2, 0, 32), device="cuda"))
    assert (g["dA"] == 0).all() and (g["dD"] == 0).all() and (g["ddelta_bias"] == 0).all()
    p = inputs((9,), 32, 16, F32, 1)
    g = vs.causal_scan_bwd(*cuda(p), torch.ones((9, 32), device="cuda"),
                           cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (g["dA"] == 0).all() and (g["du"] == 0).all()
