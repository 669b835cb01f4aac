"""The causal operators together, as a model uses them: prompts of several sequences packed into
one row, then single tokens from a captured graph, against whole sequences in fp64; and a
training step (forward, every gradient, clipping, update) against automatic differentiation
in fp64.

The block: x, z = halves of one projection; u = causal_conv(x); [delta | B | C] = u P by a
matrix product; y = causal_scan(u, delta, z, B, C).  Tolerances: fp32 throughout; the chain
of conv (1e-6), product (fp32 sums over d channels, 1e-6) and scan (1e-5 of its own inputs,
which carry the former two into Delta, B and C: each enters y at most linearly or through an
exponent of size one) stays below 1e-5 + 4 * 2e-6 = 2e-5 normwise; gradients, products of two
such chains, at twice the 5e-5 of the scan's own derivative.
"""
import pytest
import torch

import causal_ref

pytestmark = pytest.mark.gpu
D, N, W = 48, 16, 4
TOL, GRAD_TOL = 2e-5, 1e-4


@pytest.fixture(scope="module")
def vs():
    from vision_mamba_selective_b200 import vimscan

    return vimscan


@pytest.fixture(autouse=True)
def full_fp32_products():
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = before


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)
    return dict(w=(torch.rand((D, W), generator=g) * 2 - 1) / 2, b=(torch.rand(D, generator=g) * 2 - 1) / 2,
                P=torch.randn((D, D + 2 * N), generator=g) / D ** 0.5,
                A=-(torch.arange(1, N + 1).float() * torch.exp(0.2 * torch.randn((D, N), generator=g))),
                D=torch.randn(D, generator=g), bias=torch.log(torch.expm1(step)))


def reference(xz, p, cu=None):
    """fp64, differentiable: (y, (conv states, scan states))."""
    x, z = xz[..., :D], xz[..., D:]
    u, last_x = causal_ref.conv(x, p["w"], p["b"], True, cu)
    proj = u @ p["P"].double()
    y, last_h = causal_ref.scan(u, proj[..., :D], z, proj[..., D:D + N], proj[..., D + N:], p["A"], p["D"], p["bias"], cu)
    return y, last_x, last_h


def close(got, want, tol):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all()
    assert (got - want).abs().max() <= tol * want.abs().max(), ((got - want).abs().max() / want.abs().max()).item()


def test_prompts_then_tokens(vs):
    p = {k: v.cuda() for k, v in weights().items()}
    lens, more = [7, 1, 30, 2], 5                      # prompts, then five tokens of each
    g = torch.Generator().manual_seed(3)
    full = [torch.randn((n + more, 2 * D), generator=g) for n in lens]
    want = [reference(f[None], {k: v.cpu() for k, v in p.items()}) for f in full]

    n = len(lens)
    slots = torch.tensor([4, 0, 5, 2], dtype=torch.int32, device="cuda")
    conv_state = torch.full((6, W - 1, D), 9.0, device="cuda")       # stale: the prompts are fresh
    scan_state = torch.full((6, D, N), 9.0, device="cuda")
    fresh = torch.ones(n, dtype=torch.bool, device="cuda")
    cu = torch.tensor([0, 7, 8, 38, 40], dtype=torch.int32, device="cuda")
    xz = torch.cat([f[:k] for f, k in zip(full, lens)]).cuda()
    u = vs.causal_conv(xz[:, :D], p["w"], p["b"], cu_seqlens=cu, state=conv_state, slots=slots, fresh=fresh)
    proj = u @ p["P"]
    y = vs.causal_scan(u, proj[:, :D], xz[:, D:], proj[:, D:D + N], proj[:, D + N:], p["A"], p["D"], p["bias"],
                       cu_seqlens=cu, state=scan_state, slots=slots, fresh=fresh)
    for i, k in enumerate(lens):
        close(y[int(cu[i]):int(cu[i + 1])], want[i][0][0, :k], TOL)

    # tokens from a graph whose inputs are replaced between replays; one padding row
    row_slots = torch.cat([slots, torch.tensor([-1], dtype=torch.int32, device="cuda")])
    token = torch.zeros((n + 1, 2 * D), device="cuda")
    out = torch.zeros((n + 1, D), device="cuda")

    def one_token():
        u = vs.causal_conv_step(token[:, :D], p["w"], p["b"], conv_state, slots=row_slots)
        proj = u @ p["P"]
        vs.causal_scan_step(u, proj[:, :D], token[:, D:], proj[:, D:D + N], proj[:, D + N:], p["A"], p["D"], p["bias"],
                            scan_state, slots=row_slots, y=out)

    kept = conv_state.clone(), scan_state.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one_token()                                    # warm up, then put the states back
    torch.cuda.current_stream().wait_stream(side)
    conv_state.copy_(kept[0]), scan_state.copy_(kept[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_token()
    for t in range(more):
        token[:n] = torch.stack([f[k + t] for f, k in zip(full, lens)]).cuda()
        graph.replay()
        for i, k in enumerate(lens):
            close(out[i], want[i][0][0, k + t], TOL)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(conv_state[s].cpu(), full[i][-(W - 1):, :D].float())
        close(scan_state[s], want[i][2][0], TOL)
    assert (conv_state[[1, 3]] == 9).all() and (scan_state[[1, 3]] == 9).all()


@pytest.mark.parametrize("packed", [False, True])
def test_training_step(vs, packed):
    p = weights(1)
    rows = (90,) if packed else (2, 45)
    cu = [0, 3, 50, 50, 90] if packed else None
    g = torch.Generator().manual_seed(5)
    xz, target = torch.randn((*rows, 2 * D), generator=g), torch.randn((*rows, D), generator=g)
    leaf = {k: v.double().requires_grad_() for k, v in p.items()}
    want_xz = xz.double().requires_grad_()
    y, _, _ = reference(want_xz, leaf, cu)
    names = list(leaf)
    loss = ((y - target.double()) ** 2).sum() / 2
    want = dict(zip(names + ["xz"], torch.autograd.grad(loss, [leaf[k] for k in names] + [want_xz])))

    q = {k: v.cuda() for k, v in p.items()}
    x, z = xz.cuda()[..., :D], xz.cuda()[..., D:]
    off = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    u = vs.causal_conv(x, q["w"], q["b"], cu_seqlens=off)
    proj = u @ q["P"]
    args = (u, proj[..., :D], z, proj[..., D:D + N], proj[..., D + N:], q["A"], q["D"], q["bias"])
    ck = torch.empty(vs.causal_ckpt_shape(*((1, 90) if packed else rows), D, N), device="cuda")
    y = vs.causal_scan(*args, cu_seqlens=off, ckpt=ck)
    s = vs.causal_scan_bwd(*args, y - target.cuda(), cu_seqlens=off, ckpt=ck)
    dproj = torch.cat([s["ddelta"], s["dB"], s["dC"]], -1)
    du = s["du"] + dproj @ q["P"].t()
    c = vs.causal_conv_bwd(x, q["w"], q["b"], du.contiguous(), cu_seqlens=off)
    dP = u.reshape(-1, D).t() @ dproj.reshape(-1, D + 2 * N)
    got = dict(w=c["dw"], b=c["db"], P=dP, A=s["dA"], D=s["dD"], bias=s["ddelta_bias"],
               xz=torch.cat([c["dx"], s["dz"]], -1))
    for k in want:
        close(got[k], want[k], GRAD_TOL)
    # clip the parameters' gradients together, and step
    grads = {k: got[k] for k in names}
    norm = vs.clip_grad_norm(grads, 0.5)
    true = torch.sqrt(sum((want[k] ** 2).sum() for k in names))
    assert abs(norm.item() - true.item()) <= GRAD_TOL * true.item()
    assert true.item() > 0.5
    for k in names:
        close(grads[k], want[k] * (0.5 / true), 2 * GRAD_TOL)
        q[k] -= 0.1 * grads[k]
