"""Calls of the causal operators that their documentation allows and that are easily got wrong:
outputs named in another order, padding entries with kept states, values past fp32, parameters at
infinity.
"""
import math

import pytest
import torch

import causal_ref
from test_causal_scan_gpu import BF, F32, STATE_TOL, Y_TOL, close, cuda, inputs, packed_case, vs  # noqa: F401

pytestmark = pytest.mark.gpu


def test_clipping_into_a_dict_in_another_order(vs):
    """Gradients of equal shapes go to the outputs of their names."""
    g = torch.Generator().manual_seed(1)
    grads = {k: torch.randn(40, generator=g).cuda() for k in ("dD", "ddelta_bias", "db")} | {"dz": None}
    out = {k: None if grads[k] is None else torch.full((40,), 7.0, device="cuda") for k in ("dz", "db", "dD", "ddelta_bias")}
    want = [t.clone() for t in grads.values() if t is not None]
    norm = vs.clip_grad_norm(want, 0.5)                     # in place
    assert torch.equal(vs.clip_grad_norm(grads, 0.5, out=out), norm)
    for k, w in zip(("dD", "ddelta_bias", "db"), want):
        assert torch.equal(out[k], w), k
    with pytest.raises(ValueError):
        vs.clip_grad_norm(grads, 0.5, out={**out, "dz": out["db"]})
    with pytest.raises(TypeError):
        vs.clip_grad_norm(grads, 0.5, out=[t for t in out.values() if t is not None])


@pytest.mark.parametrize("d,N,dtype", [(40, 16, F32), (300, 16, BF), (1300, 16, F32), (6000, 16, BF), (24, 8, F32), (20, 2, F32)])
def test_kept_states_of_padding_entries(vs, d, N, dtype):
    """A padding slot skips the outputs and the final state of a sequence, not the states that are
    kept for the derivative: it takes every sequence that cu_seqlens lists and knows no slots."""
    lens = [21, 50, 0, 9, 33]
    p, cu = packed_case(lens, d, N, dtype, seed=d, lead=2, tail=3)
    args = cuda(p)
    dev = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    shape = vs.causal_ckpt_shape(1, cu[-1] + 3, d, N)
    plain, some, all_skipped = (torch.full(shape, float("nan"), device="cuda") for _ in range(3))
    state = torch.full((5, d, N), 7.0, device="cuda")
    y0 = torch.full_like(args[0], 3.0)
    vs.causal_scan(*args, ckpt=plain, state_out=state, y=y0, **dev)
    for slots, ck in (([4, -1, 0, 9, 2], some), ([5, -1, 7, 9, -3], all_skipped)):
        y, out = torch.full_like(args[0], 3.0), torch.full((5, d, N), 7.0, device="cuda")
        vs.causal_scan(*args, ckpt=ck, state_out=out, y=y, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), **dev)
        torch.cuda.synchronize()
        kept = ~torch.isnan(plain)
        assert torch.equal(torch.isnan(ck), torch.isnan(plain)) and torch.equal(ck[kept], plain[kept])
        used = {s for s in slots if 0 <= s < 5}
        for s, (slot, t0, t1) in enumerate(zip(slots, cu[:-1], cu[1:])):
            if slot in used:
                assert torch.equal(y[t0:t1], y0[t0:t1]) and torch.equal(out[slot], state[s])
            else:
                assert (y[t0:t1] == 3.0).all()
        assert all((out[i] == 7.0).all() for i in range(5) if i not in used)
    dout = torch.randn(args[0].shape, generator=torch.Generator().manual_seed(d)).to(dtype).cuda()
    want = vs.causal_scan_bwd(*args, dout, ckpt=plain, **dev)
    got = vs.causal_scan_bwd(*args, dout, ckpt=some, **dev)
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("dtype", [F32, BF])
def test_norm_past_fp32_scales_nothing(vs, dtype):
    """A norm that is infinite in fp32, although every gradient and the sum in fp64 are finite, is
    what the caller sees, and leaves the gradients as they are."""
    src = [torch.full((40,), 2e38, device="cuda").to(dtype), torch.ones(7, device="cuda")]
    before = [t.clone() for t in src]
    out = [torch.zeros_like(t) for t in src]
    assert vs.clip_grad_norm(src, 1.0, out=out).item() == math.inf
    assert all(torch.equal(a, b) for a, b in zip(out, before))
    assert vs.clip_grad_norm(src, 1.0).item() == math.inf
    assert all(torch.equal(a, b) for a, b in zip(src, before))


@pytest.mark.parametrize("batch,d,N,dtype", [(2, 40, 16, F32), (3, 264, 16, BF), (2, 600, 16, F32), (2, 4100, 16, F32),
                                             (2, 24, 8, F32), (1, 20, 4, F32), (2, 20, 2, F32)])
def test_a_at_minus_infinity(vs, batch, d, N, dtype):
    """States that forget everything at once: A of -infinity, or of the type's lowest value, in
    sequences whose ends lie inside a segment.  The definition has decays of exactly 0 there."""
    L = 21
    p = inputs((batch, L), d, N, dtype, seed=d)
    p["A"][1, 1], p["A"][3], p["A"][d - 1, 0] = -math.inf, -math.inf, torch.finfo(F32).min
    state = torch.empty((batch, d, N), device="cuda")
    ck = torch.full(vs.causal_ckpt_shape(batch, L, d, N), float("nan"), device="cuda")
    args = cuda(p)
    y = vs.causal_scan(*args, state_out=state, ckpt=ck)
    want, last = causal_ref.scan(p["u"], p["delta"], p["z"], p["B"], p["C"], p["A"], p["D"], p["bias"])
    close(y, want, Y_TOL[dtype], "y")
    close(state, last, STATE_TOL, "state")
    assert torch.isfinite(ck).all()
    token = [t[:, 3] for t in args[:5]]
    start = torch.randn((batch, d, N), generator=torch.Generator().manual_seed(2))
    got = start.cuda()
    vs.causal_scan_step(*token, *args[5:], got)
    one = {k: (v[:, 3:4] if k in ("u", "delta", "z", "B", "C") else v) for k, v in p.items()}
    close(got, causal_ref.scan(one["u"], one["delta"], one["z"], one["B"], one["C"], p["A"], p["D"], p["bias"],
                               starts=start)[1], STATE_TOL, "step")
    # the derivative: what -1e30, whose decays are 0 as well, gives (its slope with respect to A is 0)
    dout = torch.randn((batch, L, d), generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    near = list(args)
    near[5] = args[5].clamp(min=-1e30)
    for kept in (None, ck):
        g, w = vs.causal_scan_bwd(*args, dout, ckpt=kept), vs.causal_scan_bwd(*near, dout, ckpt=kept)
        for k in g:
            assert torch.equal(g[k], w[k]), k
        assert (g["dA"][3] == 0).all()
