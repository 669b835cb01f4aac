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
