"""Checks of the causal operators and of the binding that are made on the host, before anything
is launched: none of the calls below reaches a kernel, so they run without a GPU.
"""
import pytest
import torch

from test_causal_abi_host import FAKE, i64, scan, vs  # noqa: F401  (vs: the built library)


def test_workspace_on_the_calls_device(vs):
    """A workspace that the kernels could not write as it is described: not a tensor, host
    memory, another device, elements that share their bytes."""
    gpu = torch.device("cuda", 0)
    for bad in (torch.empty(4096, dtype=torch.uint8), 4096, torch.empty(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(TypeError):
            vs._workspace(1024, bad, gpu)
    here = torch.device("cpu")
    for bad in (torch.empty(1, dtype=torch.uint8).expand(4096), torch.empty(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            vs._workspace(1024, bad, here)
    with pytest.raises(ValueError):
        vs._workspace(1024, torch.empty(255), here)
    good = torch.empty(256)
    ws, nbytes = vs._workspace(1024, good, here)
    assert ws is good and nbytes == 1024
    assert vs._workspace(0, None, gpu) == (None, 0)


def test_parameters_of_an_empty_prompt(vs):
    """No token, but initial states to hand on: the kernel still loads A, D and delta_bias, so
    they are checked as ever."""
    none = i64(*[0] * 18)
    seqs = i64(0, 2, FAKE, FAKE, 0, 2, 0)
    for A, D, bias in ((FAKE + 4, FAKE, FAKE), (FAKE, FAKE + 2, FAKE), (FAKE, FAKE, FAKE + 2), (None, FAKE, FAKE),
                       (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert scan(vs, none, A, D, bias, L=0, seqs=seqs) == vs.VIM_ERR_INVALID_ARG, (A, D, bias)


def test_gradients_and_their_outputs_are_paired(vs):
    """Dicts by key, whatever their order; lists and tuples by place; None where the other is."""
    a, b, c, d = (torch.zeros(2) for _ in range(4))
    pairs = lambda grads, out: vs._clip_pairs("clip_grad_norm", grads, out)
    same = lambda got, want: all(len(x) == len(y) and all(p is q for p, q in zip(x, y)) for x, y in zip(got, want))
    assert same(pairs(dict(dD=a, dz=None, dA=b), dict(dA=d, dz=None, dD=c)), ([a, b], [c, d]))
    assert same(pairs([a, None, b], (c, None, d)), ([a, b], [c, d]))
    assert same(pairs(dict(dD=a, dz=None), None), ([a], [a]))
    assert same(pairs((t for t in (a, b)), None), ([a, b], [a, b]))
    assert same(pairs((t for t in (a, b)), iter([c, d])), ([a, b], [c, d]))
    assert same(pairs([], []), ([], []))
    for grads, out in ((dict(dD=a), dict(dA=c)), (dict(dD=a, dA=b), dict(dD=c)), (dict(dD=a), dict(dD=c, dA=None)),
                       (dict(dD=a, dA=None), dict(dD=None, dA=c)), ([None, a], [c, None]), ([a], [c, None]), ([a, b], [c])):
        with pytest.raises(ValueError):
            pairs(grads, out)
    for grads, out in ((dict(dD=a), [c]), ([a], dict(dD=c))):
        with pytest.raises(TypeError):
            pairs(grads, out)


def test_norm_and_workspace_of_their_own(vs):
    """The norm and the workspace are written while gradients are still read."""
    need = vs.lib.clip_grad_norm_workspace_bytes(1)
    def clip(table, norm=FAKE + (1 << 33), ws=FAKE + (1 << 34)):
        return vs.lib.clip_grad_norm(i64(*table), len(table) // 4, 1.0, norm, ws, need, None)
    in_place, apart = (FAKE, FAKE, 100, 0), (FAKE, FAKE + 4096, 100, 0)
    for table in (in_place, apart):
        for at in (FAKE, FAKE + 396):
            assert clip(table, norm=at) == vs.VIM_ERR_INVALID_ARG
        assert clip(table, ws=FAKE) == vs.VIM_ERR_INVALID_ARG
        assert clip(table, ws=FAKE + 256) == vs.VIM_ERR_INVALID_ARG
    assert clip(apart, norm=FAKE + 4096 + 200) == vs.VIM_ERR_INVALID_ARG
    assert clip(in_place, norm=FAKE + (1 << 34) + need - 4) == vs.VIM_ERR_INVALID_ARG      # in the workspace
