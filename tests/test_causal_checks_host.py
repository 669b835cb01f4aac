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
