"""Checks of the causal operators and of the binding that are made on the host, before anything
is launched: none of the calls below reaches a kernel, so they run without a GPU.
"""
import pytest
import torch

from test_causal_abi_host import FAKE, i64, rows, scan, vs  # noqa: F401  (vs: the built library)


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


def elements(start, batch, L, width, bs, rs):
    return {start + b * bs + t * rs + c for b in range(batch) for t in range(L) for c in range(width)}


def test_outputs_of_the_derivative_over_other_tensors(vs):
    """du, ddelta and dz among one another and over every activation: rows with the same strides are
    compared exactly (against the sets of their elements here), others by their first element.  The
    calls that pass are stopped by the missing workspace."""
    import random

    rng = random.Random(1)
    d, N = 5, 4
    width = dict(zip(range(9), (d, d, d, N, N, d, d, d, d)))
    refused = passed = 0
    for case in range(3000):
        batch, L = rng.choice([(1, 1), (1, 6), (3, 1), (2, 4), (3, 3), (4, 2)])
        if rng.random() < 0.5:                               # tokens of a batch item follow one another, or items of a token do
            rs = d + rng.randrange(0, 9)
            bs = L * rs + rng.choice([0, 1, 7, 3 * rs])
        else:
            bs = d + rng.randrange(0, 9)
            rs = batch * bs + rng.choice([0, 1, 7, 3 * bs])
        i, j = rng.choice([(o, k) for o in (6, 7, 8) for k in range(9) if k != o])
        start = rng.randrange(-2 * (bs + rs), 2 * (bs + rs)) if rng.random() < 0.7 else rng.randrange(-40 * rs, 40 * rs)
        place = {k: (FAKE + (k << 32), bs, rs) for k in range(9)}
        place[j] = (place[i][0] + 4 * start, bs, rs)
        meet = elements(0, batch, L, width[i], bs, rs) & elements(start, batch, L, width[j], bs, rs)
        io = i64(*[v for k in range(9) for v in place[k]])
        got = vs.lib.causal_scan_bwd(io, FAKE, FAKE, FAKE, *[FAKE + (20 << 32)] * 5, batch, L, d, N, 0, None, 0, None, None, 0, None)
        assert got == (vs.VIM_ERR_INVALID_ARG if meet else vs.VIM_ERR_WORKSPACE), (case, batch, L, bs, rs, i, j, start)
        refused, passed = refused + bool(meet), passed + (not meet)
    assert refused > 300 and passed > 300
    io = i64(*[v for k in range(9) for v in (FAKE + (min(k, 7) << 32), 100, 5 if k < 8 else 7)])   # dz at ddelta, other rows
    assert vs.lib.causal_scan_bwd(io, FAKE, FAKE, FAKE, *[FAKE + (20 << 32)] * 5, 1, 6, d, N, 0, None, 0, None, None, 0,
                                  None) == vs.VIM_ERR_INVALID_ARG


def test_outputs_over_inputs(vs):
    """y of the scan may be u, delta or z itself, that of the convolution's step x itself; a row
    further, with other strides, or over B and C it may not.  Every call is refused."""
    bad, far = vs.VIM_ERR_INVALID_ARG, [(FAKE + (k << 32), 600, 64) for k in range(6)]
    put = lambda place, **k: i64(*[v for i, p in enumerate(place) for v in k.get(f"r{i}", p)])
    for i in (0, 1, 2):
        y = far[i][0]
        for at in ((y + 128, 600, 64), (y - 1200, 600, 64), (y, 600, 66), (y, 640, 64)):
            assert scan(vs, put(far, r5=at)) == bad, (i, at)
    for i in (3, 4):
        for at in ((far[i][0], 600, 64), (far[i][0] + 128, 600, 64), (far[i][0] + 30, 600, 64)):
            assert scan(vs, put(far, r5=at)) == bad, (i, at)
    one = [(p, b, 0) for p, b, _ in far]
    step = lambda io: vs.lib.causal_scan_step(io, FAKE, FAKE, FAKE, 2, 64, 16, 1, i64(0, 2, FAKE, FAKE, 0, 2, 0), None)
    for i in (0, 1, 2):
        for at in ((one[i][0] + 1200, 600, 0), (one[i][0], 700, 0), (one[i][0] + 126, 600, 0)):
            assert step(put(one, r5=at)) == bad, (i, at)
    for i in (3, 4):
        assert step(put(one, r5=one[i])) == bad
    conv = lambda y: vs.lib.causal_conv(i64(FAKE, 600, 64, *y), FAKE, FAKE, 2, 8, 64, 4, 1, 1, None, None)
    for y in ((FAKE, 600, 64), (FAKE + 128, 600, 64), (FAKE - 2, 600, 64), (FAKE + 1200, 600, 64)):
        assert conv(y) == bad, y
    conv_step = lambda y: vs.lib.causal_conv_step(i64(FAKE, 600, 0, *y), FAKE, None, 2, 64, 4, 1, 1,
                                                  i64(0, 2, FAKE, FAKE, 0, 2, 0), None)
    for y in ((FAKE + 1200, 600, 0), (FAKE + 2, 600, 0), (FAKE, 700, 0)):
        assert conv_step(y) == bad, y
    for dx in ((FAKE + 128, 600, 64), (FAKE + (1 << 32) - 2, 600, 64), (FAKE, 640, 64)):
        io = i64(FAKE, 600, 64, FAKE + (1 << 32), 600, 64, *dx)
        assert vs.lib.causal_conv_bwd(io, FAKE, FAKE, FAKE, FAKE, 2, 8, 64, 4, 1, 1, None, 0, FAKE, 1 << 40, None) == bad, dx


def test_final_states_over_initial_ones(vs):
    """state_out is state itself or apart from it."""
    bad = vs.VIM_ERR_INVALID_ARG
    row = 64 * 16 * 4
    for out in (FAKE + 16, FAKE + row, FAKE - 16, FAKE - 2 * row + 16):
        assert scan(vs, seqs=i64(0, 2, FAKE, out, 0, 2, 0)) == bad
        assert vs.lib.causal_scan_step(rows(6, row=0), FAKE, FAKE, FAKE, 2, 64, 16, 1, i64(0, 2, FAKE, out, 0, 2, 0), None) == bad
    row = 3 * 64 * 2
    for out in (FAKE + 2, FAKE + 2 * row - 2, FAKE - 2 * row + 2):
        assert vs.lib.causal_conv(rows(2), FAKE, FAKE, 2, 8, 64, 4, 1, 1, i64(0, 2, FAKE, out, 0, 2, 0), None) == bad
        assert vs.lib.causal_conv_step(rows(2, row=0), FAKE, None, 2, 64, 4, 1, 1, i64(0, 2, FAKE, out, 0, 2, 0), None) == bad
