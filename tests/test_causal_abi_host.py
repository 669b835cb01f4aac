"""The causal entry points without a GPU: declared symbols are exported, bad arguments are
refused on the host before anything is launched, sizes of zero do nothing.  Every call below
fails a check or has nothing to do, so none reaches a launch.
"""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "vimscan_causal.h")
FAKE = 0x7f0000000000   # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def vs():
    from vision_mamba_selective_b200 import build

    build.build()
    from vision_mamba_selective_b200 import vimscan

    return vimscan


def i64(*values):
    return (ctypes.c_int64 * len(values))(*values)


def rows(n, batch=600, row=64, **other):
    """n vim_rows of FAKE data, far from one another; other: index -> (data, batch stride, row stride)."""
    v = []
    for i in range(n):
        v += other.get(f"r{i}", (FAKE + (i << 32), batch, row))
    return i64(*v)


def test_declared_functions_are_exported(vs):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:vim_status|size_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) == {"causal_scan", "causal_scan_step", "causal_scan_bwd", "causal_ckpt_bytes",
                          "causal_bwd_workspace_bytes", "causal_conv", "causal_conv_step", "causal_conv_bwd",
                          "causal_conv_bwd_workspace_bytes", "clip_grad_norm", "clip_grad_norm_workspace_bytes"}
    out = subprocess.run(["nm", "-D", "--defined-only", vs.LIB_PATH], check=True, capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(names) <= exported


def test_header_compiles_as_c():
    subprocess.run(["gcc", "-fsyntax-only", "-x", "c", "-std=c99", "-I/usr/local/cuda/include",
                    "-I" + os.path.dirname(HEADER), HEADER], check=True)


def test_package_names():
    import vision_mamba_selective_b200 as pkg

    for name in ("causal_scan", "causal_scan_step", "causal_scan_bwd", "causal_conv", "causal_conv_step",
                 "causal_conv_bwd", "clip_grad_norm"):
        assert callable(getattr(pkg, name))


def scan(vs, io=None, A=FAKE, D=FAKE, bias=FAKE, batch=2, L=8, d=64, N=16, dt=1, seqs=None, ckpt=None):
    return vs.lib.causal_scan(rows(6) if io is None else io, A, D, bias, batch, L, d, N, dt, seqs, ckpt, None)


def test_scan_refusals(vs):
    bad, uns = vs.VIM_ERR_INVALID_ARG, vs.VIM_ERR_UNSUPPORTED
    assert vs.lib.causal_scan(None, FAKE, FAKE, FAKE, 2, 8, 64, 16, 1, None, None, None) == bad
    for i in (0, 1, 3, 4, 5):
        assert scan(vs, rows(6, **{f"r{i}": (0, 600, 64)})) == bad, i              # null (z, r2, may be)
    for i in range(6):
        assert scan(vs, rows(6, **{f"r{i}": (FAKE + 1, 600, 64)})) == bad, i       # not element aligned
        assert scan(vs, rows(6, **{f"r{i}": (FAKE, -600, 64)})) == bad, i
        assert scan(vs, rows(6, **{f"r{i}": (FAKE, 600, -64)})) == bad, i
        assert scan(vs, rows(6, **{f"r{i}": (FAKE, 600, 1 << 30)})) == bad, i
    assert scan(vs, rows(6, r5=(FAKE, 600, 63))) == bad                            # y's rows overlap
    assert scan(vs, rows(6, r5=(FAKE, 511, 64))) == bad                            # y's batch items overlap
    assert scan(vs, A=None) == bad and scan(vs, A=FAKE + 4) == bad
    assert scan(vs, D=None) == bad and scan(vs, D=FAKE + 2) == bad and scan(vs, bias=None) == bad
    assert scan(vs, batch=-1) == bad and scan(vs, L=-1) == bad and scan(vs, d=-8) == bad
    assert scan(vs, dt=2) == bad
    assert scan(vs, N=3) == uns and scan(vs, N=32) == uns
    assert scan(vs, ckpt=FAKE + 4) == bad
    assert scan(vs, ckpt=FAKE, seqs=i64(0, 2, FAKE, FAKE, 0, 2, 0)) == bad         # kept states start from zeros
    assert scan(vs, L=2**31 - 8) == uns and scan(vs, d=2**31 - 8) == uns           # counted in ints with tiles
    # sequences: cu, n, state, state_out, slots, n_slots, fresh
    assert scan(vs, seqs=i64(0, 3, 0, 0, 0, 0, 0)) == bad                          # not one per batch row
    assert scan(vs, seqs=i64(FAKE, 3, 0, 0, 0, 0, 0)) == bad                       # packed, batch 2
    assert scan(vs, batch=1, seqs=i64(FAKE + 2, 3, 0, 0, 0, 0, 0)) == bad
    assert scan(vs, batch=1, seqs=i64(FAKE, -1, 0, 0, 0, 0, 0)) == bad
    assert scan(vs, seqs=i64(0, 2, 0, 0, FAKE, 4, 0)) == bad                       # slots without a state
    assert scan(vs, seqs=i64(0, 2, FAKE, FAKE, 0, 1, 0)) == bad                    # fewer rows than sequences
    assert scan(vs, seqs=i64(0, 2, FAKE + 8, FAKE, 0, 2, 0)) == bad
    assert scan(vs, seqs=i64(0, 2, FAKE, FAKE + 4, 0, 2, 0)) == bad
    assert scan(vs, seqs=i64(0, 2, FAKE, FAKE, FAKE + 1, 2, 0)) == bad
    assert scan(vs, seqs=i64(0, 2, FAKE, FAKE, 0, -2, 0)) == bad


def test_scan_with_nothing_to_do(vs):
    ok = vs.VIM_OK
    assert scan(vs, batch=0) == ok and scan(vs, d=0) == ok
    assert scan(vs, batch=1, seqs=i64(FAKE, 0, 0, 0, 0, 0, 0)) == ok
    assert vs.lib.causal_ckpt_bytes(2, 17, 24, 16) == 2 * 3 * 24 * 16 * 4
    assert vs.lib.causal_ckpt_bytes(0, 17, 24, 16) == 0 and vs.lib.causal_ckpt_bytes(2, 17, 24, 3) == 0


def step(vs, io=None, batch=2, d=64, N=16, dt=1, seqs=(0, 2, FAKE, FAKE, 0, 2, 0), A=FAKE):
    return vs.lib.causal_scan_step(rows(6, row=0) if io is None else io, A, FAKE, FAKE, batch, d, N, dt,
                                   None if seqs is None else i64(*seqs), None)


def test_step_refusals(vs):
    bad = vs.VIM_ERR_INVALID_ARG
    assert step(vs, seqs=None) == bad
    assert step(vs, seqs=(0, 2, 0, FAKE, 0, 2, 0)) == bad                          # no state to start from
    assert step(vs, seqs=(0, 1, FAKE, FAKE, 0, 2, 0)) == bad
    assert step(vs, seqs=(0, 2, FAKE, FAKE, 0, 1, 0)) == bad
    assert step(vs, rows(6, row=0, r5=(FAKE, 63, 0))) == bad                       # y's rows overlap
    assert step(vs, rows(6, row=0, r0=(0, 64, 0))) == bad
    assert step(vs, A=None) == bad
    assert step(vs, N=5) == vs.VIM_ERR_UNSUPPORTED
    assert step(vs, rows(6, row=0, r0=(FAKE, 1 << 30, 0))) == vs.VIM_ERR_UNSUPPORTED
    assert step(vs, batch=0, seqs=(0, 0, FAKE, FAKE, 0, 2, 0)) == vs.VIM_OK


def scan_bwd(vs, io=None, batch=2, L=8, d=64, N=16, dt=1, cu=None, n=0, ckpt=None, ws=FAKE, nbytes=1 << 40, grads=FAKE):
    return vs.lib.causal_scan_bwd(rows(9) if io is None else io, FAKE, FAKE, FAKE, grads, grads, grads, grads, grads,
                                  batch, L, d, N, dt, cu, n, ckpt, ws, nbytes, None)


def test_scan_bwd_refusals(vs):
    bad = vs.VIM_ERR_INVALID_ARG
    for i in (0, 1, 3, 4, 5, 6, 7):
        assert scan_bwd(vs, rows(9, **{f"r{i}": (0, 600, 64)})) == bad, i
    assert scan_bwd(vs, rows(9, r2=(0, 0, 0))) == bad                              # dz without z
    assert scan_bwd(vs, rows(9, r8=(0, 0, 0))) == bad                              # z without dz
    for i in (6, 7, 8):
        assert scan_bwd(vs, rows(9, **{f"r{i}": (FAKE, 600, 63)})) == bad, i
    for o in (6, 7, 8):
        for i in (0, 1, 2, 5):                                                     # an output over an input
            assert scan_bwd(vs, rows(9, **{f"r{o}": (FAKE, 600, 64), f"r{i}": (FAKE, 600, 64)})) == bad
    assert scan_bwd(vs, grads=None) == bad and scan_bwd(vs, grads=FAKE + 2) == bad
    assert scan_bwd(vs, ckpt=FAKE + 8) == bad
    assert scan_bwd(vs, cu=FAKE, n=2) == bad                                       # packed, batch 2
    assert scan_bwd(vs, N=6) == vs.VIM_ERR_UNSUPPORTED
    need = vs.lib.causal_bwd_workspace_bytes(2, 8, 64, 16, 0)
    assert need > vs.lib.causal_bwd_workspace_bytes(2, 8, 64, 16, 1) > 0
    for ws, nbytes in ((None, need), (FAKE, need - 1), (FAKE + 128, need)):
        assert scan_bwd(vs, ws=ws, nbytes=nbytes) == vs.VIM_ERR_WORKSPACE
    assert scan_bwd(vs, d=0) == vs.VIM_OK
    assert vs.lib.causal_bwd_workspace_bytes(2, 0, 64, 16, 0) == 0


def conv(vs, io=None, w=FAKE, b=FAKE, batch=2, L=8, ch=64, W=4, dt=1, seqs=None):
    return vs.lib.causal_conv(rows(2) if io is None else io, w, b, batch, L, ch, W, 1, dt, seqs, None)


def test_conv_refusals(vs):
    bad, uns = vs.VIM_ERR_INVALID_ARG, vs.VIM_ERR_UNSUPPORTED
    for i in range(2):
        assert conv(vs, rows(2, **{f"r{i}": (0, 600, 64)})) == bad
        assert conv(vs, rows(2, **{f"r{i}": (FAKE + 1, 600, 64)})) == bad
    assert conv(vs, rows(2, r1=(FAKE, 600, 60))) == bad
    assert conv(vs, rows(2, r1=(FAKE, 600, 64), r0=(FAKE, 600, 64))) == bad        # in place
    assert conv(vs, L=2**31 - 8) == uns
    assert conv(vs, w=None) == bad and conv(vs, w=FAKE + 2) == bad and conv(vs, b=FAKE + 1) == bad
    assert conv(vs, W=1) == uns and conv(vs, W=5) == uns
    assert conv(vs, dt=9) == bad and conv(vs, L=-1) == bad
    assert conv(vs, seqs=i64(0, 2, FAKE + 1, FAKE, 0, 2, 0)) == bad
    assert conv(vs, batch=0) == vs.VIM_OK and conv(vs, ch=0) == vs.VIM_OK
    st = lambda seqs, io=None: vs.lib.causal_conv_step(rows(2, row=0) if io is None else io, FAKE, None, 2, 64, 4, 1, 1,
                                                        seqs, None)
    assert st(None) == bad and st(i64(0, 2, 0, FAKE, 0, 2, 0)) == bad
    assert st(i64(0, 2, FAKE, FAKE, 0, 2, 0), rows(2, row=0, r1=(FAKE, 10, 0))) == bad


def test_conv_bwd_refusals(vs):
    bad = vs.VIM_ERR_INVALID_ARG
    def bwd(io=None, b=FAKE, dw=FAKE, db=FAKE, cu=None, n=0, ws=FAKE, nbytes=1 << 40, W=4, L=8, ch=64):
        return vs.lib.causal_conv_bwd(rows(3) if io is None else io, FAKE, b, dw, db, 2, L, ch, W, 1, 1, cu, n, ws, nbytes,
                                      None)
    for i in range(3):
        assert bwd(rows(3, **{f"r{i}": (0, 600, 64)})) == bad
    assert bwd(rows(3, r2=(FAKE, 600, 1))) == bad
    for i in range(2):                                                             # dx over x or dout
        assert bwd(rows(3, r2=(FAKE, 600, 64), **{f"r{i}": (FAKE, 600, 64)})) == bad
    assert bwd(dw=None) == bad and bwd(b=None) == bad and bwd(db=FAKE + 2) == bad
    assert bwd(cu=FAKE, n=2) == bad
    assert bwd(W=7) == vs.VIM_ERR_UNSUPPORTED
    need = vs.lib.causal_conv_bwd_workspace_bytes(2, 8, 64, 4)
    assert need > 0 and bwd(nbytes=need - 1) == vs.VIM_ERR_WORKSPACE and bwd(ws=None) == vs.VIM_ERR_WORKSPACE
    assert bwd(ch=0) == vs.VIM_OK


def test_clip_refusals(vs):
    bad = vs.VIM_ERR_INVALID_ARG
    need = vs.lib.clip_grad_norm_workspace_bytes(2)
    def clip(table, count, max_norm=1.0, norm=FAKE, ws=FAKE, nbytes=need):
        return vs.lib.clip_grad_norm(None if table is None else i64(*table), count, max_norm, norm, ws, nbytes, None)
    one = (FAKE, FAKE, 100, 0)
    assert clip(None, 1) == bad and clip(one, -1) == bad
    assert clip(one, 1, max_norm=-1.0) == bad and clip(one, 1, max_norm=float("nan")) == bad
    assert clip(one, 1, norm=None) == bad and clip(one, 1, norm=FAKE + 2) == bad
    assert clip((0, FAKE, 100, 0), 1) == bad and clip((FAKE, 0, 100, 0), 1) == bad
    assert clip((FAKE + 2, FAKE + 2, 100, 0), 1) == bad
    assert clip((FAKE, FAKE, -1, 0), 1) == bad and clip((FAKE, FAKE, 100, 5), 1) == bad
    assert clip(one + one, 2) == bad                                                # the same tensor twice
    assert clip(one + (FAKE + 396, FAKE + 396, 4, 0), 2) == bad                     # overlapping by an element
    assert clip((FAKE, FAKE + 4, 100, 0), 1) == bad                                 # out over its own input
    assert clip((FAKE, FAKE + 4096, 100, 0, FAKE + 4096 + 200, FAKE + 8192, 100, 1), 2) == bad   # out over another input
    assert clip((FAKE, FAKE, 1 << 60, 1), 1) == vs.VIM_ERR_UNSUPPORTED
    for ws, nbytes in ((None, need), (FAKE, need - 1), (FAKE + 8, need)):
        assert clip(one, 1, ws=ws, nbytes=nbytes) == vs.VIM_ERR_WORKSPACE
    assert vs.lib.clip_grad_norm_workspace_bytes(-1) == 0
    assert vs.lib.clip_grad_norm_workspace_bytes(121) == 2 * vs.lib.clip_grad_norm_workspace_bytes(120)


def test_binding_refuses_cpu_tensors(vs):
    """No launch, no fallback: the binding refuses tensors that are not on a GPU."""
    t = torch.zeros(2, 8, 16)
    p, v = torch.zeros(16, 16), torch.zeros(16)
    with pytest.raises(TypeError):
        vs.causal_scan(t, t, None, t, t, p, v, v)
    with pytest.raises(TypeError):
        vs.causal_scan_step(t[:, 0], t[:, 0], None, t[:, 0], t[:, 0], p, v, v, torch.zeros(2, 16, 16))
    with pytest.raises(TypeError):
        vs.causal_scan_bwd(t, t, None, t, t, p, v, v, t)
    for call in (lambda: vs.causal_conv(t, p[:, :4], v), lambda: vs.causal_conv_step(t[:, 0], p[:, :4], v, t),
                 lambda: vs.causal_conv_bwd(t, p[:, :4], v, t)):
        with pytest.raises(TypeError):
            call()
