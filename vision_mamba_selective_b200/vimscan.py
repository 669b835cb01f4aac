"""Thin ctypes binding of libvimscan.so (declared in include/vimscan.h and, for the causal
operators, include/vimscan_causal.h).

Argument marshalling only: every tensor is checked for device (the current CUDA
device), dtype, shape and contiguity before the library is called, then turned into
raw device pointers and handed to the C ABI together with
the current torch CUDA stream, or ``stream=``, which is then the current one for the whole of
the call.  Every step of the scan runs in the library's sm_100a
kernels; there is no fallback of any kind, and a missing library is an ImportError.
"""
from __future__ import annotations

import ctypes
import functools
import itertools
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvimscan.so")

VIM_OK, VIM_ERR_INVALID_ARG, VIM_ERR_UNSUPPORTED, VIM_ERR_WORKSPACE, VIM_ERR_CUDA, VIM_ERR_TIMEOUT = range(6)
VIM_F32, VIM_BF16 = 0, 1

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m vision_mamba_selective_b200.build` "
        "(nvcc, sm_100a); the selective scan has no other implementation")

lib = ctypes.CDLL(LIB_PATH)

_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
lib.vim_scan_bidir.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                               _i, _i, _i, _i, _i, _vp, _sz, _vp]
lib.vim_scan_bidir.restype = _i
lib.vmamba_cross_scan4.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _i, _i, _i, _i, _i, _i, _vp, _sz, _vp]
lib.vmamba_cross_scan4.restype = _i
lib.vim_scan_bidir_events.argtypes = lib.vim_scan_bidir.argtypes + [_vp]
lib.vim_scan_bidir_events.restype = _i
lib.vmamba_cross_scan4_events.argtypes = lib.vmamba_cross_scan4.argtypes + [_vp]
lib.vmamba_cross_scan4_events.restype = _i
lib.vim_scan_bidir_conv.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                    _i, _i, _i, _i, _i, _vp, _sz, _vp]
lib.vim_scan_bidir_conv.restype = _i
lib.vim_scan_bidir_conv_events.argtypes = lib.vim_scan_bidir_conv.argtypes + [_vp]
lib.vim_scan_bidir_conv_events.restype = _i
_u = ctypes.c_uint
lib.vim_scan_bidir_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                  _i, _i, _i, _i, _i, _u, _vp, _sz, _vp, _vp]
lib.vim_scan_bidir_ex.restype = _i
lib.vmamba_cross_scan4_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _i, _i, _i, _i, _i, _i, _u, _vp, _sz, _vp, _vp]
lib.vmamba_cross_scan4_ex.restype = _i
VIM_FLAG_ZOH_EXACT = 1
lib.vim_scan_bidir_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp]
lib.vim_scan_bidir_bwd.restype = _i
lib.vim_scan_bidir_bwd_events.argtypes = lib.vim_scan_bidir_bwd.argtypes + [_vp]
lib.vim_scan_bidir_bwd_events.restype = _i
# the _bwd arguments with `flags` before the workspace, then the events
lib.vim_scan_bidir_bwd_ex.argtypes = (lib.vim_scan_bidir_bwd.argtypes[:23] + [ctypes.c_uint]
                                      + lib.vim_scan_bidir_bwd.argtypes[23:] + [_vp])
lib.vim_scan_bidir_bwd_ex.restype = _i
# the training pair: the forward scan keeping the derivative's chunk states, and the
# derivative that takes them
lib.vim_scan_bidir_ckpt.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                    _i, _i, _i, _i, _i, _u, _vp, _sz, _vp, _vp]
lib.vim_scan_bidir_ckpt.restype = _i
lib.vim_scan_bidir_bwd_ckpt.argtypes = (lib.vim_scan_bidir_bwd_ex.argtypes[:9] + [_vp]
                                        + lib.vim_scan_bidir_bwd_ex.argtypes[9:])
lib.vim_scan_bidir_bwd_ckpt.restype = _i
lib.vim_scan_ckpt_bytes.argtypes = [_i, _i, _i, _i]
lib.vim_scan_ckpt_bytes.restype = _sz
lib.vim_scan_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
lib.vim_scan_bwd_workspace_bytes.restype = _sz
lib.vim_block_scan.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                               _vp, _sz, _vp, _vp]
lib.vim_block_scan.restype = _i
lib.vim_block_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.vim_block_workspace_bytes.restype = _sz
lib.vmamba_cross_scan4_bwd.argtypes = [_vp] * 17 + [_i, _i, _i, _i, _i, _i, _vp, _sz, _vp]
lib.vmamba_cross_scan4_bwd_ex.argtypes = [_vp] * 17 + [_i, _i, _i, _i, _i, _i, ctypes.c_uint, _vp, _sz, _vp]
lib.vmamba_cross_scan4_bwd_ex.restype = _i
lib.vmamba_cross_scan4_bwd.restype = _i
lib.vmamba_cross_scan4_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
lib.vmamba_cross_scan4_bwd_workspace_bytes.restype = _sz
lib.vim_scan_bidir_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                       _i, _i, _i, _i, _i, _vp]
lib.vim_scan_bidir_noalloc.restype = _i
VIM_NOALLOC_SCRATCH_BYTES = 8 << 20
lib.vim_scan_bidir_conv_bwd_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                           _i, _i, _i, _i, _i, _u, _vp, _sz, _vp]
lib.vim_scan_bidir_conv_bwd_ex.restype = _i
lib.vim_scan_bidir_conv_bwd.argtypes = (lib.vim_scan_bidir_conv_bwd_ex.argtypes[:27]
                                        + lib.vim_scan_bidir_conv_bwd_ex.argtypes[28:])
lib.vim_scan_bidir_conv_bwd.restype = _i
# the training pair with the convolution front
lib.vim_scan_bidir_conv_ckpt.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                         _i, _i, _i, _i, _i, _u, _vp, _sz, _vp, _vp]
lib.vim_scan_bidir_conv_ckpt.restype = _i
lib.vim_scan_bidir_conv_bwd_ckpt.argtypes = (lib.vim_scan_bidir_conv_bwd_ex.argtypes[:11] + [_vp]
                                             + lib.vim_scan_bidir_conv_bwd_ex.argtypes[11:])
lib.vim_scan_bidir_conv_bwd_ckpt.restype = _i
# the training pair of the cross-scan
lib.vmamba_cross_scan4_ckpt.argtypes = [_vp] * 10 + [_i, _i, _i, _i, _i, _i, _u, _vp, _sz, _vp, _vp]
lib.vmamba_cross_scan4_ckpt.restype = _i
lib.vmamba_cross_scan4_bwd_ckpt.argtypes = [_vp] * 18 + [_i, _i, _i, _i, _i, _i, _u, _vp, _sz, _vp]
lib.vmamba_cross_scan4_bwd_ckpt.restype = _i
lib.vmamba_cross_ckpt_bytes.argtypes = [_i, _i, _i, _i, _i]
lib.vmamba_cross_ckpt_bytes.restype = _sz
lib.vim_scan_conv_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i]
lib.vim_scan_conv_bwd_workspace_bytes.restype = _sz
lib.vim_block_scan_bwd.argtypes = [_vp] * 19 + [_i, _i, _i, _i, _i, _vp, _sz, _vp]
lib.vim_block_scan_bwd.restype = _i
lib.vim_block_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.vim_block_bwd_workspace_bytes.restype = _sz
lib.vim_scan_bidir_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                    _i, _i, _i, _i, _i, _u, _i, _vp, _sz, _vp, _vp, _vp]
lib.vim_scan_bidir_host.restype = _i
lib.vim_scan_host_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.vim_scan_host_workspace_bytes.restype = _sz
lib.cross_merge4.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
lib.cross_merge4.restype = _i
lib.vim_scan_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i]
lib.vim_scan_workspace_bytes.restype = _sz
lib.vim_status_string.argtypes = [_i]
lib.vim_status_string.restype = ctypes.c_char_p


class VimScanError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def status_string(status: int) -> str:
    return lib.vim_status_string(int(status)).decode()


def vim_scan_workspace_bytes(which: int, batch: int, L_or_H: int, W: int, channels: int, d_state: int) -> int:
    return int(lib.vim_scan_workspace_bytes(which, batch, L_or_H, W, channels, d_state))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return VIM_F32
    if t.dtype == torch.bfloat16:
        return VIM_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: fp32 or bf16")


def _ptrs(where, ref, specs):
    """Check every tensor the kernels will address and return their data pointers, in
    the order of ``specs`` (None for an absent tensor), before the library is called.

    ``ref`` fixes the device; it must be the current CUDA device (the stream the library
    launches on belongs to it).  ``specs`` holds (name, tensor or None, dtype or None,
    rule) with rule either an exact shape tuple or ("numel", n, last): at least n
    elements with last dimension ``last`` (buffers such as B/C with a per-direction
    stride).  Every tensor must be contiguous.  Raises TypeError (not a CUDA tensor, a
    wrong dtype) or ValueError (device, shape, layout).  One pass per tensor, integer
    device indices and direct size comparisons: this runs on every call, so its cost
    is part of a small problem's launch latency.
    """
    if not isinstance(ref, torch.Tensor) or not ref.is_cuda:
        raise TypeError(f"{where}: inputs must be CUDA tensors")
    dev = ref.get_device()
    cur = torch.cuda.current_device()
    if dev != cur:
        raise ValueError(f"{where}: tensors are on {ref.device} but the current device is cuda:{cur}")
    out = []
    for name, t, dtype, rule in specs:
        if t is None:
            out.append(None)
            continue
        if not isinstance(t, torch.Tensor) or t.get_device() != dev:
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{where}: {name} must be a CUDA tensor")
            raise ValueError(f"{where}: {name} is on {t.device}, the other inputs on {ref.device}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
        if rule[0] == "numel":
            _, n, last = rule
            if t.numel() < n or t.dim() == 0 or t.shape[-1] != last:
                raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}; it needs at least {n} "
                                 f"elements with last dimension {last}")
        elif t.shape != rule:
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(rule)}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
        out.append(t.data_ptr())
    return out


def _out_specs(out, io, act, bc, a_shape, d_shape):
    """The derivative outputs as _ptrs specs, in the library's argument order (none when
    there is no output dict: the inputs were refused before it could be allocated)."""
    if out is None:
        return []
    f32 = torch.float32
    return [("out['du']", out["du"], io, act), ("out['ddelta']", out["ddelta"], io, act),
            ("out['dz']", out["dz"], io, act), ("out['dB']", out["dB"], f32, bc), ("out['dC']", out["dC"], f32, bc),
            ("out['dA']", out["dA"], f32, a_shape), ("out['dD']", out["dD"], f32, d_shape),
            ("out['ddelta_bias']", out["ddelta_bias"], f32, d_shape)]


def _bc_rule(batch, L, N, bc_dir_stride):
    if bc_dir_stride < 0:
        raise ValueError("bc_dir_stride must be >= 0")
    return ("numel", int(bc_dir_stride) + batch * L * N, N)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _on_stream(entry):
    """An entry point whose ``stream=`` is the current stream for the whole of the call, so that
    what it allocates and fills is ordered before its kernels.  Memory of the caller's stream would
    not do: a fill would run there, and the allocator may take a block that kernels of that stream
    still use.  The results are recorded on the caller's stream, so that they outlive their use
    there.  (The inputs are the caller's to order, and to keep until the stream has used them.)"""
    @functools.wraps(entry)
    def call(*args, **kw):
        stream = kw.get("stream")
        if stream is None:
            return entry(*args, **kw)
        caller = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            result = entry(*args, **kw)
        for t in result.values() if isinstance(result, dict) else (result,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(caller)
        return result
    return call


def _workspace(nbytes, workspace, device):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return workspace, nbytes
    # the kernels write all of it: memory of another device, or elements that share their bytes,
    # would be written past
    if not isinstance(workspace, torch.Tensor) or workspace.device != device:
        raise TypeError(f"workspace must be a tensor on {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace too small: need {nbytes} bytes")
    return workspace, workspace.numel() * workspace.element_size()


def _events(events):
    """Raw cudaEvent_t handles of torch CUDA events (created by recording them once)."""
    handles = []
    for e in events:
        if e.cuda_event == 0:
            e.record()
        handles.append(e.cuda_event)
    return (ctypes.c_void_p * len(handles))(*handles)


def _bidir(name, u, conv_w, conv_b, delta, z, B, C, A, D, delta_bias, y, bc_dir_stride, workspace, stream,
           events, zoh, ckpt=None):
    batch, L, Di = u.shape
    N = B.shape[-1]
    dt = _dtype_code(u)
    act = (batch, L, Di)
    bc = _bc_rule(batch, L, N, bc_dir_stride)
    if y is None:
        y = torch.empty_like(u)
    conv = conv_w is not None or conv_b is not None
    f32, io = torch.float32, u.dtype
    pu, pcw, pcb, pdelta, pz, pB, pC, pA, pD, pbias, py = _ptrs(name, u, [
        ("x" if conv else "u", u, None, act), ("conv_w", conv_w, f32, (2, Di, 3)), ("conv_b", conv_b, f32, (2, Di)),
        ("delta", delta, io, act), ("z", z, io, act), ("B", B, io, bc), ("C", C, io, bc),
        ("A", A, f32, (2, Di, N)), ("D", D, f32, (2, Di)), ("delta_bias", delta_bias, f32, (2, Di)),
        ("y", y, io, act)])
    ws, ws_bytes = _workspace(vim_scan_workspace_bytes(0, batch, L, 0, Di, N), workspace, u.device)
    if ckpt is not None:
        (pk,) = _ptrs(name, u, [("ckpt", ckpt, f32, ckpt_shape(batch, L, Di, N))])
        tail = (batch, L, Di, N, dt, VIM_FLAG_ZOH_EXACT if zoh else 0, None if ws is None else ws.data_ptr(),
                ws_bytes, _stream(stream), None if events is None else _events(events))
        if conv:
            st = lib.vim_scan_bidir_conv_ckpt(pu, pcw, pcb, pdelta, pz, pB, pC, int(bc_dir_stride), pA, pD, pbias,
                                              py, pk, *tail)
        else:
            st = lib.vim_scan_bidir_ckpt(pu, pdelta, pz, pB, pC, int(bc_dir_stride), pA, pD, pbias, py, pk, *tail)
        if st != VIM_OK:
            raise VimScanError(st, name)
        return y
    pre = (pu, pcw, pcb) if conv or zoh else (pu,)
    args = pre + (pdelta, pz, pB, pC, int(bc_dir_stride), pA, pD, pbias, py, batch, L, Di, N, dt)
    tail = (None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream))
    ev = None if events is None else _events(events)
    if zoh:
        st = lib.vim_scan_bidir_ex(*args, VIM_FLAG_ZOH_EXACT, *tail, ev)
    elif conv:
        st = (lib.vim_scan_bidir_conv(*args, *tail) if ev is None
              else lib.vim_scan_bidir_conv_events(*args, *tail, ev))
    else:
        st = lib.vim_scan_bidir(*args, *tail) if ev is None else lib.vim_scan_bidir_events(*args, *tail, ev)
    if st != VIM_OK:
        raise VimScanError(st, name)
    return y


def ckpt_shape(batch, L, d_inner, d_state):
    """Shape of the checkpoints vim_scan_bidir(ckpt=...) writes and
    vim_scan_bidir_bwd(ckpt=...) reads: [batch, ceil(L / 32), 2, d_state, d_inner]."""
    return (batch, (L + 31) // 32, 2, d_state, d_inner)


@_on_stream
def vim_scan_bidir(u, delta, z, B, C, A, D, delta_bias, *, y=None, bc_dir_stride=0,
                   workspace=None, stream=None, events=None, zoh=False, ckpt=None):
    """Vim bidirectional selective scan, (y^f + y^b) * silu(z); see include/vimscan.h.

    u, delta, z: [batch, L, d_inner]; B, C: [batch, L, d_state] (or a larger buffer
    whose backward copy starts ``bc_dir_stride`` elements in); A: [2, d_inner,
    d_state] fp32; D, delta_bias: [2, d_inner] fp32.  Returns y [batch, L, d_inner].
    zoh=True takes the exact zero-order-hold Bbar (VIM_FLAG_ZOH_EXACT).  ``ckpt``, an
    fp32 tensor of ckpt_shape(...), receives the states the derivative needs
    (vim_scan_bidir_ckpt) for vim_scan_bidir_bwd(ckpt=...).
    """
    return _bidir("vim_scan_bidir", u, None, None, delta, z, B, C, A, D, delta_bias, y, bc_dir_stride,
                  workspace, stream, events, zoh, ckpt)


@_on_stream
def vim_scan_bidir_conv(x, conv_w, conv_b, delta, z, B, C, A, D, delta_bias, *, y=None, bc_dir_stride=0,
                        workspace=None, stream=None, events=None, zoh=False, ckpt=None):
    """vim_scan_bidir with the pathways' kernel-3 convolution + SiLU front fused in.

    x, delta, z: [batch, L, d_inner]; conv_w: [2, d_inner, 3] fp32; conv_b: [2, d_inner]
    fp32; the rest as in vim_scan_bidir.  Returns y [batch, L, d_inner].  A missing
    half of the front (conv_w or conv_b None) is rejected by the library.  ``ckpt`` as in
    vim_scan_bidir (vim_scan_bidir_conv_ckpt), for vim_scan_bidir_conv_bwd(ckpt=...).
    """
    return _bidir("vim_scan_bidir_conv", x, conv_w, conv_b, delta, z, B, C, A, D, delta_bias, y,
                  bc_dir_stride, workspace, stream, events, zoh, ckpt)


def vim_scan_bwd_workspace_bytes(batch, L, d_inner, d_state, separate_bc):
    return int(lib.vim_scan_bwd_workspace_bytes(batch, L, d_inner, d_state, int(bool(separate_bc))))


@_on_stream
def vim_scan_bidir_bwd(u, delta, z, B, C, A, D, delta_bias, dout, *, bc_dir_stride=0, workspace=None,
                       stream=None, out=None, events=None, zoh=False, ckpt=None):
    """Derivatives of vim_scan_bidir (first-order Bbar, or with ``zoh`` the exact
    zero-order hold) for a loss whose derivative with respect to y is ``dout``; see
    include/vimscan.h.

    Returns a dict: du, ddelta (w.r.t. the raw delta), dz (None without z), in the
    input dtype; dB and dC (fp32, shaped like B and C); dA [2, d_inner, d_state], dD
    and ddelta_bias [2, d_inner] (fp32).  ``out`` may hold those tensors from an
    earlier call to be written again; ``events`` 4 CUDA events (see
    vim_scan_bidir_bwd_events).  ``ckpt``: the checkpoints vim_scan_bidir(ckpt=...) wrote
    for the same inputs (vim_scan_bidir_bwd_ckpt), which replace the derivative's own
    forward summaries.
    """
    batch, L, Di = u.shape
    N = B.shape[-1]
    dt = _dtype_code(u)
    dev = u.device
    act = (batch, L, Di)
    bc = _bc_rule(batch, L, N, bc_dir_stride)
    if out is not None:
        if z is not None and out["dz"] is None:
            raise ValueError("vim_scan_bidir_bwd: out['dz'] is needed when z is given")
    elif isinstance(u, torch.Tensor) and u.is_cuda:
        out = dict(du=torch.empty_like(u), ddelta=torch.empty_like(u),
                   dz=torch.empty_like(u) if z is not None else None,
                   dB=torch.zeros(B.shape, dtype=torch.float32, device=dev),
                   dC=torch.zeros(C.shape, dtype=torch.float32, device=dev),
                   dA=torch.empty((2, Di, N), dtype=torch.float32, device=dev),
                   dD=torch.empty((2, Di), dtype=torch.float32, device=dev),
                   ddelta_bias=torch.empty((2, Di), dtype=torch.float32, device=dev))
    f32, io = torch.float32, u.dtype
    ptrs = _ptrs("vim_scan_bidir_bwd", u, [
        ("u", u, None, act), ("delta", delta, io, act), ("z", z, io, act), ("B", B, io, bc), ("C", C, io, bc),
        ("A", A, f32, (2, Di, N)), ("D", D, f32, (2, Di)), ("delta_bias", delta_bias, f32, (2, Di)),
        ("dout", dout, io, act)] + _out_specs(out, io, act, bc, (2, Di, N), (2, Di)))
    ws, ws_bytes = _workspace(vim_scan_bwd_workspace_bytes(batch, L, Di, N, bc_dir_stride > 0), workspace, dev)
    if ckpt is not None:
        (pk,) = _ptrs("vim_scan_bidir_bwd", u, [("ckpt", ckpt, f32, ckpt_shape(batch, L, Di, N))])
        st = lib.vim_scan_bidir_bwd_ckpt(
            *ptrs[:5], int(bc_dir_stride), *ptrs[5:8], pk, *ptrs[8:], batch, L, Di, N, dt,
            VIM_FLAG_ZOH_EXACT if zoh else 0, None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream),
            None if events is None else _events(events))
        if st != VIM_OK:
            raise VimScanError(st, "vim_scan_bidir_bwd")
        return out
    if zoh:
        fn = lib.vim_scan_bidir_bwd_ex
        flags, extra = (VIM_FLAG_ZOH_EXACT,), (None if events is None else _events(events),)
    else:
        fn = lib.vim_scan_bidir_bwd if events is None else lib.vim_scan_bidir_bwd_events
        flags, extra = (), (() if events is None else (_events(events),))
    st = fn(
        *ptrs[:5], int(bc_dir_stride), *ptrs[5:],
        batch, L, Di, N, dt, *flags, None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream), *extra)
    if st != VIM_OK:
        raise VimScanError(st, "vim_scan_bidir_bwd")
    return out


def vim_scan_conv_bwd_workspace_bytes(batch, L, d_inner, d_state, dtype_code, separate_bc):
    return int(lib.vim_scan_conv_bwd_workspace_bytes(batch, L, d_inner, d_state, dtype_code, int(bool(separate_bc))))


@_on_stream
def vim_scan_bidir_conv_bwd(x, conv_w, conv_b, delta, z, B, C, A, D, delta_bias, dout, *, bc_dir_stride=0,
                            workspace=None, stream=None, out=None, zoh=False, ckpt=None):
    """Derivatives of vim_scan_bidir_conv (first-order Bbar, or with ``zoh`` the exact
    hold) for a loss whose derivative with respect to y is ``dout``; see
    include/vimscan.h.

    Returns a dict: dx, ddelta (w.r.t. the raw delta), dz (None without z) in the input
    dtype; dconv_w [2, d_inner, 3] and dconv_b [2, d_inner] fp32; dB, dC (fp32, shaped
    like B and C), dA [2, d_inner, d_state], dD and ddelta_bias [2, d_inner] fp32.
    ``out`` may hold those tensors from an earlier call to be written again.  ``ckpt``: the
    checkpoints vim_scan_bidir_conv(ckpt=...) wrote for the same inputs
    (vim_scan_bidir_conv_bwd_ckpt).
    """
    batch, L, Di = x.shape
    N = B.shape[-1]
    dt = _dtype_code(x)
    dev = x.device
    act = (batch, L, Di)
    bc = _bc_rule(batch, L, N, bc_dir_stride)
    if out is not None:
        if z is not None and out["dz"] is None:
            raise ValueError("vim_scan_bidir_conv_bwd: out['dz'] is needed when z is given")
    elif isinstance(x, torch.Tensor) and x.is_cuda:
        e32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)
        out = dict(dx=torch.empty_like(x), ddelta=torch.empty_like(x), dz=torch.empty_like(x) if z is not None else None,
                   dconv_w=e32(2, Di, 3), dconv_b=e32(2, Di),
                   dB=torch.zeros(B.shape, dtype=torch.float32, device=dev),
                   dC=torch.zeros(C.shape, dtype=torch.float32, device=dev),
                   dA=e32(2, Di, N), dD=e32(2, Di), ddelta_bias=e32(2, Di))
    f32, io = torch.float32, x.dtype
    specs = [("x", x, None, act), ("conv_w", conv_w, f32, (2, Di, 3)), ("conv_b", conv_b, f32, (2, Di)),
             ("delta", delta, io, act), ("z", z, io, act), ("B", B, io, bc), ("C", C, io, bc),
             ("A", A, f32, (2, Di, N)), ("D", D, f32, (2, Di)), ("delta_bias", delta_bias, f32, (2, Di)),
             ("dout", dout, io, act)]
    if out is not None:
        specs += [("out['dx']", out["dx"], io, act), ("out['dconv_w']", out["dconv_w"], f32, (2, Di, 3)),
                  ("out['dconv_b']", out["dconv_b"], f32, (2, Di)), ("out['ddelta']", out["ddelta"], io, act),
                  ("out['dz']", out["dz"], io, act), ("out['dB']", out["dB"], f32, bc),
                  ("out['dC']", out["dC"], f32, bc), ("out['dA']", out["dA"], f32, (2, Di, N)),
                  ("out['dD']", out["dD"], f32, (2, Di)), ("out['ddelta_bias']", out["ddelta_bias"], f32, (2, Di))]
    ptrs = _ptrs("vim_scan_bidir_conv_bwd", x, specs)
    ws, ws_bytes = _workspace(vim_scan_conv_bwd_workspace_bytes(batch, L, Di, N, dt, bc_dir_stride > 0), workspace,
                              dev)
    if ckpt is not None:
        (pk,) = _ptrs("vim_scan_bidir_conv_bwd", x, [("ckpt", ckpt, f32, ckpt_shape(batch, L, Di, N))])
        st = lib.vim_scan_bidir_conv_bwd_ckpt(
            *ptrs[:7], int(bc_dir_stride), *ptrs[7:10], pk, *ptrs[10:], batch, L, Di, N, dt,
            VIM_FLAG_ZOH_EXACT if zoh else 0, None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream))
    else:
        st = lib.vim_scan_bidir_conv_bwd_ex(
            *ptrs[:7], int(bc_dir_stride), *ptrs[7:], batch, L, Di, N, dt, VIM_FLAG_ZOH_EXACT if zoh else 0,
            None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream))
    if st != VIM_OK:
        raise VimScanError(st, "vim_scan_bidir_conv_bwd")
    return out


@_on_stream
def vmamba_cross_scan4_bwd(u, delta, z, B, C, A, D, delta_bias, dout, *, workspace=None, stream=None, out=None,
                           zoh=False, ckpt=None):
    """Derivatives of vmamba_cross_scan4 (first-order Bbar, or with ``zoh`` the exact
    zero-order hold) for a loss whose derivative
    with respect to y is ``dout``; see include/vimscan.h.  Returns a dict: du, ddelta, dz
    (None without z) in the input dtype; dB, dC [4, batch, H*W, N], dA [4, C, N], dD and
    ddelta_bias [4, C] in fp32.  ``out`` may hold those tensors from an earlier call.
    ``ckpt``: the checkpoints vmamba_cross_scan4(ckpt=...) wrote for the same inputs
    (vmamba_cross_scan4_bwd_ckpt).
    """
    batch, H, W, Ch = u.shape
    N = B.shape[-1]
    dev = u.device
    act = (batch, H, W, Ch)
    bc = (4, batch, H * W, N)
    if out is not None:
        if z is not None and out["dz"] is None:
            raise ValueError("vmamba_cross_scan4_bwd: out['dz'] is needed when z is given")
    elif isinstance(u, torch.Tensor) and u.is_cuda:
        e32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)
        out = dict(du=torch.empty_like(u), ddelta=torch.empty_like(u), dz=torch.empty_like(u) if z is not None else None,
                   dB=e32(*B.shape), dC=e32(*C.shape), dA=e32(4, Ch, N), dD=e32(4, Ch), ddelta_bias=e32(4, Ch))
    f32, io = torch.float32, u.dtype
    ptrs = _ptrs("vmamba_cross_scan4_bwd", u, [
        ("u", u, None, act), ("delta", delta, io, act), ("z", z, io, act), ("B", B, io, bc), ("C", C, io, bc),
        ("A", A, f32, (4, Ch, N)), ("D", D, f32, (4, Ch)), ("delta_bias", delta_bias, f32, (4, Ch)),
        ("dout", dout, io, act)] + _out_specs(out, io, act, bc, (4, Ch, N), (4, Ch)))
    ws, ws_bytes = _workspace(int(lib.vmamba_cross_scan4_bwd_workspace_bytes(batch, H, W, Ch, N)), workspace, dev)
    if ckpt is not None:
        (pk,) = _ptrs("vmamba_cross_scan4_bwd", u, [("ckpt", ckpt, f32, cross_ckpt_shape(batch, H, W, Ch, N))])
        st = lib.vmamba_cross_scan4_bwd_ckpt(
            *ptrs[:8], pk, *ptrs[8:], batch, H, W, Ch, N, _dtype_code(u), VIM_FLAG_ZOH_EXACT if zoh else 0,
            None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream))
    else:
        fn = lib.vmamba_cross_scan4_bwd_ex if zoh else lib.vmamba_cross_scan4_bwd
        flags = (VIM_FLAG_ZOH_EXACT,) if zoh else ()
        st = fn(
            *ptrs,
            batch, H, W, Ch, N, _dtype_code(u), *flags, None if ws is None else ws.data_ptr(), ws_bytes,
            _stream(stream))
    if st != VIM_OK:
        raise VimScanError(st, "vmamba_cross_scan4_bwd")
    return out


def vim_block_workspace_bytes(batch, L, d_inner, d_state):
    return int(lib.vim_block_workspace_bytes(batch, L, d_inner, d_state))


@_on_stream
def vim_block_scan(x, Wx, Wdt, dt_bias, A, D, z, *, conv_w=None, conv_b=None, y=None, workspace=None,
                   stream=None, events=None):
    """The Vim block's two S6 modules from their common input x with their own
    projections (x_proj on the tensor cores, dt_proj inside the scan) and optionally
    the convolution front; see include/vimscan.h.  bf16 x, z, Wx [2, d_inner, 2N+1];
    fp32 Wdt, dt_bias, D [2, d_inner], A [2, d_inner, N].  Returns y [batch, L, d_inner].
    """
    batch, L, Di = x.shape
    N = A.shape[-1]
    act = (batch, L, Di)
    if y is None and isinstance(x, torch.Tensor) and x.is_cuda:
        y = torch.empty_like(x)
    f32, io = torch.float32, x.dtype
    ptrs = _ptrs("vim_block_scan", x, [
        ("x", x, None, act), ("conv_w", conv_w, f32, (2, Di, 3)), ("conv_b", conv_b, f32, (2, Di)),
        ("Wx", Wx, io, (2, Di, 2 * N + 1)), ("Wdt", Wdt, f32, (2, Di)), ("dt_bias", dt_bias, f32, (2, Di)),
        ("A", A, f32, (2, Di, N)), ("D", D, f32, (2, Di)), ("z", z, io, act), ("y", y, io, act)])
    ws, ws_bytes = _workspace(vim_block_workspace_bytes(batch, L, Di, N), workspace, x.device)
    st = lib.vim_block_scan(
        *ptrs,
        batch, L, Di, N, _dtype_code(x), None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream),
        None if events is None else _events(events))
    if st != VIM_OK:
        raise VimScanError(st, "vim_block_scan")
    return y


def vim_block_bwd_workspace_bytes(batch, L, d_inner, d_state):
    return int(lib.vim_block_bwd_workspace_bytes(batch, L, d_inner, d_state))


@_on_stream
def vim_block_scan_bwd(x, Wx, Wdt, dt_bias, A, D, z, dout, *, conv_w=None, conv_b=None, workspace=None, stream=None,
                       out=None):
    """Derivatives of vim_block_scan for a loss whose derivative with respect to y is
    ``dout``; see include/vimscan.h.  bf16 x, z, dout, Wx.

    Returns a dict: dx, dz (None without z) in bf16; dWx [2, d_inner, 2N+1], dWdt,
    ddt_bias, dD [2, d_inner], dA [2, d_inner, N] fp32; dconv_w [2, d_inner, 3] and
    dconv_b [2, d_inner] fp32 with the convolution front (else None).  ``out`` may hold
    those tensors from an earlier call.
    """
    batch, L, Di = x.shape
    N = A.shape[-1]
    NO = 2 * N + 1
    dev = x.device
    act = (batch, L, Di)
    conv = conv_w is not None
    if out is not None:
        if (z is not None) != (out["dz"] is not None) or conv != (out["dconv_w"] is not None):
            raise ValueError("vim_block_scan_bwd: out['dz'] and out['dconv_w'] must match z and conv_w")
    elif isinstance(x, torch.Tensor) and x.is_cuda:
        e32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)
        out = dict(dx=torch.empty_like(x), dz=torch.empty_like(x) if z is not None else None, dWx=e32(2, Di, NO),
                   dWdt=e32(2, Di), ddt_bias=e32(2, Di), dA=e32(2, Di, N), dD=e32(2, Di),
                   dconv_w=e32(2, Di, 3) if conv else None, dconv_b=e32(2, Di) if conv else None)
    f32, io = torch.float32, x.dtype
    specs = [("x", x, None, act), ("conv_w", conv_w, f32, (2, Di, 3)), ("conv_b", conv_b, f32, (2, Di)),
             ("Wx", Wx, io, (2, Di, NO)), ("Wdt", Wdt, f32, (2, Di)), ("dt_bias", dt_bias, f32, (2, Di)),
             ("A", A, f32, (2, Di, N)), ("D", D, f32, (2, Di)), ("z", z, io, act), ("dout", dout, io, act)]
    if out is not None:
        specs += [("out['dx']", out["dx"], io, act), ("out['dconv_w']", out["dconv_w"], f32, (2, Di, 3)),
                  ("out['dconv_b']", out["dconv_b"], f32, (2, Di)), ("out['dWx']", out["dWx"], f32, (2, Di, NO)),
                  ("out['dWdt']", out["dWdt"], f32, (2, Di)), ("out['ddt_bias']", out["ddt_bias"], f32, (2, Di)),
                  ("out['dA']", out["dA"], f32, (2, Di, N)), ("out['dD']", out["dD"], f32, (2, Di)),
                  ("out['dz']", out["dz"], io, act)]
    ptrs = _ptrs("vim_block_scan_bwd", x, specs)
    ws, ws_bytes = _workspace(vim_block_bwd_workspace_bytes(batch, L, Di, N), workspace, dev)
    st = lib.vim_block_scan_bwd(*ptrs, batch, L, Di, N, _dtype_code(x), None if ws is None else ws.data_ptr(),
                                ws_bytes, _stream(stream))
    if st != VIM_OK:
        raise VimScanError(st, "vim_block_scan_bwd")
    return out


@_on_stream
def vim_scan_bidir_noalloc(u, delta, z, B, C, A, D, delta_bias, *, y=None, bc_dir_stride=0, stream=None):
    """vim_scan_bidir without a workspace, for callers that cannot allocate device memory.

    The chunk carries live in a fixed buffer inside the library
    (VIM_NOALLOC_SCRATCH_BYTES), shared by every call: calls must not overlap on the GPU.
    Problems needing more scratch than that raise VimScanError (VIM_ERR_WORKSPACE).
    ``y`` must be given by callers that cannot allocate; otherwise it is allocated here.
    """
    batch, L, Di = u.shape
    N = B.shape[-1]
    dt = _dtype_code(u)
    act = (batch, L, Di)
    bc = _bc_rule(batch, L, N, bc_dir_stride)
    if y is None and isinstance(u, torch.Tensor) and u.is_cuda:
        y = torch.empty_like(u)
    f32, io = torch.float32, u.dtype
    ptrs = _ptrs("vim_scan_bidir_noalloc", u, [
        ("u", u, None, act), ("delta", delta, io, act), ("z", z, io, act), ("B", B, io, bc), ("C", C, io, bc),
        ("A", A, f32, (2, Di, N)), ("D", D, f32, (2, Di)), ("delta_bias", delta_bias, f32, (2, Di)),
        ("y", y, io, act)])
    st = lib.vim_scan_bidir_noalloc(
        *ptrs[:5], int(bc_dir_stride), *ptrs[5:],
        batch, L, Di, N, dt, _stream(stream))
    if st != VIM_OK:
        raise VimScanError(st, "vim_scan_bidir_noalloc")
    return y


def cross_ckpt_shape(batch, H, W, channels, d_state):
    """Shape of the cross-scan's checkpoints (vmamba_cross_scan4(ckpt=...),
    vmamba_cross_scan4_bwd(ckpt=...)): [2 pairs, batch, ceil(H*W / 32), 2, d_state, C]."""
    return (2,) + ckpt_shape(batch, H * W, channels, d_state)


@_on_stream
def vmamba_cross_scan4(u, delta, z, B, C, A, D, delta_bias, *, y=None, workspace=None, stream=None,
                       events=None, zoh=False, ckpt=None):
    """VMamba four-direction cross-scan with CS-Merge; see include/vimscan.h.

    u, delta, z: [batch, H, W, C]; B, C: [4, batch, H*W, d_state] by grid position;
    A: [4, C, d_state] fp32; D, delta_bias: [4, C] fp32.  Returns y [batch, H, W, C].
    zoh=True takes the exact zero-order-hold Bbar (VIM_FLAG_ZOH_EXACT).  ``ckpt``, an fp32
    tensor of cross_ckpt_shape(...), receives the states vmamba_cross_scan4_bwd(ckpt=...)
    takes (vmamba_cross_scan4_ckpt).
    """
    batch, H, W, Ch = u.shape
    N = B.shape[-1]
    dt = _dtype_code(u)
    act = (batch, H, W, Ch)
    bc = (4, batch, H * W, N)
    if y is None:
        y = torch.empty_like(u)
    f32, io = torch.float32, u.dtype
    args = tuple(_ptrs("vmamba_cross_scan4", u, [
        ("u", u, None, act), ("delta", delta, io, act), ("z", z, io, act), ("B", B, io, bc), ("C", C, io, bc),
        ("A", A, f32, (4, Ch, N)), ("D", D, f32, (4, Ch)), ("delta_bias", delta_bias, f32, (4, Ch)),
        ("y", y, io, act)])) + (batch, H, W, Ch, N, dt)
    ws, ws_bytes = _workspace(vim_scan_workspace_bytes(1, batch, H, W, Ch, N), workspace, u.device)
    tail = (None if ws is None else ws.data_ptr(), ws_bytes, _stream(stream))
    ev = None if events is None else _events(events)
    if ckpt is not None:
        (pk,) = _ptrs("vmamba_cross_scan4", u, [("ckpt", ckpt, f32, cross_ckpt_shape(batch, H, W, Ch, N))])
        st = lib.vmamba_cross_scan4_ckpt(*args[:9], pk, *args[9:], VIM_FLAG_ZOH_EXACT if zoh else 0, *tail, ev)
    elif zoh:
        st = lib.vmamba_cross_scan4_ex(*args, VIM_FLAG_ZOH_EXACT, *tail, ev)
    elif ev is None:
        st = lib.vmamba_cross_scan4(*args, *tail)
    else:
        st = lib.vmamba_cross_scan4_events(*args, *tail, ev)
    if st != VIM_OK:
        raise VimScanError(st, "vmamba_cross_scan4")
    return y


@_on_stream
def cross_merge4(ys, z, H, W, *, y=None, stream=None):
    """CS-Merge alone: ys [4, batch, H*W, C] in scan order -> y [batch, H, W, C]."""
    _, batch, L, Ch = ys.shape
    if ys.shape[0] != 4 or L != H * W:
        raise ValueError("ys must be [4, batch, H*W, C]")
    act = (batch, H, W, Ch)
    dt = _dtype_code(ys)
    if y is None and isinstance(ys, torch.Tensor) and ys.is_cuda:
        y = torch.empty((batch, H, W, Ch), dtype=ys.dtype, device=ys.device)
    pys, pz, py = _ptrs("cross_merge4", ys, [("ys", ys, None, tuple(ys.shape)), ("z", z, ys.dtype, act),
                                             ("y", y, ys.dtype, act)])
    st = lib.cross_merge4(pys, pz, py, batch, H, W, Ch, dt, _stream(stream))
    if st != VIM_OK:
        raise VimScanError(st, "cross_merge4")
    return y


def vim_scan_host_workspace_bytes(batch, L, d_inner, d_state, dtype_code, slices, two_bc):
    return int(lib.vim_scan_host_workspace_bytes(batch, L, d_inner, d_state, dtype_code, slices, int(bool(two_bc))))


_copy_streams = {}


def _host_streams(device):
    """Two non-blocking streams per device for the host entry's uploads and downloads."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if idx not in _copy_streams:
        _copy_streams[idx] = (torch.cuda.Stream(idx), torch.cuda.Stream(idx))
    return _copy_streams[idx]


@_on_stream
def vim_scan_bidir_host(u, delta, z, B, C, A, D, delta_bias, *, y=None, bc_dir_stride=0, slices=4,
                        workspace=None, stream=None, upload=None, download=None, zoh=False):
    """vim_scan_bidir for activations in host memory; see include/vimscan.h.

    u, delta, z, B, C: CPU tensors shaped as for vim_scan_bidir (pinned memory lets the
    copies overlap the scan); A, D, delta_bias: CUDA tensors on the current device.
    Returns y, a CPU tensor (pinned when allocated here), complete once ``stream``
    (default: the current stream) has reached the end of the call.
    """
    if not all(isinstance(t, torch.Tensor) for t in (u, delta, B, C)):
        raise TypeError("vim_scan_bidir_host: u, delta, B and C must be tensors")
    batch, L, Di = u.shape
    N = B.shape[-1]
    dt = _dtype_code(u)
    act = (batch, L, Di)
    bc = _bc_rule(batch, L, N, bc_dir_stride)
    if y is None:
        y = torch.empty(act, dtype=u.dtype, pin_memory=True)
    for name, t, rule in (("u", u, act), ("delta", delta, act), ("z", z, act), ("B", B, bc), ("C", C, bc),
                          ("y", y, act)):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
            raise TypeError(f"vim_scan_bidir_host: {name} must be a CPU tensor")
        if t.dtype != u.dtype:
            raise TypeError(f"vim_scan_bidir_host: {name} must be {u.dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"vim_scan_bidir_host: {name} must be contiguous")
        if rule[0] == "numel":
            if t.numel() < rule[1] or t.dim() == 0 or t.shape[-1] != rule[2]:
                raise ValueError(f"vim_scan_bidir_host: {name} has shape {tuple(t.shape)}; it needs at least "
                                 f"{rule[1]} elements with last dimension {rule[2]}")
        elif t.shape != rule:
            raise ValueError(f"vim_scan_bidir_host: {name} has shape {tuple(t.shape)}, expected {rule}")
    f32 = torch.float32
    pA, pD, pbias = _ptrs("vim_scan_bidir_host", A, [("A", A, f32, (2, Di, N)), ("D", D, f32, (2, Di)),
                                                     ("delta_bias", delta_bias, f32, (2, Di))])
    dev = A.device
    nbytes = vim_scan_host_workspace_bytes(batch, L, Di, N, dt, slices, bc_dir_stride > 0)
    ws, ws_bytes = _workspace(nbytes, workspace, dev)
    if upload is None or download is None:
        up, down = _host_streams(dev)
        upload = upload or up
        download = download or down
    st = lib.vim_scan_bidir_host(
        u.data_ptr(), delta.data_ptr(), None if z is None else z.data_ptr(), B.data_ptr(), C.data_ptr(),
        int(bc_dir_stride), pA, pD, pbias, y.data_ptr(), batch, L, Di, N, dt,
        VIM_FLAG_ZOH_EXACT if zoh else 0, int(slices), None if ws is None else ws.data_ptr(), ws_bytes,
        _stream(stream), upload.cuda_stream, download.cuda_stream)
    if st != VIM_OK:
        raise VimScanError(st, "vim_scan_bidir_host")
    return y


# ---------------------------------------------------------------------------
# causal operators
# ---------------------------------------------------------------------------
lib.causal_scan.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp]
lib.causal_scan.restype = _i
lib.causal_scan_step.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]
lib.causal_scan_step.restype = _i
lib.causal_ckpt_bytes.argtypes = [_i, _i, _i, _i]
lib.causal_ckpt_bytes.restype = _sz
lib.causal_scan_bwd.argtypes = [_vp] * 9 + [_i, _i, _i, _i, _i, _vp, _i, _vp, _vp, _sz, _vp]
lib.causal_scan_bwd.restype = _i
lib.causal_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
lib.causal_bwd_workspace_bytes.restype = _sz
lib.causal_conv.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp]
lib.causal_conv.restype = _i
lib.causal_conv_step.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp]
lib.causal_conv_step.restype = _i
lib.causal_conv_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _vp, _sz, _vp]
lib.causal_conv_bwd.restype = _i
lib.causal_conv_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.causal_conv_bwd_workspace_bytes.restype = _sz
lib.clip_grad_norm.argtypes = [_vp, _i, ctypes.c_float, _vp, _vp, _sz, _vp]
lib.clip_grad_norm.restype = _i
lib.clip_grad_norm_workspace_bytes.argtypes = [_i]
lib.clip_grad_norm_workspace_bytes.restype = _sz

# The structs of the causal entry points (vim_scan_io and the like, vim_sequences, vim_tensor)
# hold nothing but 64-bit values, so they are handed over as packed bytes of those.
_i64x = {n: struct.Struct(f"{n}q").pack for n in (6, 7, 9, 18, 27)}

_raw_stream = torch._C._cuda_getCurrentRawStream   # of a device index


def _check_ref(where, ref):
    """The device index of the call: that of ``ref``, which must be the current one."""
    if not isinstance(ref, torch.Tensor) or not ref.is_cuda:
        raise TypeError(f"{where}: inputs must be CUDA tensors")
    dev = ref.get_device()
    cur = torch.cuda.current_device()
    if dev != cur:
        raise ValueError(f"{where}: tensors are on {ref.device} but the current device is cuda:{cur}")
    return dev


def _on_device(where, name, t, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{where}: {name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{where}: {name} is on {t.device}, the other inputs on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(where, name, t, dtype, shape, dev, packed):
    """vim_rows of activation ``t``: [batch, L, c] (or [L, c] when ``packed``), or [batch, c]
    for single tokens; any strides with the channels contiguous."""
    if t is None:
        return 0, 0, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _on_device(where, name, t, dtype, shape, dev)
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{where}: the channels of {name} must be contiguous")
    if len(st) == 3:
        return t.data_ptr(), st[0], st[1]
    return (t.data_ptr(), 0, st[0]) if packed else (t.data_ptr(), st[0], 0)


def _table(where, name, t, dtype, shape, dev):
    """Address of contiguous tensor ``t`` (None for None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _on_device(where, name, t, dtype, shape, dev)
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    return t.data_ptr()


def _offsets(where, cu_seqlens):
    """Number of sequences that ``cu_seqlens`` lists (0 for None)."""
    if cu_seqlens is None:
        return 0
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError(f"{where}: cu_seqlens must be a 1-dimensional tensor of n_seqs + 1 offsets")
    return cu_seqlens.numel() - 1


def _sequences(where, dev, n_rows, cu_seqlens, state, state_out, slots, fresh, state_dtype, state_shape):
    """vim_sequences of a call on ``n_rows`` batch rows, with every table checked."""
    n = n_rows if cu_seqlens is None else _offsets(where, cu_seqlens)
    pcu = _table(where, "cu_seqlens", cu_seqlens, torch.int32, (n + 1,), dev)
    if state is None and state_out is None:
        if slots is not None or fresh is not None:
            raise ValueError(f"{where}: slots and fresh need a state")
        return None if pcu is None else _i64x[7](pcu, n, 0, 0, 0, 0, 0)
    if state is None and fresh is not None:
        raise ValueError(f"{where}: fresh needs a state")
    if state_out is None:
        state_out = state
    if state_out.dim() != 1 + len(state_shape) or tuple(state_out.shape[1:]) != state_shape:
        raise ValueError(f"{where}: state has shape {tuple(state_out.shape)}, expected (slots,) + {state_shape}")
    shape = state_out.shape
    if slots is None and shape[0] < n:
        raise ValueError(f"{where}: state has {shape[0]} rows for {n} sequences")
    if fresh is not None and fresh.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"{where}: fresh must be bool or uint8, got {fresh.dtype}")
    pout = _table(where, "state_out", state_out, state_dtype, shape, dev)
    pin = pout if state is state_out else _table(where, "state", state, state_dtype, shape, dev)
    pslots = _table(where, "slots", slots, torch.int32, (n,), dev)
    pfresh = None if fresh is None else _table(where, "fresh", fresh, fresh.dtype, (n,), dev)
    return _i64x[7](pcu or 0, n, pin or 0, pout, pslots or 0, shape[0], pfresh or 0)


def _token_shape(where, x, name, cu_seqlens):
    """(batch, L, channels) of the activations [batch, L, c], or [L, c] with cu_seqlens."""
    want = 3 if cu_seqlens is None else 2
    if x.dim() != want:
        raise ValueError(f"{where}: {name} must have {want} dimensions "
                         f"{'[batch, L, channels]' if want == 3 else '[tokens, channels] with cu_seqlens'}, "
                         f"got {tuple(x.shape)}")
    return (1, *x.shape) if want == 2 else tuple(x.shape)


def _new_like(t, zeros=False):
    """An output laid out like activation ``t``, its channels contiguous even where rows of
    ``t`` overlap (windows over one signal)."""
    make = torch.zeros_like if zeros else torch.empty_like
    y = make(t)
    return y if y.stride(-1) == 1 else make(t, memory_format=torch.contiguous_format)


def causal_ckpt_shape(batch, L, d_inner, d_state):
    """Shape of the states causal_scan(ckpt=...) keeps and causal_scan_bwd(ckpt=...) takes
    (batch 1 and L all tokens with cu_seqlens): [batch, ceil(L / 8), d_inner, d_state]."""
    return (batch, (L + 7) // 8, d_inner, d_state)


@_on_stream
def causal_scan(u, delta, z, B, C, A, D, delta_bias, *, cu_seqlens=None, state=None, state_out=None, slots=None,
                fresh=None, ckpt=None, y=None, stream=None):
    """Causal selective scan; see include/vimscan_causal.h.

    u, delta, z: [batch, L, d_inner], or [tokens, d_inner] with ``cu_seqlens`` (int32,
    n_seqs + 1 offsets of packed sequences); z may be None.  B, C: the same rows with
    d_state columns.  Rows may lie apart (a half or some columns of a wider tensor); the
    channels must be contiguous.  A: [d_inner, d_state], D, delta_bias: [d_inner], fp32.

    state: fp32 [rows, d_inner, d_state]: each sequence starts from its row and leaves its
    final state there, or in ``state_out`` when that is given (state None and state_out
    given: start from zeros).  ``slots`` (int32, one per sequence) names the rows, in
    sequence order by default; a slot outside the cache marks a padding entry, which is
    skipped.  ``fresh`` (bool, one per sequence) starts a sequence from zeros.

    ``ckpt``, fp32 of causal_ckpt_shape(...), receives the states causal_scan_bwd takes (not
    together with ``state``: the derivative starts every sequence from zeros).
    Returns y, shaped like u.  Tokens of no sequence and of padding entries keep what y held;
    where y is allocated here that is not initialised.
    """
    where = "causal_scan"
    if ckpt is not None and state is not None:
        raise ValueError(f"{where}: ckpt is for sequences that start from zeros; give state_out alone")
    dev = _check_ref(where, u)
    batch, L, Di = _token_shape(where, u, "u", cu_seqlens)
    N = B.shape[-1]
    packed = cu_seqlens is not None
    io, f32, act, bc = u.dtype, torch.float32, u.shape, (*u.shape[:-1], N)
    dt = _dtype_code(u)
    if y is None:
        y = _new_like(u)
    rows = _i64x[18](
        *_rows(where, "u", u, io, act, dev, packed), *_rows(where, "delta", delta, io, act, dev, packed),
        *_rows(where, "z", z, io, act, dev, packed), *_rows(where, "B", B, io, bc, dev, packed),
        *_rows(where, "C", C, io, bc, dev, packed), *_rows(where, "y", y, io, act, dev, packed))
    pA, pD = _table(where, "A", A, f32, (Di, N), dev), _table(where, "D", D, f32, (Di,), dev)
    pbias = _table(where, "delta_bias", delta_bias, f32, (Di,), dev)
    pk = None if ckpt is None else _table(where, "ckpt", ckpt, f32, causal_ckpt_shape(batch, L, Di, N), dev)
    seqs = _sequences(where, dev, batch, cu_seqlens, state, state_out, slots, fresh, f32, (Di, N))
    st = lib.causal_scan(rows, pA, pD, pbias, batch, L, Di, N, dt, seqs, pk, _raw_stream(dev))
    if st != VIM_OK:
        raise VimScanError(st, where)
    return y


@_on_stream
def causal_scan_step(u, delta, z, B, C, A, D, delta_bias, state, *, state_out=None, slots=None, y=None, stream=None):
    """causal_scan for one token of each sequence: u, delta, z [batch, d_inner], B, C
    [batch, d_state], state as there (required; updated in place unless ``state_out`` is
    given).  Rows whose slot is outside the cache are padding: their y is left as it was (not
    initialised where y is allocated here).  Returns y [batch, d_inner].
    """
    where = "causal_scan_step"
    dev = _check_ref(where, u)
    if u.dim() != 2:
        raise ValueError(f"{where}: u must be [batch, d_inner], got {tuple(u.shape)}")
    if state is None:
        raise ValueError(f"{where}: a state is needed")
    batch, Di = u.shape
    N = B.shape[-1]
    io, f32, act, bc = u.dtype, torch.float32, u.shape, (batch, N)
    dt = _dtype_code(u)
    if y is None:
        y = _new_like(u)
    rows = _i64x[18](
        *_rows(where, "u", u, io, act, dev, False), *_rows(where, "delta", delta, io, act, dev, False),
        *_rows(where, "z", z, io, act, dev, False), *_rows(where, "B", B, io, bc, dev, False),
        *_rows(where, "C", C, io, bc, dev, False), *_rows(where, "y", y, io, act, dev, False))
    pA, pD = _table(where, "A", A, f32, (Di, N), dev), _table(where, "D", D, f32, (Di,), dev)
    pbias = _table(where, "delta_bias", delta_bias, f32, (Di,), dev)
    seqs = _sequences(where, dev, batch, None, state, state_out, slots, None, f32, (Di, N))
    st = lib.causal_scan_step(rows, pA, pD, pbias, batch, Di, N, dt, seqs, _raw_stream(dev))
    if st != VIM_OK:
        raise VimScanError(st, where)
    return y


def causal_bwd_workspace_bytes(batch, L, d_inner, d_state, has_ckpt):
    return int(lib.causal_bwd_workspace_bytes(batch, L, d_inner, d_state, int(bool(has_ckpt))))


@_on_stream
def causal_scan_bwd(u, delta, z, B, C, A, D, delta_bias, dout, *, cu_seqlens=None, ckpt=None, workspace=None, out=None,
                    stream=None):
    """Derivatives of causal_scan, for sequences that start from zeros and whose final states
    are not used, and a loss whose derivative with respect to y is ``dout``; see
    include/vimscan_causal.h.

    Returns a dict: du, ddelta (w.r.t. the raw delta), dz (None without z), shaped like u in
    its dtype; dB and dC (fp32, contiguous, shaped like B); dA [d_inner, d_state], dD and
    ddelta_bias [d_inner] (fp32).  ``out`` may hold those tensors from an earlier call to be
    written again (du, ddelta and dz with any row strides).  Tokens of no sequence keep what
    the outputs held (zeros when allocated here).  ``ckpt``: the states causal_scan(ckpt=...)
    kept for the same inputs.  Every sequence counts, those that a padding slot made
    causal_scan skip as well: give them a dout of zero and finite inputs.
    """
    where = "causal_scan_bwd"
    dev = _check_ref(where, u)
    batch, L, Di = _token_shape(where, u, "u", cu_seqlens)
    N = B.shape[-1]
    packed = cu_seqlens is not None
    io, f32, act, bc = u.dtype, torch.float32, u.shape, (*u.shape[:-1], N)
    if out is None:
        like = lambda t: _new_like(t, packed)
        f = u.new_zeros if packed else u.new_empty
        out = dict(du=like(u), ddelta=like(u), dz=None if z is None else like(u), dB=f(bc, dtype=f32), dC=f(bc, dtype=f32),
                   dA=u.new_empty((Di, N), dtype=f32), dD=u.new_empty(Di, dtype=f32),
                   ddelta_bias=u.new_empty(Di, dtype=f32))
    elif (z is None) != (out["dz"] is None):
        raise ValueError(f"{where}: out['dz'] must be given exactly when z is")
    dt = _dtype_code(u)
    n = _offsets(where, cu_seqlens)
    tab = lambda name, t, shape, dtype=f32: _table(where, name, t, dtype, shape, dev)
    pA, pD, pbias = tab("A", A, (Di, N)), tab("D", D, (Di,)), tab("delta_bias", delta_bias, (Di,))
    pk = None if ckpt is None else tab("ckpt", ckpt, causal_ckpt_shape(batch, L, Di, N))
    pcu = tab("cu_seqlens", cu_seqlens, (n + 1,), torch.int32)
    pdB, pdC = tab("out['dB']", out["dB"], bc), tab("out['dC']", out["dC"], bc)
    pdA, pdD = tab("out['dA']", out["dA"], (Di, N)), tab("out['dD']", out["dD"], (Di,))
    pdb = tab("out['ddelta_bias']", out["ddelta_bias"], (Di,))
    r = lambda name, t, shape: _rows(where, name, t, io, shape, dev, packed)
    rows = _i64x[27](
        *r("u", u, act), *r("delta", delta, act), *r("z", z, act), *r("B", B, bc), *r("C", C, bc), *r("dout", dout, act),
        *r("out['du']", out["du"], act), *r("out['ddelta']", out["ddelta"], act), *r("out['dz']", out["dz"], act))
    ws, ws_bytes = _workspace(causal_bwd_workspace_bytes(batch, L, Di, N, ckpt is not None), workspace, u.device)
    st = lib.causal_scan_bwd(
        rows, pA, pD, pbias, pdB, pdC, pdA, pdD, pdb, batch, L, Di, N, dt, pcu, n, pk,
        None if ws is None else ws.data_ptr(), ws_bytes,
        _raw_stream(dev))
    if st != VIM_OK:
        raise VimScanError(st, where)
    return out


@_on_stream
def causal_conv(x, w, b, *, silu=True, cu_seqlens=None, state=None, state_out=None, slots=None, fresh=None, y=None,
                stream=None):
    """Short causal depthwise convolution, with SiLU unless ``silu`` is false; see
    include/vimscan_causal.h.

    x: [batch, L, channels], or [tokens, channels] with ``cu_seqlens``, any row strides.  w:
    [channels, width] fp32, width 2 to 4, the newest tap last; b: [channels] fp32 or None.
    state: [rows, width - 1, channels] in x's dtype, the last inputs of each sequence, oldest
    first; state_out, slots and fresh as in causal_scan.  Returns y, shaped like x; tokens of no
    sequence as in causal_scan.
    """
    where = "causal_conv"
    dev = _check_ref(where, x)
    batch, L, Ch = _token_shape(where, x, "x", cu_seqlens)
    W = w.shape[-1]
    packed = cu_seqlens is not None
    io, f32, act = x.dtype, torch.float32, x.shape
    if y is None:
        y = _new_like(x)
    dt = _dtype_code(x)
    rows = _i64x[6](*_rows(where, "x", x, io, act, dev, packed), *_rows(where, "y", y, io, act, dev, packed))
    pw, pb = _table(where, "w", w, f32, (Ch, W), dev), _table(where, "b", b, f32, (Ch,), dev)
    seqs = _sequences(where, dev, batch, cu_seqlens, state, state_out, slots, fresh, io, (W - 1, Ch))
    st = lib.causal_conv(rows, pw, pb, batch, L, Ch, W, int(bool(silu)), dt, seqs, _raw_stream(dev))
    if st != VIM_OK:
        raise VimScanError(st, where)
    return y


@_on_stream
def causal_conv_step(x, w, b, state, *, silu=True, state_out=None, slots=None, y=None, stream=None):
    """causal_conv for one token of each sequence: x [batch, channels]; state as there
    (required; updated in place unless ``state_out`` is given).  Rows whose slot is outside
    the cache are padding: their y is left as it was.  Returns y [batch, channels].
    """
    where = "causal_conv_step"
    dev = _check_ref(where, x)
    if x.dim() != 2:
        raise ValueError(f"{where}: x must be [batch, channels], got {tuple(x.shape)}")
    if state is None:
        raise ValueError(f"{where}: a state is needed")
    batch, Ch = x.shape
    W = w.shape[-1]
    io, f32, act = x.dtype, torch.float32, x.shape
    if y is None:
        y = _new_like(x)
    dt = _dtype_code(x)
    rows = _i64x[6](*_rows(where, "x", x, io, act, dev, False), *_rows(where, "y", y, io, act, dev, False))
    pw, pb = _table(where, "w", w, f32, (Ch, W), dev), _table(where, "b", b, f32, (Ch,), dev)
    seqs = _sequences(where, dev, batch, None, state, state_out, slots, None, io, (W - 1, Ch))
    st = lib.causal_conv_step(rows, pw, pb, batch, Ch, W, int(bool(silu)), dt, seqs, _raw_stream(dev))
    if st != VIM_OK:
        raise VimScanError(st, where)
    return y


def causal_conv_bwd_workspace_bytes(batch, L, channels, width):
    return int(lib.causal_conv_bwd_workspace_bytes(batch, L, channels, width))


@_on_stream
def causal_conv_bwd(x, w, b, dout, *, silu=True, cu_seqlens=None, workspace=None, out=None, stream=None):
    """Derivatives of causal_conv, for sequences that start from zeros and whose final states
    are not used, and a loss whose derivative with respect to y is ``dout``; see
    include/vimscan_causal.h.

    Returns a dict: dx, shaped like x in its dtype; dw [channels, width] and db [channels]
    (None without b) in fp32.  ``out`` may hold those tensors from an earlier call (dx with
    any row strides).  Tokens of no sequence keep what dx held (zeros when allocated here).
    """
    where = "causal_conv_bwd"
    dev = _check_ref(where, x)
    batch, L, Ch = _token_shape(where, x, "x", cu_seqlens)
    W = w.shape[-1]
    packed = cu_seqlens is not None
    io, f32, act = x.dtype, torch.float32, x.shape
    if out is None:
        out = dict(dx=_new_like(x, packed), dw=x.new_empty((Ch, W), dtype=f32),
                   db=None if b is None else x.new_empty(Ch, dtype=f32))
    elif (b is None) != (out["db"] is None):
        raise ValueError(f"{where}: out['db'] must be given exactly when b is")
    dt = _dtype_code(x)
    n = _offsets(where, cu_seqlens)
    tab = lambda name, t, shape, dtype=f32: _table(where, name, t, dtype, shape, dev)
    pw, pb, pcu = tab("w", w, (Ch, W)), tab("b", b, (Ch,)), tab("cu_seqlens", cu_seqlens, (n + 1,), torch.int32)
    pdw, pdb = tab("out['dw']", out["dw"], (Ch, W)), tab("out['db']", out["db"], (Ch,))
    r = lambda name, t: _rows(where, name, t, io, act, dev, packed)
    rows = _i64x[9](*r("x", x), *r("dout", dout), *r("out['dx']", out["dx"]))
    ws, ws_bytes = _workspace(causal_conv_bwd_workspace_bytes(batch, L, Ch, W), workspace, x.device)
    st = lib.causal_conv_bwd(rows, pw, pb, pdw, pdb, batch, L, Ch, W, int(bool(silu)), dt, pcu, n,
                             None if ws is None else ws.data_ptr(), ws_bytes,
                             _raw_stream(dev))
    if st != VIM_OK:
        raise VimScanError(st, where)
    return out


def clip_grad_norm_workspace_bytes(count):
    return int(lib.clip_grad_norm_workspace_bytes(count))


_CLIP_TYPES = {torch.float32: VIM_F32, torch.bfloat16: VIM_BF16}


def _refuse_gradient(where, name, t, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{where}: {name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{where}: {name} is on {t.device} but the current device is cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    if t.dtype not in _CLIP_TYPES:
        raise TypeError(f"{where}: {name}: unsupported dtype {t.dtype}: fp32 or bf16")


def _clip_pairs(where, grads, out):
    """The gradients and the output of each, as two lists: dicts are paired by key, lists and tuples
    by place; entries that are None on both sides are skipped."""
    if out is None:
        src = [t for t in (grads.values() if isinstance(grads, dict) else grads) if t is not None]
        return src, src
    if isinstance(grads, dict) != isinstance(out, dict):
        raise TypeError(f"{where}: grads and out must both be dicts, or both lists or tuples")
    if isinstance(grads, dict):
        if grads.keys() != out.keys():
            raise ValueError(f"{where}: grads has the keys {list(grads)}, out {list(out)}")
        grads, out = grads.values(), [out[k] for k in grads]
    else:
        grads, out = list(grads), list(out)
    src, dst = [t for t in grads if t is not None], [o for o in out if o is not None]
    if len(grads) != len(out) or len(src) != len(dst):
        raise ValueError(f"{where}: {len(src)} gradients and {len(dst)} outputs")
    if len(src) != len(grads) and [t is None for t in grads] != [o is None for o in out]:
        raise ValueError(f"{where}: an output must be None exactly where its gradient is")
    return src, dst


@_on_stream
def clip_grad_norm(grads, max_norm, *, out=None, norm=None, workspace=None, stream=None):
    """The common norm of many gradients, and clipping by it; see include/vimscan_causal.h.

    ``grads``: contiguous CUDA tensors, fp32 or bf16 in any mixture, as a list or tuple, or a
    dict of them as the *_bwd functions return (None entries are skipped).  They are scaled
    in place by min(1, max_norm / (norm + 1e-6)), or into ``out`` (a dict with the same keys, or
    a list or tuple in the same order; the same shapes and dtypes, None where grads has it).  A norm that is not finite scales nothing.
    max_norm may be infinite: then nothing but the norm is computed.  Returns the norm, a
    float32 tensor of one element on the device (``norm`` if given).
    """
    where = "clip_grad_norm"
    src, dst = _clip_pairs(where, grads, out)
    max_norm = float(max_norm)
    if not max_norm >= 0:
        raise ValueError(f"{where}: max_norm must be >= 0, got {max_norm}")
    dev = torch.cuda.current_device()
    try:
        # cheap checks of all at once; what is wrong is worked out only where one fails
        T = torch.Tensor
        codes = [_CLIP_TYPES.get(t.dtype) for t in src]
        good = None not in codes and set(map(T.get_device, src)) <= {dev} and all(map(T.is_contiguous, src))
        at = list(map(T.data_ptr, src))
        to = at
        if out is not None:
            good = good and set(map(T.get_device, dst)) <= {dev} and all(map(T.is_contiguous, dst)) and all(
                [o.dtype == t.dtype and o.shape == t.shape for t, o in zip(src, dst)])
            to = list(map(T.data_ptr, dst))
        table = list(itertools.chain.from_iterable(zip(at, to, map(T.numel, src), codes))) if good else None
    except (AttributeError, RuntimeError, TypeError):
        table = None
    if table is None:
        for i, (t, o) in enumerate(zip(src, dst)):
            _refuse_gradient(where, f"grads[{i}]", t, dev)
            _refuse_gradient(where, f"out[{i}]", o, dev)
            if o.dtype != t.dtype or o.shape != t.shape:
                raise ValueError(f"{where}: out[{i}] must be {t.dtype} of shape {tuple(t.shape)}, got {o.dtype} of "
                                 f"{tuple(o.shape)}")
        raise TypeError(f"{where}: grads and out must be tensors with storage")
    device = torch.device("cuda", dev)
    if norm is None:
        norm = src[0].new_empty(1, dtype=torch.float32) if src else torch.empty(1, dtype=torch.float32, device=device)
    elif not isinstance(norm, torch.Tensor) or norm.dtype != torch.float32 or norm.numel() != 1 or norm.get_device() != dev:
        raise ValueError(f"{where}: norm must be one float32 element on cuda:{dev}")
    n = len(src)
    ws, ws_bytes = _workspace(clip_grad_norm_workspace_bytes(n), workspace, device)
    st = lib.clip_grad_norm(struct.pack(f"{4 * n}q", *table), n, max_norm, norm.data_ptr(), ws.data_ptr(), ws_bytes,
                            _raw_stream(dev))
    if st != VIM_OK:
        raise VimScanError(st, where)
    return norm
