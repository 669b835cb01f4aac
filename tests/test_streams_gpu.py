"""The bidirectional and four-direction entry points given a stream= other than the current one,
while work of the current stream is still queued: outputs and workspaces that the call allocates
(the derivatives' dB and dC are zeroed first) are not touched by that work.
"""
import pytest
import torch

from test_causal_streams_gpu import QUEUE, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vs():
    from vision_mamba_selective_b200 import vimscan

    return vimscan


def calls(vs):
    g = torch.Generator().manual_seed(1)
    r = lambda *s, dtype=torch.bfloat16: torch.randn(s, generator=g).to(dtype).cuda()
    f32 = torch.float32
    b, L, d, N = 2, 300, 64, 16
    A = lambda n: (-torch.arange(1, N + 1, dtype=f32).repeat(n, d, 1)).cuda()
    bias = lambda n: torch.full((n, d), -3.0, device="cuda")
    D = lambda n: torch.ones((n, d), device="cuda")
    scan = (r(b, L, d), r(b, L, d), r(b, L, d), r(b, L, N), r(b, L, N), A(2), D(2), bias(2))
    cross = (r(b, 10, 30, d), r(b, 10, 30, d), r(b, 10, 30, d), r(4, b, L, N), r(4, b, L, N), A(4), D(4), bias(4))
    cw, cb = r(2, d, 3, dtype=f32), r(2, d, dtype=f32)
    block = (r(b, L, d), r(2, d, 2 * N + 1), r(2, d, dtype=f32), bias(2), A(2), D(2), r(b, L, d))
    do, do4, ys = r(b, L, d), r(b, 10, 30, d), r(4, b, L, d)
    return {
        "vim_scan_bidir": lambda **k: vs.vim_scan_bidir(*scan, **k),
        "vim_scan_bidir_conv": lambda **k: vs.vim_scan_bidir_conv(scan[0], cw, cb, *scan[1:], **k),
        "vim_scan_bidir_bwd": lambda **k: vs.vim_scan_bidir_bwd(*scan, do, **k),
        "vim_scan_bidir_conv_bwd": lambda **k: vs.vim_scan_bidir_conv_bwd(scan[0], cw, cb, *scan[1:], do, **k),
        "vmamba_cross_scan4": lambda **k: vs.vmamba_cross_scan4(*cross, **k),
        "vmamba_cross_scan4_bwd": lambda **k: vs.vmamba_cross_scan4_bwd(*cross, do4, **k),
        "cross_merge4": lambda **k: vs.cross_merge4(ys, cross[2], 10, 30, **k),
        "vim_block_scan": lambda **k: vs.vim_block_scan(*block, conv_w=cw, conv_b=cb, **k),
        "vim_block_scan_bwd": lambda **k: vs.vim_block_scan_bwd(*block, do, conv_w=cw, conv_b=cb, **k),
    }


@pytest.mark.parametrize("name", ["vim_scan_bidir", "vim_scan_bidir_conv", "vim_scan_bidir_bwd", "vim_scan_bidir_conv_bwd",
                                  "vmamba_cross_scan4", "vmamba_cross_scan4_bwd", "cross_merge4", "vim_block_scan",
                                  "vim_block_scan_bwd"])
def test_queued_work_of_the_current_stream(vs, name):
    call = calls(vs)[name]
    want = [t.clone() for t in values(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(QUEUE)
    old = [torch.empty_like(t) for t in want for _ in range(3)]
    for t in old:
        t.fill_(7.0)
    del old, t
    got = call(stream=side)
    torch.cuda.synchronize()
    for x, y in zip(values(got), want):
        assert torch.equal(x, y), name
