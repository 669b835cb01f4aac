"""Causal operators given a stream= other than the current one, while work of the current stream
is still queued: nothing that the call allocates, fills or returns may be touched by that work.
(The inputs are ready: both streams have finished with them before the queue is filled.)
"""
import pytest
import torch

from test_causal_scan_gpu import BF, F32, cuda, inputs, vs  # noqa: F401

pytestmark = pytest.mark.gpu
QUEUE = 100_000_000          # clocks that the current stream is kept busy: some 50 ms


def values(result):
    return [v for v in (result.values() if isinstance(result, dict) else (result,)) if v is not None]


def calls(vs):
    """name -> a call with its outputs allocated by it, packed ones (whose outputs are zeroed first)
    among them."""
    p = inputs((700,), 72, 16, BF, 1)
    a = cuda(p)
    g = torch.Generator().manual_seed(2)
    dout = torch.randn((700, 72), generator=g).to(BF).cuda()
    w, b = torch.randn((72, 4), generator=g).cuda(), torch.randn(72, generator=g).cuda()
    cu = torch.tensor([3, 300, 301, 690], dtype=torch.int32, device="cuda")
    rows = [t[None] if t.dim() == 2 and t.shape[0] == 700 else t for t in a]
    state = torch.zeros((700, 72, 16), device="cuda")
    taps = torch.zeros((700, 3, 72), dtype=BF, device="cuda")
    grads = [torch.randn(5000, generator=g).cuda(), torch.randn((40, 9), generator=g).to(BF).cuda()]
    scaled = [torch.empty_like(t) for t in grads]
    state_out, taps_out = torch.empty_like(state), torch.empty_like(taps)
    return {
        "causal_scan": lambda **k: vs.causal_scan(*rows, **k),
        "causal_scan_step": lambda **k: vs.causal_scan_step(*a, state, state_out=state_out, **k),
        "causal_scan_bwd": lambda **k: vs.causal_scan_bwd(*rows, dout[None], **k),
        "causal_scan_bwd packed": lambda **k: vs.causal_scan_bwd(*a, dout, cu_seqlens=cu, **k),
        "causal_conv": lambda **k: vs.causal_conv(rows[0], w, b, **k),
        "causal_conv_step": lambda **k: vs.causal_conv_step(a[0], w, b, taps, state_out=taps_out, **k),
        "causal_conv_bwd": lambda **k: vs.causal_conv_bwd(rows[0], w, b, dout[None], **k),
        "causal_conv_bwd packed": lambda **k: vs.causal_conv_bwd(a[0], w, b, dout, cu_seqlens=cu, **k),
        "clip_grad_norm": lambda **k: vs.clip_grad_norm(grads, 1.0, out=scaled, **k),
    }


NAMES = ["causal_scan", "causal_scan_step", "causal_scan_bwd", "causal_scan_bwd packed", "causal_conv",
         "causal_conv_step", "causal_conv_bwd", "causal_conv_bwd packed", "clip_grad_norm"]


@pytest.mark.parametrize("name", NAMES)
def test_queued_work_of_the_current_stream(vs, name):
    call = calls(vs)[name]
    want = [t.clone() for t in values(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks that the current stream still has to write, free as far as the allocator can tell
    torch.cuda._sleep(QUEUE)
    old = [torch.empty_like(t) for t in want for _ in range(3)]
    for t in old:
        t.fill_(7.0)
    del old, t
    got = call(stream=side)
    torch.cuda.synchronize()
    for x, y in zip(values(got), want):
        assert torch.equal(x, y), name


@pytest.mark.parametrize("name", NAMES)
def test_results_outlive_their_use(vs, name):
    """Results that the current stream has yet to read are not handed out again on the call's own."""
    call = calls(vs)[name]
    want = [t.clone() for t in values(call())]
    side, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    got = call(stream=side)
    cur.wait_stream(side)
    torch.cuda._sleep(QUEUE)
    read = [t.clone() for t in values(got)]
    del got
    with torch.cuda.stream(side):
        for t in [torch.empty_like(t) for t in want for _ in range(3)]:
            t.fill_(7.0)
    torch.cuda.synchronize()
    for x, y in zip(read, want):
        assert torch.equal(x, y), name


def test_stream_inside_a_capture(vs):
    """A side stream forked into a capture and joined again; replayed."""
    for name in ("causal_scan_bwd packed", "causal_conv_bwd packed", "causal_scan"):
        call = calls(vs)[name]
        want = [t.clone() for t in values(call())]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            side.wait_stream(torch.cuda.current_stream())
            got = call(stream=side)
            torch.cuda.current_stream().wait_stream(side)
        for _ in range(2):
            for t in values(got):
                t.fill_(5.0)
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip(values(got), want):
                assert torch.equal(x, y), name


def test_given_outputs(vs):
    """Outputs and workspace of the caller's, on another stream; what else their dict holds stays."""
    a = cuda(inputs((2, 130), 40, 16, F32, 3))
    dout = torch.ones((2, 130, 40), device="cuda")
    want = vs.causal_scan_bwd(*a, dout)
    out = {k: torch.full_like(v, 7.0) for k, v in want.items()} | {"name": "block 1"}
    ws = torch.empty(vs.causal_bwd_workspace_bytes(2, 130, 40, 16, False), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert vs.causal_scan_bwd(*a, dout, out=out, workspace=ws, stream=side) is out
    torch.cuda.current_stream().wait_stream(side)
    assert out.pop("name") == "block 1" and all(torch.equal(out[k], want[k]) for k in want)
