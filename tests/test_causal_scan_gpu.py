"""causal_scan and causal_scan_step against the definition in fp64.

Tolerances.  The kernels hold the state in fp32.  Per token a state takes one decay
2^(Delta A log2 e) and one fused multiply-add: the decay carries the exp2 unit's error
(at most 1.5e-7 relative, measured bias below 5e-8) and the rounding of its argument, the
multiply-add half a step (6e-8), Delta and Delta u another 3e-7 together.  Errors of
earlier tokens decay with the state itself: over a memory of m = 1 / (1 - a) tokens they add
to at most m times the per-token error, and the tests' slowest decay, Delta |A| >= 1e-3,
gives m <= 1000; as the roundings are of either sign the sum is nearer sqrt(m) times.
5e-5 normwise is the bound with that all of one sign on the slowest state (2.5e-7 * 1000 /
5, a state of that memory being one of at least five of its size in the sum); outputs are
checked at 1e-5, as everywhere in this library, final states at 2e-5.  bf16 outputs are
rounded once: half a step, 2^-8 = 3.9e-3 of the value, plus the fp32 part.
"""
import pytest
import torch

import causal_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
STATE_TOL = 2e-5
Y_TOL = {F32: 1e-5, BF: 2.0 ** -8 + 1e-5}


@pytest.fixture(scope="module")
def vs():
    from vision_mamba_selective_b200 import vimscan

    return vimscan


def inputs(rows, d, N, dtype, seed, gate=True, strided=False):
    """CPU tensors; ``rows`` is (batch, L) or (tokens,).  strided: z the second half of one
    tensor, B and C columns of another at an odd offset."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    p = dict(u=r(*rows, d).to(dtype), delta=(r(*rows, d) * 0.5).to(dtype))
    p["z"] = r(*rows, d).to(dtype) if gate else None
    p["B"], p["C"] = r(*rows, N).to(dtype), r(*rows, N).to(dtype)
    if strided:
        p["z"] = r(*rows, 2 * d).to(dtype)[..., d:] if gate else None
        proj = r(*rows, 5 + 2 * N).to(dtype)
        p["B"], p["C"] = proj[..., 5:5 + N], proj[..., 5 + N:]
    p["A"] = -(torch.arange(1, N + 1, dtype=F32) * torch.exp(0.2 * r(d, N))).contiguous()
    p["D"] = r(d)
    step = torch.exp(torch.rand(d, generator=g) * 4.6 - 6.9)      # 1e-3 .. 1e-1
    p["bias"] = torch.log(torch.expm1(step))
    return p


def cuda(p):
    """The tensors on the GPU with the same strides."""
    def move(t):
        if t is None:
            return None
        out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
        return out.copy_(t)
    return [move(p[k]) for k in ("u", "delta", "z", "B", "C", "A", "D", "bias")]


def ref(p, cu=None, starts=None):
    return causal_ref.scan(p["u"], p["delta"], p["z"], p["B"], p["C"], p["A"], p["D"], p["bias"], cu, starts)


def close(got, want, tol, name=""):
    """normwise (over everything) and per row of the last dimension, floored at the rms row"""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, name
    if not got.numel():
        return
    assert torch.isfinite(got).all(), name
    diff = got - want
    assert diff.abs().max() <= tol * max(want.abs().max().item(), 1e-30) , (name, diff.abs().max().item(), want.abs().max().item())
    norms = want.norm(dim=-1)
    floor = norms.square().mean().sqrt()
    worst = (diff.norm(dim=-1) / torch.maximum(norms, floor).clamp_min(1e-30)).max().item()
    assert worst <= tol, (name, worst)


BATCH = [
    # batch, L, d, N, dtype, gate, strided
    (1, 1, 32, 16, BF, True, False),
    (2, 5, 33, 16, F32, True, False),          # odd channel count
    (1, 31, 40, 16, BF, False, False),
    (3, 32, 24, 8, F32, True, True),
    (2, 33, 8, 4, BF, True, False),
    (1, 100, 130, 2, F32, True, False),
    (2, 197, 72, 16, F32, True, True),
    (1, 200, 7, 8, BF, True, True),
    (4, 64, 1, 16, F32, False, False),         # one channel
    (1, 130, 2400, 16, BF, True, False),       # 8 lanes a channel
    (5, 70, 2000, 16, F32, True, False),       # 4 lanes a channel
    (8, 40, 1300, 8, BF, True, False),         # N = 8, 4 lanes a channel
    (1, 300, 592, 16, BF, True, True),         # 8 lanes a channel, segments of 16
    (2, 97, 297, 16, F32, True, False),        # 4 lanes a channel, segments of 16
    (1, 300, 1184, 16, BF, True, True),
    (3, 90, 395, 16, F32, True, True),         # segments of 8
]


@pytest.mark.parametrize("case", BATCH, ids=lambda c: f"b{c[0]}_L{c[1]}_d{c[2]}_N{c[3]}_{str(c[4])[6:]}"
                         f"{'' if c[5] else '_nogate'}{'_strided' if c[6] else ''}")
def test_batch(vs, case):
    batch, L, d, N, dtype, gate, strided = case
    p = inputs((batch, L), d, N, dtype, seed=L + d, gate=gate, strided=strided)
    state = torch.full((batch, d, N), float("nan"), device="cuda")
    y = vs.causal_scan(*cuda(p), state_out=state)
    want, last = ref(p)
    close(y, want, Y_TOL[dtype], "y")
    close(state, last, STATE_TOL, "state")


def packed_case(lens, d, N, dtype, seed, lead=0, tail=0, **kw):
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    return inputs((cu[-1] + tail,), d, N, dtype, seed, **kw), cu


PACKED = [
    # lengths, d, N, dtype, tokens before the first sequence, tokens after the last
    ([1], 32, 16, BF, 0, 0),
    ([5, 0, 1, 40, 31, 1, 1, 64], 40, 16, F32, 0, 0),
    ([3, 33, 0, 0, 7], 24, 8, BF, 4, 9),
    ([100, 29, 2], 9, 16, F32, 1, 0),
    ([0, 0], 16, 4, F32, 0, 3),
    ([17] * 12, 64, 2, BF, 0, 1),
    ([200, 3, 77], 3200, 16, BF, 0, 0),
    ([150, 0, 3, 77, 16], 200, 16, F32, 5, 1),       # segments of 16, 4 lanes a channel
    ([150, 0, 3, 77, 16], 300, 16, BF, 5, 1),        # segments of 8
    ([40, 3, 77, 0, 9, 9], 3200, 16, F32, 2, 1),     # enough channels for eight states a lane
    ([(i * 7) % 5 for i in range(64)], 24, 16, F32, 0, 0),
    ([(i * 7) % 5 for i in range(70)], 24, 8, BF, 3, 0),   # more sequences than are sorted by length
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"n{len(c[0])}_d{c[1]}_N{c[2]}_{str(c[3])[6:]}_{c[4]}_{c[5]}")
def test_packed(vs, case):
    """States in a larger cache by slot, some sequences fresh; rows of no sequence, cache rows
    of no sequence and tokens of no sequence keep what they held."""
    lens, d, N, dtype, lead, tail = case
    p, cu = packed_case(lens, d, N, dtype, seed=sum(lens) + d, lead=lead, tail=tail)
    n = len(lens)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(n + 3, generator=g)[:n]
    cache = torch.randn((n + 3, d, N), generator=g)
    fresh = torch.rand(n, generator=g) < 0.4
    starts = torch.where(fresh[:, None, None], torch.zeros(()), cache[slots])
    want, last = ref(p, cu, starts)
    args = cuda(p)
    dev = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
               slots=slots.to(torch.int32).cuda(), fresh=fresh.cuda())
    for in_place in (False, True):
        state = cache.cuda()
        out = state if in_place else torch.full_like(state, 7.0)
        y = torch.full_like(args[0], 3.0)
        vs.causal_scan(*args, state=state, state_out=None if in_place else out, y=y, **dev)
        inside = slice(cu[0], cu[-1])
        close(y[inside], want[inside], Y_TOL[dtype], "y")
        assert (y[:cu[0]] == 3.0).all() and (y[cu[-1]:] == 3.0).all()
        close(out[slots.cuda()], last, STATE_TOL, "state")
        others = [i for i in range(n + 3) if i not in slots.tolist()]
        kept = cache[others] if in_place else torch.full_like(cache[others], 7.0)
        assert torch.equal(out[others].cpu(), kept)
        if not in_place:
            assert torch.equal(state.cpu(), cache)


def test_bad_tables_stay_inside(vs):
    """Decreasing and out-of-range offsets, slots outside the cache: nothing outside the named
    rows is written (the ranges themselves are the caller's error)."""
    p = inputs((50,), 32, 16, F32, 3)
    args = cuda(p)
    big = torch.full((150, 32), 3.0, device="cuda")
    cache = torch.full((30, 32, 16), 7.0, device="cuda")
    vs.causal_scan(*args, cu_seqlens=torch.tensor([-5, 20, 10, 400], dtype=torch.int32, device="cuda"),
                   state=cache[10:20], slots=torch.tensor([-1, 10, 3], dtype=torch.int32, device="cuda"),
                   y=big[50:100])
    torch.cuda.synchronize()
    assert (big[:50] == 3.0).all() and (big[100:] == 3.0).all()
    changed = (cache != 7.0).any(-1).any(-1).nonzero().flatten().tolist()
    assert changed == [13]


def test_padding_entry_is_skipped(vs):
    p = inputs((3, 20), 32, 16, BF, 5)
    args = cuda(p)
    y = torch.full_like(args[0], 3.0)
    state = torch.zeros((2, 32, 16), device="cuda")
    vs.causal_scan(*args, state=state, slots=torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda"), y=y)
    want, last = ref(p)
    close(y[[0, 2]], want[[0, 2]], Y_TOL[BF])
    assert (y[1] == 3.0).all()
    close(state, last[[2, 0]], STATE_TOL)


def test_nonfinite_outside_the_sequences(vs):
    """NaN and infinities in tokens of no sequence reach nothing."""
    p, cu = packed_case([9, 30], 40, 16, F32, seed=2, lead=3, tail=5)
    want, last = ref(p, cu)
    for k in ("u", "delta", "z", "B", "C"):
        p[k] = p[k].clone()
        p[k][:3] = float("nan")
        p[k][42:] = float("inf")
    state = torch.empty((2, 40, 16), device="cuda")
    y = torch.zeros((47, 40), device="cuda")
    vs.causal_scan(*cuda(p), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), state_out=state, y=y)
    close(y[3:42], want[3:42], Y_TOL[F32])
    close(state, last, STATE_TOL)


def test_long_decays_and_jumps(vs):
    """Steps from softplus(-20) (the state barely moves) to 30 (every state is replaced), and
    positive and zero A."""
    p = inputs((1, 90), 16, 16, F32, 8)
    p["delta"][0, :, 0:4] = torch.linspace(-12, 30, 90)[:, None]
    p["bias"][0:2] = -8.0
    p["A"][5] = 0.0
    p["A"][6] = 0.05
    state = torch.empty((1, 16, 16), device="cuda")
    y = vs.causal_scan(*cuda(p), state_out=state)
    want, last = ref(p)
    close(y, want, Y_TOL[F32])
    close(state, last, STATE_TOL)


@pytest.mark.parametrize("d,N,dtype", [(32, 16, BF), (33, 16, F32), (64, 8, BF), (70, 4, F32), (16, 2, BF), (1, 16, F32)])
@pytest.mark.parametrize("batch", [1, 9])
def test_step_follows_the_prompt(vs, batch, d, N, dtype):
    """Tokens one at a time through causal_scan_step equal the definition; slots in any order,
    a padding row between, strided rows."""
    L = 12
    p = inputs((batch, L), d, N, dtype, seed=d + batch, strided=True)
    want, last = ref(p)
    u, delta, z, B, C, A, D, bias = cuda(p)
    slots = torch.randperm(batch + 4, generator=torch.Generator().manual_seed(1))[:batch].to(torch.int32)
    if batch > 2:
        slots[1] = -1
    state = torch.zeros((batch + 4, d, N), device="cuda")
    dev = slots.cuda()
    y = torch.full((L, batch, d), 3.0, dtype=dtype, device="cuda")
    for t in range(L):
        vs.causal_scan_step(u[:, t], delta[:, t], z[:, t], B[:, t], C[:, t], A, D, bias, state, slots=dev, y=y[t])
    use = [b for b in range(batch) if slots[b] >= 0]
    close(y.permute(1, 0, 2)[use], want[use], Y_TOL[dtype])
    close(state[slots[use].long().cuda()], last[use], STATE_TOL)
    if batch > 2:
        assert (y[:, 1] == 3.0).all()
        rest = [i for i in range(batch + 4) if i not in slots.tolist()]
        assert (state[rest] == 0).all()


def test_prompt_then_steps(vs):
    """A prompt in two parts, then single tokens, equals one whole sequence; the step's
    state_out leaves the state it read."""
    p = inputs((2, 50), 48, 16, F32, 11)
    want, last = ref(p)
    u, delta, z, B, C, A, D, bias = cuda(p)
    state = torch.zeros((2, 48, 16), device="cuda")
    got = []
    for part in (slice(0, 30), slice(30, 47)):
        got.append(vs.causal_scan(u[:, part], delta[:, part], z[:, part], B[:, part], C[:, part], A, D, bias,
                                  state=state))
    for t in range(47, 50):
        new = torch.empty_like(state)
        before = state.clone()
        got.append(vs.causal_scan_step(u[:, t], delta[:, t], z[:, t], B[:, t], C[:, t], A, D, bias, state,
                                       state_out=new)[:, None])
        assert torch.equal(state, before)
        state = new
    close(torch.cat(got, 1), want, Y_TOL[F32])
    close(state, last, STATE_TOL)


def test_kept_states(vs):
    """ckpt holds the state entering every 8th token."""
    for d, N in ((40, 16), (1300, 16), (5000, 16), (40, 8), (20, 2)):
        p = inputs((2, 45), d, N, F32, d)
        ck = torch.full(vs.causal_ckpt_shape(2, 45, d, N), float("nan"), device="cuda")
        vs.causal_scan(*cuda(p), ckpt=ck)
        for i in range(6):
            part = {k: (v[:, :8 * i] if k in ("u", "delta", "z", "B", "C") else v) for k, v in p.items()}
            close(ck[:, i], ref(part)[1], STATE_TOL, f"{d} {i}")


def test_other_stream_and_graph(vs):
    p = inputs((2, 60), 64, 16, BF, 4)
    args = cuda(p)
    want, _ = ref(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = vs.causal_scan(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    close(y, want, Y_TOL[BF])
    out = torch.zeros_like(args[0])
    state = torch.zeros((2, 64, 16), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vs.causal_scan(*args, state_out=state, y=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        close(out, want, Y_TOL[BF])


def test_refusals(vs):
    p = inputs((2, 10), 32, 16, F32, 1)
    a = cuda(p)
    state = torch.zeros((2, 32, 16), device="cuda")
    bad = [
        (TypeError, lambda: vs.causal_scan(*[t.cpu() for t in a])),
        (TypeError, lambda: vs.causal_scan(a[0], a[1].bfloat16(), *a[2:])),
        (TypeError, lambda: vs.causal_scan(*[t.half() for t in a])),
        (ValueError, lambda: vs.causal_scan(a[0], a[1][:, :9], *a[2:])),
        (ValueError, lambda: vs.causal_scan(a[0], a[1], a[2], a[3][..., :8], *a[4:])),
        (ValueError, lambda: vs.causal_scan(a[0].transpose(1, 2).contiguous().transpose(1, 2), *a[1:])),
        (ValueError, lambda: vs.causal_scan(*a[:5], a[5][None], *a[6:])),
        (ValueError, lambda: vs.causal_scan(*a, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: vs.causal_scan(*a, state=state[:1])),
        (ValueError, lambda: vs.causal_scan(*a, state=state[:, :, :8])),
        (TypeError, lambda: vs.causal_scan(*a, state=state.bfloat16())),
        (ValueError, lambda: vs.causal_scan(*a, slots=torch.zeros(2, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: vs.causal_scan(*a, state_out=state, fresh=torch.zeros(2, dtype=torch.bool, device="cuda"))),
        (TypeError, lambda: vs.causal_scan(*a, state=state, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))),
        (ValueError, lambda: vs.causal_scan(*a, state=state, slots=torch.zeros(3, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: vs.causal_scan(*a, ckpt=torch.zeros((2, 1, 32, 16), device="cuda"))),
        (ValueError, lambda: vs.causal_scan(*a, state=state, ckpt=torch.zeros((2, 2, 32, 16), device="cuda"))),
        (ValueError, lambda: vs.causal_scan(*a, y=torch.zeros((2, 10, 31), device="cuda"))),
        (vs.VimScanError, lambda: vs.causal_scan(*a, y=torch.zeros((1, 10, 32), device="cuda").expand(2, 10, 32))),
        (ValueError, lambda: vs.causal_scan_step(*a, state)),
        (ValueError, lambda: vs.causal_scan_step(*[t[:, 0] for t in a[:5]], *a[5:], None)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            raise AssertionError(f"call {i} was not refused")
    assert (state == 0).all()


def test_time_major(vs):
    """Tensors that lie [L, batch, channels] in memory, outputs among them."""
    p = inputs((3, 40), 24, 16, F32, 6)
    a = cuda({k: v.transpose(0, 1).contiguous().transpose(0, 1) if v.dim() == 3 else v for k, v in p.items()})
    assert not a[0].is_contiguous()
    y = vs.causal_scan(*a)
    want, _ = ref(p)
    close(y, want, Y_TOL[F32])


def test_overlapping_rows(vs):
    """Activations that are windows over one signal: rows one element apart, shared by the batch."""
    d, L = 24, 11
    p = inputs((2, L), d, 16, F32, 9)
    signal = torch.randn(L + d, generator=torch.Generator().manual_seed(9))
    p["u"] = signal.as_strided((2, L, d), (0, 1, 1))
    a = cuda({**p, "u": p["u"].contiguous()})
    u = a[0] = signal.cuda().as_strided((2, L, d), (0, 1, 1))
    y = vs.causal_scan(*a)
    want, _ = ref(p)
    close(y, want, Y_TOL[F32])
    got = vs.causal_scan_bwd(*a, torch.ones_like(y))
    dense = vs.causal_scan_bwd(u.contiguous(), *a[1:], torch.ones_like(y))
    assert all(torch.equal(got[k], dense[k]) for k in dense)


@pytest.mark.parametrize("over", [0, 1, 2], ids=["u", "delta", "z"])
@pytest.mark.parametrize("d", [40, 300, 1300])
def test_output_over_input(vs, over, d):
    """y in the place of u, delta or z: the bits of a call with an output of its own."""
    a = cuda(inputs((2, 75), d, 16, BF, d))
    y = vs.causal_scan(*a)
    b = [t.clone() for t in a]
    assert torch.equal(vs.causal_scan(*b, y=b[over]), y)
    token = [t[:, 5] if t.dim() == 3 else t for t in a[:5]] + a[5:]
    state = torch.zeros((2, d, 16), device="cuda")
    y = vs.causal_scan_step(*token, state.clone())
    b = [t.clone() for t in token]
    assert torch.equal(vs.causal_scan_step(*b, state, y=b[over]), y)


def test_long_sequence(vs):
    """20000 tokens, few channels: many handovers, slow decays."""
    p = inputs((1, 20000), 4, 16, F32, 12)
    state = torch.empty((1, 4, 16), device="cuda")
    y = vs.causal_scan(*cuda(p), state_out=state)
    want, last = ref(p)
    close(y, want, Y_TOL[F32])
    close(state, last, STATE_TOL)


def test_offsets_past_32_bits(vs):
    """Rows 2^27 elements apart (element offsets to 2^32) and a state cache of 2.3e9 elements."""
    L, d, N, far = 34, 16, 16, 1 << 27
    p = inputs((1, L), d, N, BF, 4)
    base = torch.empty((L, far), dtype=BF, device="cuda")
    args = cuda(p)
    for i, at in ((0, 0), (1, 64), (2, 128)):
        view = base[:, at:at + d]
        view.copy_(args[i][0])
        args[i] = view[None]
    y = base[:, 256:256 + d][None]
    vs.causal_scan(*args, y=y)
    want, _ = ref(p)
    close(y, want, Y_TOL[BF])
    del base, y, args
    slots, d = 70000, 2048
    q = inputs((2, 1), d, N, BF, 5)
    want, last = ref(q)
    u, delta, z, B, C, A, D, bias = cuda(q)
    cache = torch.empty((slots, d, N), device="cuda")
    rows = torch.tensor([slots - 1, 3], dtype=torch.int32, device="cuda")
    cache[rows.long()] = 0
    y = vs.causal_scan_step(u[:, 0], delta[:, 0], z[:, 0], B[:, 0], C[:, 0], A, D, bias, cache, slots=rows)
    close(y, want[:, 0], Y_TOL[BF])
    close(cache[rows.long()], last, STATE_TOL)
    cache[rows.long()] = 0
    vs.causal_scan(u, delta, z, B, C, A, D, bias, state=cache, slots=rows)
    close(cache[rows.long()], last, STATE_TOL)


def test_empty(vs):
    p = inputs((2, 0), 32, 16, F32, 1)
    state = torch.ones((2, 32, 16), device="cuda")
    y = vs.causal_scan(*cuda(p), state=state)
    assert y.shape == (2, 0, 32) and (state == 1).all()
    out = torch.zeros_like(state)
    vs.causal_scan(*cuda(p), state=state, state_out=out)
    assert (out == 1).all()
    p = inputs((0, 5), 32, 16, F32, 1)
    assert vs.causal_scan(*cuda(p)).shape == (0, 5, 32)
    p = inputs((0,), 32, 16, F32, 1)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert vs.causal_scan(*cuda(p), cu_seqlens=none).shape == (0, 32)
