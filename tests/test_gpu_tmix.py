"""The time-mix recurrence on the GPU (rq_tmix_scan, rq_tmix_scan_bwd,
rq_tmix_step) against the recurrence written out in fp64 on the host.

Tolerances, per element.  With u = 2^-24 every value is a sum of products
computed in fp32 over at most a few hundred terms whose rounding errors the
recurrence carries on; a row of the state is multiplied by factors of at most 1
(|a| <= 1, |b| <= 1 along one direction, decay < 1), so errors add up over the
decay's memory.  The tests' decays forget within about 100 tokens (sigmoid(d)
>= 0.05 for nearly all channels) and a token adds at most about 5 roundings per
element, each relative to the largest magnitude M of the array that the result
is taken from: 500 u M in the worst case of equal signs, 3e-5 M.  The tests use
that with M the largest magnitude of the compared array (for the decay's
gradient, which is a sum of signed products of two such arrays, twice that),
plus half a step of fp16 (2^-11 of the value, 2^-25 for subnormals) where the
output is fp16.
"""
import numpy as np
import pytest
import torch

from weight_only_quantized_g64_b200 import build as rq_build
from weight_only_quantized_g64_b200 import rq

pytestmark = pytest.mark.gpu
HEAD = 64
DECAY = float(np.exp(-0.5))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rq_build.build()
    rq.lib()
    yield
    assert rq.read_device_status(reset=True) == rq.OK


def inputs(T, H, dtype, seed, wide=False):
    """r, d, k, v, a, b [T, H, 64]; wide: columns of one [T, 6 * H * 64 + 8] matrix."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda: torch.randn((T, H, HEAD), generator=g)                                    # noqa: E731
    unit = torch.nn.functional.normalize(rn(), dim=-1) if T else rn()
    xs = [0.5 * rn(), rn(), 0.5 * rn(), rn(), -unit, unit * torch.sigmoid(rn())]
    if not wide:
        return [x.to(dtype).cuda() for x in xs]
    big = torch.full((T, 6 * H * HEAD + 8), float("nan"), dtype=dtype, device="cuda")
    parts = [big[:, i * H * HEAD:(i + 1) * H * HEAD].view(T, H, HEAD) for i in range(6)]
    for p, x in zip(parts, xs):
        p.copy_(x)
    return parts


def reference(xs, starts, state, dy=None, dstate=None):
    """(y, states[, grads, dstate_in]) in fp64 on the host; tokens outside the sequences give NaN."""
    r, d, k, v, a, b = (x.double().cpu().numpy() for x in xs)
    T, H, _ = r.shape
    s = 1 / (1 + np.exp(-d))
    w = np.exp(-DECAY * s)
    y = np.full_like(r, np.nan)
    grads = [np.full_like(r, np.nan) for _ in range(6)]
    S_all = np.zeros((len(starts) - 1, H, HEAD, HEAD)) if state is None else state.double().cpu().numpy().copy()
    G_all = np.zeros_like(S_all) if dstate is None else dstate.double().cpu().numpy().copy()
    g = None if dy is None else dy.double().cpu().numpy()
    for q, (lo, hi) in enumerate(zip(starts, starts[1:])):
        S = S_all[q].copy()
        past = []
        for t in range(lo, hi):
            past.append(S)
            sa = np.einsum("hij,hj->hi", S, a[t])
            S = S * w[t][:, None, :] + sa[:, :, None] * b[t][:, None, :] + v[t][:, :, None] * k[t][:, None, :]
            y[t] = np.einsum("hij,hj->hi", S, r[t])
        S_all[q] = S
        if g is None:
            continue
        G = G_all[q].copy()
        after = S
        for t in reversed(range(lo, hi)):
            before = past.pop()
            G = G + g[t][:, :, None] * r[t][:, None, :]
            sa, gb = np.einsum("hij,hj->hi", before, a[t]), np.einsum("hij,hj->hi", G, b[t])
            grads[0][t] = np.einsum("hij,hi->hj", after, g[t])
            grads[1][t] = (G * before).sum(1) * w[t] * -DECAY * s[t] * (1 - s[t])
            grads[2][t] = np.einsum("hij,hi->hj", G, v[t])
            grads[3][t] = np.einsum("hij,hj->hi", G, k[t])
            grads[4][t] = np.einsum("hij,hi->hj", before, gb)
            grads[5][t] = np.einsum("hij,hi->hj", G, sa)
            G = G * w[t][:, None, :] + gb[:, :, None] * a[t][:, None, :]
            after = before
        G_all[q] = G
    return (y, S_all) if g is None else (y, S_all, grads, G_all)


def check(got, ref, what, times=1.0):
    half = got.dtype == torch.float16
    x = got.double().cpu().numpy()
    live = ~np.isnan(ref)
    assert live.any() or ref.size == 0, what
    if not live.any():
        return
    lim = times * 3e-5 * np.abs(ref[live]).max() + (np.abs(ref[live]) * 2.0 ** -11 + 2.0 ** -25 if half else 0.0)
    d = np.abs(x[live] - ref[live])
    assert np.all(d <= lim), f"{what}: worst {d.max():.3e}, largest value {np.abs(ref[live]).max():.3e}"


SEQS = [[0, 1], [0, 15], [0, 16], [0, 17], [0, 33, 33, 97], [0, 0, 5, 69], [3, 20, 40], [0, 300]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("H,wide", [(1, False), (3, True)])
@pytest.mark.parametrize("starts", SEQS, ids=str)
def test_scan_and_gradients(starts, H, wide, dtype):
    """Lengths from 0 and 1 to several chunks and ragged ends, tokens before and behind the sequences."""
    T, S = starts[-1] + 3, len(starts) - 1
    xs = inputs(T, H, dtype, seed=T + H, wide=wide)
    g = torch.Generator().manual_seed(T)
    state = (0.3 * torch.randn((S, H, HEAD, HEAD), generator=g)).cuda()
    dstate = (0.1 * torch.randn((S, H, HEAD, HEAD), generator=g)).cuda()
    dy = torch.randn((T, H, HEAD), generator=g).to(dtype).cuda()
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")
    y = torch.full((T, H, HEAD), 7.0, dtype=dtype, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], S)
    out, end = rq.tmix_scan(*xs, seq, state=state, y=y, ckpt=ckpt)
    grads = tuple(torch.full_like(y, 7.0) for _ in range(6))
    got, dstart = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, dstate_out=dstate, grads=grads)
    torch.cuda.synchronize()
    ref_y, ref_S, ref_g, ref_G = reference(xs, starts, state, dy, dstate)
    check(out, ref_y, "y")
    check(end, ref_S, "state")
    for n, x, ref in zip(("r", "d", "k", "v", "a", "b"), got, ref_g):
        check(x, ref, "d" + n, times=2.0 if n == "d" else 1.0)
    check(dstart, ref_G, "dstate")
    outside = [t for t in range(T) if t < starts[0] or t >= starts[-1]]
    for x in (out, *got):
        assert torch.all(x[outside] == 7.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("H,lens", [(1, [(7 * i) % 50 for i in range(70)]), (66, [1, 0, 15, 16, 17, 50]),
                                    (40, [33, 31, 130])], ids=["70x1", "6x66", "3x40"])
def test_many_heads(H, lens, dtype):
    """Enough heads of all sequences together for the kernel on the tensor cores; more sequences than it orders, too."""
    starts = np.cumsum([0] + lens).tolist()
    T, S = starts[-1], len(lens)
    xs = inputs(T, H, dtype, seed=T + H, wide=H == 40)
    g = torch.Generator().manual_seed(T)
    state = (0.3 * torch.randn((S, H, HEAD, HEAD), generator=g)).cuda()
    dstate = (0.1 * torch.randn((S, H, HEAD, HEAD), generator=g)).cuda()
    dy = torch.randn((T, H, HEAD), generator=g).to(dtype).cuda()
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], S)
    out, end = rq.tmix_scan(*xs, seq, state=state, ckpt=ckpt)
    got, dstart = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, dstate_out=dstate)
    ref_y, ref_S, ref_g, ref_G = reference(xs, starts, state, dy, dstate)
    check(out, ref_y, "y")
    check(end, ref_S, "state")
    for n, x, ref in zip("rdkvab", got, ref_g):
        check(x, ref, "d" + n, times=2.0 if n == "d" else 1.0)
    check(dstart, ref_G, "dstate")
    again, end2 = rq.tmix_scan(*xs, seq, state=state)
    assert torch.equal(out, again) and torch.equal(end, end2)


@pytest.mark.parametrize("name", ["r", "d", "k", "v", "a", "b"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("H", [2, 66])
def test_non_finite_and_huge_inputs_reach_no_earlier_token(name, value, H):
    """One element at token 21: the tokens before it, the other heads and the other sequence keep their values (the
    head's own chunk may be taken another way: within the tolerance)."""
    starts = [0, 40, 60]
    xs = inputs(60, H, torch.float32, seed=11)
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")
    clean, _ = rq.tmix_scan(*xs, seq)
    xs["rdkvab".index(name)][21, 1, 9] = value
    y, end = rq.tmix_scan(*xs, seq)
    rest = torch.ones(60, H, dtype=torch.bool)
    rest[:40, 1] = False
    assert torch.equal(y[rest.cuda()], clean[rest.cuda()])
    check(y[:21, 1], clean[:21, 1].double().cpu().numpy(), "earlier tokens")
    if np.isnan(value):
        assert torch.isnan(y[21, 1, 9] if name == "v" else y[21, 1]).all()


def test_scan_without_states():
    starts = [0, 40, 50]
    xs = inputs(50, 2, torch.float32, seed=1)
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")
    y, end = rq.tmix_scan(*xs, seq)
    ref_y, ref_S = reference(xs, starts, None)
    check(y, ref_y, "y")
    check(end, ref_S, "state")
    dy = torch.ones_like(y)
    ckpt = rq.tmix_ckpt(y, 2)
    rq.tmix_scan(*xs, seq, ckpt=ckpt)
    got, dstart = rq.tmix_scan_bwd(*xs, seq, ckpt, dy)
    _, _, ref_g, ref_G = reference(xs, starts, None, dy)
    for n, x, ref in zip("rdkvab", got, ref_g):
        check(x, ref, "d" + n, times=2.0 if n == "d" else 1.0)
    check(dstart, ref_G, "dstate")


def test_no_tokens():
    """T = 0: the states pass through, forwards and backwards."""
    xs = inputs(0, 2, torch.float16, seed=1)
    seq = torch.zeros(4, dtype=torch.int32, device="cuda")
    state = torch.randn((3, 2, HEAD, HEAD), device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], 3)
    y, end = rq.tmix_scan(*xs, seq, state=state, ckpt=ckpt)
    assert y.shape == (0, 2, HEAD) and torch.equal(end, state)
    grads, dstart = rq.tmix_scan_bwd(*xs, seq, ckpt, y, dstate_out=state)
    assert torch.equal(dstart, state)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (33, 2)])
def test_step_in_a_pool(B, H, dtype):
    """One token each, states in a pool, in place; some requests have no state."""
    xs = inputs(B, H, dtype, seed=B)
    pool = torch.randn((B + 4, H, HEAD, HEAD), device="cuda")
    slots = torch.randperm(B + 4, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32)
    if B > 1:
        slots[1] = -1
    start = pool.clone()
    y, out = rq.tmix_step(*xs, state=pool, state_out=pool, slots=slots.cuda())
    assert out is pool
    picked = torch.stack([start[s] if s >= 0 else torch.zeros_like(start[0]) for s in slots.tolist()])
    ref_y, ref_S = reference(xs, list(range(B + 1)), picked)
    check(y, ref_y, "y")
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            check(pool[s], ref_S[i], "state")
    rest = [i for i in range(B + 4) if i not in slots.tolist()]
    assert torch.equal(pool[rest], start[rest])


def test_steps_are_the_scan():
    """A sequence token by token and at once, with states in a pool."""
    T, H = 37, 2
    xs = inputs(T, H, torch.float32, seed=9, wide=True)
    pool = torch.zeros((5, H, HEAD, HEAD), device="cuda")
    slots = torch.tensor([3], dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y, _ = rq.tmix_scan(*xs, seq, state=pool, state_out=pool, slots=slots)
    one = torch.zeros((1, H, HEAD, HEAD), device="cuda")
    for t in range(T):
        yt, _ = rq.tmix_step(*(x[t:t + 1] for x in xs), state=one, state_out=one)
        check(y[t:t + 1], yt.double().cpu().numpy(), f"y[{t}]")
    check(pool[3], one[0].double().cpu().numpy(), "state")
    assert torch.all(pool[[0, 1, 2, 4]] == 0)


def test_bad_offsets_and_slots_are_skipped():
    """Offsets that fall or leave the tokens, slots behind the pool: a status, and nothing written for them."""
    xs = inputs(20, 1, torch.float32, seed=3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 8, 4, 21], dtype=torch.int32, device="cuda")
    y = torch.full((20, 1, HEAD), 7.0, device="cuda")
    end = torch.full((3, 1, HEAD, HEAD), 5.0, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], 3)
    rq.tmix_scan(*xs, seq, state_out=end, y=y, ckpt=ckpt, dev_status=status)
    grads = tuple(torch.full_like(y, 7.0) for _ in range(6))
    rq.tmix_scan_bwd(*xs, seq, ckpt, torch.ones_like(y), grads=grads, dev_status=status)
    assert status.item() == rq.ERR_RANGE
    ref_y, ref_S = reference([x[:8] for x in xs], [0, 8], None)
    check(y[:8], ref_y, "y")
    check(end[:1], ref_S, "state")
    for x in (y, *grads):
        assert torch.all(x[8:] == 7.0)
    assert torch.all(end[1:] == 5.0)
    status.zero_()
    pool = torch.full((2, 1, HEAD, HEAD), 5.0, device="cuda")
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    y1, _ = rq.tmix_step(*(x[:1] for x in xs), state=pool, state_out=pool, slots=slots, dev_status=status)
    assert status.item() == rq.ERR_RANGE and torch.all(pool == 5.0)
    check(y1, reference([x[:1] for x in xs], [0, 1], None)[0], "y without a state")


def test_bad_offsets_among_many_heads():
    """The kernel that takes sequences in the order of their lengths: a bad pair changes no other sequence."""
    T, H = 80, 40
    xs = inputs(T, H, torch.float16, seed=11)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 5, 40, 95, 60, 75], dtype=torch.int32, device="cuda")       # (40, 95) and (95, 60) are bad
    y = torch.full((T, H, HEAD), 7.0, dtype=torch.float16, device="cuda")
    end = torch.full((5, H, HEAD, HEAD), 5.0, device="cuda")
    rq.tmix_scan(*xs, seq, state_out=end, y=y, dev_status=status)
    assert status.item() == rq.ERR_RANGE
    for i, lo, hi in ((0, 0, 5), (1, 5, 40), (4, 60, 75)):
        ref_y, ref_S = reference([x[lo:hi] for x in xs], [0, hi - lo], None)
        check(y[lo:hi], ref_y, "y")
        check(end[i:i + 1], ref_S, "state")
    assert torch.all(end[2:4] == 5.0) and torch.all(y[40:60] == 7.0) and torch.all(y[75:] == 7.0)


def test_gradients_against_differences():
    """dL along random directions against central differences of the fp64 recurrence."""
    starts, T, H = [0, 21, 40], 40, 1
    xs = inputs(T, H, torch.float32, seed=5)
    g = torch.Generator().manual_seed(6)
    state = (0.3 * torch.randn((2, H, HEAD, HEAD), generator=g)).cuda()
    dy = torch.randn((T, H, HEAD), generator=g).cuda()
    dS = torch.randn((2, H, HEAD, HEAD), generator=g).cuda()
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], 2)
    rq.tmix_scan(*xs, seq, state=state, ckpt=ckpt)
    grads, dstart = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, dstate_out=dS)

    def loss(ys, st):
        y, S = reference(ys, starts, st)
        return (y * dy.double().cpu().numpy()).sum() + (S * dS.double().cpu().numpy()).sum()

    eps = 1e-5
    for i in range(7):
        base = xs[i] if i < 6 else state
        way = torch.randn(base.shape, generator=g, dtype=torch.float64)
        plus, minus = ([x.double().cpu() for x in xs] for _ in range(2))
        sp, sm = state.double().cpu(), state.double().cpu()
        if i < 6:
            plus[i] = plus[i] + eps * way
            minus[i] = minus[i] - eps * way
        else:
            sp, sm = sp + eps * way, sm - eps * way
        diff = (loss(plus, sp) - loss(minus, sm)) / (2 * eps)
        grad = (grads[i] if i < 6 else dstart).double().cpu()
        # each element within 6e-5 of the largest, as above, plus eps^2 of curvature
        bound = 6e-5 * float(grad.abs().max()) * float(way.abs().sum()) + 1e-6 * abs(diff)
        assert abs(float((grad * way).sum()) - diff) <= bound, i


def test_non_finite_stays_in_its_head():
    """A NaN value channel spoils its own row only; the other head and sequence are untouched."""
    starts = [0, 20, 40]
    xs = inputs(40, 2, torch.float32, seed=8)
    clean, _ = rq.tmix_scan(*xs, torch.tensor(starts, dtype=torch.int32, device="cuda"))
    xs[3][5, 1, 7] = float("nan")
    y, _ = rq.tmix_scan(*xs, torch.tensor(starts, dtype=torch.int32, device="cuda"))
    bad = torch.isnan(y)
    assert bad[5:20, 1, 7].all()
    bad[5:20, 1, 7] = False
    assert not bad.any()
    keep = torch.ones_like(bad)
    keep[5:20, 1, 7] = False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_same_bits_every_time(dtype):
    xs = inputs(333, 6, dtype, seed=2)
    seq = torch.tensor([0, 200, 333], dtype=torch.int32, device="cuda")
    dy = torch.randn((333, 6, HEAD), device="cuda").to(dtype)
    first = None
    for _ in range(10):
        ckpt = rq.tmix_ckpt(xs[0], 2)
        y, end = rq.tmix_scan(*xs, seq, ckpt=ckpt)
        grads, dstart = rq.tmix_scan_bwd(*xs, seq, ckpt, dy)
        now = [x.clone() for x in (y, end, *grads, dstart)]
        first = first or now
        assert all(torch.equal(p, q) for p, q in zip(first, now))


@pytest.mark.parametrize("H", [2, 40])
def test_other_stream_and_capture(H):
    """On a stream of its own, and captured and replayed on new values."""
    xs = inputs(70, H, torch.float16, seed=4)
    seq = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    dy = torch.randn((70, H, HEAD), device="cuda").half()
    ckpt = rq.tmix_ckpt(xs[0], 2)
    y0, s0 = rq.tmix_scan(*xs, seq, ckpt=ckpt)
    g0, d0 = rq.tmix_scan_bwd(*xs, seq, ckpt, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y1, s1 = rq.tmix_scan(*xs, seq, ckpt=ckpt, stream=side)
    g1, d1 = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(s0, s1) and torch.equal(d0, d1)
    assert all(torch.equal(p, q) for p, q in zip(g0, g1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ck2 = rq.tmix_ckpt(xs[0], 2)
        y2, s2 = rq.tmix_scan(*xs, seq, ckpt=ck2)
        g2, d2 = rq.tmix_scan_bwd(*xs, seq, ck2, dy)
    new = inputs(70, H, torch.float16, seed=40)
    for x, n in zip(xs, new):
        x.copy_(n)
    graph.replay()
    y3, s3 = rq.tmix_scan(*xs, seq, ckpt=ckpt)
    g3, d3 = rq.tmix_scan_bwd(*xs, seq, ckpt, dy)
    torch.cuda.synchronize()
    assert torch.equal(y2, y3) and torch.equal(s2, s3) and torch.equal(d2, d3)
    assert all(torch.equal(p, q) for p, q in zip(g2, g3))
    del graph


@pytest.mark.parametrize("H", [1, 40])
def test_two_at_once(H):
    """Two calls on two streams, each with its own memory, give what they give one after the other."""
    calls = []
    for i in range(2):
        xs = inputs(600, H, torch.float32, seed=60 + i)
        calls.append((xs, torch.tensor([0, 450, 600], dtype=torch.int32, device="cuda"), rq.tmix_ckpt(xs[0], 2),
                      torch.randn((600, H, HEAD), device="cuda"), torch.cuda.Stream()))

    def both(streams):
        got = []
        for xs, seq, ckpt, dy, side in calls:
            s = side if streams else None
            y, end = rq.tmix_scan(*xs, seq, ckpt=ckpt, stream=s)
            grads, start = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, stream=s)
            got += [y, end, start, *grads]
        torch.cuda.synchronize()
        return got

    torch.cuda.synchronize()
    for p, q in zip(both(False), both(True)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("H", [1, 40])
def test_offsets_past_32_bits(H):
    """The last tokens of a matrix with more than 2^31 elements before them."""
    T, last, ld = 33000, 24, 65536
    big = torch.empty((T, ld), dtype=torch.float16, device="cuda")
    small = inputs(last, H, torch.float16, seed=9)
    parts = [big[:, (i + 1) * H * HEAD:(i + 2) * H * HEAD].unflatten(1, (H, HEAD)) for i in range(6)]
    for p, x in zip(parts, small):
        p[T - last:] = x
    seq = torch.tensor([T - last, T], dtype=torch.int32, device="cuda")
    ckpt = rq.tmix_ckpt(parts[0], 1)
    dy = torch.ones((T, H, HEAD), dtype=torch.float16, device="cuda")
    y, end = rq.tmix_scan(*parts, seq, ckpt=ckpt)
    grads, start = rq.tmix_scan_bwd(*parts, seq, ckpt, dy)
    own = torch.tensor([0, last], dtype=torch.int32, device="cuda")
    few = rq.tmix_ckpt(small[0], 1)
    y1, end1 = rq.tmix_scan(*small, own, ckpt=few)
    grads1, start1 = rq.tmix_scan_bwd(*small, own, few, dy[:last])
    assert torch.equal(y[T - last:], y1) and torch.equal(end, end1) and torch.equal(start, start1)
    for p, q in zip(grads, grads1):
        assert torch.equal(p[T - last:], q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("lens", [[33], [48], [64], [65, 0, 129], [400]], ids=str)
def test_gradients_of_many_heads_by_chunks(lens, dtype):
    """From the first chunk that a preparing group takes while its last one may still be in use: against fp64, and the
    same bits every time."""
    starts = np.cumsum([0] + lens).tolist()
    T, S, H = starts[-1], len(lens), 40
    xs = inputs(T, H, dtype, seed=T)
    g = torch.Generator().manual_seed(T)
    dstate = (0.1 * torch.randn((S, H, HEAD, HEAD), generator=g)).cuda()
    dy = torch.randn((T, H, HEAD), generator=g).to(dtype).cuda()
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], S)
    out, end = rq.tmix_scan(*xs, seq, ckpt=ckpt)
    got, dstart = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, dstate_out=dstate)
    ref_y, ref_S, ref_g, ref_G = reference(xs, starts, None, dy, dstate)
    check(out, ref_y, "y")
    check(end, ref_S, "state")
    for n, x, ref in zip("rdkvab", got, ref_g):
        check(x, ref, "d" + n, times=2.0 if n == "d" else 1.0)
    check(dstart, ref_G, "dstate")
    for _ in range(20):
        again, dagain = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, dstate_out=dstate)
        assert torch.equal(dstart, dagain) and all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("H", [2, 40])
def test_slow_decays(H, dtype):
    """Decays near 1, the same in every token of a long sequence: what a rounding of each would lose adds up.

    The keys 32 .. 63 have a = b = 0, so every element of their states is w S + v k in each token; d runs over them
    from -12 to -7, v k is small against the first state, and the outputs read these keys alone.  With u = 2^-24 and M
    the largest magnitude of a state, a chunk of 16 tokens rounds an element twice (the sum, the decay) and a pair or
    a single token at most three times for two: 3 u M T / 2 if every rounding has one sign in the worst form, 2 u M T /
    16 in the chunks.  log w, off by at most (|d| + 6) u of itself, adds T |log w| w^T (|d| + 6) u <= 18 u.  The
    products v k are kept to 2^-21: T of them, together at most 2^-21 T max|v| max|k| (backwards dy, r).  An output is a
    sum of 32 products, each kept to 2^-21 as well.
    """
    T, u = 4096, 2.0 ** -24
    g = torch.Generator().manual_seed(H)
    r, d, k, v, a, b = inputs(T, H, torch.float32, seed=H)
    v, d = 0.01 * v, d.clone()
    d[:, :, 32:] = torch.linspace(-12, -7, 32)
    for x in (a, b):
        x[:, :, 32:] = 0
    r[:, :, :32] = 0
    xs = [x.to(dtype) for x in (r, d, k, v, a, b)]
    dy = (0.01 * torch.randn((T, H, HEAD), generator=g)).to(dtype).cuda()
    state, dstate = ((10 * torch.randn((1, H, HEAD, HEAD), generator=g)).cuda() for _ in range(2))
    seq = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], 1)
    y, end = rq.tmix_scan(*xs, seq, state=state, ckpt=ckpt)
    _, start = rq.tmix_scan_bwd(*xs, seq, ckpt, dy, dstate_out=dstate)
    n = 2                                    # heads that are compared
    R, D, K, V, dY = (x[:, :n].double().cpu().numpy() for x in (*xs[:4], dy))
    w = np.exp(-DECAY / (1 + np.exp(-D)))[:, :, None, 32:]
    S, G = (x[0, :n, :, 32:].double().cpu().numpy() for x in (state, dstate))
    M, N = np.abs(S).max(), np.abs(G).max()
    rounds = 2 * T / 16 if H == 40 else 1.5 * T
    lim = (rounds + 18) * u * M + 2.0 ** -21 * T * np.abs(V).max() * np.abs(K).max()
    out = y[:, :n].double().cpu().numpy()
    for t in range(T):
        S = S * w[t] + V[t][:, :, None] * K[t][:, None, 32:]
        ref, r1 = np.einsum("hij,hj->hi", S, R[t][:, 32:]), np.abs(R[t]).sum(1, keepdims=True)
        half = np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 if dtype == torch.float16 else 0.0
        assert np.all(np.abs(out[t] - ref) <= r1 * (lim + 2.0 ** -20 * M) + half), t
    for t in reversed(range(T)):
        G = (G + dY[t][:, :, None] * R[t][:, None, 32:]) * w[t]
    for got, ref, top, f in ((end, S, M, np.abs(V).max() * np.abs(K).max()), (start, G, N, np.abs(dY).max() * np.abs(R).max())):
        e = np.abs(got[0, :n, :, 32:].double().cpu().numpy() - ref).max()
        assert e <= (rounds + 18) * u * top + 2.0 ** -21 * T * f, (e, top)


@pytest.mark.parametrize("H", [2, 40])
def test_strong_decays(H):
    """States that do nothing but decay, through products of down to 6e-5 in 16 tokens, element by element: with
    u = 2^-24 a token multiplies by w, off by 0.61 * 2^-21 (the sigmoid's error) and rounded, and rounds the product: at
    most 7 u.  The chunks of 16 add up log2 w instead, at most 14 and so with roundings of 8 u in four sums, and take 2^x,
    good to 4 u: 5 u a token and 40 u a chunk."""
    T = 75
    xs = inputs(T, H, torch.float32, seed=H)
    for i in (2, 3, 4, 5):
        xs[i].zero_()
    xs[1][:] = torch.linspace(-4, 20, HEAD)
    g = torch.Generator().manual_seed(H)
    state, dstate = (torch.randn((1, H, HEAD, HEAD), generator=g).cuda() for _ in range(2))
    seq = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], 1)
    _, end = rq.tmix_scan(*xs, seq, state=state, ckpt=ckpt)
    _, start = rq.tmix_scan_bwd(*xs, seq, ckpt, torch.zeros_like(xs[0]), dstate_out=dstate)
    w = torch.exp(-DECAY * T * torch.sigmoid(xs[1][0, 0].double()))
    for got, first in ((end, state), (start, dstate)):
        ref = first.double() * w
        assert torch.all((got.double() - ref).abs() <= 8 * T * 2.0 ** -24 * ref.abs())


def test_gradient_of_strong_and_weak_decays():
    """dd = dlogw * -c s (1 - s) where either factor is small, element by element: sequences of one token with k = v =
    dy = 0, so that dlogw_j = w_j sum_i G_ij S_ij, here of positive terms.

    With u = 2^-24: the sum of 64 products in fp32 is off by at most 66 u of itself, w by 2 u; e^-|d| by 2 |d| u + 4 u (its
    argument rounded once, beside log2(e); 2^x good to 2^-22), 1 / (1 + e) by that and 3 u; their products add 3 u.
    Together (66 + 2 + 6 |d| + 24) u."""
    T, H = 256, 1
    xs = inputs(T, H, torch.float32, seed=21)
    for i in (2, 3):
        xs[i].zero_()
    xs[1][:] = torch.linspace(-30, 30, T * HEAD).view(T, H, HEAD)
    g = torch.Generator().manual_seed(21)
    state, dstate = ((0.1 + torch.rand((T, H, HEAD, HEAD), generator=g)).cuda() for _ in range(2))
    xs[4].zero_(), xs[5].zero_()
    seq = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    ckpt = rq.tmix_ckpt(xs[0], T)
    rq.tmix_scan(*xs, seq, state=state, ckpt=ckpt)
    grads, _ = rq.tmix_scan_bwd(*xs, seq, ckpt, torch.zeros_like(xs[0]), dstate_out=dstate)
    d = xs[1].double().cpu().numpy()
    s, c = 1 / (1 + np.exp(-d)), 1 / (1 + np.exp(d))
    sums = (state.double() * dstate.double()).sum(2).cpu().numpy()
    ref = sums * np.exp(-DECAY * s) * -DECAY * s * c
    off = np.abs(grads[1].double().cpu().numpy() / ref - 1)
    lim = (92 + 6 * np.abs(d)) * 2.0 ** -24
    assert np.all(off <= lim), f"worst {(off / lim).max():.2f} of the bound at d = {d.flat[(off / lim).argmax()]}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_scan_of_many_heads_in_a_pool(dtype):
    """States of a pool updated in place by the kernel for many heads; an empty sequence, and one without a state."""
    H, starts = 30, [0, 40, 40, 57, 90]
    T, S = starts[-1], len(starts) - 1
    xs = inputs(T, H, dtype, seed=31)
    pool = (0.3 * torch.randn((7, H, HEAD, HEAD), generator=torch.Generator().manual_seed(1))).cuda()
    slots = [5, 2, -1, 0]
    first = pool.clone()
    y, out = rq.tmix_scan(*xs, torch.tensor(starts, dtype=torch.int32, device="cuda"), state=pool, state_out=pool,
                          slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert out is pool
    state = torch.stack([first[s] if s >= 0 else torch.zeros_like(first[0]) for s in slots])
    ref_y, ref_S = reference(xs, starts, state)
    check(y, ref_y, "y")
    for i, s in enumerate(slots):
        if s >= 0:
            check(pool[s], ref_S[i], "state")
    assert torch.equal(pool[[1, 2, 3, 4, 6]], first[[1, 2, 3, 4, 6]])


@pytest.mark.parametrize("name", ["r", "d", "k", "v", "a", "b", "dy"])
@pytest.mark.parametrize("H", [2, 66])
def test_non_finite_and_gradients(name, H):
    """A NaN at token 21 of one head: outside its 16 tokens every gradient that the formula keeps finite keeps its
    value, and so do the other head's and the other sequence's in full."""
    starts, h = [0, 50, 70], 1
    xs = inputs(70, H, torch.float32, seed=12)
    dy = torch.randn((70, H, HEAD), generator=torch.Generator().manual_seed(3)).cuda()
    dstate = torch.randn((2, H, HEAD, HEAD), generator=torch.Generator().manual_seed(4)).cuda()
    seq = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def run():
        ckpt = rq.tmix_ckpt(xs[0], 2)
        rq.tmix_scan(*xs, seq, ckpt=ckpt)
        return rq.tmix_scan_bwd(*xs, seq, ckpt, dy, dstate_out=dstate)

    clean, clean_start = run()
    (dy if name == "dy" else xs["rdkvab".index(name)])[21, h, 9] = float("nan")
    got, start = run()
    one = [x[:, h:h + 1] for x in xs]
    _, _, ref, _ = reference(one, starts, None, dy[:, h:h + 1], dstate[:, h:h + 1])
    rest = torch.ones(70, H, dtype=torch.bool)
    rest[:50, h] = False
    assert torch.equal(start[1], clean_start[1]) and torch.equal(start[0, [0]], clean_start[0, [0]])
    for i, n in enumerate("rdkvab"):
        assert torch.equal(got[i][rest.cuda()], clean[i][rest.cuda()]), n
        values = ref[i].copy()
        values[16:32] = np.nan               # (check leaves NaN of the formula out)
        values[50:] = np.nan
        live = ~np.isnan(values)
        x = got[i][:, h:h + 1].double().cpu().numpy()
        lim = (2 if n == "d" else 1) * 3e-5 * clean[i][:50, h].abs().max().item()
        assert not live.any() or np.all(np.abs(x[live] - values[live]) <= lim), n
