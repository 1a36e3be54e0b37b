"""The operators between the projections together, as a time-mix block uses
them: norm, R/K/V products with an adapter, recurrence, head norm and gate, O
product, residual and the next norm -- a prefill of two sequences, then decode
steps of both from a pool of states, eager and replayed from a graph.

Every stage is checked against fp64 on the values that the stage before it
gave, with that stage's own tolerance: products 2e-3 sum |x||w| (the products'
own), adapters, norms and the recurrence as in their tests (loosened to 1e-4 of
the largest value here, against their 3e-5 and less, since the stages are only
to be the same operators), fp16 outputs plus half a step.
"""
import numpy as np
import pytest
import torch

import oracle
from weight_only_quantized_g64_b200 import build as rq_build
from weight_only_quantized_g64_b200 import rq, synth

pytestmark = pytest.mark.gpu
H, D, R, L = 3, 192, 8, 2
LENS = [23, 17]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rq_build.build()
    rq.lib()
    yield
    assert rq.read_device_status(reset=True) == rq.OK


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, what, extra=0.0):
    lim = 1e-4 * np.abs(ref).max() + extra
    if got.dtype == torch.float16:
        lim = lim + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
    assert np.all(np.abs(f64(got) - ref) <= lim), what


class Block:
    """Weights of one block; every call checks its result if it is told to."""

    def __init__(self):
        self.w, self.host = {}, {}
        for i, n in enumerate("rkvo"):
            c, s, st = oracle.quantize_g64(synth.weights(D, D, seed=60 + i).numpy() * 3, 4)
            assert st == 0
            self.host[n] = (c, s)
            self.w[n] = (torch.from_numpy(c).cuda(), torch.from_numpy(s.view(np.int16)).cuda())
        g = torch.Generator().manual_seed(1)
        rn = lambda *s: torch.randn(s, generator=g)                                        # noqa: E731
        self.A = (rn(L, R, D) * D ** -0.5).half().cuda()
        self.B = (rn(L, D, R) * 0.3).half().cuda()
        self.w1, self.b1, self.w2, self.b2 = ((1 + 0.1 * rn(D)).cuda() if i % 2 == 0 else (0.1 * rn(D)).cuda()
                                              for i in range(4))
        self.decay, self.bonus = (rn(D) - 2).cuda(), (0.3 * rn(D)).cuda()

    def product(self, x, name, check, stacked=None):
        y = stacked if stacked is not None else (
            rq.gemv_wq(x, *self.w[name], D, 4) if x.shape[0] <= rq.MAX_DECODE_M else rq.gemm_wq(x, *self.w[name], D, 4))
        if check:
            ref, budget = oracle.matmul(x.cpu().numpy(), *self.host[name], 4)
            assert np.all(np.abs(f64(y) - ref) <= 2e-3 * budget), name
        return y

    def run(self, h, ids, scan, check):
        """h [M, D] fp32 -> (h', x' fp16); scan(r, d, k, v, a, b) -> y [M, H, 64]."""
        M = h.shape[0]
        _, x = rq.norm_residual(h, pre="layer", pre_weight=self.w1, pre_bias=self.b1)
        if check:
            u = f64(h)
            z = (u - u.mean(1, keepdims=True)) / np.sqrt(u.var(1, keepdims=True) + 1e-5)
            near(x, z * f64(self.w1) + f64(self.b1), "first norm")
        if M <= rq.MAX_DECODE_M:
            ys = rq.rkv_fused3(x, x, x, self.w["r"], self.w["k"], self.w["v"], D, 4)
            r, k, v = (self.product(x, n, check, y) for n, y in zip("rkv", ys))
        else:
            r, k, v = (self.product(x, n, check) for n in "rkv")
        plain = r.clone()
        r = rq.lora_add(x, self.A, self.B, ids, r, out=r)
        if check:
            ref = f64(plain)
            for m, a in enumerate(ids.tolist()):
                if a >= 0:
                    ref[m] += f64(self.B[a]) @ (f64(self.A[a]) @ f64(x[m]))
            near(r, ref, "adapter")
        heads = lambda t: t.view(M, H, 64)                                                 # noqa: E731
        r, k, v, d = heads(r), heads(k), heads(v), heads(self.decay + 0.1 * k)
        unit = torch.nn.functional.normalize(k, dim=-1)
        y = scan(r, d.contiguous(), k, v, -unit, 0.5 * unit)
        bonus = ((r * k * heads(self.bonus.expand(M, D))).sum(-1, keepdim=True) * v).reshape(M, D)
        gate = torch.sigmoid(h)
        _, x = rq.norm_residual(y.view(M, D), post="layer", post_group=64, post_weight=self.w2, post_bias=self.b2,
                                add=bonus, gate=gate)
        if check:
            u = f64(y)
            z = (u - u.mean(2, keepdims=True)) / np.sqrt(u.var(2, keepdims=True) + 1e-5)
            near(x, (z.reshape(M, D) * f64(self.w2) + f64(self.b2) + f64(bonus)) * f64(gate), "head norm and gate")
        o = self.product(x, "o", check)
        h2, x2 = rq.norm_residual(o, h=h, pre="layer", pre_weight=self.w1, pre_bias=self.b1)
        if check:
            u = f64(o) + f64(h)
            z = (u - u.mean(1, keepdims=True)) / np.sqrt(u.var(1, keepdims=True) + 1e-5)
            near(h2, u, "residual")
            near(x2, z * f64(self.w1) + f64(self.b1), "second norm")
        return h2, x2


def recurrence(xs, S):
    """One token of one sequence in fp64: (y, S)."""
    r, d, k, v, a, b = xs
    w = np.exp(-np.exp(-0.5) / (1 + np.exp(-d)))
    sa = np.einsum("hij,hj->hi", S, a)
    S = S * w[:, None, :] + sa[:, :, None] * b[:, None, :] + v[:, :, None] * k[:, None, :]
    return np.einsum("hij,hj->hi", S, r), S


def test_prefill_and_decode():
    block = Block()
    T = sum(LENS)
    g = torch.Generator().manual_seed(2)
    h = torch.randn((T, D), generator=g).cuda()
    ids = torch.tensor([0] * LENS[0] + [1] * LENS[1], dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, LENS[0], T], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool = torch.zeros((5, H, 64, 64), device="cuda")
    states = [np.zeros((H, 64, 64)) for _ in LENS]

    def prefill(*xs):
        y, _ = rq.tmix_scan(*xs, seq, state=pool, state_out=pool, slots=slots)
        ref, n = np.zeros((T, H, 64)), [f64(x) for x in xs]
        for q, (lo, hi) in enumerate(((0, LENS[0]), (LENS[0], T))):
            for t in range(lo, hi):
                ref[t], states[q] = recurrence([x[t] for x in n], states[q])
        near(y, ref, "scan")
        return y

    block.run(h, ids, prefill, True)
    for q, s in enumerate(slots.tolist()):
        near(pool[s], states[q], "state after the prefill")

    ids = torch.tensor([0, -1], dtype=torch.int32, device="cuda")

    def step(*xs):
        y, _ = rq.tmix_step(*xs, state=pool, state_out=pool, slots=slots)
        return y

    def checked_step(*xs):
        y = step(*xs)
        n = [f64(x) for x in xs]
        ref = []
        for q in range(2):
            out, states[q] = recurrence([x[q] for x in n], states[q])
            ref.append(out)
        near(y, np.stack(ref), "step")
        return y

    tokens = [torch.randn((2, D), generator=g).cuda() for _ in range(3)]
    block.run(tokens[0], ids, checked_step, True)
    for q, s in enumerate(slots.tolist()):
        near(pool[s], states[q], "state after a step")
    assert torch.all(pool[[0, 2, 4]] == 0)

    # the next two steps: eager, and the same from one graph replayed on new inputs
    start = pool.clone()
    eager = [block.run(t, ids, step, False) for t in tokens[1:]]
    end = pool.clone()
    pool.copy_(start)
    fixed = tokens[1].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block.run(fixed, ids, step, False)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.run(fixed, ids, step, False)
    pool.copy_(start)
    for t, want in zip(tokens[1:], eager):
        fixed.copy_(t)
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert torch.equal(pool, end)
    del graph
