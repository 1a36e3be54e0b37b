"""The norm / gate / residual step on the GPU (rq_norm_residual) against the
formula in fp64.

Tolerance per element, from the arithmetic, with u = 2^-24.  A norm of G values
v with mean m and deviation s computes (v - m) / s: the mean is off by at most
(G / 8 + 16) u max|v| (sums of at most G / 8 partial sums, joined), the mean
square by twice that relatively, so the normed value z by
  e(z) = ((G / 8 + 16) u max|v| / s + u |v| / s + (G / 8 + 20) u |z|),
times the weight, plus 3 u of the result.  The tests use 8 u per rounding
of u, gate (e^-x within 2 u, the division 1 u) and residual on the magnitudes
that enter, carry e through Norm_pre with its own e and 1 / s, and add half a
step of fp16 (2^-11 of the value, 2^-25 for subnormals) where an output is fp16.
"""
import types

import numpy as np
import pytest
import torch

from weight_only_quantized_g64_b200 import build as rq_build
from weight_only_quantized_g64_b200 import rq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rq_build.build()
    rq.lib()
    yield


def normed(v, e, kind, group, w, b, eps):
    """(value, error bound) of a norm of v, known to within e."""
    if kind == "none":
        return v, e
    M, D = v.shape
    G = group or D
    g, ge = v.reshape(-1, G), e.reshape(-1, G)
    m = g.mean(1, keepdims=True) if kind == "layer" else np.zeros((g.shape[0], 1))
    s = np.sqrt(((g - m) ** 2).mean(1, keepdims=True) + eps)
    z = (g - m) / s
    top = np.abs(g).max(1, keepdims=True)
    off = ge.max(1, keepdims=True)
    # the inputs' own errors move the value, the mean and (relatively) the deviation
    ez = ((G / 8 + 16) * U * top + U * np.abs(g) + ge + off) / s + ((G / 8 + 20) * U + off / s) * np.abs(z)
    z, ez = z.reshape(M, D), ez.reshape(M, D)
    wv = np.ones(D) if w is None else w.double().cpu().numpy()
    bv = np.zeros(D) if b is None else b.double().cpu().numpy()
    out = z * wv + bv
    return out, ez * np.abs(wv) + 3 * U * (np.abs(z * wv) + np.abs(out))


def reference(y, post="none", post_group=0, post_weight=None, post_bias=None, eps_post=1e-5, add=None, gate=None,
              gate_act="identity", h=None, alpha=None, pre="none", pre_weight=None, pre_bias=None, eps_pre=1e-5):
    d = lambda t: t.double().cpu().numpy()                                                 # noqa: E731
    u = d(y)
    u, e = normed(u, np.zeros_like(u), post, post_group, post_weight, post_bias, eps_post)
    if add is not None:
        u, e = u + d(add), e + 8 * U * (np.abs(u) + np.abs(d(add)))
    if gate is not None:
        q = d(gate)
        f = q if gate_act == "identity" else (q if gate_act == "silu" else 1.0) / (1 + np.exp(-q))
        u, e = u * f, e * np.abs(f) + 8 * U * np.abs(u * f)
    if alpha is not None:
        u, e = u * d(alpha), e * np.abs(d(alpha)) + 8 * U * np.abs(u * d(alpha))
    if h is not None:
        e = e + 8 * U * (np.abs(u) + np.abs(d(h)))
        u = u + d(h)
    x, ex = normed(u, e, pre, 0, pre_weight, pre_bias, eps_pre)
    return u, e, x, ex


def check(got, ref, e, what):
    if got.dtype == torch.float16:
        e = e + (np.abs(ref) + e) * 2.0 ** -11 + 2.0 ** -25
    d = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(d <= e), f"{what}: worst {(d / np.maximum(e, 1e-300)).max():.2f} of the bound"


def tensors(M, D, dtype, seed, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    rows = lambda: torch.randn((M, D), generator=g).to(dtype).cuda()                       # noqa: E731
    cols = lambda: torch.randn(D, generator=g).cuda()                                      # noqa: E731
    return dict(y=(2 * torch.randn((M, D), generator=g) + mean).to(dtype).cuda(), add=rows(), gate=rows(), h=rows(),
                alpha=cols(), post_weight=cols(), post_bias=cols(), pre_weight=cols(), pre_bias=cols())


def run(kw, **more):
    kw = {**kw, **more}
    h, x = rq.norm_residual(**kw)
    u, e, rx, ex = reference(**kw)
    if h is not None:
        check(h, u, e, "h")
    check(x, rx, ex, "x")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("M,D", [(1, 64), (3, 128), (2, 320), (17, 768), (5, 2560), (2, 4096), (3, 4160), (2, 8192),
                                 (1, 10240), (2, 16384)])
def test_sizes_and_norms(M, D, dtype):
    t = tensors(M, D, dtype, seed=M + D)
    for post in ("none", "layer", "rms"):
        for pre in ("none", "layer", "rms"):
            for group in ((0, 64, 8) if post != "none" else (0,)):
                run(t, post=post, post_group=group, pre=pre, gate_act="silu")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("left_out", ["add", "gate", "h", "alpha", "post_weight", "post_bias", "pre_weight",
                                      "pre_bias"])
def test_absent_parts(left_out, dtype):
    t = tensors(4, 512, dtype, seed=1)
    t.pop(left_out)
    run(t, post="layer", post_group=64, pre="layer", gate_act="sigmoid")
    run(dict(y=t["y"]), pre="rms")
    run(dict(y=t["y"]))


@pytest.mark.parametrize("group", [8, 16, 32, 64, 128, 256, 512])
def test_groups(group):
    t = tensors(3, 512, torch.float32, seed=group)
    run(t, post="layer", post_group=group, gate_act="identity")
    run(t, post="rms", post_group=group, gate_act="sigmoid")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_strided_rows_and_in_place(dtype):
    """y, add and gate as columns of wider matrices; h updated in place; x and h_out given."""
    M, D = 6, 256
    t = tensors(M, D, dtype, seed=2)
    wide = torch.full((M, 3 * D + 40), float("nan"), dtype=dtype, device="cuda")
    for i, n in enumerate(("y", "add", "gate")):
        wide[:, 8 + i * D:8 + (i + 1) * D] = t[n]
        t[n] = wide[:, 8 + i * D:8 + (i + 1) * D]
    kw = dict(post="rms", pre="layer", gate_act="sigmoid")
    run(t, **kw)
    h1, x1 = rq.norm_residual(**t, **kw)
    mine = t["h"].clone()
    x = torch.empty((M, D), dtype=torch.float16, device="cuda")
    h2, x2 = rq.norm_residual(**{**t, "h": mine}, h_out=mine, x=x, **kw)
    assert h2 is mine and x2 is x and torch.equal(h1, mine) and torch.equal(x1, x)


def test_hard_rows():
    """A mean far above the deviation, constant rows, zeros, one large value, eps of 0."""
    D = 1024
    y = torch.randn((5, D), generator=torch.Generator().manual_seed(4))
    y[0] += 1e4
    y[1] = 3.0
    y[2] = 0.0
    y[3, 17] = 6e4
    y = y.cuda()
    for kind in ("layer", "rms"):
        run(dict(y=y), pre=kind)
        run(dict(y=y[3:]), pre=kind, eps_pre=0.0)


def test_non_finite_stays_in_its_row():
    t = tensors(4, 256, torch.float32, seed=5)
    clean_h, clean_x = rq.norm_residual(**t, post="layer", pre="layer")
    t["y"][2, 5] = float("inf")
    h, x = rq.norm_residual(**t, post="layer", pre="layer")
    for got, clean in ((h, clean_h), (x, clean_x)):
        assert torch.isnan(got[2]).all()
        assert torch.equal(got[[0, 1, 3]], clean[[0, 1, 3]])


def test_stream_capture_and_bits():
    t = tensors(9, 768, torch.float16, seed=6)
    kw = dict(post="layer", post_group=64, pre="rms", gate_act="silu")
    h, x = rq.norm_residual(**t, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = t.pop("y")
    h2, x2 = rq.norm_residual(y, **t, **kw, stream=side)
    side.synchronize()
    assert torch.equal(h, h2) and torch.equal(x, x2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, x3 = rq.norm_residual(y, **t, **kw)
    y.copy_(tensors(9, 768, torch.float16, seed=7)["y"])
    graph.replay()
    h4, x4 = rq.norm_residual(y, **t, **kw)
    assert torch.equal(h3, h4) and torch.equal(x3, x4)
    del graph


def test_offsets_past_32_bits():
    """Rows behind more than 2^31 elements of a wide matrix."""
    M, D, ld, last = 33000, 128, 65536, 9
    big = torch.empty((M, ld), dtype=torch.float16, device="cuda")
    y = big[:, 64:64 + D]
    y[:] = 1.0
    y[M - last:] = torch.randn((last, D), device="cuda").half()
    h = torch.randn((M, D), device="cuda").half()
    h1, x1 = rq.norm_residual(y, post="layer", h=h, pre="rms")
    h2, x2 = rq.norm_residual(y[M - last:].contiguous(), post="layer", h=h[M - last:], pre="rms")
    assert torch.equal(h1[M - last:], h2) and torch.equal(x1[M - last:], x2)


@pytest.mark.parametrize("D", [512, 8192])
def test_silu_of_large_and_very_negative_gates(D):
    """u * gate alone would overflow; the sigmoid by itself is 0 from about -87 on.

    silu is off by at most (2 |g| + 16) u of itself above -87, and below 2^-126 |g| there."""
    M = 3
    y = torch.full((M, D), 1e37, device="cuda")
    y[1] = -3e30
    gate = torch.linspace(-120, -60, M * D).view(M, D).cuda()
    gate[2, ::2] = 20.0
    y[2] = 1e25
    h, _ = rq.norm_residual(y, gate=gate, gate_act="silu", h=torch.zeros_like(y))
    g, v = gate.double().cpu().numpy(), y.double().cpu().numpy()
    ref = v * g / (1 + np.exp(-g))
    lim = np.where(g > -87, (2 * np.abs(g) + 16) * U * np.abs(ref), np.abs(v * g) * 2.0 ** -126)
    d = np.abs(h.double().cpu().numpy() - ref)
    assert np.all(d <= lim), f"worst at gate {g.flat[np.nanargmax(d / lim)]}"


@pytest.mark.parametrize("first", [dict(post="rms"), dict(x=None), dict(eps_pre=1e-5), {}], ids=str)
def test_stream_with_keywords_in_any_order(first, monkeypatch):
    t = tensors(4, 128, torch.float32, seed=1)
    side = torch.cuda.Stream()
    seen, real = [], rq._stream_of
    monkeypatch.setattr(rq, "_stream_of", lambda at: seen.append(real(at)) or seen[-1])
    torch.cuda.synchronize()
    rq.norm_residual(**first, y=t["y"], stream=side)
    side.synchronize()
    assert seen == [side.cuda_stream]


def test_stream_of_another_device_is_refused():
    t = tensors(4, 128, torch.float32, seed=1)
    with pytest.raises(rq.RQError) as e:
        rq.norm_residual(t["y"], stream=types.SimpleNamespace(device_index=t["y"].get_device() + 1))
    assert e.value.status == rq.ERR_SHAPE


MANY = [(18945, 64), (3789, 320), (2369, 512), (475, 2560), (297, 4096)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("M,D", MANY)
def test_many_rows(M, D, dtype):
    """Enough rows to be taken two at a time, the last one by itself; four fp32 tensors of 4096 one at a time all the
    same."""
    t = tensors(M, D, dtype, seed=D)
    run(t, post="layer", post_group=64, pre="rms", gate_act="silu")
    run(t, post="rms", post_group=8, pre="layer", gate_act="identity")
    run(t, post="layer", pre="layer", gate_act="sigmoid")
    run(dict(y=t["y"], h=t["h"], gate=t["gate"]), post="rms", pre="rms", gate_act="silu")
    run(dict(y=t["y"], h=t["h"]), pre="layer")
    run(dict(y=t["y"], add=t["add"], post_weight=t["post_weight"]), post="layer", post_group=32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("M,D", [(2369, 512), (297, 4096), (149, 8192)])
def test_many_rows_strided_and_in_place(M, D, dtype):
    t = tensors(M, D, dtype, seed=3)
    kw = dict(post="rms", pre="layer", gate_act="sigmoid")
    h1, x1 = rq.norm_residual(**t, **kw)
    wide = torch.full((M, 3 * D + 40), float("nan"), dtype=dtype, device="cuda")
    for i, n in enumerate(("y", "add", "gate")):
        wide[:, 8 + i * D:8 + (i + 1) * D] = t[n]
        t[n] = wide[:, 8 + i * D:8 + (i + 1) * D]
    mine = t["h"].clone()
    h2, x2 = rq.norm_residual(**{**t, "h": mine}, h_out=mine, **kw)
    assert h2 is mine and torch.equal(h1, mine) and torch.equal(x1, x2)


def test_many_rows_non_finite_stays_in_its_row():
    M, D = 2369, 512
    t = tensors(M, D, torch.float32, seed=5)
    clean_h, clean_x = rq.norm_residual(**t, post="layer", pre="layer")
    t["y"][7, 5] = float("inf")
    t["y"][M - 1, 9] = float("nan")
    h, x = rq.norm_residual(**t, post="layer", pre="layer")
    rest = [i for i in range(M) if i not in (7, M - 1)]
    for got, clean in ((h, clean_h), (x, clean_x)):
        assert torch.isnan(got[[7, M - 1]]).all() and torch.equal(got[rest], clean[rest])
