"""Low-rank adapters on the GPU (rq_lora_add) against the formula in fp64.

Tolerance per output, from the arithmetic: with u = 2^-24, the fp32 sum over K
exact products is off by at most (K / 16 + 20) u of sum |A||x| (the terms are
added in at most K / 16 partial sums of 16, or in 256 lanes of K / 256, then
joined); t is then kept to 2^-22 of its token's largest; the sum over R terms
adds (R + 2) u, the scale and the sum with y one u each.  So
  |out - ref| <= ((K / 16 + R + 32) u + 2^-22 R) * s sum_r |B| T_r + 2 u |y|,
T_r = sum_k |A||x| -- and for the second term the largest T_r of the token --
before the epilogue; max(v, 0)^2 turns e into e (2 |v| + e), and its own
rounding into u of the value; fp16 adds 2^-11 of the value (2^-25 for
subnormals).
"""
import numpy as np
import pytest
import torch

import oracle
from weight_only_quantized_g64_b200 import build as rq_build
from weight_only_quantized_g64_b200 import rq, synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rq_build.build()
    rq.lib()
    yield
    assert rq.read_device_status(reset=True) == rq.OK


def adapters(M, K, N, R, L, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g).half().cuda()
    A = (torch.randn((L, R, K), generator=g) * K ** -0.5).half().cuda()
    B = (torch.randn((L, N, R), generator=g) * 0.1).half().cuda()
    y = torch.randn((M, N), generator=g).to(dtype).cuda()
    ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda()
    scale = (0.5 + torch.rand(L, generator=g)).cuda()
    return x, A, B, ids, y, scale


def check(out, x, A, B, ids, y, scale=None, ranks=None, relu_sq=False, what=""):
    xd, yd = x.double().cpu().numpy(), y.double().cpu().numpy()
    M, K = xd.shape
    R = A.shape[1]
    v, lim = yd.copy(), 2 * U * np.abs(yd)
    for m, a in enumerate(ids.tolist()):
        if a < 0 or a >= A.shape[0]:
            continue
        n = R if ranks is None else min(max(int(ranks[a]), 0), R)
        if n == 0:
            continue
        s = 1.0 if scale is None else float(scale[a])
        Ad, Bd = A[a, :n].double().cpu().numpy(), B[a, :, :n].double().cpu().numpy()
        v[m] += s * (Bd @ (Ad @ xd[m]))
        T = np.abs(Ad) @ np.abs(xd[m])
        lim[m] += abs(s) * ((K / 16 + R + 32) * U * (np.abs(Bd) @ T) + 2.0 ** -22 * T.max() * np.abs(Bd).sum(1))
    if relu_sq:
        lim = lim * (2 * np.abs(v) + lim)
        v = np.maximum(v, 0) ** 2
        lim += 2 * U * v
    if out.dtype == torch.float16:
        lim = lim + (np.abs(v) + lim) * 2.0 ** -11 + 2.0 ** -25
    d = np.abs(out.double().cpu().numpy() - v)
    assert np.all(d <= lim), f"{what}: worst {d.max():.3e} (limit {lim.flat[d.argmax()]:.3e})"


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("R", [8, 16, 24, 40, 64, 128])
@pytest.mark.parametrize("M,K,N", [(1, 64, 1), (1, 2048, 768), (5, 72, 129), (32, 768, 2051), (33, 256, 127),
                                   (64, 520, 300), (131, 1024, 257), (200, 8, 64)])
def test_sizes(M, K, N, R, dtype):
    """From one token and one output to several tiles; odd sizes; every token any adapter or none."""
    x, A, B, ids, y, scale = adapters(M, K, N, R, 5, dtype, seed=M + K + N + R)
    out = rq.lora_add(x, A, B, ids, y, scale=scale)
    check(out, x, A, B, ids, y, scale, what="out")
    out = rq.lora_add(x, A, B, ids, y, epilogue=rq.EPI_RELU_SQ)
    check(out, x, A, B, ids, y, relu_sq=True, what="squared ReLU")
    mine = y.clone()
    assert rq.lora_add(x, A, B, ids, mine, out=mine, scale=scale) is mine
    assert torch.equal(mine, rq.lora_add(x, A, B, ids, y, scale=scale))


@pytest.mark.parametrize("M", [90, 1300, 2500])
def test_many_adapters_in_a_tile(M):
    """16 tokens of up to 16 adapters, whichever number of CTAs they are dealt over; the number changes no bit."""
    x, A, B, ids, y, scale = adapters(M, 64, 24, 8, 20, torch.float32, seed=M)
    out = rq.lora_add(x, A, B, ids, y, scale=scale)
    check(out, x, A, B, ids, y, scale, what="out")
    few = rq.lora_add(x[:80], A, B, ids[:80], y[:80], scale=scale)
    assert torch.equal(few, out[:80])


@pytest.mark.parametrize("M", [1, 7, 32, 33, 150])
def test_ranks_and_what_lies_behind_them(M):
    """Ranks of 0, odd, full, out of range; NaN behind a rank and in adapters that no token uses."""
    x, A, B, ids, y, scale = adapters(M, 256, 200, 16, 6, torch.float32, seed=M)
    ranks = torch.tensor([0, 1, 7, 13, 99, -3], dtype=torch.int32, device="cuda")
    ids = (torch.arange(M) % 6).to(torch.int32).cuda()
    for a, n in enumerate(ranks.tolist()):
        n = min(max(n, 0), 16)
        A[a, n:] = float("nan")
        B[a, :, n:] = float("inf")
    out = rq.lora_add(x, A, B, ids, y, scale=scale, ranks=ranks)
    check(out, x, A, B, ids, y, scale, ranks, what="ranks")


@pytest.mark.parametrize("M", [4, 70])
def test_other_adapters_values_do_not_leak(M):
    """An adapter with infinities and NaN spoils its own tokens only; ids out of range set the status."""
    x, A, B, ids, y, _ = adapters(M, 128, 96, 8, 4, torch.float32, seed=M)
    ids = (torch.arange(M) % 4).to(torch.int32).cuda()
    clean = rq.lora_add(x, A, B, ids, y)
    A[2] = float("nan")
    B[2] = float("inf")
    out = rq.lora_add(x, A, B, ids, y)
    ok = (ids != 2).cpu()
    assert torch.equal(out.cpu()[ok], clean.cpu()[ok]) and torch.isnan(out.cpu()[~ok]).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids[1] = 4
    out = rq.lora_add(x, A, B, ids, y, dev_status=status)
    assert status.item() == rq.ERR_RANGE and torch.equal(out[1], y[1])
    ids[:] = -1
    assert torch.equal(rq.lora_add(x, A, B, ids, y), y)


@pytest.mark.parametrize("M", [3, 80])
@pytest.mark.parametrize("size", [1e-6, 1.0, 1e4])
def test_large_and_small_sums(M, size):
    """Sums t far above fp16's range and far below its normal numbers."""
    x, A, B, ids, y, _ = adapters(M, 512, 64, 16, 3, torch.float32, seed=M)
    A = (A * 16).half()
    x = (x * size).half()
    check(rq.lora_add(x, A, B, ids, y), x, A, B, ids, y, what=f"x of {size}")


def test_many_adapters_in_a_tile_and_one_for_all():
    x, A, B, _, y, scale = adapters(128, 256, 130, 8, 128, torch.float32, seed=1)
    for ids in (torch.randperm(128, generator=torch.Generator().manual_seed(2)), torch.full((128,), 77)):
        ids = ids.to(torch.int32).cuda()
        check(rq.lora_add(x, A, B, ids, y, scale=scale), x, A, B, ids, y, scale)


def test_tokens_and_tiles_agree():
    """The two forms (up to 32 tokens one by one, more in tiles) on the same tokens."""
    x, A, B, ids, y, scale = adapters(64, 2048, 512, 32, 5, torch.float32, seed=3)
    many = rq.lora_add(x, A, B, ids, y, scale=scale)
    few = torch.cat([rq.lora_add(x[i:i + 32], A, B, ids[i:i + 32], y[i:i + 32], scale=scale) for i in (0, 32)])
    check(few, x, A, B, ids, y, scale)
    check(many, x, A, B, ids, y, scale)


@pytest.mark.parametrize("M", [16, 100])
def test_same_bits_stream_and_capture(M):
    x, A, B, ids, y, scale = adapters(M, 1024, 768, 16, 8, torch.float16, seed=5)
    first = rq.lora_add(x, A, B, ids, y, scale=scale)
    for _ in range(10):
        assert torch.equal(first, rq.lora_add(x, A, B, ids, y, scale=scale))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = rq.lora_add(x, A, B, ids, y, scale=scale, stream=side)
    side.synchronize()
    assert torch.equal(first, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rq.lora_add(x, A, B, ids, y, scale=scale)
    x2, _, _, ids2, y2, _ = adapters(M, 1024, 768, 16, 8, torch.float16, seed=6)
    x.copy_(x2), ids.copy_(ids2), y.copy_(y2)
    graph.replay()
    assert torch.equal(out, rq.lora_add(x, A, B, ids, y, scale=scale))
    del graph


@pytest.mark.parametrize("M", [4, 48])
def test_beside_a_quantized_projection(M):
    """As it is used: the channel-mix key, its adapters and the squared ReLU."""
    N, K, bits = 512, 256, 4
    W = synth.weights(N, K, seed=7)
    codes, scales, st = oracle.quantize_g64(W.numpy(), bits)
    assert st == 0
    cd, sd = torch.from_numpy(codes).cuda(), torch.from_numpy(scales.view(np.int16)).cuda()
    x, A, B, ids, _, scale = adapters(M, K, N, 8, 3, torch.float32, seed=8)
    y = rq.gemv_wq(x, cd, sd, N, bits) if M <= rq.MAX_DECODE_M else rq.gemm_wq(x, cd, sd, N, bits)
    out = rq.lora_add(x, A, B, ids, y, scale=scale, epilogue=rq.EPI_RELU_SQ)
    check(out, x, A, B, ids, y, scale, relu_sq=True)
    ref, budget = oracle.matmul(x.cpu().numpy(), codes, scales, bits)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= 2e-3 * budget)


@pytest.mark.parametrize("M", [8, 64])
def test_between_products_with_programmatic_launch(M):
    """Products that may start while the call before them runs: the same bits as without."""
    K = 512
    codes, scales = rq.quantize_g64(synth.weights(K, K, seed=3, device="cuda") * 20, 4)
    x, A, B, ids, _, scale = adapters(M, K, K, 16, 4, torch.float32, seed=M)
    product = rq.gemv_wq if M <= 32 else rq.gemm_wq

    def chain():
        v = x
        for _ in range(3):
            y = product(v, codes, scales, K, 4)
            out = rq.lora_add(v, A, B, ids, y, scale=scale)
            _, v = rq.norm_residual(out, pre="rms")
        return out, v

    first = chain()
    rq.set_pdl(True)
    try:
        for _ in range(20):
            for p, q in zip(first, chain()):
                assert torch.equal(p, q)
    finally:
        rq.set_pdl(False)


@pytest.mark.parametrize("M", [20, 200])
def test_two_at_once(M):
    """Two calls on two streams, each with its own workspace, give what they give one after the other."""
    calls = [adapters(M, 2048, 2048, 32, 6, torch.float32, seed=70 + i) for i in range(2)]
    alone = [rq.lora_add(x, A, B, ids, y, scale=scale) for x, A, B, ids, y, scale in calls]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = [rq.lora_add(x, A, B, ids, y, scale=scale, stream=s) for (x, A, B, ids, y, scale), s in zip(calls, sides)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(alone, got))


def test_offsets_past_32_bits():
    """Tokens behind more than 2^31 elements of x."""
    M, K, last = 33008, 65536, 48
    x = torch.empty((M, K), dtype=torch.float16, device="cuda")
    x[M - last:] = torch.randn((last, K), device="cuda").half()
    _, A, B, ids, y, scale = adapters(last, K, 16, 8, 2, torch.float32, seed=2)
    none = torch.full((M - last,), -1, dtype=torch.int32, device="cuda")
    out = rq.lora_add(x, A, B, torch.cat([none, ids]), torch.cat([torch.zeros((M - last, 16), device="cuda"), y]), scale=scale)
    assert torch.equal(out[M - last:], rq.lora_add(x[M - last:], A, B, ids, y, scale=scale))
    assert torch.all(out[:M - last] == 0)
