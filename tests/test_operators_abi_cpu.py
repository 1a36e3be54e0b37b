"""Argument errors of the calls between the projections: found before any CUDA
call, so these tests launch nothing and need no GPU."""
import pytest
import torch

from weight_only_quantized_g64_b200 import build as rq_build
from weight_only_quantized_g64_b200 import rq

FAKE = 1 << 20          # aligned, non-null; never dereferenced because validation fails first


@pytest.fixture(scope="module")
def L():
    rq_build.build()
    return rq.lib()


def test_tmix_ckpt_bytes(L):
    assert L.rq_tmix_ckpt_bytes(0, 1, 1) == 16384
    assert L.rq_tmix_ckpt_bytes(333, 3, 12) == (333 // 16 + 3) * 12 * 16384
    assert L.rq_tmix_ckpt_bytes(-1, 1, 1) == 0
    assert L.rq_tmix_ckpt_bytes(16, 0, 1) == 0
    assert L.rq_tmix_ckpt_bytes(16, 1, 0) == 0


def scan_args(**kw):
    a = dict(r=FAKE, d=FAKE, k=FAKE, v=FAKE, a=FAKE, b=FAKE, T=10, H=2, ld=128, dtype=0, seq=FAKE, S=1, si=FAKE,
             so=FAKE, slots=None, ns=1, y=FAKE, ckpt=None, status=None, stream=None)
    a.update(kw)
    return list(a.values())


def bwd_args(**kw):
    a = dict(r=FAKE, d=FAKE, k=FAKE, v=FAKE, a=FAKE, b=FAKE, T=10, H=2, ld=128, dtype=0, seq=FAKE, S=1, ckpt=FAKE,
             dy=FAKE, dso=None, dsi=None, dr=FAKE, dd=FAKE, dk=FAKE, dv=FAKE, da=FAKE, db=FAKE, work=FAKE,
             status=None, stream=None)
    a.update(kw)
    return list(a.values())


def step_args(**kw):
    a = dict(r=FAKE, d=FAKE, k=FAKE, v=FAKE, a=FAKE, b=FAKE, T=10, H=2, ld=128, dtype=0, si=FAKE, so=FAKE,
             slots=None, ns=1, y=FAKE, status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("call,args", [("rq_tmix_scan", scan_args), ("rq_tmix_scan_bwd", bwd_args),
                                       ("rq_tmix_step", step_args)])
def test_tmix_argument_errors(L, call, args):
    f = getattr(L, call)
    for bad in (dict(dtype=2), dict(dtype=-1)):
        assert f(*args(**bad)) == rq.ERR_RANGE, bad
    for bad in (dict(T=-1), dict(T=1 << 30), dict(H=0), dict(ld=120), dict(ld=132), dict(H=1 << 40),
                dict(T=(1 << 30) - 1, H=64, ld=4096)):
        assert f(*args(**bad)) == rq.ERR_SHAPE, bad
    tokens = ["r", "d", "k", "v", "a", "b"] + (["dy", "dr", "dd", "dk", "dv", "da", "db"] if "bwd" in call else ["y"])
    for n in tokens:
        assert f(*args(**{n: None})) == rq.ERR_NULL, n
        assert f(*args(**{n: FAKE + 8})) == rq.ERR_ALIGN, n
    if "step" in call:
        assert f(*args(T=0)) == rq.ERR_SHAPE
        assert f(*args(si=FAKE + 4)) == rq.ERR_ALIGN
    else:
        assert f(*args(seq=None)) == rq.ERR_NULL
        assert f(*args(seq=FAKE + 2)) == rq.ERR_ALIGN
        assert f(*args(S=0)) == rq.ERR_SHAPE
    if "bwd" in call:
        for n in ("ckpt", "work"):
            assert f(*args(**{n: None})) == rq.ERR_NULL
            assert f(*args(**{n: FAKE + 8})) == rq.ERR_ALIGN
    else:
        assert f(*args(slots=FAKE, ns=0)) == rq.ERR_SHAPE
        assert f(*args(slots=FAKE + 1)) == rq.ERR_ALIGN
    assert f(*args(status=FAKE + 2)) == rq.ERR_ALIGN


def heads(T=4, H=2, dtype=torch.float32):
    return [torch.zeros(T, H, 64, dtype=dtype) for _ in range(6)]


def refused(status, fn, *a, **kw):
    with pytest.raises(rq.RQError) as e:
        fn(*a, **kw)
    assert e.value.status == status, e.value


def test_tmix_binding_refuses(L):
    """Types, shapes and strides that the C call cannot see."""
    seq = torch.tensor([0, 4], dtype=torch.int32)
    refused(rq.ERR_RANGE, rq.tmix_scan, *heads(dtype=torch.float64), seq)
    refused(rq.ERR_RANGE, rq.tmix_step, *heads(dtype=torch.bfloat16))
    xs = heads()
    refused(rq.ERR_SHAPE, rq.tmix_scan, *(x[:, :, :32] for x in xs), seq)
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs[:5], xs[5].half(), seq)
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs[:5], xs[5].transpose(0, 1).contiguous().transpose(0, 1), seq)
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq.long())
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq[:1])
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq, state=torch.zeros(2, 2, 64, 64))
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq, state=torch.zeros(1, 2, 64, 64).mT)
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq, slots=torch.zeros(1, dtype=torch.int32))
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq, y=torch.zeros(3, 2, 64))
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq, ckpt=torch.zeros(5))
    refused(rq.ERR_SHAPE, rq.tmix_scan_bwd, *xs, seq, rq.tmix_ckpt(xs[0], 1), torch.zeros(4, 2, 64).half())
    refused(rq.ERR_SHAPE, rq.tmix_scan_bwd, *xs, seq, rq.tmix_ckpt(xs[0], 2), torch.zeros(4, 2, 64))
    refused(rq.ERR_SHAPE, rq.tmix_step, *xs, state=torch.zeros(4, 2, 64, 64, dtype=torch.float64))
    # good arguments, but on the host
    refused(rq.ERR_SHAPE, rq.tmix_scan, *xs, seq)
    refused(rq.ERR_SHAPE, rq.tmix_step, *xs, state=torch.zeros(4, 2, 64, 64))
