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


def lora_args(**kw):
    a = dict(x=FAKE, M=40, K=64, A=FAKE, B=FAKE, L=2, R=16, ids=FAKE, ranks=None, scale=None, y=FAKE, out=FAKE, N=33,
             dtype=0, epi=0, work=FAKE, status=None, stream=None)
    a.update(kw)
    return list(a.values())


def test_lora_argument_errors(L):
    f = L.rq_lora_add
    for bad in (dict(dtype=2), dict(dtype=-1), dict(epi=2), dict(epi=-1)):
        assert f(*lora_args(**bad)) == rq.ERR_RANGE, bad
    for bad in (dict(M=0), dict(M=4194241), dict(K=0), dict(K=12), dict(N=0), dict(N=1 << 31), dict(L=0), dict(R=0),
                dict(R=12), dict(R=136)):
        assert f(*lora_args(**bad)) == rq.ERR_SHAPE, bad
    for n in ("x", "A", "B", "ids", "y", "out", "work"):
        assert f(*lora_args(**{n: None})) == rq.ERR_NULL, n
    for n in ("x", "A", "B", "y", "out", "work"):
        assert f(*lora_args(**{n: FAKE + 8})) == rq.ERR_ALIGN, n
    for n in ("ids", "ranks", "scale", "status"):
        assert f(*lora_args(**{n: FAKE + 2})) == rq.ERR_ALIGN, n
    assert L.rq_lora_work_bytes(32, 64) == 0
    assert L.rq_lora_work_bytes(33, 64) == 3 * (4 * 1024 + 64)
    assert L.rq_lora_work_bytes(33, 12) == 0


def test_lora_binding_refuses(L):
    x, A, B = torch.zeros(4, 64).half(), torch.zeros(2, 8, 64).half(), torch.zeros(2, 10, 8).half()
    ids, y = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 10)
    refused(rq.ERR_RANGE, rq.lora_add, x, A, B, ids, y.double())
    refused(rq.ERR_SHAPE, rq.lora_add, x.float(), A, B, ids, y)
    refused(rq.ERR_SHAPE, rq.lora_add, x, A[:, :, :32], B, ids, y)
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B.mT, ids, y)
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B[:1], ids, y)
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B, ids.long(), y)
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B, ids[:3], y)
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B, ids, y[:, :9])
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B, ids, y, out=y.half())
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B, ids, y, scale=torch.zeros(3))
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B, ids, y, ranks=torch.zeros(2))
    refused(rq.ERR_SHAPE, rq.lora_add, x, A, B, ids, y)          # on the host


def norm_args(**kw):
    a = dict(y=FAKE, ldy=128, M=3, D=128, dtype=0, post=1, group=64, pw=FAKE, pb=FAKE, ep=1e-5, add=FAKE, lda=128,
             gate=FAKE, ldg=128, act=1, h=FAKE, alpha=FAKE, pre=2, w=FAKE, b=FAKE, e=1e-5, ho=FAKE, x=FAKE, stream=None)
    a.update(kw)
    return list(a.values())


def test_norm_argument_errors(L):
    f = L.rq_norm_residual
    for bad in (dict(dtype=2), dict(post=3), dict(post=-1), dict(pre=3), dict(act=3), dict(act=-1), dict(ep=-1.0),
                dict(e=float("nan"))):
        assert f(*norm_args(**bad)) == rq.ERR_RANGE, bad
    for bad in (dict(M=0), dict(D=0), dict(D=100), dict(D=16448, ldy=1 << 20), dict(group=4), dict(group=48),
                dict(group=512), dict(group=256), dict(ldy=120), dict(ldy=132), dict(lda=64), dict(ldg=129)):
        assert f(*norm_args(**bad)) == rq.ERR_SHAPE, bad
    assert f(*norm_args(y=None)) == rq.ERR_NULL
    assert f(*norm_args(ho=None, x=None)) == rq.ERR_NULL
    for n in ("y", "pw", "pb", "add", "gate", "h", "alpha", "w", "b", "ho", "x"):
        assert f(*norm_args(**{n: FAKE + 8})) == rq.ERR_ALIGN, n


def test_norm_binding_refuses(L):
    y = torch.zeros(4, 128)
    refused(rq.ERR_RANGE, rq.norm_residual, y.double())
    refused(rq.ERR_RANGE, rq.norm_residual, y, post="batch")
    refused(rq.ERR_RANGE, rq.norm_residual, y, gate=y, gate_act="relu")
    refused(rq.ERR_SHAPE, rq.norm_residual, y[0])
    refused(rq.ERR_SHAPE, rq.norm_residual, torch.zeros(128, 4).T)
    refused(rq.ERR_SHAPE, rq.norm_residual, y, gate=y.half())
    refused(rq.ERR_SHAPE, rq.norm_residual, y, add=y[:3])
    refused(rq.ERR_SHAPE, rq.norm_residual, y, h=torch.zeros(4, 256)[:, :128])
    refused(rq.ERR_SHAPE, rq.norm_residual, y, alpha=torch.zeros(64))
    refused(rq.ERR_SHAPE, rq.norm_residual, y, pre="rms", pre_weight=torch.zeros(128).half())
    refused(rq.ERR_SHAPE, rq.norm_residual, y, x=torch.zeros(4, 128))
    refused(rq.ERR_SHAPE, rq.norm_residual, y)                   # on the host
