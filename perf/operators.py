"""Cases of the operators that stand between the projections: low-rank adapters
beside a product, the norm / gate / residual step, and the time-mix recurrence
(single token, sequences, sequences with gradients).

``run`` computes a case in its plain form, with elementary torch operations, or
(``own``) through the calls of this package.  Sizes are those of the RWKV-7
shapes of the package's workloads: widths 768 to 4096, channel-mix 4x, heads of
64, decode batches 1 to 32, prefill to 4096 tokens.
"""
import math

import torch

own = False

HEAD = 64
DECAY = math.exp(-0.5)
TYPES = {"fp16": torch.float16, "fp32": torch.float32}
CHUNK = 16          # tokens that the plain form of the recurrence takes at once


def listed():
    return [
        # one request with its adapter beside the O projection of the 1.5B shape
        dict(name="lora 1 token 2048", op="lora", M=1, K=2048, N=2048, R=16, L=8, runs=1, type="fp32", relu_sq=False),
        # a decode batch, every request its own adapter, beside the channel-mix key (squared ReLU, fp16 out)
        dict(name="lora 32 tokens key", op="lora", M=32, K=4096, N=16384, R=32, L=64, runs=32, type="fp16",
             relu_sq=True),
        # a chunk of prefill tokens of some requests, odd count, small ranks
        dict(name="lora 517 tokens 2560", op="lora", M=517, K=2560, N=2560, R=8, L=16, runs=9, type="fp32",
             relu_sq=False),
        # a full prefill batch with large ranks
        dict(name="lora 2048 tokens 4096", op="lora", M=2048, K=4096, N=4096, R=64, L=8, runs=6, type="fp32",
             relu_sq=False),
        # one decode token: residual, channel scale and the norm of the next block
        dict(name="norm 1 token 2560", op="norm", M=1, D=2560, post="none", group=0, add=False, gate="none",
             residual=True, alpha=True, pre="layer", type="fp32"),
        # after the recurrence: norm of each head, bonus, gate; the input of the O projection
        dict(name="norm heads 2049x2048", op="norm", M=2049, D=2048, post="layer", group=64, add=True,
             gate="identity", residual=False, alpha=False, pre="none", type="fp16"),
        # prefill with norms before and after the block and a silu gate
        dict(name="norm 4096x4096", op="norm", M=4096, D=4096, post="rms", group=0, add=False, gate="silu",
             residual=True, alpha=True, pre="rms", type="fp16"),
        # one token of 32 requests on the 4096-wide shape
        dict(name="step 32 requests 4096", op="step", B=32, H=64, type="fp16"),
        # one short sequence of the 768-wide shape
        dict(name="scan 129 tokens 768", op="scan", T=129, S=1, H=12, type="fp32"),
        # prefill of five requests of unlike lengths on the 4096-wide shape
        dict(name="scan 8192 tokens 4096", op="scan", T=8192, S=5, H=64, type="fp16"),
        # gradients over three short sequences, one of them empty
        dict(name="grad 333 tokens 768", op="grad", T=333, S=3, H=12, type="fp32"),
        # gradients over a calibration batch of the 2048-wide shape
        dict(name="grad 2048 tokens 2048", op="grad", T=2048, S=2, H=32, type="fp16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["lora", "norm", "step", "scan", "grad"])
    t = rng.choice(["fp16", "fp32"])
    if op == "lora":
        M = _log_int(rng, 1, 2048)
        big = M > 64
        return dict(op=op, M=M, K=_log_int(rng, 256, 4096, 64), N=_log_int(rng, 256, 4096 if big else 16384),
                    R=rng.choice([8, 16, 24, 32, 64]), L=rng.randint(1, 16 if big else 64),
                    runs=rng.randint(1, min(M, 32)), type=t, relu_sq=rng.random() < 0.3)
    if op == "norm":
        post = rng.choice(["none", "layer", "rms"])
        return dict(op=op, M=_log_int(rng, 1, 4096), D=_log_int(rng, 256, 4096, 64), post=post,
                    group=rng.choice([0, 64]) if post != "none" else 0, add=rng.random() < 0.5,
                    gate=rng.choice(["none", "identity", "sigmoid", "silu"]), residual=rng.random() < 0.7,
                    alpha=rng.random() < 0.5, pre=rng.choice(["none", "layer", "rms"]), type=t)
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 64), H=_log_int(rng, 1, 64), type=t)
    top = 8192 if op == "scan" else 2048
    T = _log_int(rng, 1, top)
    return dict(op=op, T=T, S=rng.randint(1, 8), H=_log_int(rng, 1, 64 if op == "scan" else 32), type=t)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _starts(T, S, seed):
    """Offsets of S sequences over T tokens, of unlike lengths; with three or more, the second is empty."""
    g = torch.Generator().manual_seed(seed)
    full = S - 1 if S >= 3 else S
    cuts = torch.sort(torch.randint(0, T + 1, (full - 1,), generator=g)).values.tolist()
    at = [0] + cuts + [T]
    if S >= 3:
        at = at[:2] + at[1:]
    return at


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    t = TYPES[case["type"]]
    if case["op"] == "lora":
        M, K, N, R, L = (case[k] for k in ("M", "K", "N", "R", "L"))
        s["x"] = _randn(g, M, K).half()
        s["A"] = (_randn(g, L, R, K) * K ** -0.5).half()
        s["B"] = (_randn(g, L, N, R) * 0.1).half()
        s["y"] = _randn(g, M, N).to(t)
        s["scale"] = 0.5 + torch.rand(L, generator=g, device="cuda")
        c = torch.Generator().manual_seed(seed)
        ends = torch.sort(torch.randperm(M - 1, generator=c)[: case["runs"] - 1] + 1).values if M > 1 else \
            torch.empty(0, dtype=torch.int64)
        of_run = torch.randint(-1, L, (ends.numel() + 1,), generator=c)     # -1: a request without an adapter
        if case["runs"] == M and M <= L:
            of_run = torch.randperm(L, generator=c)[:M]                      # each request its own adapter
        run_of = torch.searchsorted(ends, torch.arange(M), right=True)
        s["ids"] = of_run[run_of].to(torch.int32).cuda()
    elif case["op"] == "norm":
        M, D = case["M"], case["D"]
        s["y"] = (_randn(g, M, D) * 2 + 0.3).to(t)
        s["post_w"], s["post_b"] = 1 + 0.2 * _randn(g, D), 0.1 * _randn(g, D)
        s["add_t"] = _randn(g, M, D).to(t) if case["add"] else None
        s["gate_t"] = _randn(g, M, D).to(t) if case["gate"] != "none" else None
        s["h"] = (_randn(g, M, D) * 3).to(t) if case["residual"] else None
        s["alpha_t"] = 0.5 + 0.2 * _randn(g, D) if case["alpha"] else None
        s["pre_w"], s["pre_b"] = 1 + 0.2 * _randn(g, D), 0.1 * _randn(g, D)
    else:
        H = case["H"]
        T = case["B"] if case["op"] == "step" else case["T"]
        S = case["B"] if case["op"] == "step" else case["S"]
        unit = torch.nn.functional.normalize(_randn(g, T, H, HEAD), dim=-1)
        s["r"], s["k"] = (0.5 * _randn(g, T, H, HEAD)).to(t), (0.5 * _randn(g, T, H, HEAD)).to(t)
        s["v"], s["d"] = _randn(g, T, H, HEAD).to(t), (1.5 * _randn(g, T, H, HEAD) - 2).to(t)
        s["a"] = (-unit).to(t)
        s["b"] = (unit * torch.sigmoid(_randn(g, T, H, HEAD))).to(t)
        s["state"] = 0.3 * _randn(g, S, H, HEAD, HEAD)
        if case["op"] != "step":
            s["starts"] = _starts(T, S, seed)           # the host's own copy of the offsets
            s["seq_start"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
        if case["op"] == "grad":
            s["dy"] = _randn(g, T, H, HEAD).to(t)
            s["dstate"] = 0.1 * _randn(g, S, H, HEAD, HEAD)
    return s


# ---- plain forms ----------------------------------------------------------------------------------

def _lora(s):
    x, A, B, y = s["x"].float(), s["A"], s["B"], s["y"].float()
    M, (L, R, K) = x.shape[0], A.shape
    has = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    scale = torch.where(has, s["scale"][ids], torch.zeros_like(s["scale"][ids]))
    if M <= 64:                                          # each token's own adapter, gathered
        t = torch.bmm(A[ids].float(), x[:, :, None])[:, :, 0]
        delta = torch.bmm(B[ids].float(), t[:, :, None])[:, :, 0]
    else:                                                # all adapters at once, the others' parts zero
        t = (x @ A.float().view(L * R, K).T).view(M, L, R)
        t = t * (ids[:, None] == torch.arange(L, device=x.device))[:, :, None]
        delta = t.view(M, L * R) @ B.float().permute(0, 2, 1).reshape(L * R, -1)
    out = y + scale[:, None] * delta
    if s["relu_sq"]:
        out = out.clamp(min=0).square()
    return out.to(s["y"].dtype)


def _normed(u, kind, group, w, b):
    if kind == "none":
        return u
    D = u.shape[-1]
    v = u.view(*u.shape[:-1], -1, group or D)
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5)
    v = v.view_as(u) * w
    return v + b if kind == "layer" else v


def _norm(s):
    u = _normed(s["y"].float(), s["post"], s["group"], s["post_w"], s["post_b"])
    if s["add_t"] is not None:
        u = u + s["add_t"].float()
    if s["gate_t"] is not None:
        gate = s["gate_t"].float()
        act = {"identity": gate, "sigmoid": torch.sigmoid(gate), "silu": gate * torch.sigmoid(gate)}[s["gate"]]
        u = u * act
    if s["alpha_t"] is not None:
        u = u * s["alpha_t"]
    if s["h"] is not None:
        u = u + s["h"].float()
    x = _normed(u, s["pre"], 0, s["pre_w"], s["pre_b"]).half()
    return (u.to(s["h"].dtype), x) if s["h"] is not None else (x,)


def _decay_log(d):
    return -DECAY * torch.sigmoid(d)


def _step(s):
    r, k, v, a, b = (s[n].float() for n in "rkvab")
    w = torch.exp(_decay_log(s["d"].float()))
    S = s["state"]
    sa = (S * a[:, :, None, :]).sum(-1)
    S = S * w[:, :, None, :] + sa[..., None] * b[:, :, None, :] + v[..., None] * k[:, :, None, :]
    return (S * r[:, :, None, :]).sum(-1).to(s["r"].dtype), S


def _in_chunks(x, at):
    """[T, H, 64] -> [S, H, chunks, CHUNK, 64]: sequences padded with zeros to whole chunks."""
    S, n = at.shape
    x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[at]
    return x.view(S, n // CHUNK, CHUNK, *x.shape[2:]).permute(0, 3, 1, 2, 4)


def _chunked(r, d, k, v, a, b, state, starts):
    """The recurrence by chunks of CHUNK tokens: inside a chunk as products of matrices, from chunk to chunk in turn."""
    T, H, _ = r.shape
    st = torch.tensor(starts, device=r.device)
    lens = st[1:] - st[:-1]
    n = max(1, -(-max(j - i for i, j in zip(starts, starts[1:])) // CHUNK)) * CHUNK
    pos = torch.arange(n, device=r.device)
    inside = pos[None] < lens[:, None]
    at = torch.where(inside, st[:-1, None] + pos[None], torch.full_like(pos, T)[None])
    r, lw, k, v, a, b = (_in_chunks(x, at) for x in (r, _decay_log(d), k, v, a, b))
    cum = lw.double().cumsum(-2)                         # far positions: 64 bits for the exponents
    grow, shrink, last = torch.exp(cum).float(), torch.exp(-cum).float(), torch.exp(cum[..., -1:, :]).float()
    R, Kt, At, Bt = r * grow, k * shrink, a * torch.exp(cum - lw.double()).float(), b * shrink
    low = torch.ones(CHUNK, CHUNK, device=r.device).tril()
    strict = low.tril(-1)
    Aab, Aak = (At @ Bt.mT) * strict, (At @ Kt.mT) * strict
    Arb, Ark = (R @ Bt.mT) * low, (R @ Kt.mT) * low
    eye = torch.eye(CHUNK, device=r.device).expand_as(Aab)
    rows = [eye[..., 0, :]]
    for i in range(1, CHUNK):                            # rows of (1 - Aab)^-1
        rows.append(eye[..., i, :] + (Aab[..., i, :i, None] * torch.stack(rows, -2)).sum(-2))
    inv = torch.stack(rows, -2)
    of_state, of_v = inv @ At, inv @ (Aak @ v)
    y_v = Ark @ v
    kv = v.mT @ Kt
    S, ys = state, []
    for c in range(n // CHUNK):
        U = of_state[:, :, c] @ S.mT + of_v[:, :, c]
        ys.append(R[:, :, c] @ S.mT + Arb[:, :, c] @ U + y_v[:, :, c])
        S = (S + U.mT @ Bt[:, :, c] + kv[:, :, c]) * last[:, :, c]
    y = torch.stack(ys, 2).permute(0, 2, 3, 1, 4).reshape(len(starts) - 1, n, H, HEAD)
    return y[inside], S                                  # sequences follow one another, so the order is the tokens'


def _scan(s):
    y, S = _chunked(*(s[n].float() for n in "rdkvab"), s["state"], s["starts"])
    return y.to(s["r"].dtype), S


def _grad(s):
    leaves = [s[n].float().requires_grad_() for n in "rdkvab"] + [s["state"].clone().requires_grad_()]
    with torch.enable_grad():
        y, S = _chunked(*leaves, s["starts"])
        grads = torch.autograd.grad([y, S], leaves, [s["dy"].float(), s["dstate"]])
    t = s["r"].dtype
    return y.detach().to(t), S.detach(), [x.to(t) for x in grads[:6]], grads[6]


def _run_own(s):
    from weight_only_quantized_g64_b200 import rq
    if s["op"] == "lora":
        return rq.lora_add(s["x"], s["A"], s["B"], s["ids"], s["y"], scale=s["scale"],
                           epilogue=rq.EPI_RELU_SQ if s["relu_sq"] else rq.EPI_NONE)
    if s["op"] == "norm":
        h, x = rq.norm_residual(s["y"], post=s["post"], post_group=s["group"], post_weight=s["post_w"],
                                post_bias=s["post_b"] if s["post"] == "layer" else None, add=s["add_t"],
                                gate=s["gate_t"], gate_act=s["gate"] if s["gate"] != "none" else "identity",
                                h=s["h"], alpha=s["alpha_t"], pre=s["pre"], pre_weight=s["pre_w"],
                                pre_bias=s["pre_b"] if s["pre"] == "layer" else None)
        return (h, x) if h is not None else (x,)
    ins = [s[n] for n in "rdkvab"]
    if s["op"] == "step":
        return rq.tmix_step(*ins, s["state"])
    if s["op"] == "scan":
        return rq.tmix_scan(*ins, s["seq_start"], state=s["state"])
    ckpt = rq.tmix_ckpt(s["r"], s["S"])
    y, state = rq.tmix_scan(*ins, s["seq_start"], state=s["state"], ckpt=ckpt)
    grads, dstate = rq.tmix_scan_bwd(*ins, s["seq_start"], ckpt, s["dy"], dstate_out=s["dstate"])
    return y, state, list(grads), dstate


def run(state):
    if own:
        return _run_own(state)
    return {"lora": _lora, "norm": _norm, "step": _step, "scan": _scan, "grad": _grad}[state["op"]](state)


def work(case):
    e = 2 if case["type"] == "fp16" else 4
    if case["op"] == "lora":
        M, K, N, R, L = (case[k] for k in ("M", "K", "N", "R", "L"))
        used = min(L, case["runs"])
        return {"bytes": 2 * M * K + 2 * used * R * (K + N) + 2 * e * M * N + 4 * (M + L), "flops": 2 * M * R * (K + N)}
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        wide = 1 + case["add"] + (case["gate"] != "none") + 2 * case["residual"]
        vecs = case["alpha"] + sum({"none": 0, "layer": 2, "rms": 1}[case[k]] for k in ("post", "pre"))
        return {"bytes": M * D * (e * wide + 2) + 4 * D * vecs, "flops": 20 * M * D}
    H = case["H"]
    if case["op"] == "step":
        return {"bytes": case["B"] * H * (7 * HEAD * e + 8 * HEAD * HEAD), "flops": 10 * case["B"] * H * HEAD * HEAD}
    T, S = case["T"], case["S"]
    if case["op"] == "scan":
        return {"bytes": T * H * 7 * HEAD * e + S * H * 8 * HEAD * HEAD, "flops": 10 * T * H * HEAD * HEAD}
    return {"bytes": T * H * 14 * HEAD * e + S * H * 16 * HEAD * HEAD, "flops": 34 * T * H * HEAD * HEAD}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        out = s["y"].double()
        for a in range(case["L"]):
            m = torch.nonzero(s["ids"] == a)[:, 0]
            out[m] += s["scale"][a].double() * ((s["x"][m].double() @ s["A"][a].double().T) @ s["B"][a].double().T)
        return torch.relu(out) ** 2 if case["relu_sq"] else out
    if case["op"] == "norm":
        def norm(u, kind, group, w, b):
            if kind == "none":
                return u
            p = u.reshape(-1, group or u.shape[1])
            if kind == "rms":
                q = p / (p.pow(2).sum(1, keepdim=True) / p.shape[1] + 1e-5).sqrt()
                return q.reshape(u.shape) * w.double()
            q = (p - p.mean(1, keepdim=True)) / (p.var(1, keepdim=True, unbiased=False) + 1e-5).sqrt()
            return q.reshape(u.shape) * w.double() + b.double()
        u = norm(s["y"].double(), case["post"], case["group"], s["post_w"], s["post_b"])
        u = u + s["add_t"].double() if case["add"] else u
        if case["gate"] != "none":
            q = s["gate_t"].double()
            u = u * (q if case["gate"] == "identity" else (q if case["gate"] == "silu" else 1) / (1 + torch.exp(-q)))
        u = u * s["alpha_t"].double() if case["alpha"] else u
        u = u + s["h"].double() if case["residual"] else u
        x = norm(u, case["pre"], 0, s["pre_w"], s["pre_b"])
        return (u, x) if case["residual"] else (x,)

    r, d, k, v, a, b = (s[n].double() for n in "rdkvab")
    gate = 1 / (1 + torch.exp(-d))
    w = torch.exp(-DECAY * gate)
    col, row = (lambda x: x[..., :, None]), (lambda x: x[..., None, :])
    if case["op"] == "step":
        S = s["state"].double()
        S = S * row(w) + torch.matmul(S, col(a)) * row(b) + col(v) * row(k)
        return torch.matmul(S, col(r))[..., 0], S
    y, ends = torch.zeros_like(r), s["state"].double()
    grads = [torch.zeros_like(r) for _ in range(6)]
    dstate = s["dstate"].double() if case["op"] == "grad" else None
    for q in range(case["S"]):
        lo, hi = s["starts"][q], s["starts"][q + 1]
        S, past = ends[q].clone(), []
        for t in range(lo, hi):
            if case["op"] == "grad":
                past.append(S)
            S = S * row(w[t]) + torch.matmul(S, col(a[t])) * row(b[t]) + col(v[t]) * row(k[t])
            y[t] = torch.matmul(S, col(r[t]))[..., 0]
        ends[q] = S
        if case["op"] != "grad":
            continue
        G = dstate[q]
        for t in range(hi - 1, lo - 1, -1):
            P, dy = past.pop(), s["dy"][t].double()
            G = G + col(dy) * row(r[t])
            sa, gb = torch.matmul(P, col(a[t])), torch.matmul(G, col(b[t]))
            grads[0][t] = torch.matmul(row(dy), S)[..., 0, :]
            grads[1][t] = (G * P).sum(-2) * w[t] * -DECAY * gate[t] * (1 - gate[t])
            grads[2][t] = torch.matmul(row(v[t]), G)[..., 0, :]
            grads[3][t] = torch.matmul(G, col(k[t]))[..., 0]
            grads[4][t] = torch.matmul(gb.mT, P)[..., 0, :]
            grads[5][t] = torch.matmul(sa.mT, G)[..., 0, :]
            G = G * row(w[t]) + gb * row(a[t])
            S = P
        dstate[q] = G
    if case["op"] == "scan":
        return y, ends
    return y, ends, grads, dstate
