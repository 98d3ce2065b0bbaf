"""Cases of the recurrent-block operators: what is measured, the operators'
plain forms, and the same results in 64 bits.

The operators: the gated linear recurrence (``scan``), the causal depthwise
convolution (``conv``), the residual + root-mean-square norm with an 8-bit
output (``norm``) and the 8-bit matrix product (``matmul``).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
DECAY = 8.0
EPS = 1e-6


def listed():
    return [
        # one generated token for each of 16 sequences: latency
        {"name": "scan_step", "op": "scan", "dir": "fwd", "dtype": "bf16", "B": 16, "T": 1, "D": 2048, "ragged": False},
        # one long prompt: few channels for the whole GPU, a long axis to scan
        {"name": "scan_prompt", "op": "scan", "dir": "fwd", "dtype": "bf16", "B": 1, "T": 32768, "D": 2048, "ragged": False},
        # a training step's forward and backward pass
        {"name": "scan_train", "op": "scan", "dir": "train", "dtype": "bf16", "B": 8, "T": 2048, "D": 2048, "ragged": False},
        # a small 32-bit training batch of padded sequences, odd sizes, one sequence empty
        {"name": "scan_train_ragged", "op": "scan", "dir": "train", "dtype": "f32", "B": 3, "T": 1537, "D": 700, "ragged": True},
        # one generated token for each of 64 sequences
        {"name": "conv_step", "op": "conv", "dir": "fwd", "dtype": "f16", "B": 64, "T": 1, "D": 2048, "K": 4, "ragged": False},
        # two long prompts
        {"name": "conv_prompt", "op": "conv", "dir": "fwd", "dtype": "bf16", "B": 2, "T": 16384, "D": 2048, "K": 4, "ragged": False},
        # a training step on padded sequences, odd length, one sequence empty
        {"name": "conv_train_ragged", "op": "conv", "dir": "train", "dtype": "bf16", "B": 8, "T": 1999, "D": 2048, "K": 4, "ragged": True},
        # one generated token for each of 16 sequences
        {"name": "norm_step", "op": "norm", "dtype": "bf16", "M": 16, "D": 2048},
        # a long prompt's tokens
        {"name": "norm_prompt", "op": "norm", "dtype": "f16", "M": 16384, "D": 4096},
        # one generated token for each of 4 sequences: the weights' bytes count
        {"name": "matmul_step", "op": "matmul", "dtype": "bf16", "M": 4, "N": 8192, "K": 2048},
        # a ragged batch of a few hundred tokens, a width that no tile divides
        {"name": "matmul_batch", "op": "matmul", "dtype": "f16", "M": 197, "N": 5000, "K": 2048},
        # a long prompt's tokens: the tensor cores count
        {"name": "matmul_prompt", "op": "matmul", "dtype": "bf16", "M": 8192, "N": 8192, "K": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A channel count: mostly a multiple of 64, sometimes odd."""
    d = _log(rng, lo, hi)
    return d if rng.random() < 0.3 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["scan", "scan", "conv", "conv", "norm", "matmul", "matmul"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("scan", "conv"):
        d = _width(rng, 256, 4096)
        b = _log(rng, 1, 32)
        t = 1 if rng.random() < 0.25 else _log(rng, 2, 32768)
        t = max(1, min(t, (1 << 26) // (b * d * (2 if dtype == "f32" else 1))))
        train = t > 1 and b * t * d <= 1 << 25 and rng.random() < 0.5
        c = {"op": op, "dir": "train" if train else "fwd", "dtype": dtype, "B": b, "T": t, "D": d,
             "ragged": t > 1 and rng.random() < 0.4}
        if op == "conv":
            c["K"] = rng.choice([2, 3, 4, 4])
        return c
    if op == "norm":
        d = _width(rng, 256, 8192)
        return {"op": op, "dtype": dtype, "M": _log(rng, 1, (1 << 26) // d if dtype != "f32" else (1 << 25) // d), "D": d}
    n, k = _width(rng, 256, 8192), _width(rng, 256, 4096)
    return {"op": op, "dtype": dtype, "M": _log(rng, 1, min(8192, (1 << 36) // (n * k))), "N": n, "K": k}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _inputs(case, seed):
    """The case's tensors on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda") * std + mean

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {}
    op = case["op"]
    if op in ("scan", "conv"):
        B, T, D = case["B"], case["T"], case["D"]
        s["x"] = normal(B, T, D).to(dt)
        s["lens"] = None
        if case["ragged"]:
            lens = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            lens[0] = T
            if B > 2:
                lens[1] = 0
            s["lens"] = lens
    if op == "scan":
        s["r"] = normal(B, T, D).to(dt)
        s["i"] = normal(B, T, D).to(dt)
        # a channel's slowest decay, e^(-DECAY softplus(lam)), lies in 0.9 ... 0.999
        s["lam"] = torch.log(torch.expm1(-torch.log(uniform(0.9, 0.999, D)) / DECAY))
        s["h0"] = normal(B, D, std=0.5)
        if case["dir"] == "train":
            s["dy"] = normal(B, T, D).to(dt)
            s["dhT"] = normal(B, D)
    elif op == "conv":
        K = case["K"]
        s["w"] = normal(D, K, std=K ** -0.5).to(dt)
        s["bias"] = uniform(-0.1, 0.1, D).to(dt)
        s["state"] = normal(B, K - 1, D).to(dt)
        if case["dir"] == "train":
            s["dy"] = normal(B, T, D, std=0.1).to(dt)
            s["dstate_out"] = normal(B, K - 1, D, std=0.1).to(dt)
    elif op == "norm":
        M, D = case["M"], case["D"]
        s["x"] = normal(M, D).to(dt)
        s["res"] = normal(M, D, std=2.0).to(dt)
        s["w"] = uniform(0.5, 1.5, D).to(dt)
        s["values"] = torch.empty(M, D, dtype=torch.bfloat16 if dt == torch.float32 else dt, device="cuda")
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["xq"] = torch.clamp(torch.round(normal(M, K, std=40.0)), -127, 127).to(torch.int8)
        s["wq"] = torch.clamp(torch.round(normal(N, K, std=40.0)), -127, 127).to(torch.int8)
        s["sx"] = uniform(0.01, 0.03, M)
        s["sw"] = uniform(0.5, 1.5, N) * (0.02 / K ** 0.5)
        s["bias"] = uniform(-0.1, 0.1, N).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _plan(s, case)
    return s


def _plan(s, case):
    """Problem records, outputs and workspaces, as a user's program keeps them."""
    import depthwise_convolution_forward_gb300 as gc

    op, code = case["op"], gc.DTYPE_CODES[case["dtype"]]
    s["gc"], s["code"] = gc, code

    def like(t, dtype=None):
        return torch.empty_like(t, dtype=dtype or t.dtype)

    def scratch(n):
        return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")

    if op == "scan":
        p = s["p"] = gc.make_scan_problem(case["B"], case["T"], case["D"], DECAY)
        s["y"], s["hT"] = like(s["x"]), like(s["h0"])
        if case["dir"] == "train":
            s["saved"] = scratch(gc.gconv_gated_scan_saved_size(p, code))
            s["ws"] = scratch(gc.gconv_gated_scan_bwd_workspace_size(p, code))
            s["dx"], s["dr"], s["di"] = like(s["x"]), like(s["r"]), like(s["i"])
            s["dlam"], s["dh0"] = like(s["lam"]), like(s["h0"])
    elif op == "conv":
        p = s["p"] = gc.make_conv1d_problem(case["B"], case["T"], case["D"], case["K"], gc.ACT_SILU)
        s["y"], s["state_out"] = like(s["x"]), like(s["state"])
        if case["dir"] == "train":
            s["ws"] = scratch(gc.gconv_causal_conv1d_bwd_workspace_size(p, code))
            s["dx"], s["dw"], s["dbias"], s["dstate"] = like(s["x"]), like(s["w"]), like(s["bias"]), like(s["state"])
    elif op == "norm":
        s["p"] = gc.make_norm_problem(case["M"], case["D"], EPS)
        s["res_out"], s["q"] = like(s["res"]), like(s["x"], torch.int8)
        s["scale"] = torch.empty(case["M"], device="cuda")
    else:
        s["p"] = gc.make_matmul_q8_problem(case["M"], case["N"], case["K"])
        s["y"] = torch.empty(case["M"], case["N"], dtype=DTYPES[case["dtype"]], device="cuda")


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return _OWN[case["op"]](s, case)
    return _PLAIN[case["op"]](s, case)


def _own_scan(s, case):
    gc, train = s["gc"], case["dir"] == "train"
    st = torch.cuda.current_stream()
    gc.gconv_gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["h0"], s["lens"], s["y"], s["hT"],
                            s["saved"] if train else None, s["p"], s["code"], st)
    if not train:
        return {"y": s["y"], "hT": s["hT"]}
    gc.gconv_gated_scan_bwd(s["dy"], s["dhT"], s["x"], s["r"], s["i"], s["lam"], s["lens"], s["saved"], s["dx"], s["dr"],
                            s["di"], s["dlam"], s["dh0"], s["p"], s["code"], s["ws"], 0, st)
    return {k: s[k] for k in ("y", "hT", "dx", "dr", "di", "dlam", "dh0")}


def _own_conv(s, case):
    gc = s["gc"]
    st = torch.cuda.current_stream()
    gc.gconv_causal_conv1d_fwd(s["x"], s["w"], s["bias"], s["state"], s["lens"], s["y"], s["state_out"], s["p"], s["code"],
                               st)
    if case["dir"] != "train":
        return {"y": s["y"], "state": s["state_out"]}
    gc.gconv_causal_conv1d_bwd(s["dy"], s["dstate_out"], s["x"], s["w"], s["bias"], s["state"], s["lens"], s["dx"], s["dw"],
                               s["dbias"], s["dstate"], s["p"], s["code"], s["ws"], 0, st)
    return {"y": s["y"], "state": s["state_out"], "dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"], "dstate": s["dstate"]}


def _own_norm(s, case):
    gc = s["gc"]
    gc.gconv_rms_norm_q8(s["x"], s["res"], s["w"], s["res_out"], None, s["q"], s["scale"], s["p"], s["code"],
                         torch.cuda.current_stream())
    return {"residual": s["res_out"], "scale": s["scale"], "q": _values(s, s["q"], s["scale"])}


def _own_matmul(s, case):
    gc = s["gc"]
    gc.gconv_matmul_q8(s["xq"], s["sx"], s["wq"], s["sw"], s["bias"], s["y"], s["p"], s["code"], torch.cuda.current_stream())
    return s["y"]


def _values(s, q, scale):
    """The values that 8-bit numbers and their rows' scales stand for, in a
    16-bit type; part of both sides' pass."""
    return torch.mul(q, scale[:, None], out=s["values"])


def _valid(s, case):
    """[B, T, 1]: tokens inside their sequence, or None when all are."""
    if s["lens"] is None:
        return None
    return (torch.arange(case["T"], device="cuda")[None, :] < s["lens"][:, None])[..., None]


def _scan_time(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, h_{-1} = 0, by doubling."""
    step, T = 1, a.shape[1]
    while step < T:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _plain_scan(s, case):
    dt = DTYPES[case["dtype"]]
    x, h0, mask = s["x"].float(), s["h0"], _valid(s, case)
    sr, si = torch.sigmoid(s["r"].float()), torch.sigmoid(s["i"].float())
    decay = DECAY * torch.log1p(torch.exp(s["lam"]))
    la = -decay * sr
    a = torch.exp(la)
    beta = torch.sqrt(-torch.expm1(2 * la))
    b = beta * si * x
    if mask is not None:
        a, b = torch.where(mask, a, 1.0), torch.where(mask, b, 0.0)
    first = b[:, :1] + a[:, :1] * h0[:, None]
    h = _scan_time(a, torch.cat([first, b[:, 1:]], 1))
    y = h if mask is None else torch.where(mask, h, 0.0)
    out = {"y": y.to(dt), "hT": h[:, -1]}
    if case["dir"] != "train":
        return out
    dy = s["dy"].float()
    if mask is not None:
        dy = torch.where(mask, dy, 0.0)
    # g_t = dy_t + a_{t+1} g_{t+1}, with the final state's gradient at the end
    dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dhT"][:, None]], 1)
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _scan_time(later.flip(1), dy.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    dh0 = a[:, 0] * g[:, 0]
    dla = a * g * before - a * a / beta * g * si * x
    grads = {"dx": g * beta * si, "dr": dla * la * (1 - sr), "di": g * beta * x * si * (1 - si)}
    if mask is not None:
        grads = {k: torch.where(mask, v, 0.0) for k, v in grads.items()}
        dla = torch.where(mask, dla, 0.0)
    dlam = (dla * sr).sum((0, 1)) * -DECAY * torch.sigmoid(s["lam"])
    return {**out, **{k: v.to(dt) for k, v in grads.items()}, "dlam": dlam, "dh0": dh0}


def _last_rows(s, case, ext):
    """The K - 1 rows of ``ext`` (K - 1 carried rows, then the sequence) that
    end at each sequence's end, and their places."""
    K, T = case["K"], case["T"]
    at = torch.arange(K - 1, device="cuda")[None, :] + (s["lens"][:, None].long() if s["lens"] is not None else T)
    at = at.expand(case["B"], K - 1)[..., None].expand(-1, -1, case["D"])
    return at, torch.gather(ext, 1, at)


def _plain_conv(s, case):
    dt, K, T = DTYPES[case["dtype"]], case["K"], case["T"]
    mask, w = _valid(s, case), s["w"].float()
    ext = torch.cat([s["state"].float(), s["x"].float()], 1)
    u = s["bias"].float() + sum(ext[:, j:j + T] * w[:, j] for j in range(K))
    sig = torch.sigmoid(u)
    y = u * sig
    y = y if mask is None else torch.where(mask, y, 0.0)
    at, last = _last_rows(s, case, ext)
    out = {"y": y.to(dt), "state": last.to(dt)}
    if case["dir"] != "train":
        return out
    du = s["dy"].float() * sig * (1 + u * (1 - sig))
    du = du if mask is None else torch.where(mask, du, 0.0)
    pad = torch.nn.functional.pad(du, (0, 0, K - 1, K - 1))
    dext = sum(pad[:, K - 1 - j:K - 1 - j + T + K - 1] * w[:, j] for j in range(K))
    dext = dext.scatter_add(1, at, s["dstate_out"].float())
    dw = torch.stack([(ext[:, j:j + T] * du).sum((0, 1)) for j in range(K)], 1)
    return {**out, "dx": dext[:, K - 1:].to(dt), "dw": dw.to(dt), "dbias": du.sum((0, 1)).to(dt),
            "dstate": dext[:, :K - 1].to(dt)}


def _plain_norm(s, case):
    dt = DTYPES[case["dtype"]]
    res = (s["x"].float() + s["res"].float()).to(dt)
    h = res.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
    scale = y.abs().amax(1) / 127
    q = torch.round(y / scale[:, None]).to(torch.int8)
    return {"residual": res, "scale": scale, "q": _values(s, q, scale)}


def _plain_matmul(s, case):
    acc = s["xq"].float() @ s["wq"].float().t()
    return (acc * s["sx"][:, None] * s["sw"] + s["bias"].float()).to(DTYPES[case["dtype"]])


_OWN = {"scan": _own_scan, "conv": _own_conv, "norm": _own_norm, "matmul": _own_matmul}
_PLAIN = {"scan": _plain_scan, "conv": _plain_conv, "norm": _plain_norm, "matmul": _plain_matmul}


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = {k: v.double() if torch.is_tensor(v) and k != "lens" else v for k, v in _inputs(case, seed).items()}
    return {"scan": _exact_scan, "conv": _exact_conv, "norm": _exact_norm, "matmul": _exact_matmul}[case["op"]](s, case)


def _lengths(s, case):
    return [case["T"]] * case["B"] if s["lens"] is None else s["lens"].tolist()


def _exact_scan(s, case):
    """The recurrence token by token, and its adjoint in reverse."""
    T = case["T"]
    x, h = s["x"], s["h0"]
    gate, inp = 1 / (1 + torch.exp(-s["r"])), 1 / (1 + torch.exp(-s["i"]))
    rate = DECAY * torch.nn.functional.softplus(s["lam"])
    keep = torch.exp(-rate * gate)
    root = (-torch.expm1(-2 * rate * gate)).sqrt()
    live = torch.ones(case["B"], T, 1, device=x.device, dtype=torch.bool)
    for b, n in enumerate(_lengths(s, case)):
        live[b, n:] = False
    whole = s["lens"] is None
    put = root * inp * x
    hs = [h]
    for t in range(T):
        new = torch.addcmul(put[:, t], keep[:, t], h)
        h = new if whole else torch.where(live[:, t], new, h)
        hs.append(h)
    hs = torch.stack(hs, 1)
    out = {"y": hs[:, 1:] * live, "hT": h}
    if case["dir"] != "train":
        return out
    g, gs = s["dhT"], [None] * T
    for t in reversed(range(T)):
        here = g + s["dy"][:, t]
        gs[t] = here if whole else torch.where(live[:, t], here, torch.zeros_like(here))
        g = here * keep[:, t] if whole else torch.where(live[:, t], here * keep[:, t], g)
    gs = torch.stack(gs, 1)
    dkeep = gs * hs[:, :-1] - gs * inp * x * keep / root
    dlog = dkeep * keep
    out["dx"] = gs * root * inp
    out["di"] = gs * root * x * inp * (1 - inp)
    out["dr"] = dlog * -rate * gate * (1 - gate)
    out["dlam"] = (dlog * -DECAY * gate).sum((0, 1)) * torch.sigmoid(s["lam"])
    out["dh0"] = g
    return out


def _exact_conv(s, case):
    """Sequence by sequence, through torch's own differentiation."""
    K, D = case["K"], case["D"]
    train = case["dir"] == "train"
    w, bias = s["w"].requires_grad_(train), s["bias"].requires_grad_(train)
    y = torch.zeros_like(s["x"])
    state = torch.zeros_like(s["state"])
    dx, dstate, dw, dbias = torch.zeros_like(s["x"]), torch.zeros_like(s["state"]), torch.zeros_like(w), torch.zeros_like(bias)
    with torch.set_grad_enabled(train):
        for b, n in enumerate(_lengths(s, case)):
            row = torch.cat([s["state"][b], s["x"][b, :n]]).requires_grad_(train)
            u = (row.unfold(0, K, 1) * w).sum(2) + bias if n else row[:0] * bias
            v = u / (1 + torch.exp(-u))
            y[b, :n] = v.detach()
            state[b] = row[n:n + K - 1].detach()
            if train:
                loss = (v * s["dy"][b, :n]).sum() + (row[n:] * s["dstate_out"][b]).sum() + 0 * (w.sum() + bias.sum())
                grow, gw, gb = torch.autograd.grad(loss, (row, w, bias))
                dstate[b], dx[b, :n] = grow[:K - 1], grow[K - 1:]
                dw, dbias = dw + gw, dbias + gb
    out = {"y": y, "state": state}
    return {**out, "dx": dx, "dw": dw, "dbias": dbias, "dstate": dstate} if train else out


def _exact_norm(s, case):
    """The stored residual is the rounded sum: exact() starts from it."""
    dt = DTYPES[case["dtype"]]
    res = (s["x"] + s["res"]).float().to(dt).double()
    y = res / (res.square().mean(1, keepdim=True) + EPS).sqrt() * s["w"]
    scale = y.abs().amax(1) / 127
    return {"residual": res, "scale": scale, "q": torch.round(y / scale[:, None]) * scale[:, None]}


def _exact_matmul(s, case):
    return torch.einsum("mk,nk->mn", s["xq"], s["wq"]) * torch.outer(s["sx"], s["sw"]) + s["bias"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op == "scan":
        n, bd = case["B"] * case["T"] * case["D"], case["B"] * case["D"]
        byt, flops = 4 * n * e + 8 * bd + 4 * case["D"], 20 * n
        if case["dir"] == "train":
            byt, flops = byt + 7 * n * e + 8 * bd + 8 * case["D"], flops + 50 * n
    elif op == "conv":
        n, K = case["B"] * case["T"] * case["D"], case["K"]
        st, wb = case["B"] * (K - 1) * case["D"] * e, case["D"] * (K + 1) * e
        byt, flops = 2 * n * e + 2 * st + wb, n * (2 * K + 5)
        if case["dir"] == "train":
            byt, flops = byt + 3 * n * e + 3 * st + 2 * wb, flops + n * (6 * K + 12)
    elif op == "norm":
        m, d = case["M"], case["D"]
        byt, flops = m * d * (3 * e + 1) + 4 * m + d * e, 9 * m * d
    else:
        m, n, k = case["M"], case["N"], case["K"]
        byt, flops = m * k + n * k + m * n * e + 4 * (m + n) + n * e, 2 * m * n * k
    return {"bytes": byt, "flops": flops}
