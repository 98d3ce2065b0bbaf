"""Cases of the selective-block operators: what is measured, the operators'
plain forms, and the same results in 64 bits.

The operators: the selective state space scan (``scan``), the product of 8-bit
floating-point matrices with a scale for each block of 128 (``matmul``), rows
and columns to that form (``quant``), and the residual + root-mean-square norm
with an output in that form (``norm``).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# largest value, bits of the significand, exponent of the smallest normal number
F8_TOP = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}
BLOCK = 128
LEAST = 2.0 ** -110  # a block's largest magnitude counts as no less
EPS = 1e-6


def listed():
    return [
        # one generated token for each of 64 sequences: the states' bytes count
        {"name": "scan_step", "op": "scan", "dir": "fwd", "dtype": "bf16", "B": 64, "T": 1, "D": 2048, "N": 16, "G": 1,
         "gate": True, "ragged": False},
        # one long prompt: few channels for the whole GPU, a long axis to walk
        {"name": "scan_prompt", "op": "scan", "dir": "fwd", "dtype": "bf16", "B": 1, "T": 32768, "D": 2048, "N": 16, "G": 1,
         "gate": True, "ragged": False},
        # a training step's forward and backward pass
        {"name": "scan_train", "op": "scan", "dir": "train", "dtype": "bf16", "B": 8, "T": 2048, "D": 2048, "N": 16, "G": 1,
         "gate": True, "ragged": False},
        # a small 32-bit training batch of padded sequences, odd sizes, one sequence empty, two groups of channels
        {"name": "scan_train_ragged", "op": "scan", "dir": "train", "dtype": "f32", "B": 3, "T": 1537, "D": 700, "N": 16,
         "G": 2, "gate": False, "ragged": True},
        # one generated token for each of 4 sequences: the weights' bytes count
        {"name": "matmul_step", "op": "matmul", "dtype": "bf16", "M": 4, "N": 8192, "K": 2048, "xf": "e4m3", "wf": "e4m3",
         "square": True},
        # a ragged batch of a few hundred tokens, a width that no tile divides
        {"name": "matmul_batch", "op": "matmul", "dtype": "f16", "M": 197, "N": 5000, "K": 2048, "xf": "e4m3", "wf": "e4m3",
         "square": True},
        # a long prompt's tokens: the tensor cores count
        {"name": "matmul_prompt", "op": "matmul", "dtype": "bf16", "M": 8192, "N": 8192, "K": 2048, "xf": "e4m3",
         "wf": "e4m3", "square": True},
        # a weight's gradient over 8192 tokens: both sides scaled in 1 x 128, gradients in the wider format
        {"name": "matmul_weight_grad", "op": "matmul", "dtype": "f32", "M": 4096, "N": 2048, "K": 8192, "xf": "e5m2",
         "wf": "e4m3", "square": False},
        # a long prompt's activations before a product
        {"name": "quant_prompt", "op": "quant", "dtype": "bf16", "M": 16384, "D": 4096, "f8": "e4m3", "square": False,
         "both": False},
        # a training step's output gradients, for the input's and for the weight's gradient: rows and columns, odd sizes
        {"name": "quant_train", "op": "quant", "dtype": "f16", "M": 8191, "D": 2050, "f8": "e5m2", "square": False,
         "both": True},
        # one generated token for each of 16 sequences
        {"name": "norm_step", "op": "norm", "dtype": "bf16", "M": 16, "D": 2048},
        # a long prompt's tokens
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "M": 16384, "D": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A channel count: mostly a multiple of 64, sometimes odd."""
    d = _log(rng, lo, hi)
    return d if rng.random() < 0.3 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["scan", "scan", "matmul", "matmul", "quant", "norm"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "scan":
        g = rng.choice([1, 1, 1, 2])
        d = max(1, _width(rng, 256, 4096) // g) * g
        n = rng.choice([8, 16, 16, 16, 32, _log(rng, 4, 64)])
        b = _log(rng, 1, 64)
        t = 1 if rng.random() < 0.25 else _log(rng, 2, 32768)
        train = t > 1 and rng.random() < 0.5
        t = max(1, min(t, 8192 if train else t, (1 << (29 if train else 30)) // (b * d * n)))
        return {"op": op, "dir": "train" if train else "fwd", "dtype": dtype, "B": b, "T": t, "D": d, "N": n, "G": g,
                "gate": rng.random() < 0.7, "ragged": t > 1 and rng.random() < 0.4}
    if op == "matmul":
        n, k = _width(rng, 256, 8192), _width(rng, 256, 8192)
        square = rng.random() < 0.7
        return {"op": op, "dtype": dtype, "M": _log(rng, 1, min(8192, (1 << 36) // (n * k))), "N": n, "K": k,
                "xf": "e4m3" if square else rng.choice(["e4m3", "e5m2"]), "wf": "e4m3", "square": square}
    d = _width(rng, 256, 8192)
    m = _log(rng, 1, (1 << (25 if dtype == "f32" else 26)) // d)
    if op == "norm":
        return {"op": op, "dtype": dtype, "M": m, "D": d}
    square = rng.random() < 0.3
    return {"op": op, "dtype": dtype, "M": m, "D": d, "f8": "e4m3" if square else rng.choice(["e4m3", "e5m2"]),
            "square": square, "both": rng.random() < 0.5}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _up(n, to):
    return -(-n // to) * to


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
    if op == "scan":
        B, T, D, N, G = (case[k] for k in "BTDNG")
        s["x"] = normal(B, T, D).to(dt)
        s["delta"] = normal(B, T, D, std=0.5).to(dt)
        # a channel's ordinary step, softplus(bias), lies in 0.001 ... 0.1
        s["bias"] = torch.log(torch.expm1(torch.exp(uniform(math.log(0.001), math.log(0.1), D))))
        s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(normal(D, N, std=0.1))
        s["Bm"] = normal(B, T, G * N).to(dt)
        s["Cm"] = normal(B, T, G * N).to(dt)
        s["skip"] = normal(D, std=0.1, mean=1.0)
        s["z"] = normal(B, T, D).to(dt) if case["gate"] else None
        s["h0"] = normal(B, D, N, std=0.5)
        s["lens"] = None
        if case["ragged"]:
            lens = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            lens[0] = T
            if B > 2:
                lens[1] = 0
            s["lens"] = lens
        if case["dir"] == "train":
            s["dy"] = normal(B, T, D).to(dt)
            s["dhT"] = normal(B, D, N)
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb, pitch = -(-K // BLOCK), _up(K, 16)

        def codes(rows, f8):  # blocks of normal values whose largest one is near the format's
            top = F8_TOP[f8][0]
            v = torch.clamp(normal(rows, pitch, std=top / 3.5), -top, top).to(F8[f8])
            return v.view(torch.uint8)

        s["xq"], s["wq"] = codes(M, case["xf"]), codes(N, case["wf"])
        s["sx"] = uniform(0.5, 1.5, kb, M) * (3.5 / F8_TOP[case["xf"]][0])
        s["sw"] = uniform(0.5, 1.5, kb, -(-N // BLOCK) if case["square"] else N) * (3.5 / F8_TOP[case["wf"]][0] / K ** 0.5)
        s["bias"] = uniform(-0.1, 0.1, N).to(dt) if case["square"] else None
    elif op == "quant":
        s["x"] = (normal(case["M"], case["D"]) * torch.exp(normal(case["M"], 1))).to(dt)
    else:
        M, D = case["M"], case["D"]
        s["x"] = normal(M, D).to(dt)
        s["res"] = normal(M, D, std=2.0).to(dt)
        s["w"] = uniform(0.5, 1.5, D).to(dt)
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
        return None if t is None else torch.empty_like(t, dtype=dtype or t.dtype)

    def scratch(n):
        return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")

    def blocks(rows, width, square):  # a matrix in 8 bits and its blocks' scales
        q = torch.empty(rows, gc.f8_pitch(width), dtype=torch.uint8, device="cuda")
        return q, torch.empty(-(-width // BLOCK), -(-rows // BLOCK) if square else rows, device="cuda")

    if op == "scan":
        p = s["p"] = gc.make_ssm_problem(case["B"], case["T"], case["D"], case["N"], case["G"], softplus=True)
        s["y"], s["hT"], s["saved"] = like(s["x"]), like(s["h0"]), None
        s["ws"] = scratch(gc.gconv_selective_scan_fwd_workspace_size(p, code))
        if case["dir"] == "train":
            s["saved"] = scratch(gc.gconv_selective_scan_saved_size(p, code))
            s["ws_bwd"] = scratch(gc.gconv_selective_scan_bwd_workspace_size(p, code))
            for k in ("x", "delta", "A", "Bm", "Cm", "skip", "z", "bias", "h0"):
                s["d" + k] = like(s[k])
    elif op == "matmul":
        rows = BLOCK if case["square"] else 1
        s["p"] = gc.make_matmul_f8_problem(case["M"], case["N"], case["K"], gc.F8_CODES[case["xf"]], gc.F8_CODES[case["wf"]], rows)
        s["y"] = torch.empty(case["M"], case["N"], dtype=DTYPES[case["dtype"]], device="cuda")
    elif op == "quant":
        M, D = case["M"], case["D"]
        s["p"] = gc.make_quant_f8_problem(M, D, gc.F8_CODES[case["f8"]], BLOCK if case["square"] else 1)
        s["q"], s["scale"] = blocks(M, D, case["square"])
        s["qt"], s["scale_t"] = blocks(D, M, case["square"]) if case["both"] else (None, None)
    else:
        s["p"] = gc.make_norm_problem(case["M"], case["D"], EPS)
        s["res_out"] = like(s["res"])
        s["q"], s["scale"] = blocks(case["M"], case["D"], False)


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
    gc.gconv_selective_scan_fwd(s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], s["skip"], s["z"], s["bias"], s["h0"], s["lens"],
                                s["y"], s["hT"], s["saved"], s["p"], s["code"], s["ws"], 0, st)
    out = {"y": s["y"], "hT": s["hT"]}
    if train:
        gc.gconv_selective_scan_bwd(s["dy"], s["dhT"], s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], s["skip"], s["z"],
                                    s["bias"], s["lens"], s["saved"], s["dx"], s["ddelta"], s["dA"], s["dBm"], s["dCm"],
                                    s["dskip"], s["dz"], s["dbias"], s["dh0"], s["p"], s["code"], s["ws_bwd"], 0, st)
        out.update({k: s[k] for k in ("dx", "ddelta", "dA", "dBm", "dCm", "dskip", "dbias", "dh0")})
        if case["gate"]:
            out["dz"] = s["dz"]
    return out


def _own_matmul(s, case):
    gc = s["gc"]
    gc.gconv_matmul_f8(s["xq"], s["sx"], s["wq"], s["sw"], s["bias"], s["y"], s["p"], s["code"], torch.cuda.current_stream())
    return s["y"]


def _own_quant(s, case):
    gc = s["gc"]
    gc.gconv_quantize_f8(s["x"], s["q"], s["scale"], s["qt"], s["scale_t"], s["p"], s["code"], torch.cuda.current_stream())
    # a byte of q is an 8-bit floating-point number, and read as one
    out = {"q": s["q"].view(F8[case["f8"]])[:, :case["D"]], "scale": s["scale"]}
    if case["both"]:
        out["qt"], out["scale_t"] = s["qt"].view(F8[case["f8"]])[:, :case["M"]], s["scale_t"]
    return out


def _own_norm(s, case):
    gc = s["gc"]
    gc.gconv_rms_norm_f8(s["x"], s["res"], s["w"], s["res_out"], None, s["q"], s["scale"], gc.F8_CODES["e4m3"], s["p"],
                         s["code"], torch.cuda.current_stream())
    return {"residual": s["res_out"], "q": s["q"].view(F8["e4m3"])[:, :case["D"]], "scale": s["scale"]}


def _valid(s, case):
    """[B, T, 1]: tokens inside their sequence, or None when all are."""
    if s["lens"] is None:
        return None
    return (torch.arange(case["T"], device="cuda")[None, :] < s["lens"][:, None])[..., None]


def _scan_time(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, h_{-1} = 0, by doubling; in place of a and b."""
    step, T = 1, a.shape[1]
    while step < T:
        b[:, step:] += a[:, step:] * b[:, :-step]
        a[:, step:] *= a[:, :-step].clone()
        step *= 2
    return b


def _states(m, case):
    """[B, T, G N] of the groups as [B, T, D, N] for their channels."""
    B, T, D, N, G = (case[k] for k in "BTDNG")
    return m.float().view(B, T, G, 1, N).expand(B, T, G, D // G, N).reshape(B, T, D, N)


def _groups(v, case):
    """[B, T, D, N] summed over each group's channels: [B, T, G N]."""
    B, T, D, N, G = (case[k] for k in "BTDNG")
    return v.view(B, T, G, D // G, N).sum(3).reshape(B, T, G * N)


def _plain_scan(s, case):
    dt = DTYPES[case["dtype"]]
    x, A, mask = s["x"].float(), s["A"], _valid(s, case)
    v = s["delta"].float() + s["bias"]
    step = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    if mask is not None:
        step, x = torch.where(mask, step, 0.0), torch.where(mask, x, 0.0)
    Bm, Cm = _states(s["Bm"], case), _states(s["Cm"], case)
    u = step * x
    a = torch.exp(step[..., None] * A)
    b = u[..., None] * Bm
    b[:, 0] += a[:, 0] * s["h0"]
    h = _scan_time(a.clone(), b)
    o = (h * Cm).sum(-1) + s["skip"] * x
    sig = None if s["z"] is None else torch.sigmoid(s["z"].float())
    y = o if sig is None else o * s["z"].float() * sig
    y = y if mask is None else torch.where(mask, y, 0.0)
    out = {"y": y.to(dt), "hT": h[:, -1]}
    if case["dir"] != "train":
        return out
    dy = s["dy"].float()
    if mask is not None:
        dy = torch.where(mask, dy, 0.0)
    grads = {}
    if sig is not None:
        z = s["z"].float()
        grads["dz"] = dy * o * sig * (1 + z * (1 - sig))
        dy = dy * z * sig
    # g_t = C_t dy_t + a_{t+1} g_{t+1}, with the final state's gradient at the end
    put = Cm * dy[..., None]
    put[:, -1] += s["dhT"]
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _scan_time(later.flip(1), put.flip(1)).flip(1)
    grads["dCm"] = _groups(h * dy[..., None], case)
    grads["dBm"] = _groups(g * u[..., None], case)
    du = (g * Bm).sum(-1)
    before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    dl = g * before * a
    dstep = (dl * A).sum(-1) + du * x
    grads["dx"] = du * step + dy * s["skip"]
    grads["ddelta"] = dstep * torch.sigmoid(v)
    if mask is not None:
        grads = {k: torch.where(mask, w, 0.0) for k, w in grads.items()}
    sums = {"dA": (dl * step[..., None]).sum((0, 1)), "dskip": (dy * x).sum((0, 1)), "dbias": grads["ddelta"].sum((0, 1)),
            "dh0": a[:, 0] * g[:, 0]}
    return {**out, **{k: w.to(dt) for k, w in grads.items()}, **sums}


def _widened(q, scale, f8, width, square):
    """The values of a matrix in 8 bits: [rows, width], 32 bits."""
    v = q.view(F8[f8])[:, :width].float()
    by = scale.t().repeat_interleave(BLOCK, 1)[:, :width]
    return v * (by.repeat_interleave(BLOCK, 0)[:len(v)] if square else by)


def _plain_matmul(s, case):
    x = _widened(s["xq"], s["sx"], case["xf"], case["K"], False)
    y = x @ _widened(s["wq"], s["sw"], case["wf"], case["K"], case["square"]).t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(DTYPES[case["dtype"]])


def _to_f8(v, f8):
    """64-bit values to the nearest number of the format, ties to the even one."""
    top, bits, least = F8_TOP[f8]
    binade = torch.where(v == 0, 0.0, v / torch.frexp(v)[0] / 2)  # the power of two at or below |v|
    step = torch.clamp(binade, min=2.0 ** least) * 2.0 ** -bits
    return torch.clamp(torch.round(v / step) * step, -top, top).to(F8[f8])


def _block_top(v, rows):
    """The largest magnitude of each block of rows x 128: [row blocks, column blocks]."""
    M, D = v.shape
    v = torch.nn.functional.pad(v.abs(), (0, _up(D, BLOCK) - D, 0, _up(M, rows) - M))
    top = v.view(-1, rows, _up(D, BLOCK) // BLOCK, BLOCK).amax((1, 3))
    return torch.clamp(top, min=LEAST)


def _quantised(v, top, rows, f8):
    """Rows of v (fp32) by their blocks' factors, which are 32-bit numbers; next to a border 64 bits decide."""
    M, D = v.shape
    factor = torch.full_like(top, F8_TOP[f8][0]).div(top).repeat_interleave(BLOCK, 1)[:, :D].repeat_interleave(rows, 0)[:M]
    return _to_f8(v.double() * factor.double(), f8)


def _plain_quant(s, case):
    x, rows, f8 = s["x"].float(), BLOCK if case["square"] else 1, case["f8"]
    top = _block_top(x, rows)
    out = {"q": _quantised(x, top, rows, f8), "scale": (top / F8_TOP[f8][0]).t().contiguous()}
    if case["both"]:
        x = x.t().contiguous()
        top = _block_top(x, rows)
        out["qt"], out["scale_t"] = _quantised(x, top, rows, f8), (top / F8_TOP[f8][0]).t().contiguous()
    return out


def _plain_norm(s, case):
    res = (s["x"].float() + s["res"].float()).to(DTYPES[case["dtype"]])
    h = res.float()
    v = h * s["w"].float()
    top = _block_top(v, 1)
    root = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    return {"residual": res, "q": _quantised(v, top, 1, "e4m3"), "scale": (top * root / F8_TOP["e4m3"][0]).t().contiguous()}


_OWN = {"scan": _own_scan, "matmul": _own_matmul, "quant": _own_quant, "norm": _own_norm}
_PLAIN = {"scan": _plain_scan, "matmul": _plain_matmul, "quant": _plain_quant, "norm": _plain_norm}


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    return {"scan": _exact_scan, "matmul": _exact_matmul, "quant": _exact_quant, "norm": _exact_norm}[case["op"]](
        _inputs(case, seed), case)


def _exact_scan(s, case):
    """The recurrence token by token, and its adjoint in reverse."""
    B, T, D, N, G = (case[k] for k in "BTDNG")
    if T > 40000:
        return None
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    live = torch.zeros(B, T, 1, device="cuda", dtype=torch.float64)
    for b, n in enumerate(lens):
        live[b, :n] = 1
    x, raw, A, h = s["x"].double(), s["delta"].double() + s["bias"].double(), s["A"].double(), s["h0"].double()
    dt = torch.nn.functional.softplus(raw, threshold=700.0) * live
    in_, out_ = (s[k].double().view(B, T, G, 1, N) for k in ("Bm", "Cm"))

    def per_channel(m, t):
        return m[:, t].expand(B, G, D // G, N).reshape(B, D, N)

    train = case["dir"] == "train"
    hs, o = [h], torch.empty_like(x)
    for t in range(T):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * per_channel(in_, t)
        o[:, t] = torch.einsum("bdn,bdn->bd", h, per_channel(out_, t))
        if train:
            hs.append(h)
    o += s["skip"].double() * x
    z = None if s["z"] is None else s["z"].double()
    out = {"y": (o if z is None else o * z / (1 + torch.exp(-z))) * live, "hT": h}
    if not train:
        return out
    dy = s["dy"].double() * live
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        out["dz"] = dy * o * (sig + z * sig * (1 - sig))
        dy = dy * z * sig
    g = s["dhT"].double()
    dx, dstep = dy * s["skip"].double(), torch.zeros_like(x)
    dA = torch.zeros_like(A)
    dB, dC = torch.zeros(B, T, G, N, device="cuda", dtype=torch.float64), torch.zeros(B, T, G, N, device="cuda", dtype=torch.float64)
    for t in reversed(range(T)):
        a = torch.exp(dt[:, t, :, None] * A)
        g = g + per_channel(out_, t) * dy[:, t, :, None]
        du = torch.einsum("bdn,bdn->bd", g, per_channel(in_, t))
        dx[:, t] += du * dt[:, t]
        dB[:, t] = (g * (dt[:, t] * x[:, t])[..., None]).view(B, G, -1, N).sum(2)
        dC[:, t] = (hs[t + 1] * dy[:, t, :, None]).view(B, G, -1, N).sum(2)
        g = g * a
        late = g * hs[t]
        dA += (late * dt[:, t, :, None]).sum(0)
        dstep[:, t] = (late * A).sum(-1) + du * x[:, t]
    out["ddelta"] = dstep * torch.sigmoid(raw) * live
    out["dx"] = dx * live
    out["dBm"], out["dCm"] = ((m * live[..., None]).reshape(B, T, G * N) for m in (dB, dC))
    out["dA"], out["dskip"], out["dbias"], out["dh0"] = dA, (dy * x).sum((0, 1)), out["ddelta"].sum((0, 1)), g
    return out


def _exact_matmul(s, case):
    """Block by block of the summed axis."""
    M, N, K = case["M"], case["N"], case["K"]
    x, w = s["xq"].view(F8[case["xf"]])[:, :K].double(), s["wq"].view(F8[case["wf"]])[:, :K].double()
    y = torch.zeros(M, N, device="cuda", dtype=torch.float64)
    for k in range(-(-K // BLOCK)):
        at = slice(k * BLOCK, (k + 1) * BLOCK)
        side = s["sw"][k].double()
        if case["square"]:
            side = side[torch.arange(N, device="cuda") // BLOCK]
        y += torch.einsum("mk,nk->mn", x[:, at], w[:, at]) * torch.outer(s["sx"][k].double(), side)
    return y if s["bias"] is None else y + s["bias"].double()


def _nearest(v, f8):
    """Nearest number of the format among all of them, ties to the even code."""
    codes = torch.arange(127 if f8 == "e4m3" else 124, device="cuda").to(torch.uint8).view(F8[f8]).double()
    middle = (codes[1:] + codes[:-1]) / 2
    m = v.abs()
    at = torch.bucketize(m, middle)  # a value in the middle has the lower code
    up = (at < len(middle)) & (at % 2 == 1) & (m == middle[torch.clamp(at, max=len(middle) - 1)])
    return torch.copysign(codes[at + up.long()], v)


def _exact_blocks(v, rows, f8):
    """(values, largest magnitudes); the factor of a block is a 32-bit number by definition."""
    M, D = v.shape
    q, top = torch.empty_like(v), torch.empty(-(-M // rows), -(-D // BLOCK), device="cuda", dtype=torch.float64)
    most = F8_TOP[f8][0]
    for k in range(top.shape[1]):
        part = v[:, k * BLOCK:(k + 1) * BLOCK]
        mag = part.abs().amax(1)
        if rows > 1:
            mag = torch.stack([c.max() for c in mag.split(rows)])
        top[:, k] = torch.clamp(mag, min=LEAST)
        factor = torch.full_like(top[:, k].float(), most).div(top[:, k].float()).double()[torch.arange(M, device="cuda") // rows]
        q[:, k * BLOCK:(k + 1) * BLOCK] = _nearest(part * factor[:, None], f8)
    return q, top


def _exact_quant(s, case):
    x, rows = s["x"].double(), BLOCK if case["square"] else 1
    most = F8_TOP[case["f8"]][0]
    q, top = _exact_blocks(x, rows, case["f8"])
    out = {"q": q, "scale": top.t() / most}
    if case["both"]:
        q, top = _exact_blocks(x.t().contiguous(), rows, case["f8"])
        out["qt"], out["scale_t"] = q, top.t() / most
    return out


def _exact_norm(s, case):
    """The stored residual is the rounded sum: exact() starts from it."""
    res = (s["x"].double() + s["res"].double()).float().to(DTYPES[case["dtype"]]).double()
    q, top = _exact_blocks(res * s["w"].double(), 1, "e4m3")
    root = (res.square().mean(1) + EPS).sqrt()
    return {"residual": res, "q": q, "scale": top.t() / root / F8_TOP["e4m3"][0]}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op == "scan":
        B, T, D, N, G = (case[k] for k in "BTDNG")
        n, state, mixes, gate = B * T * D, B * D * N * 4, 2 * B * T * G * N, int(case["gate"])
        small = D * N * 4 + 8 * D
        byt, flops = n * e * (3 + gate) + mixes * e + 2 * state + small, n * (7 * N + 20)
        if case["dir"] == "train":  # dy, x, delta, z, B, C in; dx, ddelta, dz, dB, dC out
            byt, flops = byt + n * e * (5 + 2 * gate) + 2 * mixes * e + 2 * state + 2 * small, flops + n * (22 * N + 50)
    elif op == "matmul":
        m, n, k = case["M"], case["N"], case["K"]
        kb = -(-k // BLOCK)
        byt = m * k + n * k + m * n * e + 4 * kb * (m + (-(-n // BLOCK) if case["square"] else n)) + n * e * int(case["square"])
        flops = 2 * m * n * k
    elif op == "quant":
        m, d = case["M"], case["D"]
        per = BLOCK * BLOCK if case["square"] else BLOCK
        byt, flops = m * d * (e + (1 + 4 / per) * (2 if case["both"] else 1)), 4 * m * d * (2 if case["both"] else 1)
    else:
        m, d = case["M"], case["D"]
        byt, flops = m * d * (3 * e + 1 + 4 / BLOCK) + d * e, 9 * m * d
    return {"bytes": byt, "flops": flops}
