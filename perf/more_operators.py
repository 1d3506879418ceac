"""Operators of a dense MLP's training step and of its calls for few tokens: what is measured.

Each case names one pass (`kind`) and its sizes:
  linear        y = act(x w^T + bias) + residual
  linear_back   its gradients: of x (joined by a skip connection's), of w and of the bias (added up over micro-batches)
  gated         h = act(x w_gate^T) * (x w_up^T), the pre-activations kept or not
  gated_back    its gradients, from the kept pre-activations or from x and w alone
  adamw         one AdamW step over many tensors, moments in 32 bits or in 8

With `own` false, run() computes the plain form in elementary torch operations (32 bits, rounded once at the end);
with `own` true it makes the calls of mxfp4_precision_numerics_amd.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64, I64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.uint8
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def listed():
    return [
        # a decode step of one request: a square projection, bias and residual added to it (the weights are read once: bandwidth)
        dict(name="linear_token", kind="linear", tokens=1, hidden=4096, features=4096, act="none", bias=True,
             residual=True, keep=False, out="bf16"),
        # a few requests at ragged sizes
        dict(name="linear_few", kind="linear", tokens=23, hidden=2880, features=5000, act="gelu", bias=True,
             residual=False, keep=False, out="bf16"),
        # a training batch's down-projection into a residual stream of 32 bits (matrix units)
        dict(name="linear_down", kind="linear", tokens=8192, hidden=14336, features=4096, act="none", bias=False,
             residual=True, keep=False, out="f32"),
        # the gradients of a layer with bias and activation
        dict(name="linear_back", kind="linear_back", tokens=4096, hidden=4096, features=14336, act="gelu_tanh", bias=True,
             add=False, accumulate=False, out="bf16"),
        # a micro-batch's gradients at ragged sizes, added in 32 bits to those of the ones before it, the skip connection's joined
        dict(name="linear_back_ragged", kind="linear_back", tokens=2011, hidden=2880, features=1000, act="none", bias=True,
             add=True, accumulate=True, out="f32"),
        # one token through a shared expert's gate and up projections
        dict(name="gated_token", kind="gated", tokens=1, hidden=7168, inter=2048, act="silu", keep=False),
        # a few tokens through a dense layer's
        dict(name="gated_few", kind="gated", tokens=48, hidden=4096, inter=14336, act="silu", keep=False),
        # a training batch, the pre-activations kept for the backward pass
        dict(name="gated_batch", kind="gated", tokens=8192, hidden=4096, inter=14336, act="silu", keep=True),
        # its backward pass
        dict(name="gated_back", kind="gated_back", tokens=8192, hidden=4096, inter=14336, act="silu", keep=True, add=False),
        # the same with the pre-activations computed again (activation memory saved), ragged sizes
        dict(name="gated_back_again", kind="gated_back", tokens=2011, hidden=2880, inter=5000, act="gelu_tanh", keep=False,
             add=True),
        # a small dense model's layer: ragged matrices, many short vectors; all in 32 bits (launches count)
        dict(name="adamw_ragged", kind="adamw", matrices=7, rows=1001, cols=771, vectors=150, length=771, params="f32",
             copies=False, states="f32", clip=True),
        # 16 experts' matrices and their norms: 32-bit weights with bf16 copies, bf16 gradients, moments in 8 bits
        dict(name="adamw_experts", kind="adamw", matrices=16, rows=4096, cols=7168, vectors=40, length=7168, params="f32",
             copies=True, states="8bit", clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST = 8192 * 4096 * 14336  # tokens x hidden x features of the largest case


def draw(rng):
    kind = rng.choice(["linear", "linear_back", "gated", "gated_back", "adamw", "adamw"])
    if kind == "adamw":
        matrices = rng.randint(1, 64)
        rows = min(_log(rng, 16, 8192), max(16, 400_000_000 // (matrices * 4096)))
        return dict(kind=kind, matrices=matrices, rows=rows, cols=_log(rng, 17, 4096),
                    vectors=rng.randint(0, 300), length=_log(rng, 1, 8192), params=rng.choice(["f32", "bf16"]),
                    copies=rng.random() < 0.5, states=rng.choice(["f32", "8bit"]), clip=rng.random() < 0.5)
    hidden = 8 * _log(rng, 8, 1024)
    width = 8 * _log(rng, 8, 1792)
    tokens = min(_log(rng, 1 if kind in ("linear", "gated") else 16, 8192), MOST // (hidden * width * (2 if "gated" in kind else 1)))
    flip = lambda: rng.random() < 0.5
    if kind == "linear":
        return dict(kind=kind, tokens=tokens, hidden=hidden, features=width,
                    act=rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]), bias=flip(), residual=flip(),
                    keep=flip(), out=rng.choice(["bf16", "f32"]))
    if kind == "linear_back":
        act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"])
        # with an activation the weights' gradient is wanted in the weights' type
        return dict(kind=kind, tokens=tokens, hidden=hidden, features=width, act=act, bias=flip(), add=flip(),
                    accumulate=flip(), out="bf16" if act != "none" else rng.choice(["bf16", "f32"]))
    if kind == "gated":
        return dict(kind=kind, tokens=tokens, hidden=hidden, inter=width, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                    keep=flip())
    return dict(kind=kind, tokens=tokens, hidden=hidden, inter=width, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                keep=flip(), add=flip())


# the optimizer's settings, as a program has them in the middle of a training
STEP, RATE, BETAS, EPS, DECAY, MAX_NORM, SEED = 1000, 3e-4, (0.9, 0.95), 1e-8, 0.1, 1.0, 20
CHUNK, BLOCK = 8192, 128  # elements that one entry of the chunk list, and one scale of an 8-bit moment, covers


def _dtype(name):
    return BF16 if name == "bf16" else F32


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std
    kind, s = case["kind"], dict(case=case)
    if kind == "adamw":
        return _prepare_adamw(case, rn, s)
    T, H = case["tokens"], case["hidden"]
    N = case["features"] if "features" in case else 2 * case["inter"]
    s["x"] = rn(T, H).to(BF16)
    s["w"] = rn(N, H, std=1 / math.sqrt(H)).to(BF16)
    s["workspaces"] = {}
    if kind in ("linear", "linear_back"):
        bias = rn(N, std=0.2) if case["bias"] else None
    if kind == "linear":
        s["bias"] = bias
        s["residual"] = rn(T, N).to(_dtype(case["out"])) if case["residual"] else None
        s["y"] = torch.empty(T, N, dtype=_dtype(case["out"]), device=DEV)
        s["z"] = torch.empty(T, N, dtype=BF16, device=DEV) if case["keep"] else None
    elif kind == "gated":
        s["h"] = torch.empty(T, N // 2, dtype=BF16, device=DEV)
        s["z"] = torch.empty(T, N, dtype=BF16, device=DEV) if case["keep"] else None
    else:
        # what the forward pass kept
        if kind == "gated_back" and case["keep"] or kind == "linear_back" and case["act"] != "none":
            s["z"] = torch.mm(s["x"], s["w"].t())
            if kind == "linear_back" and bias is not None:
                s["z"] = (s["z"].float() + bias).to(BF16)
        else:
            s["z"] = None
        s["dy"] = rn(T, N if kind == "linear_back" else N // 2, std=1e-3).to(BF16)
        out = _dtype(case.get("out", "bf16"))
        s["add"] = rn(T, H, std=1e-3).to(BF16) if case["add"] else None
        s["dx"] = torch.empty(T, H, dtype=BF16, device=DEV)
        s["dw"] = rn(N, H, std=1e-3).to(out)  # the gradients so far, where they are added up
        s["dbias"] = rn(N, std=1e-3) if case.get("bias") else None
    return s


def _quantized(x, kind):
    """An 8-bit moment that a training has left: codes and a scale for each BLOCK of a row."""
    n, e = x.shape
    top = 448.0 if kind is E4M3 else 57344.0
    b = torch.nn.functional.pad(x, (0, -e % BLOCK)).view(n, -1, BLOCK)
    scale = (b.abs().amax(2) / top).clamp(min=2.0 ** -120)
    q = (b / scale[..., None]).clamp(-top, top).to(kind).view(n, -1)[:, :e].contiguous()
    return q.view(U8), scale


def _prepare_adamw(case, rn, s):
    sizes = [(case["matrices"], case["rows"] * case["cols"]), (case["vectors"], case["length"])]
    s["groups"] = []
    first = 0
    for k, (n, e) in enumerate(sizes):
        if n == 0:
            continue
        p = BF16 if k == 0 and case["params"] == "bf16" else F32
        q = dict(first=first, decay=k == 0, param=rn(n, e, std=0.02).to(p))
        q["grad"] = rn(n, e, std=1e-3).to(BF16 if k == 0 and (case["copies"] or p == BF16) else F32)
        q["copy"] = torch.empty(n, e, dtype=BF16, device=DEV) if k == 0 and case["copies"] and p == F32 else None
        m, v = rn(n, e, std=2e-4), rn(n, e, std=1e-3).square_().add_(1e-9)
        if case["states"] == "8bit":
            (q["m"], q["m_scale"]), (q["v"], q["v_scale"]) = _quantized(m, E4M3), _quantized(v, E5M2)
        else:
            q["m"], q["v"] = m, v
        s["groups"].append(q)
        first += n * -(-e // CHUNK)
    s["norm"] = torch.full((1,), 2.5, device=DEV) if case["clip"] else None
    s["handles"] = {}
    return s


def run(s):
    return (_own if own else _plain)(s)


def _outputs(s):
    keys = dict(linear=("y", "z"), linear_back=("dx", "dw", "dbias"), gated=("h", "z"), gated_back=("dx", "dw"))
    return {k: s[k] for k in keys[s["case"]["kind"]] if s[k] is not None}


def _states(groups):
    """What an optimizer step leaves: 8-bit moments as the values that their codes stand for."""
    out = []
    for q in groups:
        o = {k: q[k] for k in ("param", "copy") if q[k] is not None}
        if "m_scale" in q:
            o |= dict(m=q["m"].view(E4M3), v=q["v"].view(E5M2), m_scale=q["m_scale"], v_scale=q["v_scale"])
        else:
            o |= dict(m=q["m"], v=q["v"])
        out.append(o)
    return out


def _own(s):
    import mxfp4_precision_numerics_amd as mxq
    case, kind = s["case"], s["case"]["kind"]
    if kind == "adamw":
        if not s["handles"]:
            rows = lambda key: [t for q in s["groups"] for t in (q[key].unbind(0) if q.get(key) is not None else [None] * len(q["param"]))]
            eight = case["states"] == "8bit"
            s["handles"]["set"] = mxq.AdamW(
                rows("param"), rows("grad"), rows("m"), rows("v"), rows("m_scale") if eight else None,
                rows("v_scale") if eight else None, copies=rows("copy"),
                decay=[q["decay"] for q in s["groups"] for _ in q["param"]])
        s["handles"]["set"].step(STEP, RATE, BETAS, EPS, DECAY, norm=s["norm"], max_norm=MAX_NORM, seed=SEED)
        return _states(s["groups"])
    act = dict(none=mxq.ACT_NONE, relu=mxq.ACT_RELU, silu=mxq.ACT_SILU, gelu=mxq.ACT_GELU, gelu_tanh=mxq.ACT_GELU_TANH)[case["act"]]
    T, H = s["x"].shape
    if not s["workspaces"]:  # sized once per shape, as a program keeps it
        if "linear" in kind:
            size = mxq.linear_workspace(T, H, case["features"], backward=kind == "linear_back")
        else:
            size = mxq.gated_linear_workspace(T, H, case["inter"], backward=kind == "gated_back")
        s["workspaces"]["w"] = torch.empty(size, dtype=U8, device=DEV)
    ws = s["workspaces"]["w"]
    if kind == "linear":
        mxq.linear(s["x"], s["w"], s["y"], bias=s["bias"], activation=act, residual=s["residual"], z=s["z"], workspace=ws)
    elif kind == "linear_back":
        mxq.linear_backward(s["x"], s["w"], s["dy"], s["dx"], s["dw"], dbias=s["dbias"], activation=act, z=s["z"],
                            add=s["add"], accumulate=case["accumulate"], workspace=ws)
    elif kind == "gated":
        mxq.gated_linear(s["x"], s["w"], s["h"], activation=act, z=s["z"], workspace=ws)
    else:
        mxq.gated_linear_backward(s["x"], s["w"], s["dy"], s["dx"], s["dw"], activation=act, z=s["z"], add=s["add"],
                                  workspace=ws)
    return _outputs(s)


C0, C1 = math.sqrt(2 / math.pi), 0.044715  # of the tanh form of the GELU


def _act(z, name):
    """(act(z), act'(z))"""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + (-z).exp())
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * (-0.5 * z * z).exp() / math.sqrt(2 * math.pi)
    t = torch.tanh(C0 * (z + C1 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C0 * (1 + 3 * C1 * z * z)


def _gradients(s, dz):
    case = s["case"]
    dx, dw = dz @ s["w"].float(), dz.t() @ s["x"].float()
    if s["add"] is not None:
        dx += s["add"].float()
    if case.get("accumulate"):
        dw += s["dw"].float()
    s["dx"].copy_(dx)
    s["dw"].copy_(dw)


def _plain(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind == "adamw":
        for q in s["groups"]:
            _plain_adamw(q, s["norm"])
        return _states(s["groups"])
    if kind in ("linear", "gated"):
        z = s["x"].float() @ s["w"].float().t()
        if kind == "linear" and s["bias"] is not None:
            z += s["bias"]
        if s["z"] is not None:
            s["z"].copy_(z)
        if kind == "gated":
            gate, up = z.chunk(2, 1)
            s["h"].copy_(_act(gate, case["act"])[0] * up)
        else:
            y = _act(z, case["act"])[0]
            s["y"].copy_(y if s["residual"] is None else y + s["residual"].float())
        return _outputs(s)
    dy = s["dy"].float()
    if kind == "linear_back":
        dz = dy if case["act"] == "none" else dy * _act(s["z"].float(), case["act"])[1]
        if s["dbias"] is not None:
            s["dbias"].copy_(dz.sum(0) + s["dbias"] if case["accumulate"] else dz.sum(0))
    else:
        z = s["z"].float() if s["z"] is not None else s["x"].float() @ s["w"].float().t()
        gate, up = z.chunk(2, 1)
        a, d = _act(gate, case["act"])
        dz = torch.cat([dy * up * d, dy * a], 1)
    _gradients(s, dz)
    return _outputs(s)


U32 = 0xFFFFFFFF


def _words(step, seed):
    """The first random word of a step: the top of a 64-bit counter's avalanche."""
    m = (1 << 64) - 1
    x = (seed + step * 0x9E3779B97F4A7C15) & m
    x = ((x ^ x >> 30) * 0xBF58476D1CE4E5B9) & m
    x = ((x ^ x >> 27) * 0x94D049BB133111EB) & m
    return (x ^ x >> 31) & U32


def _bits(q):
    """16 random bits for each element: an avalanche of the pair's place in the list, halved between the two."""
    n, e = q["param"].shape
    at = (q["first"] + torch.arange(n, device=DEV) * -(-e // CHUNK))[:, None] * (CHUNK // 2) + torch.arange((e + 1) // 2, device=DEV)
    r = at & U32 ^ _words(STEP, SEED) ^ ((at >> 32) * 0x9E3779B1 & U32)
    r = ((r ^ r >> 16) * 0x85EBCA6B) & U32
    r = ((r ^ r >> 13) * 0xC2B2AE35) & U32
    r = r ^ r >> 16
    return torch.stack([r & 0xFFFF, r >> 16], 2).view(n, -1)[:, :e]


def _decoded(codes, scale, kind):
    n, e = codes.shape
    return (torch.nn.functional.pad(codes.view(kind).float(), (0, -e % BLOCK)).view(n, -1, BLOCK) * scale[..., None]).view(n, -1)[:, :e]


def _encode(x, codes, scale, kind, bits=None):
    n, e = x.shape
    top = 448.0 if kind is E4M3 else 57344.0
    b = torch.nn.functional.pad(x, (0, -e % BLOCK)).view(n, -1, BLOCK)
    scale.copy_((b.abs().amax(2) / top).clamp(min=2.0 ** -120))
    y = (b / scale[..., None]).view(n, -1)[:, :e].clamp(-top, top)
    if bits is not None:  # two bits of mantissa, the rest rounded by chance, nothing to zero
        unit = torch.ldexp(torch.ones_like(y), torch.frexp(y.clamp(min=2.0 ** -14)).exponent - 3)
        r = (torch.floor(y / unit + bits * 2.0 ** -16) * unit).clamp(max=top)
        y = torch.where((y > 0) & (r == 0), 2.0 ** -16, r)
    codes.copy_(y.to(kind).view(U8))


def _plain_adamw(q, norm):
    (b1, b2), eight = BETAS, "m_scale" in q
    g = q["grad"].float()
    if norm is not None:
        g = g * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    m, v = (_decoded(q["m"], q["m_scale"], E4M3), _decoded(q["v"], q["v_scale"], E5M2)) if eight else (q["m"], q["v"])
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = q["param"].float()
    if q["decay"]:
        p = p * (1 - RATE * DECAY)
    p = p - RATE / (1 - b1 ** STEP) * m / ((v / (1 - b2 ** STEP)).sqrt() + EPS)
    q["param"].copy_(p)
    if q["copy"] is not None:
        q["copy"].copy_(p)
    if eight:
        _encode(m, q["m"], q["m_scale"], E4M3)
        _encode(v, q["v"], q["v_scale"], E5M2, _bits(q))
    else:
        q["m"].copy_(m)
        q["v"].copy_(v)


def work(case):
    kind = case["kind"]
    if kind == "adamw":
        n, m = case["matrices"] * case["rows"] * case["cols"], case["vectors"] * case["length"]
        eight, p = case["states"] == "8bit", 2 if case["params"] == "bf16" else 4
        state = 4 * (1 + 4 / BLOCK) if eight else 16  # both moments, read and written
        copy = 2 if case["copies"] and p == 4 else 0
        grad = 2 if case["copies"] or p == 2 else 4
        return {"bytes": n * (2 * p + grad + copy + state) + m * (12 + state), "flops": 15 * (n + m)}
    T, H = case["tokens"], case["hidden"]
    if kind == "linear":
        N, out = case["features"], 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * (T + N) * H + 4 * N * case["bias"] + T * N * (out * (1 + case["residual"]) + 2 * case["keep"]),
                "flops": 2 * T * H * N}
    if kind == "linear_back":
        N, out = case["features"], 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * (T + N) * H + 2 * T * N * (1 + (case["act"] != "none")) + 4 * N * case["bias"] +
                2 * T * H * (1 + case["add"]) + N * H * out * (1 + case["accumulate"]), "flops": 4 * T * H * N}
    I = case["inter"]
    if kind == "gated":
        return {"bytes": 2 * (T + 2 * I) * H + 2 * T * I * (1 + 2 * case["keep"]), "flops": 4 * T * H * I}
    return {"bytes": 2 * (T + 4 * I) * H + 2 * T * I * (1 + 2 * case["keep"]) + 2 * T * H * (1 + case["add"]),
            "flops": (8 if case["keep"] else 12) * T * H * I}


def exact(case, seed):
    """The definitions in 64 bits; the gradients of the activations by differentiation, not by the plain form's formulas."""
    s, kind = prepare(case, seed), case["kind"]
    if kind == "adamw":
        return [_exact_adamw(q, s["norm"]) for q in s["groups"]]
    x, w = s["x"].double(), s["w"].double()
    act = dict(none=lambda z: z, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu,
               gelu_tanh=lambda z: torch.nn.functional.gelu(z, approximate="tanh"))[case["act"]]
    product = lambda: torch.mm(x, w.t().contiguous())
    out = {}
    if kind == "linear":
        z = product()
        if s["bias"] is not None:
            z += s["bias"].double()
        if case["keep"]:
            out["z"] = z
        out["y"] = act(z) + (s["residual"].double() if case["residual"] else 0.0)
        return out
    if kind == "gated":
        z = product()
        if case["keep"]:
            out["z"] = z
        out["h"] = act(z[:, :case["inter"]]) * z[:, case["inter"]:]
        return out
    dy = s["dy"].double()
    if kind == "linear_back" and case["act"] == "none":
        dz = dy
    else:
        z = (s["z"].double() if s["z"] is not None else product()).requires_grad_()
        h = act(z) if kind == "linear_back" else act(z[:, :case["inter"]]) * z[:, case["inter"]:]
        dz = torch.autograd.grad(h, z, dy)[0]
    if case.get("bias"):
        out["dbias"] = dz.sum(0) + (s["dbias"].double() if case["accumulate"] else 0.0)
    out["dx"] = torch.mm(dz, w) + (s["add"].double() if case["add"] else 0.0)
    out["dw"] = torch.mm(dz.t().contiguous(), x) + (s["dw"].double() if case.get("accumulate") else 0.0)
    return out


def _exact_adamw(q, norm):
    n, e = q["param"].shape
    eight = "m_scale" in q
    spread = lambda scale: scale.double().repeat_interleave(BLOCK, 1)[:, :e]
    g = q["grad"].double()
    if norm is not None:
        g *= min(1.0, MAX_NORM / (float(norm) + 1e-6))
    m = q["m"].view(E4M3).double() * spread(q["m_scale"]) if eight else q["m"].double()
    v = q["v"].view(E5M2).double() * spread(q["v_scale"]) if eight else q["v"].double()
    m = m + (1 - BETAS[0]) * (g - m)
    v = v + (1 - BETAS[1]) * (g * g - v)
    del g
    step = m / (1 - BETAS[0] ** STEP) / (torch.sqrt(v / (1 - BETAS[1] ** STEP)) + EPS)
    p = q["param"].double()
    p = p - RATE * (step + (DECAY * p if q["decay"] else 0.0))
    del step
    out = dict(param=p) | (dict(copy=p) if q["copy"] is not None else {})
    if not eight:
        return out | dict(m=m, v=v)
    for name, x, top, least, digits in (("m", m, 448.0, -6, 3), ("v", v, 57344.0, -14, 2)):
        scale = torch.zeros(n, -(-e // BLOCK), dtype=F64, device=DEV)
        scale.scatter_reduce_(1, (torch.arange(e, device=DEV) // BLOCK).expand(n, e), x.abs(), "amax")
        out[name + "_scale"] = scale = (scale / top).clamp(min=2.0 ** -120)
        y = (x.abs() / spread(scale.float())).clamp(max=top)  # codes are relative to the scale as it is stored
        unit = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** least))) - digits)
        k = torch.round(y / unit) if name == "m" else torch.floor(y / unit + _bits(q).double() / 65536)
        k = (k * unit).clamp(max=top)
        out[name] = k * torch.sign(x) if name == "m" else torch.where((y > 0) & (k == 0), 2.0 ** -16, k)
    return out
