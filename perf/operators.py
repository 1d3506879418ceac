"""Operators of a mixture-of-experts training step around the scaled GEMMs: what is measured.

Each case names one pass (`kind`) and its sizes:
  route          router top-k (softmax weights) and the sort of the chosen assignments by local expert
  route_back     the router's gradient: dweights -> dlogits
  dispatch       token rows into expert order, quantized to MX E4M3 on the way
  combine        expert rows back into token order, weighted (or the plain sum: dispatch's gradient)
  combine_back   the weighted combine's gradient: expert rows' and weights' gradients
  loss           softmax cross entropy of hidden states against a vocabulary projection, no gradient
  loss_grad      the same with the gradients of the hidden states and of the projection
  clip           global gradient norm over many tensors, and the clipped gradients

With `own` false, run() computes the plain form in elementary torch operations (32 bits, rounded once at the end);
with `own` true it makes the calls of mxfp4_precision_numerics_amd.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def listed():
    return [
        # a decode step of 16 requests on one expert-parallel rank: top-8 of 256 experts, 32 of them local
        dict(name="route_decode", kind="route", tokens=16, experts=256, topk=8, local=32, renorm=True, dtype="f32"),
        # the prompt / training batch of the same layer, every expert local
        dict(name="route_batch", kind="route", tokens=8192, experts=256, topk=8, local=256, renorm=True, dtype="bf16"),
        # the router's gradient of a training batch
        dict(name="route_back_batch", kind="route_back", tokens=8192, experts=256, topk=8, renorm=False, dtype="f32"),
        # the rank's share of a batch (32 of 256 experts), quantized for the grouped up-projection
        dict(name="dispatch_share", kind="dispatch", tokens=8192, cols=7168, experts=256, topk=8, local=32),
        # every expert on one GPU: each token's row goes to 8 places
        dict(name="dispatch_all", kind="dispatch", tokens=4096, cols=4096, experts=64, topk=8, local=64),
        # a batch's weighted sum, every expert local
        dict(name="combine_batch", kind="combine", tokens=4096, cols=7168, experts=256, topk=8, local=256, weighted=True,
             dtype="bf16"),
        # its gradient at an odd token count
        dict(name="combine_back_ragged", kind="combine_back", tokens=4001, cols=4096, experts=64, topk=6, local=64,
             dtype="bf16"),
        # scoring a few tokens against a large vocabulary (the projection is read once: bandwidth)
        dict(name="loss_few_tokens", kind="loss", tokens=48, hidden=4096, vocab=131072, ignored=0.0),
        # a training step at ragged sizes, a fifth of the tokens masked (prompt tokens, padding)
        dict(name="loss_grad_ragged", kind="loss_grad", tokens=2011, hidden=2880, vocab=50021, ignored=0.2),
        # a training batch over a large vocabulary (matrix units)
        dict(name="loss_grad_large", kind="loss_grad", tokens=8192, hidden=4096, vocab=131072, ignored=0.05),
        # the gradients of a small dense model's layer: ragged matrices, many short vectors, the launch counts
        dict(name="clip_ragged", kind="clip", matrices=7, rows=1001, cols=771, vectors=150, length=771),
        # the gradients of 16 experts and their router and norms: large bf16 matrices and small fp32 vectors
        dict(name="clip_experts", kind="clip", matrices=32, rows=4096, cols=7168, vectors=40, length=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "route_back", "dispatch", "combine", "combine_back", "loss", "loss_grad", "loss_grad",
                       "clip", "clip"])
    dtype = rng.choice(["f32", "bf16"])
    if kind in ("route", "route_back"):
        experts = _log(rng, 4, 512)
        case = dict(kind=kind, tokens=_log(rng, 1, 16384), experts=experts, topk=min(experts, rng.randint(1, 10)),
                    renorm=rng.random() < 0.5, dtype=dtype)
        if kind == "route":
            case["local"] = rng.randint(1, experts)
        return case
    if kind in ("dispatch", "combine", "combine_back"):
        experts = _log(rng, 4, 256)
        topk = min(experts, rng.randint(1, 8))
        cols = 32 * _log(rng, 4, 256)
        tokens = min(_log(rng, 1, 8192), 8192 * 7168 // (cols * topk) + 1)
        case = dict(kind=kind, tokens=tokens, cols=cols, experts=experts, topk=topk, local=rng.randint(1, experts))
        if kind != "dispatch":
            case["dtype"] = dtype
        if kind == "combine":
            case["weighted"] = rng.random() < 0.7
        return case
    if kind in ("loss", "loss_grad"):
        return dict(kind=kind, tokens=_log(rng, 1, 4096), hidden=8 * _log(rng, 32, 640), vocab=_log(rng, 300, 131072),
                    ignored=rng.choice([0.0, 0.1, 0.5, 1.0]) if rng.random() < 0.5 else 0.02)
    return dict(kind="clip", matrices=rng.randint(1, 64), rows=_log(rng, 16, 4096), cols=_log(rng, 17, 4096),
                vectors=rng.randint(0, 300), length=_log(rng, 1, 8192))


def _dtype(case):
    return BF16 if case.get("dtype", "bf16") == "bf16" else F32


def _routing(case, g):
    """The places of the local assignments in expert order: what a program holds after the sort. Each token has
    distinct random experts of skewed popularity; the rows' buffers have a fixed capacity, and what is past it is dropped."""
    T, k, E, G = case["tokens"], case["topk"], case["experts"], case["local"]
    keys = torch.rand(T, E, generator=g, device=DEV) + 0.3 * torch.rand(E, generator=g, device=DEV)
    ids = keys.argsort(1, descending=True)[:, :k].to(I32)
    flat = ids.reshape(-1).to(I64)
    kept = flat < G
    order = torch.where(kept, flat, G).sort(stable=True).indices
    capacity = min(T * k, int(1.3 * T * k * G / E) + 8)
    R = min(int(kept.sum()), capacity)
    pos = torch.full((T * k,), -1, dtype=I32, device=DEV)
    pos[order[:R]] = torch.arange(R, dtype=I32, device=DEV)
    return pos.view(T, k), capacity


def _sort_outputs(T, k, G):
    return (torch.empty(G + 1, dtype=I64, device=DEV), torch.empty(T * k, dtype=I32, device=DEV),
            torch.empty(T, k, dtype=I32, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std
    kind, s = case["kind"], dict(case=case)
    if kind in ("route", "route_back"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        s["logits"] = (rn(T, E) + rn(E, std=0.5)).to(_dtype(case))
        s["ids"] = s["logits"].float().sort(dim=1, descending=True, stable=True).indices[:, :k].to(I32).contiguous()
        if kind == "route":
            s["weights"] = torch.empty(T, k, device=DEV)
            s["off"], s["src"], s["pos"] = _sort_outputs(T, k, case["local"])
            s["ids_out"] = torch.empty(T, k, dtype=I32, device=DEV)
            s["workspace"] = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
        else:
            s["dweights"] = rn(T, k)
            s["dlogits"] = torch.empty_like(s["logits"])
    elif kind in ("dispatch", "combine", "combine_back"):
        T, C, k = case["tokens"], case["cols"], case["topk"]
        s["pos"], R = _routing(case, g)
        if kind == "dispatch":
            s["x"] = rn(T, C).to(BF16)
            s["x"][:, torch.randperm(C, generator=g, device=DEV)[:max(1, C // 100)]] *= 50  # outlier channels
            s["q"] = torch.zeros(R, C, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros(R, C // 32, dtype=torch.uint8, device=DEV)
        else:
            s["rows"] = rn(R, C).to(_dtype(case))
            s["weights"] = torch.rand(T, k, generator=g, device=DEV) + 0.05
            s["weights"] /= s["weights"].sum(1, keepdim=True)
            if kind == "combine":
                s["y"] = torch.empty(T, C, dtype=_dtype(case), device=DEV)
            else:
                s["dy"] = rn(T, C, std=1e-3).to(_dtype(case))
                s["drows"], s["dweights"] = torch.zeros_like(s["rows"]), torch.empty_like(s["weights"])
    elif kind in ("loss", "loss_grad"):
        T, H, V = case["tokens"], case["hidden"], case["vocab"]
        s["x"] = rn(T, H).to(BF16)
        s["w"] = rn(V, H, std=1.5 / math.sqrt(H)).to(BF16)
        targets = torch.randint(0, V, (T,), generator=g, device=DEV)
        masked = torch.rand(T, generator=g, device=DEV) < case["ignored"]
        s["targets"] = torch.where(masked, -100, targets)
        s["loss"], s["lse"] = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        s["dloss"] = (~masked).float() / (~masked).sum().clamp(min=1)  # the mean over the tokens that count
        if kind == "loss_grad":
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        s["workspaces"] = {}
    else:
        n, r, c, m, v = case["matrices"], case["rows"], case["cols"], case["vectors"], case["length"]
        s["flat"] = [rn(n * r * c, std=1e-3).to(BF16), rn(m * v, std=1e-2)]
        s["grads"] = [*s["flat"][0].view(n, r, c).unbind(0), *s["flat"][1].view(m, v).unbind(0)]
        s["clipped"] = [torch.empty_like(f) for f in s["flat"]]
        s["out"] = [*s["clipped"][0].view(n, r, c).unbind(0), *s["clipped"][1].view(m, v).unbind(0)]
        s["norm"] = torch.empty(1, device=DEV)
        s["handles"] = {}
    return s


MAX_NORM = 1.0  # the usual clipping threshold


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import mxfp4_precision_numerics_amd as mxq
    case, kind = s["case"], s["case"]["kind"]
    if kind == "route":
        mxq.moe_topk(s["logits"], s["ids_out"], s["weights"], renormalize=case["renorm"])
        mxq.moe_sort(s["ids_out"], case["local"], s["off"], s["src"], s["pos"], s["workspace"])
        return s["ids_out"], s["weights"], s["off"], s["src"], s["pos"]
    if kind == "route_back":
        mxq.moe_topk_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], renormalize=case["renorm"])
        return s["dlogits"]
    if kind == "dispatch":
        mxq.moe_dispatch_mx(s["x"], s["pos"], mxq.E4M3, s["q"], s["scales"])
        return s["q"].view(torch.float8_e4m3fn), s["scales"].view(torch.float8_e8m0fnu)
    if kind == "combine":
        mxq.moe_combine(s["rows"], s["pos"], s["y"], weights=s["weights"] if case["weighted"] else None)
        return s["y"]
    if kind == "combine_back":
        mxq.moe_combine_backward(s["dy"], s["pos"], s["drows"], weights=s["weights"], rows=s["rows"],
                                 dweights=s["dweights"])
        return s["drows"], s["dweights"]
    if kind in ("loss", "loss_grad"):
        if not s["workspaces"]:  # sized once per shape, as a program keeps it
            size = mxq.linear_cross_entropy_workspace(case["tokens"], case["hidden"], case["vocab"],
                                                      backward=kind == "loss_grad")
            s["workspaces"]["w"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        ws = s["workspaces"]["w"]
        mxq.linear_cross_entropy(s["x"], s["w"], s["targets"], s["loss"], s["lse"], ws)
        if kind == "loss":
            return s["loss"], s["lse"]
        mxq.linear_cross_entropy_backward(s["x"], s["w"], s["targets"], s["lse"], s["dloss"], s["dx"], s["dw"], ws)
        return s["loss"], s["lse"], s["dx"], s["dw"]
    if not s["handles"]:
        s["handles"]["set"] = mxq.GradientSet(s["grads"], s["out"])
    s["handles"]["set"].clip(MAX_NORM, s["norm"])
    return s["norm"], s["clipped"]


def _take(table, pos):
    """Rows of `table` at `pos`, zero where pos is -1."""
    padded = torch.cat([table, table.new_zeros(1, *table.shape[1:])])
    return padded[torch.where(pos < 0, table.shape[0], pos.to(I64))]


def _plain(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind == "route":
        T, k, G = case["tokens"], case["topk"], case["local"]
        top = s["logits"].float().sort(dim=1, descending=True, stable=True)
        e = (top.values - top.values[:, :1]).exp()
        weights = e[:, :k] / (e[:, :k] if case["renorm"] else e).sum(1, keepdim=True)
        ids = top.indices[:, :k]
        flat = ids.reshape(-1)
        order = torch.where(flat < G, flat, G).sort(stable=True)
        off = torch.searchsorted(order.values, torch.arange(G + 1, device=DEV))
        row = torch.arange(T * k, device=DEV)
        in_group = row < off[-1]
        src = torch.where(in_group, order.indices // k, -1).to(I32)
        pos = torch.empty_like(src)
        pos[order.indices] = torch.where(in_group, row, -1).to(I32)
        return ids.to(I32), weights, off, src, pos.view(T, k)
    if kind == "route_back":
        z, ids, g = s["logits"].float(), s["ids"].to(I64), s["dweights"]
        if case["renorm"]:
            z = torch.full_like(z, -math.inf).scatter(1, ids, z.gather(1, ids))
        e = (z - z.amax(1, keepdim=True)).exp()
        p = e / e.sum(1, keepdim=True)
        full = torch.zeros_like(p).scatter(1, ids, g)
        return (p * (full - (full * p).sum(1, keepdim=True))).to(s["logits"].dtype)
    if kind == "dispatch":
        T, C, R = case["tokens"], case["cols"], s["q"].shape[0]
        b = s["x"].float().view(T, C // 32, 32)
        e = (torch.frexp(b.abs().amax(2)).exponent - 1 - 8).clamp(min=-127)
        q = torch.ldexp(b, -e[..., None]).clamp(-448, 448).view(T, C).to(torch.float8_e4m3fn).view(torch.uint8)
        at = s["pos"].reshape(-1).to(I64)
        token = torch.arange(at.numel(), device=DEV) // case["topk"]
        src = torch.full((R + 1,), -1, device=DEV).scatter(0, torch.where(at < 0, R, at), token)[:R]
        return _take(q, src).view(torch.float8_e4m3fn), _take((e + 127).to(torch.uint8), src).view(torch.float8_e8m0fnu)
    if kind == "combine":
        rows = _take(s["rows"].float(), s["pos"])
        return (rows * s["weights"][..., None] if case["weighted"] else rows).sum(1).to(s["rows"].dtype)
    if kind == "combine_back":
        dy, pos, R, C = s["dy"].float(), s["pos"], s["rows"].shape[0], case["cols"]
        dweights = (_take(s["rows"].float(), pos) * dy[:, None]).sum(2)
        drows = torch.zeros(R + 1, C, device=DEV)
        drows[torch.where(pos < 0, R, pos.to(I64)).reshape(-1)] = (s["weights"][..., None] * dy[:, None]).view(-1, C)
        return drows[:R].to(s["rows"].dtype), dweights
    if kind in ("loss", "loss_grad"):
        x, w, t = s["x"].float(), s["w"].float(), s["targets"]
        z = x @ w.t()
        m = z.amax(1, keepdim=True)
        lse = (z - m).exp().sum(1).log() + m[:, 0]
        valid, at = t >= 0, t.clamp(min=0)[:, None]
        loss = torch.where(valid, lse - z.gather(1, at)[:, 0], 0.0)
        if kind == "loss":
            return loss, lse
        g = (z - lse[:, None]).exp()
        g.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        g *= torch.where(valid, s["dloss"], 0.0)[:, None]
        return loss, lse, (g @ w).to(BF16), (g.t() @ x).to(BF16)
    flat = torch.cat([v.reshape(-1).float() for v in s["grads"]])
    norm = flat.double().square().sum().sqrt()
    coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    a = s["flat"][0].numel()
    return norm.float().view(1), [(flat[:a] * coef).to(BF16), flat[a:] * coef]


def work(case):
    kind = case["kind"]
    b = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if kind in ("route", "route_back"):
        n, k = case["tokens"] * case["experts"], case["tokens"] * case["topk"]
        if kind == "route":
            return {"bytes": n * b + k * 16 + (case["local"] + 1) * 8, "flops": 3 * n}
        return {"bytes": (1 if case["renorm"] else 2) * n * b + k * 8 + (n * b if case["renorm"] else 0), "flops": 6 * n}
    if kind in ("dispatch", "combine", "combine_back"):
        T, C, k = case["tokens"], case["cols"], case["topk"]
        R = T * k * case["local"] / case["experts"]  # the share that is local
        if kind == "dispatch":
            return {"bytes": 2 * T * C + R * C * (1 + 1 / 32) + T * k * 4, "flops": 4 * T * C}
        if kind == "combine":
            return {"bytes": R * C * b + T * C * b + T * k * 8, "flops": 2 * R * C}
        return {"bytes": T * C * b + 2 * R * C * b + T * k * 12, "flops": 3 * R * C}
    if kind in ("loss", "loss_grad"):
        T, H, V = case["tokens"], case["hidden"], case["vocab"]
        if kind == "loss":
            return {"bytes": 2 * (T + V) * H + 16 * T, "flops": 2 * T * H * V}
        return {"bytes": 4 * (T + V) * H + 20 * T, "flops": 6 * T * H * V}
    n, m = case["matrices"] * case["rows"] * case["cols"], case["vectors"] * case["length"]
    return {"bytes": 4 * n + 8 * m, "flops": 3 * (n + m)}


def exact(case, seed):
    """The definitions in 64 bits (whole numbers by counting, not by the sorts of the plain form)."""
    s, kind = prepare(case, seed), case["kind"]
    if kind == "route":
        T, k, G, E = case["tokens"], case["topk"], case["local"], case["experts"]
        z = s["logits"].double()
        ids = torch.empty(T, k, dtype=I32, device=DEV)
        left, index = z.clone(), torch.arange(E, device=DEV)
        for j in range(k):
            best = left.amax(1, keepdim=True)
            first = torch.where(left == best, index, E).amin(1)
            ids[:, j] = first.to(I32)
            left.scatter_(1, first[:, None], -math.inf)
        p = torch.softmax(z, 1).gather(1, ids.to(I64))
        weights = p / p.sum(1, keepdim=True) if case["renorm"] else p
        flat = ids.reshape(-1).to(I64)
        off = torch.zeros(G + 1, dtype=I64, device=DEV)
        src = torch.full((T * k,), -1, dtype=I32, device=DEV)
        pos = torch.full((T * k,), -1, dtype=I32, device=DEV)
        for e in range(G):
            at = (flat == e).nonzero()[:, 0]
            off[e + 1] = off[e] + at.numel()
            src[int(off[e]):int(off[e + 1])] = (at // k).to(I32)
            pos[at] = torch.arange(int(off[e]), int(off[e + 1]), dtype=I32, device=DEV)
        return ids, weights, off, src, pos.view(T, k)
    if kind == "route_back":
        z, ids = s["logits"].double().requires_grad_(), s["ids"].to(I64)
        p = torch.softmax(z, 1).gather(1, ids)
        p = p / p.sum(1, keepdim=True) if case["renorm"] else p
        p.backward(s["dweights"].double())
        return z.grad
    if kind == "dispatch":
        T, C, R = case["tokens"], case["cols"], s["q"].shape[0]
        b = s["x"].double().view(T, -1, 32)
        top = b.abs().amax(2)
        e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 8, -127.0).clamp(min=-127)
        v = b / torch.exp2(e)[..., None]
        mag = v.abs().clamp(max=448)
        step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
        q = (torch.round(mag / step) * step).clamp(max=448) * torch.sign(v)
        rows = torch.zeros(R, C, dtype=torch.float64, device=DEV)
        scales = torch.full((R, C // 32), 2.0 ** -127, dtype=torch.float64, device=DEV)  # an unused row's byte 0
        for j in range(case["topk"]):
            p = s["pos"][:, j].to(I64)
            rows[p[p >= 0]], scales[p[p >= 0]] = q.view(T, C)[p >= 0], torch.exp2(e)[p >= 0]
        return rows, scales
    if kind == "combine":
        y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            p = s["pos"][:, j].to(I64)
            at = (p >= 0).nonzero()[:, 0]
            w = s["weights"][at, j, None].double() if case["weighted"] else 1.0
            y[at] += w * s["rows"][p[at]].double()
        return y
    if kind == "combine_back":
        drows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=DEV)
        dweights = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            p = s["pos"][:, j].to(I64)
            at = (p >= 0).nonzero()[:, 0]
            dy = s["dy"][at].double()
            drows[p[at]] = s["weights"][at, j, None].double() * dy
            dweights[at, j] = (s["rows"][p[at]].double() * dy).sum(1)
        return drows, dweights
    if kind in ("loss", "loss_grad"):
        T, V = case["tokens"], case["vocab"]
        x, w, t = s["x"].double(), s["w"].double(), s["targets"]
        z = torch.mm(x, w.t().contiguous())
        lse = torch.logsumexp(z, 1)
        at = (t >= 0).nonzero()[:, 0]
        loss = torch.zeros(T, dtype=torch.float64, device=DEV)
        loss[at] = lse[at] - z[at, t[at]]
        if kind == "loss":
            return loss, lse
        z.sub_(lse[:, None]).exp_()
        z[at, t[at]] -= 1
        z.mul_(torch.where(t >= 0, s["dloss"], 0.0).double()[:, None])
        return loss, lse, torch.mm(z, w), torch.mm(z.t().contiguous(), x)
    norm = math.sqrt(sum(float((v.double() ** 2).sum()) for v in s["grads"]))
    coef = min(1.0, MAX_NORM / (norm + 1e-6))
    return torch.tensor([norm], dtype=torch.float64, device=DEV), [f.double() * coef for f in s["flat"]]
