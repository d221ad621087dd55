"""The Muon step of a sharded unit and the RMS norm of its blocks: cases, plain forms and 64-bit values.

Kinds of case:

* ``orthogonalize``: Newton-Schulz orthogonalisation of a list of matrices (the gathered momentum of a unit);
* ``momentum``: the ranks' bf16 gradient rows folded into a rank's window, its momentum, and the bf16 update;
* ``apply``: a rank's window of the orthogonalised matrices subtracted from the fp32 master weights;
* ``norm``: RMS norm of ``x + residual``, with an output of x's type or in 8 bits with a scale for each row;
* ``norm_backward``: its gradients.

``own`` selects the library's kernels (True) or the plain torch forms (False).
"""

import itertools
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS_NS = 1e-7
EPS_NORM = 1e-6
LR, MU, WD = 0.02, 0.95, 0.01
E4M3_MAX = 448.0

TINY = "256x1024,1024,1024x256,256"
BLK7 = "4096x4096,4096x4096,4096x4096,4096x4096,11008x4096,11008x4096,4096x11008"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the two matrices of the two-layer MLP unit: a small model's step, where each product is a few tiles and latency counts
        {"name": "orthogonalize tiny unit", "op": "orthogonalize", "shapes": "256x1024,1024x256", "type": "bf16"},
        # the key and value projections of the 70B block: few rows, long inner axis
        {"name": "orthogonalize 70B k, v", "op": "orthogonalize", "shapes": "1024x8192,1024x8192", "type": "bf16"},
        # matrices of odd sizes, wide and tall, gathered in fp32
        {"name": "orthogonalize odd sizes", "op": "orthogonalize", "shapes": "515x1373,2049x771,1000x1000", "type": "f32"},
        # every matrix of the 7B block: the ordinary step of a large unit
        {"name": "orthogonalize 7B block", "op": "orthogonalize", "shapes": BLK7, "type": "bf16"},
        # the MLP unit over 4 ranks, a middle rank
        {"name": "momentum tiny unit", "op": "momentum", "shapes": TINY, "F": 4, "rank": 1, "nesterov": True},
        # the 7B block's matrices over 8 ranks
        {"name": "momentum 7B block", "op": "momentum", "shapes": BLK7, "F": 8, "rank": 0, "nesterov": True},
        {"name": "apply tiny unit", "op": "apply", "shapes": TINY, "F": 4, "rank": 1},
        # the last rank of 8, whose window lies in the last matrix
        {"name": "apply 7B block", "op": "apply", "shapes": BLK7, "F": 8, "rank": 7},
        # one token through a norm of the 7B block
        {"name": "norm one token", "op": "norm", "rows": 1, "dim": 4096, "pitch": 4096, "type": "bf16", "residual": True, "bits8": False},
        # 8192 tokens, in 8 bits for the products that follow
        {"name": "norm 8192 tokens 8 bits", "op": "norm", "rows": 8192, "dim": 4096, "pitch": 4096, "type": "bf16", "residual": True, "bits8": True},
        # a ragged batch in fp32 whose rows are parts of wider ones
        {"name": "norm backward odd f32", "op": "norm_backward", "rows": 777, "dim": 1027, "pitch": 1100, "type": "f32", "residual": False},
        # a training batch of the 7B block, with the residual stream's gradient
        {"name": "norm backward 8192 tokens", "op": "norm_backward", "rows": 8192, "dim": 4096, "pitch": 4096, "type": "bf16", "residual": True},
    ]


def draw(rng):
    spread = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["orthogonalize", "momentum", "apply", "norm", "norm_backward"])
    if op == "orthogonalize":
        top = 0.6 * work(listed()[3])["flops"]
        while True:
            c = {"op": op, "type": rng.choice(["bf16", "f32"]),
                 "shapes": ",".join("%dx%d" % (spread(64, 11008), spread(64, 11008)) for _ in range(rng.randint(1, 6)))}
            if work(c)["flops"] <= top:
                return c
    if op in ("momentum", "apply"):
        F = rng.choice([1, 2, 4, 7, 8, 11, 16])
        while True:
            shapes = ["%dx%d" % (spread(64, 8192), spread(64, 8192)) for _ in range(rng.randint(1, 8))]
            if rng.random() < 0.3:
                shapes.insert(rng.randint(0, len(shapes)), str(spread(64, 8192)))
            c = {"op": op, "shapes": ",".join(shapes), "F": F, "rank": rng.randrange(F)}
            if sum(_numel(c)) * F <= 202_375_168 * 8:
                break
        return {**c, "nesterov": rng.random() < 0.7} if op == "momentum" else c
    dim = spread(64, 16384)
    c = {"op": op, "dim": dim, "type": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.6}
    c["rows"] = min(spread(1, 32768), max(1, 8192 * 2048 // dim))
    c["pitch"] = dim + (rng.randint(1, 200) if rng.random() < 0.4 else 0)
    return {**c, "bits8": rng.random() < 0.5} if op == "norm" else c


def _shapes(case):
    return [tuple(int(d) for d in s.split("x")) for s in case["shapes"].split(",")]


def _numel(case):
    return [math.prod(s) for s in _shapes(case)]


def _window(case):
    """This rank's slice of the unit laid end to end: begin and length."""
    total = sum(_numel(case))
    share = -(-total // case["F"])
    begin = case["rank"] * share
    return begin, max(0, min(share, total - begin))


def _scale(shape):
    """The step's scale for a matrix: sqrt(max(1, rows / columns)); 1 for anything else."""
    return math.sqrt(max(1.0, shape[0] / shape[1])) if len(shape) == 2 else 1.0


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _gradient(gen, r, c):
    """A momentum matrix: a few strong directions of falling strength over noise, as gradients of a batch are."""
    k = max(1, min(64, min(r, c) // 16))
    fall = torch.logspace(0, -1.5, k, device="cuda")
    return 1e-3 * ((_randn(gen, r, k) * fall) @ _randn(gen, k, c) * (2.0 / math.sqrt(k)) + 0.3 * _randn(gen, r, c))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if own:
        import sharded_flatparameter_flatten_amd as fsdp
        s["fsdp"] = fsdp
    if op == "orthogonalize":
        s["mats"] = [_gradient(gen, r, c).to(TYPES[case["type"]]) for r, c in _shapes(case)]
        if own:
            s["outs"] = [torch.empty(m.shape, dtype=torch.bfloat16, device="cuda") for m in s["mats"]]
            need = fsdp.orthogonalize_workspace(s["mats"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    elif op in ("momentum", "apply"):
        total = sum(_numel(case))
        begin, n = _window(case)
        if own:
            s["unit"] = fsdp.Unit(_shapes(case), case["F"], case["rank"])
        if op == "momentum":
            s["grads"] = [(1e-3 * _randn(gen, total)).to(torch.bfloat16) for _ in range(case["F"])]
            s["momentum"] = 1e-3 * _randn(gen, n)
            if own:
                s["update"] = torch.empty(n, dtype=torch.bfloat16, device="cuda")
                s["hp"] = fsdp.MuonHparams(lr=LR, momentum=MU, nesterov=case["nesterov"], weight_decay=WD)
        else:
            s["flat"] = (_randn(gen, total) / 64).to(torch.bfloat16)
            s["tensors"] = list(torch.split(s["flat"], _numel(case)))
            s["scales"] = [_scale(shape) for shape in _shapes(case)]
            s["master"] = 0.02 * _randn(gen, n)
            if own:
                s["param"] = torch.empty(n, dtype=torch.bfloat16, device="cuda")
                s["hp"] = fsdp.MuonHparams(lr=LR, momentum=MU, nesterov=True, weight_decay=WD)
    else:
        rows, dim, pitch, t = case["rows"], case["dim"], case["pitch"], TYPES[case["type"]]
        rows_of = lambda scale: (scale * _randn(gen, rows, pitch)).to(t)[:, :dim]  # noqa: E731
        empty = lambda t: torch.empty(rows, dim, dtype=t, device="cuda")  # noqa: E731
        s["weight"] = (1.0 + 0.1 * _randn(gen, dim)).to(t)
        s["x"] = rows_of(1.0)
        s["x"][:, :: max(1, dim // 7)] *= 20.0  # a few channels of a hidden state are far larger than the others
        if op == "norm":
            s["residual"] = rows_of(2.0) if case["residual"] else None
            if own:
                s["sum"] = empty(t) if case["residual"] else None
                s["out"] = empty(torch.float8_e4m3fn if case["bits8"] else t)
                s["scales"] = torch.empty(rows, device="cuda") if case["bits8"] else None
                s["rstd"] = torch.empty(rows, device="cuda")
        else:
            s["dy"] = rows_of(1e-2)
            s["dresidual"] = rows_of(1e-2) if case["residual"] else None
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS_NORM).float()
            if own:
                s["dx"], s["dweight"] = empty(t), torch.empty(dim, dtype=t, device="cuda")
                need = fsdp.rms_norm_backward_workspace(rows, dim)
                s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["case"]["op"]](s)


# --- the library's operators, as a training step calls them -----------------------------------------------------------


def _own_orthogonalize(s):
    s["fsdp"].orthogonalize(s["mats"], s["outs"], s["workspace"], steps=STEPS, coeffs=COEFFS, eps=EPS_NS)
    return s["outs"]


def _own_momentum(s):
    s["fsdp"].reduce_momentum_shard(s["unit"], s["grads"], s["momentum"], s["update"], s["hp"])
    return {"momentum": s["momentum"], "update": s["update"]}


def _own_apply(s):
    s["fsdp"].muon_apply_shard(s["unit"], s["tensors"], s["scales"], s["master"], s["param"], s["hp"])
    return {"master": s["master"], "param": s["param"]}


def _own_norm(s):
    s["fsdp"].rms_norm(s["x"], s["weight"], s["out"], eps=EPS_NORM, residual=s["residual"], residual_out=s["sum"],
                       rstd=s["rstd"], scales=s["scales"])
    return {"out": s["out"], "rstd": s["rstd"], "sum": s["sum"], "scales": s["scales"]}


def _own_norm_backward(s):
    s["fsdp"].rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], s["dweight"], s["workspace"],
                                dresidual=s["dresidual"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


# --- the plain forms, in 32 bits --------------------------------------------------------------------------------------


def _newton_schulz(g):
    a, b, c = COEFFS
    x = g.float()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (torch.linalg.vector_norm(x, dtype=torch.float64) + EPS_NS).float()
    for _ in range(STEPS):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.T if tall else x).to(torch.bfloat16).contiguous()


def _plain_orthogonalize(s):
    return [_newton_schulz(g) for g in s["mats"]]


def _plain_momentum(s):
    begin, n = _window(s["case"])
    g = torch.stack([row[begin:begin + n] for row in s["grads"]]).float().sum(0) * (1.0 / len(s["grads"]))
    m = s["momentum"].mul_(MU).add_(g)
    return {"momentum": m, "update": (g + MU * m if s["case"]["nesterov"] else m).to(torch.bfloat16)}


def _plain_apply(s):
    begin, n = _window(s["case"])
    ends = list(itertools.accumulate(_numel(s["case"])))
    part = lambda t, end: t.reshape(-1)[max(0, begin - end + t.numel()):max(0, begin + n - end + t.numel())]  # noqa: E731
    u = torch.cat([k * part(t, end).float() for k, t, end in zip(s["scales"], s["tensors"], ends)])
    p = s["master"]
    p.sub_(LR * (u + WD * p))
    return {"master": p, "param": p.to(torch.bfloat16)}


def _plain_norm(s):
    t = s["x"].dtype
    h = s["x"].float()
    total = None
    if s["residual"] is not None:
        total = (h + s["residual"].float()).to(t)
        h = total.float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS_NORM)
    y = h * rstd[:, None] * s["weight"].float()
    scales = None
    if s["case"]["bits8"]:
        scales = (y.abs().amax(1) / E4M3_MAX).clamp_min(2.0 ** -126)
        out = (y / scales[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    else:
        out = y.to(t)
    return {"out": out, "rstd": rstd, "sum": total, "scales": scales}


def _plain_norm_backward(s):
    t, dim = s["x"].dtype, s["case"]["dim"]
    dy = s["dy"].float()
    xhat = s["x"].float() * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - xhat * ((g * xhat).sum(1, keepdim=True) / dim))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(t), "dweight": (dy * xhat).sum(0).to(t)}


_RUN_OWN = {"orthogonalize": _own_orthogonalize, "momentum": _own_momentum, "apply": _own_apply, "norm": _own_norm,
            "norm_backward": _own_norm_backward}
_RUN_PLAIN = {"orthogonalize": _plain_orthogonalize, "momentum": _plain_momentum, "apply": _plain_apply, "norm": _plain_norm,
              "norm_backward": _plain_norm_backward}


# --- the definitions in 64 bits ---------------------------------------------------------------------------------------


def _exact_polar(g):
    """The composed polynomial acts on the small side's Gram matrix S alone: X_k = Q_k X_0 with Q_0 = I,
    A_k = Q_k S Q_k (all are polynomials of S and commute) and Q_(k+1) = (a + b A_k + c A_k^2) Q_k."""
    g = g.double()
    tall = g.size(0) > g.size(1)
    x = (g.mT if tall else g).contiguous()
    x = x / (x.square().sum().sqrt() + EPS_NS)
    gram = torch.mm(x, x.mT.contiguous())
    eye = torch.eye(len(x), dtype=torch.float64, device=x.device)
    q = eye
    for _ in range(STEPS):
        ak = torch.mm(torch.mm(q, gram), q)
        q = torch.mm(torch.addmm(COEFFS[1] * ak + COEFFS[0] * eye, ak, ak, alpha=COEFFS[2]), q)
    x = torch.mm(q, x)
    return x.mT.contiguous() if tall else x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "orthogonalize":
        return [_exact_polar(g) for g in s["mats"]]
    if op in ("momentum", "apply"):
        begin, n = _window(case)
        here = slice(begin, begin + n)
        if op == "momentum":
            mean = torch.zeros(n, dtype=torch.float64, device="cuda")
            for row in s["grads"]:
                mean += row[here].double() / case["F"]
            m = s["momentum"].double() * MU + mean
            return {"momentum": m, "update": mean + m * MU if case["nesterov"] else m}
        flat = torch.empty(sum(_numel(case)), dtype=torch.float64, device="cuda")
        at = 0
        for k, t in zip(s["scales"], s["tensors"]):
            flat[at:at + t.numel()] = t.double().reshape(-1) * k
            at += t.numel()
        p = s["master"].double()
        p = p * (1.0 - LR * WD) - flat[here] * LR
        return {"master": p, "param": p}
    x, w, dim = s["x"].double(), s["weight"].double(), case["dim"]
    if op == "norm":
        h = x if s["residual"] is None else (x + s["residual"].double()).to(s["x"].dtype).double()
        rstd = 1.0 / (h.pow(2).sum(1) / dim + EPS_NORM).sqrt()
        y = h * torch.outer(rstd, w)
        scales = y.abs().max(1).values / E4M3_MAX if case["bits8"] else None
        return {"out": y / scales[:, None] if case["bits8"] else y, "rstd": rstd,
                "sum": None if s["residual"] is None else h, "scales": scales}
    r = s["rstd"].double()[:, None]
    dy = s["dy"].double()
    dot = (dy * w * x).sum(1, keepdim=True) * r ** 3 / dim
    dx = dy * w * r - x * dot
    if s["dresidual"] is not None:
        dx += s["dresidual"].double()
    return {"dx": dx, "dweight": (x * r * dy).sum(0)}


def work(case):
    """Inputs read once and outputs written once; a symmetric product counts each of its values once."""
    op = case["op"]
    if op == "orthogonalize":
        size = {"bf16": 2, "f32": 4}[case["type"]]
        ends = [(min(s), max(s)) for s in _shapes(case)]
        return {"bytes": sum((size + 2) * m * n for m, n in ends),
                "flops": STEPS * sum(m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n for m, n in ends)}
    if op in ("momentum", "apply"):
        n = _window(case)[1]
        return {"bytes": max(1, n * (2 * case["F"] + 10 if op == "momentum" else 12)), "flops": n * (case["F"] + 5 if op == "momentum" else 4)}
    e, t = case["rows"] * case["dim"], 2 if case["type"] == "bf16" else 4
    if op == "norm":
        per = t + (2 * t if case["residual"] else 0) + (1 if case["bits8"] else t)
        return {"bytes": e * per + case["dim"] * t + case["rows"] * (8 if case["bits8"] else 4), "flops": 4 * e}
    return {"bytes": e * t * (4 if case["residual"] else 3) + 2 * case["dim"] * t + 4 * case["rows"], "flops": 8 * e}
