"""More operators around one MoE layer, as they are measured: the whole layer for a few tokens, with the experts'
weights in bf16 or in 4 bits with a scale for each 32 values, and the step of an optimiser that orthogonalises each
matrix's update by Newton-Schulz products.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's calls.  A case's
``op`` names the operator.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one token of a decoding stream: the router's choice among 64 experts, and eight experts read for one row each
        {"name": "moe one token", "op": "moe", "weights": "bf16", "tokens": 1, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "score": "sigmoid", "bias": True, "normalize": True, "closed": 0.0, "activation": "silu"},
        # a small layer: launches and latencies count
        {"name": "moe tiny", "op": "moe", "weights": "bf16", "tokens": 4, "hidden": 256, "inter": 512, "experts": 8,
         "top_k": 2, "score": "softmax", "bias": False, "normalize": True, "closed": 0.0, "activation": "silu"},
        # odd sizes: partial tiles in every direction, closed experts
        {"name": "moe odd", "op": "moe", "weights": "bf16", "tokens": 13, "hidden": 2056, "inter": 1000, "experts": 24,
         "top_k": 3, "score": "softmax", "bias": False, "normalize": False, "closed": 0.8, "activation": "gelu"},
        # a small decoding batch: nearly every expert is read
        {"name": "moe batch", "op": "moe", "weights": "bf16", "tokens": 32, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "score": "sigmoid", "bias": True, "normalize": True, "closed": 0.0, "activation": "silu"},
        # the same three with the weights in 4 bits, the batch at its largest
        {"name": "moe 4 bit one token", "op": "moe", "weights": "mxfp4", "tokens": 1, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "score": "sigmoid", "bias": True, "normalize": True, "closed": 0.0, "activation": "silu"},
        {"name": "moe 4 bit odd", "op": "moe", "weights": "mxfp4", "tokens": 7, "hidden": 2080, "inter": 992, "experts": 24,
         "top_k": 3, "score": "softmax", "bias": False, "normalize": True, "closed": 0.8, "activation": "gelu"},
        {"name": "moe 4 bit batch", "op": "moe", "weights": "mxfp4", "tokens": 64, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "score": "sigmoid", "bias": True, "normalize": True, "closed": 0.0, "activation": "silu"},
        # the gate and up matrices of a small layer, one call
        {"name": "orthogonalize tiny", "op": "orthogonalize", "batch": 16, "rows": 512, "cols": 256, "input": "bfloat16",
         "rank": 16},
        # odd sizes, wide
        {"name": "orthogonalize odd", "op": "orthogonalize", "batch": 6, "rows": 777, "cols": 1001, "input": "float32",
         "rank": 40},
        # a layer's small projections: matrices of several shapes, an odd one among them
        {"name": "muon small", "op": "muon", "shapes": "1x512x2048,1x2048x512,2x1000x300,1x1024x1024", "param": "bfloat16",
         "grad": "bfloat16", "copy": False, "rank": 64},
        # gate and up matrices of eight experts: float32 masters, bf16 gradients and working copy
        {"name": "muon gate up", "op": "muon", "shapes": "16x2048x7168", "param": "float32", "grad": "bfloat16", "copy": True,
         "rank": 256},
        # their down matrices
        {"name": "muon down", "op": "muon", "shapes": "8x7168x2048", "param": "float32", "grad": "bfloat16", "copy": True,
         "rank": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "moe", "moe4", "moe4", "orthogonalize", "muon"])
    if op == "orthogonalize":
        rows, cols = _log(rng, 16, 4000), _log(rng, 16, 4000)
        batch = _log(rng, 1, max(1, min(64, int(1e8 / (rows * cols)))))
        return {"op": op, "batch": batch, "rows": rows, "cols": cols, "input": rng.choice(["float32", "bfloat16"]),
                "rank": _log(rng, 1, min(rows, cols))}
    if op == "muon":
        shapes = []
        for _ in range(rng.randint(1, 5)):
            rows, cols = _log(rng, 16, 3500), _log(rng, 16, 3500)
            shapes.append("%dx%dx%d" % (_log(rng, 1, max(1, min(24, int(2e7 / (rows * cols))))), rows, cols))
        param = rng.choice(["float32", "bfloat16"])
        return {"op": op, "shapes": ",".join(shapes), "param": param, "grad": rng.choice(["float32", "bfloat16"]),
                "copy": param == "float32" and rng.random() < 0.5, "rank": _log(rng, 1, 256)}
    experts = _log(rng, 1, 256)
    top_k = rng.randint(1, min(8, experts))
    unit = 32 if op == "moe4" else 8
    hidden, inter = unit * _log(rng, 64 // unit, 7168 // unit), unit * _log(rng, 64 // unit, 2400 // unit)
    while experts * hidden * inter * 3 > 2.8e9:
        hidden, inter = max(64, hidden // (2 * unit) * unit), max(64, inter // (2 * unit) * unit)
    score = rng.choice(["softmax", "sigmoid"])
    return {"op": "moe", "weights": "mxfp4" if op == "moe4" else "bf16", "tokens": _log(rng, 1, 64), "hidden": hidden,
            "inter": inter, "experts": experts, "top_k": top_k, "score": score,
            "bias": score == "sigmoid" and rng.random() < 0.5, "normalize": rng.random() < 0.7,
            "closed": rng.choice([0.0, 0.1, 0.7]), "activation": rng.choice(["silu", "gelu"])}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _encode(w):
    """4-bit codes, two a byte with the lower index in the lower half, and an exponent byte for each 32 values of a
    float32 matrix: the least power of two under which none is larger than 6, ties of a value to the even code."""
    blocks = w.view(*w.shape[:-1], -1, 32)
    mantissa, exponent = torch.frexp(blocks.abs().amax(-1))             # top = mantissa * 2^exponent, mantissa in [1/2, 1)
    e = exponent - 3 + (mantissa > 0.75).to(exponent.dtype)             # 6 = 0.75 * 2^3
    x = torch.ldexp(blocks, -e.unsqueeze(-1))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    a = x.abs().contiguous()
    up, down = torch.bucketize(a, edges, right=True), torch.bucketize(a, edges)
    code = torch.where(up % 2 == 0, up, down) + 8 * (x < 0)
    code = code.view(*w.shape[:-1], -1, 2).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _experts(c, g, rows, cols):
    """The experts' matrices [experts, rows, cols], or their codes and scales."""
    E = c["experts"]
    if c["weights"] == "bf16":
        return _normal(g, (E, rows, cols), cols ** -0.5)
    codes = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, rows, cols // 32, dtype=torch.uint8, device=DEV)
    for e in range(E):
        codes[e], scales[e] = _encode(_normal(g, (rows, cols), cols ** -0.5, torch.float32))
    return codes, scales


def _prepare_moe(c, g):
    T, E, H, I = c["tokens"], c["experts"], c["hidden"], c["inter"]
    logits = _normal(g, (T, E), 2.0, torch.float32)
    if c["closed"] > 0:
        logits.masked_fill_(torch.rand(T, E, device=DEV, generator=g) < c["closed"], float("-inf"))
    s = {"op": "moe", "case": c, "logits": logits, "x": _normal(g, (T, H)),
         "bias": _normal(g, (E,), 0.1, torch.float32) if c["bias"] else None,
         "scale": 2.5 if c["score"] == "sigmoid" else 1.0,
         "w_gate_up": _experts(c, g, 2 * I, H), "w_down": _experts(c, g, H, I)}
    return s


def _gradient(g, batch, rows, cols, rank):
    """Matrices like an update's: a few strong directions over noise."""
    r = max(1, min(rank, rows, cols))
    strength = torch.arange(1, r + 1, device=DEV).float() ** -0.5
    m = torch.bmm(_normal(g, (batch, rows, r), 1.0, torch.float32) * strength, _normal(g, (batch, r, cols), 1.0, torch.float32))
    return m.add_(_normal(g, (batch, rows, cols), 0.5, torch.float32)).mul_(1e-3)


def _prepare_orthogonalize(c, g):
    x = _gradient(g, c["batch"], c["rows"], c["cols"], c["rank"])
    return {"op": "orthogonalize", "case": c, "x": x.to(getattr(torch, c["input"]))}


def _shapes(c):
    return [tuple(int(n) for n in s.split("x")) for s in c["shapes"].split(",")]


def _prepare_muon(c, g):
    s = {"op": "muon", "case": c, "params": [], "grads": [], "momenta": [], "copies": [] if c["copy"] else None}
    for shape in _shapes(c):
        s["params"].append(_normal(g, shape, 0.02, getattr(torch, c["param"])))
        s["grads"].append(_gradient(g, *shape, c["rank"]).to(getattr(torch, c["grad"])))
        s["momenta"].append(_gradient(g, *shape, c["rank"]))
        if c["copy"]:
            s["copies"].append(torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
    return s


def prepare(case, seed):
    g = _generator(seed)
    return {"moe": _prepare_moe, "orthogonalize": _prepare_orthogonalize, "muon": _prepare_muon}[case["op"]](case, g)


HYPER = {"lr": 3e-4, "momentum": 0.95, "weight_decay": 0.1, "steps": 5}
COEFFICIENTS = (3.4445, -4.775, 2.0315)


# -------------------------------------------------------------- plain forms --

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode(codes, scales):
    """float32 values of 4-bit codes [..., n / 2] and their exponents [..., n / 32]."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = table[both.int()]
    scale = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return (v.view(*scales.shape, 32) * scale.unsqueeze(-1)).flatten(-2)


def _matrices(w, which=None):
    """The experts' matrices in float32, all or those of `which`."""
    if isinstance(w, tuple):
        return _decode(*w) if which is None else _decode(w[0][which], w[1][which])
    return (w if which is None else w[which]).float()


def _act(x, kind):
    if kind == "silu":
        return x / (1.0 + torch.exp(-x))
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _choice(s):
    """The chosen experts (-1: none) and their weights."""
    c, logits = s["case"], s["logits"]
    K = c["top_k"]
    is_open = logits > float("-inf")
    key = logits.double()               # the order next to a border needs more than 32 bits
    if c["score"] == "sigmoid":
        key = 1.0 / (1.0 + torch.exp(-key))
        if s["bias"] is not None:
            key = key + s["bias"].double()
    key = torch.where(is_open, key, torch.full_like(key, float("-inf")))
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    chosen = torch.gather(is_open, 1, idx)
    if c["score"] == "softmax":
        top = logits.amax(1, keepdim=True)
        e = torch.where(is_open, torch.exp(logits - torch.where(top > float("-inf"), top, torch.zeros_like(top))),
                        torch.zeros_like(logits))
        p = e / e.sum(1, keepdim=True).clamp_min(1e-30)
    else:
        p = torch.where(is_open, 1.0 / (1.0 + torch.exp(-logits)), torch.zeros_like(logits))
    w = torch.gather(p, 1, idx)
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
    return torch.where(chosen, idx, torch.full_like(idx, -1)), w * s["scale"]


def _plain_moe(s):
    c, x = s["case"], s["x"].float()
    T, E, K, I, H = c["tokens"], c["experts"], c["top_k"], c["inter"], c["hidden"]
    idx, w = _choice(s)
    if T * K <= E:          # few tokens: the matrices of each slot
        which = idx.clamp_min(0).flatten()
        rows = x.repeat_interleave(K, 0).unsqueeze(2)
        gu = torch.bmm(_matrices(s["w_gate_up"], which), rows).squeeze(2)
        o = torch.bmm(_matrices(s["w_down"], which), (_act(gu[:, :I], c["activation"]) * gu[:, I:]).unsqueeze(2))
        y = (o.view(T, K, H) * w.unsqueeze(2)).sum(1)
    else:                   # every expert on every token, weighted by the choice
        gu = torch.matmul(_matrices(s["w_gate_up"]), x.t())
        o = torch.bmm(_matrices(s["w_down"]), _act(gu[:, :I], c["activation"]) * gu[:, I:])     # [E, H, T]
        share = torch.zeros(T, E, device=x.device).scatter_add_(1, idx.clamp_min(0), torch.where(idx >= 0, w, torch.zeros_like(w)))
        y = (o * share.t().unsqueeze(1)).sum(0).t()
    return {"y": y.contiguous().to(torch.bfloat16), "topk_idx": idx.to(torch.int32), "topk_weights": w}


def _newton_schulz(x):
    """x [batch, rows, cols] in float32: `steps` times a x + (b g + c g g) x with g = x x^T, from x over its norm."""
    a, b, c = COEFFICIENTS
    wide = x.shape[1] <= x.shape[2]
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + 1e-7)
    x = x if wide else x.transpose(1, 2).contiguous()
    for _ in range(HYPER["steps"]):
        g = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * g + c * torch.bmm(g, g), x)
    return x if wide else x.transpose(1, 2)


def _plain_orthogonalize(s):
    return {"out": _newton_schulz(s["x"].float()).contiguous().to(torch.bfloat16)}


def _plain_matrix_step(s, i):
    h, p, m, g = HYPER, s["params"][i], s["momenta"][i], s["grads"][i].float()
    m.copy_(h["momentum"] * m + (1.0 - h["momentum"]) * g)
    u = _newton_schulz((1.0 - h["momentum"]) * g + h["momentum"] * m)
    new = p.float() * (1.0 - h["lr"] * h["weight_decay"]) - h["lr"] * 0.2 * math.sqrt(max(p.shape[1:])) * u
    p.copy_(new)
    if s["copies"] is not None:
        s["copies"][i].copy_(new)


def _plain_muon(s):
    [_plain_matrix_step(s, i) for i in range(len(s["params"]))]


# ---------------------------------------------------- the framework's calls --

def _own_moe(s):
    import combine_ep_layout_amd as ep
    c = s["case"]
    up, down = (ep.Mxfp4(*w) if isinstance(w, tuple) else w for w in (s["w_gate_up"], s["w_down"]))
    y, idx, w = ep.moe_tokens(s["x"], up, down, logits=s["logits"], top_k=c["top_k"], score=c["score"], bias=s["bias"],
                              normalize=c["normalize"], scale=s["scale"], activation=c["activation"])
    return {"y": y, "topk_idx": idx, "topk_weights": w}


def _own_orthogonalize(s):
    import combine_ep_layout_amd as ep
    return {"out": ep.orthogonalize(s["x"], steps=HYPER["steps"], coefficients=COEFFICIENTS)}


def _own_muon(s):
    import combine_ep_layout_amd as ep
    ep.muon(s["params"], s["grads"], s["momenta"], copies=s["copies"], coefficients=COEFFICIENTS, **HYPER)


def run(state):
    op = state["op"]
    if op == "moe":
        return _own_moe(state) if own else _plain_moe(state)
    if op == "orthogonalize":
        return _own_orthogonalize(state) if own else _plain_orthogonalize(state)
    if own:
        _own_muon(state)
    else:
        _plain_muon(state)
    return {k: state[k] for k in ("params", "momenta", "copies")}


# -------------------------------------------------------------------- work --

def _products(batch, rows, cols):
    """Multiplications and additions of the steps: x x^T and g g are symmetric."""
    m, n = min(rows, cols), max(rows, cols)
    return batch * HYPER["steps"] * (m * m * n + m * m * m + 2.0 * m * m * n)


def work(case):
    c = case
    if c["op"] == "orthogonalize":
        n = c["batch"] * c["rows"] * c["cols"]
        return {"bytes": n * (4 if c["input"] == "float32" else 2) + n * 2, "flops": _products(c["batch"], c["rows"], c["cols"])}
    if c["op"] == "muon":
        n = sum(b * r * k for b, r, k in _shapes(c))
        each = 8 + (8 if c["param"] == "float32" else 4) + (4 if c["grad"] == "float32" else 2) + (2 if c["copy"] else 0)
        return {"bytes": n * each, "flops": sum(_products(*t) for t in _shapes(c))}
    T, H, I, E, K = c["tokens"], c["hidden"], c["inter"], c["experts"], c["top_k"]
    k = min(K, E * (1.0 - c["closed"]))                         # open slots of a token, about
    used = E * (1.0 - (1.0 - k / E) ** T)                       # experts with a row, for even routing
    each = 3.0 * H * I * (2 if c["weights"] == "bf16" else 0.5 + 1 / 32)
    return {"bytes": used * each + T * (4 * H + 4 * E + 8 * K), "flops": 6.0 * T * k * H * I}


# ------------------------------------------------------------ in 64 bits --

def _exact_matrix(w, e):
    """One expert's matrix in float64; a code's value from its sign, exponent and mantissa bits."""
    if not isinstance(w, tuple):
        return w[e].double()
    codes, scales = w[0][e].long(), w[1][e].double()
    n = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    n[:, 0::2] = codes.remainder(16)
    n[:, 1::2] = codes.div(16, rounding_mode="floor")
    exponent, mantissa = (n % 8).div(2, rounding_mode="floor"), n % 2
    v = torch.where(exponent > 0, (2 + mantissa).double() * 2.0 ** (exponent - 2).double(), mantissa.double() / 2)
    return torch.where(n >= 8, -v, v) * (2.0 ** (scales - 127.0)).repeat_interleave(32, 1)


def _exact_moe(s):
    c = s["case"]
    f = torch.nn.functional
    l, x, I = s["logits"].double(), s["x"].double(), c["inter"]
    shut = torch.isinf(l)
    if c["score"] == "softmax":
        some = ~shut.all(1, keepdim=True)
        rank = l.clone()
        p = torch.softmax(torch.where(some, l, torch.zeros_like(l)), 1) * ~shut
    else:
        p = torch.sigmoid(l) * ~shut
        rank = p + (0 if s["bias"] is None else s["bias"].double())
    rank[shut] = float("-inf")
    idx = rank.argsort(dim=1, descending=True, stable=True)[:, :c["top_k"]]
    w = p.gather(1, idx)
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    w = w * s["scale"]
    idx = idx.masked_fill(shut.gather(1, idx), -1)
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in sorted(set(idx.flatten().tolist()) - {-1}):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        gu = f.linear(x[t], _exact_matrix(s["w_gate_up"], e))
        a = (f.silu(gu[:, :I]) if c["activation"] == "silu" else f.gelu(gu[:, :I], approximate="tanh")) * gu[:, I:]
        y.index_add_(0, t, f.linear(a, _exact_matrix(s["w_down"], e)) * w[t, k].unsqueeze(1))
    return {"y": y, "topk_idx": idx.to(torch.int32), "topk_weights": w}


def _exact_newton_schulz(x):
    """The same polynomial of the singular values with the powers on the other side: x (a + (b + c k) k), k = x^T x,
    over the shorter side."""
    a, b, c = COEFFICIENTS
    tall = x if x.shape[-2] >= x.shape[-1] else x.mT.contiguous()
    tall = tall / (torch.linalg.matrix_norm(tall, keepdim=True) + 1e-7)
    one = torch.eye(tall.shape[-1], dtype=torch.float64, device=x.device)
    for _ in range(HYPER["steps"]):
        k = tall.mT.contiguous() @ tall
        tall = tall @ (a * one + (b * one + c * k) @ k)
    return tall if x.shape[-2] >= x.shape[-1] else tall.mT


def _exact_muon(s):
    h, out = HYPER, {"params": [], "momenta": []}
    if s["copies"] is not None:
        out["copies"] = []
    for p, g, m in zip(s["params"], s["grads"], s["momenta"]):
        m1 = torch.lerp(m.double(), g.double(), 1.0 - h["momentum"])
        o = torch.stack([_exact_newton_schulz(u) for u in torch.lerp(g.double(), m1, h["momentum"])])
        p1 = p.double() - h["lr"] * (h["weight_decay"] * p.double() + 0.2 * max(p.shape[1:]) ** 0.5 * o)
        out["params"].append(p1)
        out["momenta"].append(m1)
        if s["copies"] is not None:
            out["copies"].append(p1)
    return out


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "moe":
        return _exact_moe(s)
    if case["op"] == "orthogonalize":
        return {"out": torch.stack([_exact_newton_schulz(x.double()) for x in s["x"]])}
    return _exact_muon(s)
