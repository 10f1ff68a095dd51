"""The operators around one MoE layer's dispatch and combine, as they are measured:
the router, the experts' gated feed-forward over the dispatched pool, its training
form with the backward pass, and the AdamW step over many tensors.

``own`` chooses between the plain form (elementary torch operations in 32 bits)
and the framework's calls.  A case's ``op`` names the operator.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # router of a decoding step: sigmoid scores, a selection bias, float32 logits
        {"name": "route decode", "op": "route", "train": False, "tokens": 256, "experts": 256, "top_k": 8,
         "score": "sigmoid", "bias": True, "normalize": True, "logits": "float32", "closed": 0.0},
        # router of a training step over the prefill batch, with the gradient of its logits
        {"name": "route train", "op": "route", "train": True, "tokens": 16384, "experts": 256, "top_k": 8,
         "score": "softmax", "bias": False, "normalize": True, "logits": "float32", "closed": 0.02},
        # one token of a decoding stream: eight experts read for one row each
        {"name": "ffn one token", "op": "ffn", "train": False, "tokens": 1, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "block_m": 64, "routing": "uniform", "masked": 0.0, "activation": "silu"},
        # a decoding batch: every expert's weights read for some 32 rows
        {"name": "ffn decode", "op": "ffn", "train": False, "tokens": 256, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "block_m": 64, "routing": "uniform", "masked": 0.0, "activation": "silu"},
        # odd sizes: a ragged batch, partial tiles in every direction, masked slots, tiles of 100 rows
        {"name": "ffn odd", "op": "ffn", "train": False, "tokens": 777, "hidden": 2056, "inter": 1000, "experts": 24,
         "top_k": 3, "block_m": 100, "routing": "zipf", "masked": 0.05, "activation": "gelu"},
        # prompt processing: 16384 tokens over 256 unevenly loaded experts
        {"name": "ffn prefill", "op": "ffn", "train": False, "tokens": 16384, "hidden": 7168, "inter": 2048, "experts": 256,
         "top_k": 8, "block_m": 128, "routing": "zipf", "masked": 0.0, "activation": "silu"},
        # a small layer trained on a small batch: launches and latencies count
        {"name": "train tiny", "op": "ffn", "train": True, "tokens": 128, "hidden": 256, "inter": 512, "experts": 8,
         "top_k": 2, "block_m": 16, "routing": "uniform", "masked": 0.0, "activation": "silu"},
        # a ragged training batch over odd widths, unevenly loaded
        {"name": "train odd", "op": "ffn", "train": True, "tokens": 1999, "hidden": 2008, "inter": 1096, "experts": 12,
         "top_k": 4, "block_m": 64, "routing": "zipf", "masked": 0.1, "activation": "silu"},
        # one GPU's share of a training step: 32 experts, 2048 rows each
        {"name": "train share", "op": "ffn", "train": True, "tokens": 8192, "hidden": 7168, "inter": 2048, "experts": 32,
         "top_k": 8, "block_m": 128, "routing": "uniform", "masked": 0.0, "activation": "silu"},
        # the experts' tensors of a layer: float32 masters and states, bf16 gradients, bf16 working copy
        {"name": "adamw experts", "op": "adamw", "tensors": 16, "smallest": 7340032, "largest": 14680064, "state": "float32",
         "param": "float32", "grad": "bfloat16", "copy": True},
        # the same with the states in 8 bits
        {"name": "adamw 8 bit", "op": "adamw", "tensors": 16, "smallest": 7340032, "largest": 14680064, "state": "8bit",
         "param": "float32", "grad": "bfloat16", "copy": True},
        # norms, biases and small projections of a model: many short tensors of odd lengths
        {"name": "adamw many", "op": "adamw", "tensors": 300, "smallest": 1, "largest": 30000, "state": "float32",
         "param": "bfloat16", "grad": "bfloat16", "copy": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "ffn", "ffn", "train", "adamw"])
    if op == "route":
        experts = _log(rng, 2, 1024)
        score, top_k = rng.choice(["softmax", "sigmoid"]), rng.randint(1, min(16, experts))
        return {"op": "route", "train": rng.random() < 0.5, "tokens": _log(rng, 1, 16384), "experts": experts,
                "top_k": top_k, "score": score, "bias": score == "sigmoid" and rng.random() < 0.5,
                "normalize": top_k > 1 and rng.random() < 0.7,      # one weight alone, normalised, is a constant
                "logits": rng.choice(["float32", "bfloat16"]), "closed": rng.choice([0.0, 0.1, 0.7])}
    if op == "adamw":
        tensors = _log(rng, 1, 400)
        top = max(64, min(16000000, 120000000 // tensors))
        largest = _log(rng, 64, top)
        param = rng.choice(["float32", "bfloat16"])
        return {"op": "adamw", "tensors": tensors, "smallest": _log(rng, 1, largest), "largest": largest,
                "state": rng.choice(["float32", "8bit"]), "param": param, "grad": rng.choice(["float32", "bfloat16"]),
                "copy": param == "float32" and rng.random() < 0.5}
    experts = _log(rng, 1, 128)
    top_k = rng.randint(1, min(8, experts))
    hidden, inter = 8 * _log(rng, 8, 900), 8 * _log(rng, 8, 300)
    most = 1.5e9 if op == "train" else 3e9            # weights
    while experts * hidden * inter * 3 > most:
        hidden, inter = max(64, hidden // 16 * 8), max(64, inter // 16 * 8)
    flops = 6.0 * hidden * inter * top_k * (3 if op == "train" else 1)
    tokens = _log(rng, 1, max(2, min(16384, int(4e12 / flops))))
    return {"op": "ffn", "train": op == "train", "tokens": tokens, "hidden": hidden, "inter": inter, "experts": experts,
            "top_k": top_k, "block_m": rng.choice([1, 16, 64, 100, 128]), "routing": rng.choice(["uniform", "zipf"]),
            "masked": rng.choice([0.0, 0.05, 0.5]), "activation": rng.choice(["silu", "gelu"])}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _prepare_route(c, g):
    T, E, K = c["tokens"], c["experts"], c["top_k"]
    logits = _normal(g, (T, E), 2.0, torch.float32)
    if c["closed"] > 0:
        logits.masked_fill_(torch.rand(T, E, device=DEV, generator=g) < c["closed"], float("-inf"))
    s = {"op": "route", "case": c, "logits": logits.to(getattr(torch, c["logits"])), "bias": None,
         "scale": 2.5 if c["score"] == "sigmoid" else 1.0}
    if c["bias"]:
        s["bias"] = _normal(g, (E,), 0.1, torch.float32)
    if c["train"]:
        s["grad_weights"] = _normal(g, (T, K), 1.0, torch.float32)
    return s


def _routing(c, g):
    """K distinct experts a token, some slots masked with -1."""
    T, E, K = c["tokens"], c["experts"], c["top_k"]
    score = -torch.log(-torch.log(torch.rand(T, E, device=DEV, generator=g).clamp_(1e-7, 1 - 1e-7)))
    if c["routing"] == "zipf":
        rank = torch.randperm(E, device=DEV, generator=g).float()
        score = score - 1.2 * torch.log(rank + 1.0)
    idx = score.topk(K, dim=1).indices.to(torch.int32)
    if c["masked"] > 0:
        idx.masked_fill_(torch.rand(T, K, device=DEV, generator=g) < c["masked"], -1)
    return idx.contiguous()


def _prepare_ffn(c, g):
    T, H, I, E, K, BM = c["tokens"], c["hidden"], c["inter"], c["experts"], c["top_k"], c["block_m"]
    idx = _routing(c, g)
    weights = torch.softmax(torch.randn(T, K, device=DEV, generator=g), dim=1)
    x = _normal(g, (T, H))
    # the pool of the dispatch: rows grouped by expert in slot order, each expert's region padded to block_m
    flat = idx.flatten().long()
    slots = torch.nonzero(flat >= 0).flatten()
    slots = slots[torch.sort(flat[slots], stable=True).indices]
    counts = torch.bincount(flat[slots], minlength=E)
    starts = ((counts + BM - 1) // BM).cumsum(0) * BM - (counts + BM - 1) // BM * BM
    rank = torch.arange(len(slots), device=DEV) - (counts.cumsum(0) - counts)[flat[slots]]
    rows = starts[flat[slots]] + rank
    capacity = T * K + E * (BM - 1)
    pool = torch.zeros(capacity, H, dtype=torch.bfloat16, device=DEV)
    pool[rows] = x[slots // K]
    s = {"op": "ffn", "case": c, "pool": pool,
         "w_gate_up": _normal(g, (E, 2 * I, H), H ** -0.5), "w_down": _normal(g, (E, H, I), I ** -0.5),
         "out": torch.zeros_like(pool),
         "regions": [(e, a, n) for e, (a, n) in enumerate(zip(starts.tolist(), counts.tolist())) if n]}
    if c["train"]:
        s["grad_out"] = torch.zeros_like(pool)
        s["grad_out"][rows] = _normal(g, (len(slots), H))
        s["grad_pool"] = torch.zeros_like(pool)
        s["grad_w_gate_up"] = torch.empty_like(s["w_gate_up"])
        s["grad_w_down"] = torch.empty_like(s["w_down"])
    if own:
        import combine_ep_layout_amd as ep
        s["handle"] = ep.EpHandle(T, K, E, BM)
        s["epoch"] = s["handle"].layout(idx, weights)
    return s


HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}


def _slices(flat, sizes, align):
    """Tensors of these lengths out of one buffer, each at a multiple of `align` values."""
    at = 0
    out = []
    for k in sizes:
        out.append(flat[at:at + k])
        at += -(-k // align) * align
    return out


def _prepare_adamw(c, g):
    n, lo, hi = c["tensors"], c["smallest"], c["largest"]
    # lengths spread evenly over their logarithm; the tensors lie in one buffer of each kind
    sizes = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    whole = sum(-(-k // 128) * 128 for k in sizes)
    s = {"op": "adamw", "case": c, "step": 100}
    flat = {"params": _normal(g, (whole,), 0.02, getattr(torch, c["param"]))}
    s["grads"] = _slices(_normal(g, (whole,), 0.01, getattr(torch, c["grad"])), sizes, 128)
    flat["exp_avgs"] = _normal(g, (whole,), 0.002, torch.float32)
    root = _normal(g, (whole,), 0.01, torch.float32).abs_().add_(1e-4)      # of the second moment
    if c["state"] == "8bit":
        flat["exp_avgs"], flat["exp_avg_scales"] = _encode(flat["exp_avgs"])
        flat["exp_avg_sqs"], flat["exp_avg_sq_scales"] = _encode(root)
    else:
        flat["exp_avg_sqs"] = root.square_()
    if c["copy"]:
        flat["copies"] = torch.zeros(whole, dtype=torch.bfloat16, device=DEV)
    blocks = [-(-k // 128) for k in sizes]
    for k in ("params", "exp_avgs", "exp_avg_sqs", "copies"):
        s[k] = _slices(flat[k], sizes, 128) if k in flat else None
    for k in ("exp_avg_scales", "exp_avg_sq_scales"):       # one for each 128 values
        s[k] = _slices(flat[k], blocks, 1) if k in flat else None
    s["flat"] = flat
    return s


def prepare(case, seed):
    g = _generator(seed)
    return {"route": _prepare_route, "ffn": _prepare_ffn, "adamw": _prepare_adamw}[case["op"]](case, g)


# -------------------------------------------------------------- plain forms --

def _blocks(a):
    """Values in rows of 128, the last one filled with zeros."""
    n = a.numel()
    full = torch.zeros((n + 127) // 128 * 128, dtype=a.dtype, device=a.device)
    full[:n] = a
    return full.view(-1, 128)


def _encode(a):
    """e4m3 codes (bytes) of a float32 vector and a float32 scale for each 128 values; no value but zero becomes zero
    in a vector of nothing negative (the roots of second moments keep their least code)."""
    b = _blocks(a)
    top = b.abs().amax(1, keepdim=True).clamp_min(448.0 * 2.0 ** -126)
    codes = (b * (448.0 / top)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten()[:a.numel()].contiguous(), (top / 448.0).flatten()


def _keep(codes, values):
    """The least code in the place of a zero that stands for more than zero."""
    return torch.where((codes == 0) & (values > 0), torch.ones_like(codes), codes)


def _decode(codes, scales):
    return (_blocks(codes).view(torch.float8_e4m3fn).float() * scales[:, None]).flatten()[:codes.numel()]


def _plain_route(s):
    c = s["case"]
    logits = s["logits"].float()
    K, scale = c["top_k"], s["scale"]
    is_open = logits > float("-inf")
    key = logits.double()
    if c["score"] == "sigmoid":         # the order next to a border needs more than 32 bits
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
    q = w / w.sum(1, keepdim=True).clamp_min(1e-30) if c["normalize"] else w
    out = {"topk_idx": torch.where(chosen, idx, torch.full_like(idx, -1)).to(torch.int32), "topk_weights": scale * q}
    if c["train"]:
        gw = torch.where(chosen, s["grad_weights"], torch.zeros_like(q)) * scale
        rest = 1.0 / (1.0 + torch.exp(torch.gather(logits, 1, idx)))       # 1 - sigmoid
        if c["normalize"]:
            gl = q * (gw - (q * gw).sum(1, keepdim=True))
            if c["score"] == "sigmoid":
                gl = gl * rest
            grad = torch.zeros_like(p).scatter_(1, idx, gl)
        elif c["score"] == "sigmoid":
            grad = torch.zeros_like(p).scatter_(1, idx, gw * w * rest)
        else:
            grad = p * (torch.zeros_like(p).scatter_(1, idx, gw) - (w * gw).sum(1, keepdim=True))
        out["grad_logits"] = grad.to(s["logits"].dtype)
    return out


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def _plain_expert(s, e, a, n):
    """One expert's rows, and in training its gradients."""
    c = s["case"]
    I = c["inter"]
    x, wgu, wd = s["pool"][a:a + n].float(), s["w_gate_up"][e].float(), s["w_down"][e].float()
    gu = x @ wgu.t()
    act, slope = _act(gu[:, :I], c["activation"])
    h = act * gu[:, I:]
    s["out"][a:a + n] = h @ wd.t()
    if c["train"]:
        do = s["grad_out"][a:a + n].float()
        dh = do @ wd
        dgu = torch.cat([dh * gu[:, I:] * slope, dh * act], 1)
        s["grad_pool"][a:a + n] = dgu @ wgu
        s["grad_w_gate_up"][e] = dgu.t() @ x
        s["grad_w_down"][e] = do.t() @ h


def _ffn_outputs(s):
    return {k: s[k] for k in (("out", "grad_pool", "grad_w_gate_up", "grad_w_down") if s["case"]["train"] else ("out",))}


def _plain_ffn(s):
    if s["case"]["train"] and len(s["regions"]) < s["case"]["experts"]:
        s["grad_w_gate_up"].zero_()         # experts without a row
        s["grad_w_down"].zero_()
    [_plain_expert(s, e, a, n) for e, a, n in s["regions"]]
    return _ffn_outputs(s)


def _plain_tensor(s, i, bc1, bc2):
    """One tensor's step, in place."""
    h = HYPER
    p, g = s["params"][i].float(), s["grads"][i].float()
    if s["exp_avg_scales"] is not None:
        m = _decode(s["exp_avgs"][i], s["exp_avg_scales"][i])
        v = _decode(s["exp_avg_sqs"][i], s["exp_avg_sq_scales"][i]).square()
    else:
        m, v = s["exp_avgs"][i], s["exp_avg_sqs"][i]
    m = h["beta1"] * m + (1.0 - h["beta1"]) * g
    v = h["beta2"] * v + (1.0 - h["beta2"]) * (g * g)
    r = torch.sqrt(v)
    p = p * (1.0 - h["lr"] * h["weight_decay"]) - (h["lr"] / bc1) * (m / (r / math.sqrt(bc2) + h["eps"]))
    s["params"][i].copy_(p)
    if s["copies"] is not None:
        s["copies"][i].copy_(p)
    if s["exp_avg_scales"] is not None:
        codes, scales = _encode(m)
        s["exp_avgs"][i].copy_(codes)
        s["exp_avg_scales"][i].copy_(scales)
        codes, scales = _encode(r)
        s["exp_avg_sqs"][i].copy_(_keep(codes, r))
        s["exp_avg_sq_scales"][i].copy_(scales)
    else:
        s["exp_avgs"][i].copy_(m)
        s["exp_avg_sqs"][i].copy_(v)


def _plain_adamw(s):
    bc1, bc2 = 1.0 - HYPER["beta1"] ** s["step"], 1.0 - HYPER["beta2"] ** s["step"]
    [_plain_tensor(s, i, bc1, bc2) for i in range(len(s["params"]))]


def _adamw_outputs(s):
    """The buffers that the updated tensors lie in; 8-bit codes as the e4m3 values that they are, beside their scales."""
    f = dict(s["flat"])
    if s["exp_avg_scales"] is not None:
        f["exp_avgs"], f["exp_avg_sqs"] = (f[k].view(torch.float8_e4m3fn) for k in ("exp_avgs", "exp_avg_sqs"))
    return f


# ---------------------------------------------------- the framework's calls --

def _own_route(s):
    import combine_ep_layout_amd as ep
    c = s["case"]
    how = {"score": c["score"], "normalize": c["normalize"], "scale": s["scale"]}
    idx, w = ep.route(s["logits"], c["top_k"], bias=s["bias"], **how)
    out = {"topk_idx": idx, "topk_weights": w}
    if c["train"]:
        out["grad_logits"] = ep.route_backward(s["logits"], idx, s["grad_weights"], **how)
    return out


def _own_ffn(s):
    c, h = s["case"], s["handle"]
    if not c["train"]:
        h.expert_ffn(s["epoch"], s["pool"], s["w_gate_up"], s["w_down"], activation=c["activation"], out=s["out"])
    else:
        _, saved = h.expert_ffn(s["epoch"], s["pool"], s["w_gate_up"], s["w_down"], activation=c["activation"],
                                out=s["out"], save=True)
        h.expert_ffn_backward(s["epoch"], s["grad_out"], s["pool"], s["w_gate_up"], s["w_down"], saved,
                              activation=c["activation"], grad_pool=s["grad_pool"],
                              grad_w_gate_up=s["grad_w_gate_up"], grad_w_down=s["grad_w_down"])
    return _ffn_outputs(s)


def _own_adamw(s):
    import combine_ep_layout_amd as ep
    ep.adamw(s["params"], s["grads"], s["exp_avgs"], s["exp_avg_sqs"], step=s["step"], copies=s["copies"],
             exp_avg_scales=s["exp_avg_scales"], exp_avg_sq_scales=s["exp_avg_sq_scales"], **HYPER)


def run(state):
    op = state["op"]
    if op == "route":
        return _own_route(state) if own else _plain_route(state)
    if op == "ffn":
        return _own_ffn(state) if own else _plain_ffn(state)
    state["step"] += 1
    if own:
        _own_adamw(state)
    else:
        _plain_adamw(state)
    return _adamw_outputs(state)


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "route":
        T, E, K = c["tokens"], c["experts"], c["top_k"]
        size = 4 if c["logits"] == "float32" else 2
        b = T * E * size + T * K * 8
        if c["train"]:
            b += T * K * 8 + 2 * T * E * size       # logits again, their gradient
        return {"bytes": b, "flops": 5 * T * E}
    if c["op"] == "adamw":
        n, lo, hi = c["tensors"], c["smallest"], c["largest"]
        total = sum(int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n))
        state = 16.0 if c["state"] == "float32" else 4.0 + 16.0 / 128
        each = state + (8 if c["param"] == "float32" else 4) + (4 if c["grad"] == "float32" else 2) + (2 if c["copy"] else 0)
        return {"bytes": total * each, "flops": 15 * total}
    T, H, I, E, K = c["tokens"], c["hidden"], c["inter"], c["experts"], c["top_k"]
    rows = T * K * (1.0 - c["masked"])
    used = E * (1.0 - (1.0 - min(1.0, K * (1.0 - c["masked"]) / E)) ** T)       # experts with a row, for even routing
    weights = 3.0 * I * H * 2
    if not c["train"]:
        return {"bytes": 2 * rows * H * 2 + used * weights, "flops": 6.0 * rows * H * I}
    # in: rows, gradient rows, weights; out: rows, gradient rows, gradients of the weights
    return {"bytes": 4 * rows * H * 2 + used * weights + E * weights, "flops": 18.0 * rows * H * I}


# ------------------------------------------------------------ in 64 bits --

def _exact_route(s):
    c = s["case"]
    l = s["logits"].double().requires_grad_(c["train"])
    T, E = l.shape
    K = c["top_k"]
    shut = torch.isinf(l)
    if c["score"] == "softmax":
        rank = l.detach().clone()
        some = ~shut.all(1, keepdim=True)
        p = torch.softmax(torch.where(some, l, torch.zeros_like(l)), 1) * ~shut
    else:
        p = torch.sigmoid(l) * ~shut
        rank = p.detach() + (0 if s["bias"] is None else s["bias"].double())
    rank[shut] = float("-inf")
    idx = rank.argsort(dim=1, descending=True, stable=True)[:, :K]
    w = p.gather(1, idx)
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    w = w * s["scale"]
    shut_k = shut.gather(1, idx)
    out = {"topk_idx": idx.masked_fill(shut_k, -1).to(torch.int32), "topk_weights": w.detach()}
    if c["train"]:
        w.backward(s["grad_weights"].double().masked_fill(shut_k, 0.0))
        out["grad_logits"] = torch.nan_to_num(l.grad)
    return out


def _exact_ffn(s):
    c = s["case"]
    I, train = c["inter"], c["train"]
    f = torch.nn.functional
    out = {k: torch.zeros(v.shape, dtype=torch.float64, device=DEV) for k, v in _ffn_outputs(s).items()}
    for e, a, n in s["regions"]:
        x, up, down = (t.double().requires_grad_(train) for t in (s["pool"][a:a + n], s["w_gate_up"][e], s["w_down"][e]))
        y = f.linear(x, up)
        y = (f.silu(y[:, :I]) if c["activation"] == "silu" else f.gelu(y[:, :I], approximate="tanh")) * y[:, I:]
        y = f.linear(y, down)
        out["out"][a:a + n] = y.detach()
        if train:
            y.backward(s["grad_out"][a:a + n].double())
            out["grad_pool"][a:a + n] = x.grad
            out["grad_w_gate_up"][e] = up.grad
            out["grad_w_down"][e] = down.grad
    return out


def _exact_adamw(s):
    c, f = s["case"], s["flat"]
    grads = torch.zeros(f["params"].shape, dtype=torch.float64, device=DEV)
    real = torch.zeros(f["params"].shape, dtype=torch.bool, device=DEV)
    at = 0
    for g in s["grads"]:            # the tensors' places in the buffers
        grads[at:at + g.numel()] = g.double()
        real[at:at + g.numel()] = True
        at += (g.numel() + 127) // 128 * 128
    eight = c["state"] == "8bit"
    if eight:
        per = lambda k: f[k].double().repeat_interleave(128)  # noqa: E731
        m = f["exp_avgs"].view(torch.float8_e4m3fn).double() * per("exp_avg_scales")
        v = (f["exp_avg_sqs"].view(torch.float8_e4m3fn).double() * per("exp_avg_sq_scales")) ** 2
    else:
        m, v = f["exp_avgs"].double(), f["exp_avg_sqs"].double()
    t = s["step"] + 1
    h = HYPER
    m1 = m.lerp(grads, 1.0 - h["beta1"])
    v1 = v * h["beta2"] + grads ** 2 * (1.0 - h["beta2"])
    p = f["params"].double()
    step = (m1 / (1.0 - h["beta1"] ** t)) / ((v1 / (1.0 - h["beta2"] ** t)).sqrt() + h["eps"])
    p1 = p - h["lr"] * h["weight_decay"] * p - h["lr"] * step
    out = {"params": torch.where(real, p1, p)}
    if not eight:       # codes in 8 bits have no value of their own in 64
        out.update(exp_avgs=torch.where(real, m1, m), exp_avg_sqs=torch.where(real, v1, v))
    if c["copy"]:
        out["copies"] = torch.where(real, p1, torch.zeros_like(p1))
    return out


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    return {"route": _exact_route, "ffn": _exact_ffn, "adamw": _exact_adamw}[case["op"]](s)
