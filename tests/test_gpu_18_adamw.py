"""The AdamW step over many tensors on the GPU against float64: every type of
parameter, gradient and state, lengths off every vector and block, more tensors
than one launch holds, steps and gradient factors read on the device, values
that are no numbers."""
import math

import pytest
import torch

from gpu_helpers import say, dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
LENGTHS = [1, 2, 3, 4, 5, 127, 128, 129, 255, 1023, 4097, 8191, 8192, 8193, 8197, 20001, 0, 1024 * 33]
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05)


def encode(x):
    """Codes and scales of each 128 values, in the fp32 operations of the definition (torch's quotient of a number by a
    tensor is the number times the reciprocal, and its quotient by a number the product with that number's reciprocal)."""
    n = x.numel()
    b = torch.zeros((n + 127) // 128 * 128, device=x.device)
    b[:n] = x
    b = b.view(-1, 128)
    top = b.abs().amax(1, keepdim=True).clamp_min(448.0 * 2.0 ** -126)
    codes = (b * (448.0 / top)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten()[:n].clone(), (top / 448.0).flatten()


def decode(codes, scales):
    n = codes.numel()
    return codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128)[:n]


def make(lengths, p_dtype, g_dtype, eight, copy, seed=0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    r = lambda n, s: torch.randn(n, device=dev(), generator=g) * s
    s = dict(params=[r(n, 1.0).to(p_dtype) for n in lengths], grads=[r(n, 0.3).to(g_dtype) for n in lengths])
    m, root = [r(n, 0.1) for n in lengths], [r(n, 0.2).abs() for n in lengths]
    s["exp_avg_scales"] = s["exp_avg_sq_scales"] = None
    if eight:
        em, er = [encode(x) for x in m], [encode(x) for x in root]
        s["exp_avgs"], s["exp_avg_scales"] = [a for a, _ in em], [b for _, b in em]
        s["exp_avg_sqs"], s["exp_avg_sq_scales"] = [a for a, _ in er], [b for _, b in er]
    else:
        s["exp_avgs"], s["exp_avg_sqs"] = m, [x * x for x in root]
    s["copies"] = [torch.empty(n, dtype=BF16, device=dev()).fill_(9) for n in lengths] if copy else None
    return s


def clone(s):
    return {k: None if v is None else [t.clone() for t in v] for k, v in s.items()}


def expected(s, i, step, scale=1.0):
    """(m, v, p) in float64 and bounds of the fp32 arithmetic."""
    h = HYPER
    g = s["grads"][i].double() * scale
    if s["exp_avg_scales"] is not None:
        m0 = decode(s["exp_avgs"][i], s["exp_avg_scales"][i])
        v0 = decode(s["exp_avg_sqs"][i], s["exp_avg_sq_scales"][i]) ** 2
    else:
        m0, v0 = s["exp_avgs"][i].double(), s["exp_avg_sqs"][i].double()
    m = h["beta1"] * m0 + (1 - h["beta1"]) * g
    v = h["beta2"] * v0 + (1 - h["beta2"]) * g * g
    p0 = s["params"][i].double()
    den = v.sqrt() / math.sqrt(1 - h["beta2"] ** step) + h["eps"]
    size = h["lr"] / (1 - h["beta1"] ** step)
    p = p0 * (1 - h["lr"] * h["weight_decay"]) - size * m / den
    # at most eight roundings of 2^-24 stand in each term (the constants' own, products, sums, root, quotients)
    u = 8 * 2.0 ** -24
    em = u * (h["beta1"] * m0.abs() + (1 - h["beta1"]) * g.abs())
    ev = u * v
    epd = u * p0.abs() + size * (em + 2 * u * m.abs()) / den
    return m, em, v, ev, p, epd


def within(got, want, bound, least=2.0 ** -126):
    off = (got.double() - want).abs()
    assert bool((off <= bound + least).all()), float((off - bound).max())


def check(s, before, step, scale=1.0):
    for i, p0 in enumerate(before["params"]):
        if p0.numel() == 0:
            continue
        m, em, v, ev, p, epd = expected(before, i, step, scale)
        half = 2.0 ** -8 if p0.dtype == BF16 else 2.0 ** -24
        within(s["params"][i], p, epd + half * (p.abs() + epd))
        if s["copies"] is not None:
            assert torch.equal(s["copies"][i], s["params"][i].to(BF16))
        assert torch.equal(s["grads"][i], before["grads"][i])
        if s["exp_avg_scales"] is None:
            within(s["exp_avgs"][i], m, em)
            within(s["exp_avg_sqs"][i], v, ev)
            continue
        n = p0.numel()
        for codes, scales, x, e in ((s["exp_avgs"][i], s["exp_avg_scales"][i], m, em),
                                    (s["exp_avg_sqs"][i], s["exp_avg_sq_scales"][i], v.sqrt(), v.sqrt() * 4 * 2.0 ** -24)):
            b = torch.zeros(2, scales.numel() * 128, dtype=torch.float64, device=dev())
            b[0, :n], b[1, :n] = x.abs(), e
            top, off = b.view(2, -1, 128).amax(2)
            # |max |a| - max |b|| <= max |a - b|: the two terms of m may cancel, so that a block's largest value is off
            # by more than a few steps of itself (e counts steps of the terms); then one rounded quotient
            within(scales, top / 448, (off + 2 * 2.0 ** -24 * top) / 448)
            # a code is half a step of four significant bits off (2^-4), or half the least step 2^-9 of the scale
            unit = scales.double().repeat_interleave(128)[:n]
            within(decode(codes, scales), x, e + x.abs() * (2.0 ** -4 + 2.0 ** -20) + unit * 2.0 ** -10)
        root = decode(s["exp_avg_sqs"][i], s["exp_avg_sq_scales"][i])
        assert bool((root[v > 0] > 0).all())


@pytest.mark.parametrize("eight", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("p_dtype,g_dtype,copy", [(F32, F32, False), (F32, BF16, True), (BF16, BF16, False), (BF16, F32, False),
                                                  (F32, F32, True)])
def test_step(p_dtype, g_dtype, copy, eight):
    import combine_ep_layout_amd as ep
    say(f"[adamw] {p_dtype} {g_dtype} {copy} {eight}")
    s = make(LENGTHS, p_dtype, g_dtype, eight, copy)
    for step in (1, 2, 1000):
        before = clone(s)
        ep.adamw(**s, step=step, **HYPER)
        check(s, before, step)


def test_codes_are_those_of_the_definition():
    """Bit for bit over some 30 million values: one code off by one would show here, and in every later step."""
    import combine_ep_layout_amd as ep
    h = HYPER
    for seed in range(3):
        s = make([5_000_000, 77], F32, BF16, True, False, seed=seed)
        before = clone(s)
        ep.adamw(**s, step=9, **HYPER)
        for i in range(2):
            g = before["grads"][i].float()
            value = lambda k, t: (before[k][i].view(torch.float8_e4m3fn).float() *
                                  before[t][i].repeat_interleave(128)[: g.numel()])
            m = h["beta1"] * value("exp_avgs", "exp_avg_scales") + (1 - h["beta1"]) * g
            v = h["beta2"] * value("exp_avg_sqs", "exp_avg_sq_scales").square() + (1 - h["beta2"]) * (g * g)
            root = torch.sqrt(v)
            codes, scales = encode(m)
            assert torch.equal(s["exp_avg_scales"][i], scales)
            assert torch.equal(s["exp_avgs"][i], codes)
            codes, scales = encode(root)
            assert torch.equal(s["exp_avg_sq_scales"][i], scales)
            assert torch.equal(s["exp_avg_sqs"][i], torch.where((codes == 0) & (root > 0), torch.ones_like(codes), codes))


def test_more_tensors_than_a_launch_and_lists_of_one():
    import combine_ep_layout_amd as ep
    for lengths in ([7 * i % 300 + 1 for i in range(161)], [5]):
        for eight in (False, True):
            s = make(lengths, F32, BF16, eight, True, seed=1)
            before = clone(s)
            ep.adamw(**s, step=3, **HYPER)
            check(s, before, 3)


def test_shaped_tensors_and_what_lies_beside_them():
    """Slices of one buffer, 16-byte aligned: the values between them keep."""
    import combine_ep_layout_amd as ep
    flat = {k: torch.full((4096,), 0.5, device=dev()) for k in ("params", "grads", "exp_avgs", "exp_avg_sqs")}
    s = {k: [v[0:129], v[132:132 + 700].view(7, 100), v[1000:1001]] for k, v in flat.items()}
    before = {**{k: [t.clone().flatten() for t in v] for k, v in s.items()}, "exp_avg_scales": None, "copies": None}
    ep.adamw(**s, step=5, **HYPER)
    check({**{k: [t.flatten() for t in v] for k, v in s.items()}, "exp_avg_scales": None, "copies": None}, before, 5)
    outside = torch.ones(4096, dtype=torch.bool, device=dev())
    for a, b in ((0, 129), (132, 832), (1000, 1001)):
        outside[a:b] = False
    for v in flat.values():
        assert bool((v[outside] == 0.5).all())


def test_step_and_factor_on_the_device():
    import combine_ep_layout_amd as ep
    s = make([1000, 17], F32, F32, False, False)
    before = clone(s)
    ep.adamw(**s, step=torch.tensor([7], device=dev()), grad_scale=torch.tensor(0.25, device=dev()), **HYPER)
    check(s, before, 7, 0.25)
    t = clone(before)
    ep.adamw(**t, step=7, grad_scale=0.25, **HYPER)
    for a, b in zip(s["params"], t["params"]):
        within(a, b.double(), 2.0 ** -22 * b.double().abs())


def test_captured_steps_follow_the_step_on_the_device():
    import combine_ep_layout_amd as ep
    s = make([5000, 33, 128], F32, BF16, True, True, seed=4)
    eager = clone(s)
    step = torch.zeros(1, dtype=torch.int64, device=dev())
    start = clone(s)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step.add_(1)
        ep.adamw(**s, step=step, **HYPER)
    for k, v in start.items():
        if v is not None:
            for a, b in zip(s[k], v):
                a.copy_(b)
    step.zero_()
    for t in range(1, 5):
        for grad, other in zip(s["grads"], eager["grads"]):         # new gradients for every replay
            grad.mul_(-0.7)
            other.copy_(grad)
        g.replay()
        torch.cuda.synchronize()
        on_device = torch.tensor([t], device=dev())
        ep.adamw(**eager, step=on_device, **HYPER)
        torch.cuda.synchronize()
        for k in s:
            if s[k] is not None:
                for a, b in zip(s[k], eager[k]):
                    assert torch.equal(a, b), (k, t)


def test_zero_gradients_and_values_that_are_no_numbers():
    import combine_ep_layout_amd as ep
    s = make([300], F32, F32, False, False)
    for k in ("grads", "exp_avgs", "exp_avg_sqs"):
        s[k][0].zero_()
    before = clone(s)
    ep.adamw(**s, step=1, **HYPER)
    check(s, before, 1)                     # nothing but the decay: 0 / (0 + eps) = 0
    s["grads"][0][5], s["grads"][0][6] = float("nan"), float("inf")
    ep.adamw(**s, step=2, **HYPER)
    bad = s["params"][0].isnan()
    assert bad[5] and bad[6] and int(bad.sum()) == 2        # inf / inf
    e = make([300], F32, F32, True, False)
    e["grads"][0][5] = float("nan")
    ep.adamw(**e, step=1, **HYPER)
    nan = decode(e["exp_avgs"][0], e["exp_avg_scales"][0]).isnan()
    assert nan[5] and int(nan.sum()) == 1                   # NaN takes no part in its block's scale
    e["grads"][0][5] = 0.0
    e["grads"][0][140] = float("inf")
    ep.adamw(**e, step=2, **HYPER)
    nan = decode(e["exp_avgs"][0], e["exp_avg_scales"][0]).isnan()
    assert bool(nan[128:256].all()) and not bool(nan[256:].any())


def test_codes_are_read_by_the_cast_back():
    import combine_ep_layout_amd as ep
    s = make([128 * 6], F32, F32, True, False)
    ep.adamw(**s, step=1, **HYPER)
    back = ep.cast_back(s["exp_avgs"][0].view(2, 384), s["exp_avg_scales"][0].view(2, 3), "f32")
    want = (s["exp_avgs"][0].view(torch.float8_e4m3fn).float() * s["exp_avg_scales"][0].repeat_interleave(128)).to(BF16)
    assert torch.equal(back.flatten(), want)


def test_refusals():
    import combine_ep_layout_amd as ep
    def fresh(**kw):
        s = make([256, 100], F32, F32, False, False)
        s.update(kw)
        return s
    def refused(s, **kw):
        before = [t.clone() for t in s["params"]]
        with pytest.raises((TypeError, ValueError, ep.EpError)):
            ep.adamw(**s, **{**dict(step=1), **HYPER, **kw})
        assert all(torch.equal(a, b) for a, b in zip(before, s["params"]))
    s = fresh()
    refused({**s, "params": [s["params"][0], s["params"][0]], "grads": [s["grads"][0]] * 2,
             "exp_avgs": [s["exp_avgs"][0]] * 2, "exp_avg_sqs": [s["exp_avg_sqs"][0]] * 2})      # a tensor twice
    refused({**s, "grads": s["params"]})                                    # written and read
    refused(s, step=0)
    refused(s, beta1=1.0)
    refused(s, eps=-1.0)
    refused(s, lr=float("nan"))
    refused(fresh(grads=s["grads"][:1]))
    refused({**s, "grads": [s["grads"][0][:255], s["grads"][1]]})
    refused({**s, "exp_avgs": [t.to(BF16) for t in s["exp_avgs"]]})
    refused({**s, "params": [torch.randn(256, 2, device=dev())[:, 0], s["params"][1]]})        # not contiguous
    refused({**s, "params": [torch.randn(257, device=dev())[1:], s["params"][1]]})             # not aligned
    refused({**s, "copies": [torch.empty(256, device=dev()), torch.empty(100, device=dev())]})
    refused({**s, "exp_avg_scales": [torch.ones(2, device=dev()), torch.ones(1, device=dev())]})
    refused({**s, "params": [t.half() for t in s["params"]]})
    b = make([256], BF16, F32, False, False)
    refused({**b, "copies": [torch.empty(256, dtype=BF16, device=dev())]})
    ep.adamw([], [], [], [], step=1)
