"""The router and its backward pass on the GPU against float64: every number of
experts a lane, ties, closed experts, rows without an open expert, bf16 and
strided logits, extreme values, biases, duplicates in the given choice."""
import pytest
import torch

from gpu_helpers import say, dev

pytestmark = pytest.mark.gpu

NEG = float("-inf")
SHAPES = [(1, 1, 1), (1, 8, 8), (3, 2, 1), (5, 63, 7), (4, 64, 32), (129, 65, 2), (64, 128, 6), (33, 200, 8), (16, 256, 8),
          (7, 257, 9), (9, 500, 1), (6, 513, 32), (5, 1023, 10), (17, 1024, 16),
          # many tokens, four a wave; then many that do not take that form
          (8193, 3, 2), (8200, 64, 16), (9003, 100, 7), (8199, 256, 8), (8194, 129, 1), (8193, 256, 17), (8193, 300, 8)]
FORMS = [("softmax", True, False), ("softmax", False, False), ("sigmoid", True, False), ("sigmoid", False, True),
         ("sigmoid", True, True)]


def make(T, E, seed, dtype, spread=3.0, closed=0.2):
    g = torch.Generator(device=dev()).manual_seed(seed)
    l = torch.randn(T, E, device=dev(), generator=g) * spread
    l[torch.rand(T, E, device=dev(), generator=g) < closed] = NEG
    l[:, : E // 3] = l[:, E // 3: 2 * (E // 3)]         # ties in every row
    if T > 2:
        l[1] = NEG                                      # a row without an open expert
        l[2, : E - 1] = NEG                             # and one with at most one
    return l.to(dtype), torch.randn(E, device=dev(), generator=g) * 0.1


def reference(l, K, score, normalize, bias, scale):
    """(idx, weights, all weights, q, spread) in float64."""
    l = l.double()
    l = torch.where(l.isnan(), torch.full_like(l, NEG), l.clamp(max=3.402823466e38))
    shut = l == NEG
    rank = l.clone()
    if score == "sigmoid" and bias is not None:
        rank = torch.sigmoid(l) + bias.double()
        rank[rank.isnan()] = NEG
        rank[shut] = NEG
    order = torch.sort(rank, dim=1, descending=True, stable=True)
    idx, on = order.indices[:, :K], order.values[:, :K] > NEG
    lk = torch.gather(l, 1, idx)
    if score == "softmax":
        top = torch.where(shut.all(1), torch.zeros_like(l[:, 0]), l.amax(1))[:, None]
        e = torch.where(shut, torch.zeros_like(l), torch.exp(l - top))
        p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = torch.where(shut, torch.zeros_like(l), torch.sigmoid(l))
    w = torch.where(on, torch.gather(p, 1, idx), torch.zeros_like(lk))
    q = w
    if normalize:       # of the logarithms: the ratio lives where the sum underflows
        logp = torch.nn.functional.logsigmoid(lk) if score == "sigmoid" else lk
        logp = torch.where(on, logp, torch.full_like(lk, NEG))
        q = torch.where(on.any(1, keepdim=True), torch.softmax(logp, 1), torch.zeros_like(lk))
        q = torch.nan_to_num(q)
    fin = torch.where(shut, torch.zeros_like(l), l)
    spread = (fin.amax(1) - fin.amin(1))[:, None]
    return torch.where(on, idx, torch.full_like(idx, -1)).int(), scale * q, p, q, spread


def near(got, want, rel, extra=0.0):
    off = (got.double() - want).abs()
    bound = rel * want.abs() + extra + 2.0 ** -125
    assert bool((off <= bound).all()), (float((off - bound).max()), float(off.max()))


@pytest.mark.parametrize("score,normalize,biased", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_route(shape, dtype, score, normalize, biased):
    import combine_ep_layout_amd as ep
    T, E, K = shape
    say(f"[route] {shape} {dtype} {score} {normalize} {biased}")
    l, bias = make(T, E, 3, dtype)
    bias = bias if biased else None
    idx, w = ep.route(l, K, score=score, bias=bias, normalize=normalize, scale=1.5)
    want_idx, want_w, p, q, spread = reference(l, K, score, normalize, bias, 1.5)
    assert torch.equal(idx, want_idx)
    # exp of a difference d, itself rounded: d * 2^-24; exp, sums of 1024 in a tree, quotient: under 16 steps
    rel = (spread + 32) * 2.0 ** -23
    near(w, want_w, rel)

    g = torch.Generator(device=dev()).manual_seed(9)
    gw = torch.randn(T, K, device=dev(), generator=g)
    got = ep.route_backward(l, idx, gw, score=score, normalize=normalize, scale=1.5)
    on = idx >= 0
    gq = torch.where(on, gw.double() * 1.5, torch.zeros_like(q))
    dot, mag = (q * gq).sum(1, keepdim=True), (q * gq.abs()).sum(1, keepdim=True)
    lk = torch.gather(l.double(), 1, idx.clamp_min(0).long())
    rest = torch.where(on, torch.sigmoid(-lk), torch.zeros_like(q))
    want, size = torch.zeros_like(p), torch.zeros_like(p)
    at = idx.clamp_min(0).long()
    if normalize:
        d, s = q * (gq - dot), q * (gq.abs() + mag)
        if score == "sigmoid":
            d, s = d * rest, s * rest
    else:
        d, s = (gq * q * rest, gq.abs() * q * rest) if score == "sigmoid" else (q * gq, q * gq.abs())
    d, s = torch.where(on, d, torch.zeros_like(d)), torch.where(on, s, torch.zeros_like(s))
    want.scatter_add_(1, at, d)
    size.scatter_add_(1, at, s)
    if not normalize and score == "softmax":
        want -= p * dot
        size += p * mag
    rounding = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert got.dtype == dtype
    near(got, want, rounding, extra=2 * (spread + 32) * 2.0 ** -23 * size)


def test_extreme_logits():
    import combine_ep_layout_amd as ep
    inf, nan = float("inf"), float("nan")
    rows = [[inf, 1, inf, 0], [nan, nan, 2, NEG], [nan] * 4, [NEG] * 4, [-200, -300, -201, -1e30], [3e38, -3e38, 0, 3e38],
            [-0.0, 0.0, -0.0, 0.0], [100, 100, 100, 99]]
    l = torch.tensor(rows, device=dev())
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            idx, w = ep.route(l, 2, score=score, normalize=normalize)
            want_idx, want_w, *_ = reference(l, 2, score, normalize, None, 1.0)
            assert torch.equal(idx, want_idx), (score, idx, want_idx)
            # differences up to 100 here; each costs half a step of the exponent
            assert bool(w.isfinite().all())
            near(w, want_w, 200 * 2.0 ** -23)
            got = ep.route_backward(l, idx, torch.ones_like(w), score=score, normalize=normalize)
            assert bool(got.isfinite().all())


def test_bias_chooses_but_does_not_weigh():
    import combine_ep_layout_amd as ep
    l = torch.tensor([[2.0, 1.0, 0.0, -1.0]], device=dev())
    idx, w = ep.route(l, 2, score="sigmoid", bias=torch.tensor([0.0, NEG, 0.0, 5.0], device=dev()), normalize=False)
    assert idx.tolist() == [[3, 0]]
    near(w, torch.sigmoid(l.double()[:, [3, 0]]), 8 * 2.0 ** -23)
    idx, w = ep.route(l, 3, score="sigmoid", bias=torch.tensor([float("nan"), NEG, NEG, 0.0], device=dev()))
    assert idx.tolist() == [[3, -1, -1]] and w.tolist() == [[1.0, 0.0, 0.0]]


def test_strided_rows_and_many_tokens():
    import combine_ep_layout_amd as ep
    wide = torch.randn(9001, 100, device=dev())
    l = wide[:, 10:43]
    idx, w = ep.route(l, 4)
    a, b = ep.route(l.contiguous(), 4)
    assert torch.equal(idx, a) and torch.equal(w, b)
    gw = torch.randn_like(w)
    grad = torch.full_like(wide, 7.0)
    ep.route_backward(l, idx, gw, grad_logits=grad[:, 10:43])
    assert torch.equal(grad[:, 10:43].contiguous(), ep.route_backward(l.contiguous(), idx, gw))
    assert bool((grad[:, :10] == 7).all()) and bool((grad[:, 43:] == 7).all())


def test_given_choice_with_repeats_and_bad_numbers():
    """A choice that the router did not make: a repeated expert's terms add up, numbers outside count as masked."""
    import combine_ep_layout_amd as ep
    l = torch.tensor([[1.0, 2.0, 0.5, -1.0]], device=dev())
    idx = torch.tensor([[1, 1, 77, -5]], dtype=torch.int32, device=dev())
    got = ep.route_backward(l, idx, torch.tensor([[1.0, 2.0, 3.0, 4.0]], device=dev()), score="sigmoid", normalize=False)
    s = torch.sigmoid(torch.tensor(2.0, dtype=torch.float64))
    want = torch.zeros(1, 4, dtype=torch.float64, device=dev())
    want[0, 1] = 3 * float(s * (1 - s))
    near(got, want, 16 * 2.0 ** -23)


def test_no_tokens_and_refusals():
    import combine_ep_layout_amd as ep
    idx, w = ep.route(torch.empty(0, 8, device=dev()), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    l = torch.randn(4, 8, device=dev())
    for bad in (lambda: ep.route(l.half(), 2), lambda: ep.route(l.t(), 2), lambda: ep.route(l, 2, score="tanh"),
                lambda: ep.route(l, 9), lambda: ep.route(l, 0), lambda: ep.route(l, 2, bias=torch.zeros(8, device=dev())),
                lambda: ep.route(l[:1].expand(4, 8), 2), lambda: ep.route(l.cpu(), 2),
                lambda: ep.route(torch.zeros(4, 1025, device=dev()), 2),
                lambda: ep.route_backward(l, torch.zeros(4, 2, device=dev()), torch.zeros(4, 2, device=dev()))):
        with pytest.raises((TypeError, ValueError, ep.EpError)):
            bad()


def test_gradient_against_differences():
    import combine_ep_layout_amd as ep
    g = torch.Generator(device=dev()).manual_seed(2)
    l = torch.randn(6, 40, device=dev(), generator=g)
    gw = torch.randn(6, 4, device=dev(), generator=g)
    for score, normalize in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        idx, _ = ep.route(l, 4, score=score, normalize=normalize)
        got = ep.route_backward(l, idx, gw, score=score, normalize=normalize)
        v = torch.randn(6, 40, dtype=torch.float64, device=dev(), generator=g)

        def value(eps):
            x = l.double() + eps * v
            p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
            w = torch.gather(p, 1, idx.long())
            return ((w / w.sum(1, keepdim=True) if normalize else w) * gw.double()).sum()

        slope = float((value(1e-5) - value(-1e-5)) / 2e-5)
        terms = got.double() * v
        assert abs(float(terms.sum()) - slope) <= 64 * 2.0 ** -23 * float(terms.abs().sum()) + 1e-8
