"""The whole layer for a few tokens (moe_tokens), with bf16 and 4-bit weights, against float64 with bounds on what
rounding may add: token counts on both sides of the 16-token tiles, experts that every token chooses or none, masked
and repeated slots, odd widths, strided rows, NaN rows, graphs and streams."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
from gpu_helpers import dev, say
from mxfp4_reference import decode, encode

pytestmark = pytest.mark.gpu


def weights(E, H, I, four, seed):
    """(w_gate_up, w_down) as the call takes them, and their float64 values."""
    import combine_ep_layout_amd as ep
    g = torch.Generator(device=dev()).manual_seed(seed)
    n = lambda *s: torch.randn(s, device=dev(), generator=g)
    up, down = n(E, 2 * I, H) * H ** -0.5, n(E, H, I) * I ** -0.5
    if not four:
        up, down = up.bfloat16(), down.bfloat16()
        return (up, down), (up.double(), down.double())
    q = [ep.Mxfp4(*(torch.from_numpy(a).to(dev()) for a in encode(w.cpu().numpy()))) for w in (up, down)]
    return tuple(q), tuple(torch.from_numpy(decode(w.codes.cpu().numpy(), w.scales.cpu().numpy())).to(dev()) for w in q)


def check_y(y, x, idx, w, up, down, kind):
    """Every row of y within its bounds, from the choice and its fp32 weights."""
    T, K = idx.shape
    H, I = up.shape[2], down.shape[2]
    value, bound, size = (torch.zeros(T, H, dtype=torch.float64, device=dev()) for _ in range(3))
    for e in range(up.shape[0]):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        a, e_a = ref.expert(x[t].double(), up[e], down[e], kind)["act"]
        wt = w[t, k].double().unsqueeze(1)
        out = a @ down[e].T
        # an eighth of the sum a wave, then the waves': still at most inter additions and a few more
        e_out = e_a @ down[e].abs().T + (I + 8) * ref.U_SUM * ((a.abs() + e_a) @ down[e].abs().T)
        value.index_add_(0, t, wt * out)
        bound.index_add_(0, t, wt.abs() * e_out)
        size.index_add_(0, t, wt.abs() * ((a.abs() + e_a) @ down[e].abs().T))
    bound += (K + 8 + 2) * ref.U_SUM * size
    ref.check("y", y, value, bound + ref.H_BF16 * (value.abs() + bound))


def routing(T, E, K, seed, masked=0.0):
    g = torch.Generator(device=dev()).manual_seed(seed + 1000)
    idx = torch.rand(T, E, device=dev(), generator=g).topk(K, 1).indices.to(torch.int32)
    if masked:
        idx.masked_fill_(torch.rand(T, K, device=dev(), generator=g) < masked, -1)
    return idx.contiguous(), torch.randn(T, K, device=dev(), generator=g)


def rows(T, H, seed):
    return torch.randn(T, H, device=dev(), generator=torch.Generator(device=dev()).manual_seed(seed + 2000)).bfloat16()


CASES = [  # T, E, K, H, I, masked
    (1, 8, 2, 256, 512, 0.0), (1, 1, 1, 32, 32, 0.0), (2, 5, 3, 96, 64, 0.0), (3, 300, 8, 160, 96, 0.3),
    (7, 24, 3, 2080, 992, 0.2), (8, 64, 8, 512, 128, 0.0), (9, 64, 8, 128, 544, 0.0), (16, 3, 3, 1056, 160, 0.0),
    (17, 2, 1, 192, 288, 0.0), (31, 1024, 32, 64, 32, 0.5), (32, 2, 2, 128, 96, 0.0), (33, 1, 1, 320, 64, 0.0),
    (64, 1, 1, 544, 1120, 0.0), (64, 7, 5, 224, 64, 0.6), (64, 40, 32, 64, 64, 0.0)]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_given_choice(case, four):
    import combine_ep_layout_amd as ep
    T, E, K, H, I, masked = case
    say(f"[moe tokens] {case} {'4 bit' if four else 'bf16'}")
    q, (up, down) = weights(E, H, I, four, T)
    x, (idx, w) = rows(T, H, T), routing(T, E, K, T, masked)
    for kind in ("silu", "gelu"):
        y, got_idx, got_w = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w, activation=kind)
        assert got_idx is idx and got_w is w
        check_y(y, x, idx, w, up, down, kind)
    again = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w, activation=kind)[0]
    assert torch.equal(again, y)


@pytest.mark.parametrize("H,I", [(8, 8), (8, 200), (264, 16), (72, 1000), (2056, 104), (136, 24)])
def test_odd_widths(H, I):
    """Multiples of 8 that end inside a step and inside a row tile."""
    import combine_ep_layout_amd as ep
    say(f"[moe tokens] widths {H} {I}")
    q, (up, down) = weights(6, H, I, False, H)
    x, (idx, w) = rows(19, H, I), routing(19, 6, 2, H, 0.1)
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    check_y(y, x, idx, w, up, down, "silu")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T,E,K", [(1, 64, 8), (1, 8, 2), (5, 256, 8), (8, 33, 4), (8, 257, 8), (9, 64, 8), (40, 16, 2), (4, 32, 32)])
def test_choice_from_logits(T, E, K, four):
    """The choice is the router's own, weights too, wherever it is made."""
    import combine_ep_layout_amd as ep
    say(f"[moe tokens] logits {T} {E} {K} {four}")
    H, I = 192, 96
    q, (up, down) = weights(E, H, I, four, E)
    x = rows(T, H, E)
    g = torch.Generator(device=dev()).manual_seed(K)
    logits = torch.randn(T, E, device=dev(), generator=g) * 2
    logits[torch.rand(T, E, device=dev(), generator=g) < 0.3] = float("-inf")
    logits[0] = 0.25                                # ties: the lowest experts
    logits[-1, 1:] = float("-inf")                  # one open expert, or none
    bias = torch.randn(E, device=dev(), generator=g)
    for how in ({"score": "softmax"}, {"score": "softmax", "normalize": False}, {"score": "sigmoid", "scale": 2.5},
                {"score": "sigmoid", "bias": bias, "normalize": False}):
        for l in (logits, logits.bfloat16(), torch.cat([logits, logits], 1)[:, :E]):
            y, idx, w = ep.moe_tokens(x, *q, logits=l, top_k=K, **how)
            want_idx, want_w = ep.route(l, K, **how)
            assert torch.equal(idx, want_idx)
            # the sums of a softmax may go in another order: of up to 1024 terms that add up to 1
            assert bool(((w - want_w).abs() <= 16 * 2.0 ** -24 * want_w.abs() + 1e-37).all())
            check_y(y, x, idx, w, up, down, "silu")


def test_no_open_expert_no_token_and_unknown_ids():
    import combine_ep_layout_amd as ep
    q, (up, down) = weights(4, 64, 32, False, 1)
    x = rows(3, 64, 1)
    y, idx, w = ep.moe_tokens(x, *q, logits=torch.full((3, 4), float("-inf"), device=dev()), top_k=2)
    assert not y.any() and bool((idx == -1).all()) and not w.any()
    y, idx, w = ep.moe_tokens(x[:0], *q, logits=torch.zeros(0, 4, device=dev()), top_k=2)
    assert y.shape == (0, 64) and idx.shape == (0, 2)
    ids = torch.tensor([[0, 4], [-7, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device=dev())
    w = torch.ones(3, 2, device=dev())
    y = ep.moe_tokens(x, *q, topk_idx=ids, topk_weights=w)[0]
    check_y(y, x, ids, w, up, down, "silu")
    assert not y[2].any()


@pytest.mark.parametrize("four", [False, True])
def test_an_expert_named_twice(four):
    import combine_ep_layout_amd as ep
    q, (up, down) = weights(5, 96, 64, four, 2)
    x = rows(20, 96, 2)
    idx = torch.randint(0, 3, (20, 6), device=dev(), generator=torch.Generator(device=dev()).manual_seed(0)).to(torch.int32)
    w = torch.randn(20, 6, device=dev(), generator=torch.Generator(device=dev()).manual_seed(1))
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    check_y(y, x, idx, w, up, down, "silu")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("K", [1, 2, 7, 32])
def test_one_token_names_experts_twice_and_none(K, four):
    """One token's slots are found by one wave: repeats, masked slots, all of them one expert, all masked."""
    import combine_ep_layout_amd as ep
    q, (up, down) = weights(9, 96, 160, four, K)
    x = rows(1, 96, K)
    g = torch.Generator(device=dev()).manual_seed(K)
    w = torch.randn(1, K, device=dev(), generator=g)
    ids = torch.randint(-2, 11, (1, K), device=dev(), generator=g).to(torch.int32)       # 9 and 10 are no experts
    for idx in (ids, torch.full_like(ids, 8), torch.full_like(ids, -1)):
        y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
        check_y(y, x, idx, w, up, down, "silu")
    assert not y.any()


def test_a_part_of_the_experts():
    """Slices of the experts' matrices are matrices as well."""
    import combine_ep_layout_amd as ep
    q, (up, down) = weights(7, 160, 96, True, 9)
    part = [ep.Mxfp4(w.codes[3:6], w.scales[3:6]) for w in q]
    x, (idx, w) = rows(5, 160, 9), routing(5, 3, 2, 9)
    check_y(ep.moe_tokens(x, *part, topk_idx=idx, topk_weights=w)[0], x, idx, w, up[3:6], down[3:6], "silu")


def test_rows_of_nan_and_infinity_stay_apart():
    """Padding rows of a batch may hold anything; strided rows leave what lies between them out."""
    import combine_ep_layout_amd as ep
    q, (up, down) = weights(6, 128, 96, True, 3)
    T = 18
    wide = torch.full((T, 256), float("nan"), dtype=torch.bfloat16, device=dev())
    x = wide[:, 64:192]
    x.copy_(rows(T, 128, 3))
    idx, w = routing(T, 6, 2, 3)
    idx[4] = -1
    clean = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    check_y(clean, x, idx, w, up, down, "silu")
    x[4], x[7], x[9] = float("nan"), float("nan"), float("inf")
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    others = [t for t in range(T) if t not in (7, 9)]
    assert torch.equal(y[others], clean[others]) and not y[4].any()
    assert bool(torch.isnan(y[7]).all()) and not bool(torch.isfinite(y[9]).any())


def test_nan_blocks_and_extreme_scales():
    """An exponent byte of 255 makes its products NaN; bytes 0 and 254 are the powers they stand for."""
    import combine_ep_layout_amd as ep
    q, (up, down) = weights(2, 64, 32, True, 4)
    x = rows(2, 64, 4)
    idx, w = torch.tensor([[0], [1]], dtype=torch.int32, device=dev()), torch.ones(2, 1, device=dev())
    clean = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    q[1].scales[1, 5, 0] = 255
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    assert bool(torch.isnan(y[1, 5])) and torch.equal(y[0], clean[0])
    assert torch.equal(y[1, torch.arange(64, device=dev()) != 5], clean[1, torch.arange(64, device=dev()) != 5])
    q[1].scales[1, 5, 0] = 0                # 2^-127: next to nothing of the sum
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    assert abs(float(y[1, 5])) < 1e-30
    assert torch.equal(y[0], clean[0])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T", [1, 6, 24])
def test_captured_and_replayed(T, four):
    """A graph of the call on new inputs, with eager calls between the replays."""
    import combine_ep_layout_amd as ep
    E, K, H, I = 16, 4, 160, 128
    q, _ = weights(E, H, I, four, 5)
    x, logits = rows(T, H, 5), torch.randn(T, E, device=dev())
    call = lambda: ep.moe_tokens(x, *q, logits=logits, top_k=K)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(4):
        x.copy_(rows(T, H, 50 + seed))
        logits.copy_(torch.randn(T, E, device=dev(), generator=torch.Generator(device=dev()).manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, call()):
            assert torch.equal(a, b)


def test_another_stream_and_a_given_result():
    import combine_ep_layout_amd as ep
    q, _ = weights(8, 256, 64, False, 6)
    x, (idx, w) = rows(12, 256, 6), routing(12, 8, 2, 6)
    want = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(want)
    results = [ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w, y=y if i == 0 else None, stream=side)[0] for i in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert results[0] is y and all(torch.equal(r, want) for r in results)


def test_against_the_pool_path():
    """The same layer through layout, dispatch, expert_ffn and combine: equal but for roundings."""
    import combine_ep_layout_amd as ep
    T, E, K, H, I = 48, 16, 4, 512, 256
    q, _ = weights(E, H, I, False, 7)
    x, logits = rows(T, H, 7), torch.randn(T, E, device=dev())
    y, idx, w = ep.moe_tokens(x, *q, logits=logits, top_k=K, score="sigmoid", scale=2.5)
    h = ep.EpHandle(T, K, E, 16)
    epoch = h.layout(*ep.route(logits, K, score="sigmoid", scale=2.5))
    pool, _ = h.new_pool(H)
    h.dispatch(x, pool)
    other = h.combine(epoch, h.expert_ffn(epoch, pool, *q))
    h.close()
    # y: two roundings (of a, of y), there three; each at most 2^-8 of what it rounds, far less in the norm
    assert float((y.double() - other.double()).norm() / other.double().norm()) <= 2.0 ** -8


def test_binding_refusals():
    import combine_ep_layout_amd as ep
    q, _ = weights(4, 64, 32, False, 8)
    q4, _ = weights(4, 64, 32, True, 8)
    x, (idx, w) = rows(3, 64, 8), routing(3, 4, 2, 8)
    logits = torch.randn(3, 4, device=dev())
    for kind, args, kw in (
            (ValueError, (x, *q), {}), (ValueError, (x, *q), {"logits": logits}), (ValueError, (x, *q), {"topk_idx": idx}),
            (ValueError, (x, *q), {"logits": logits, "top_k": 2, "topk_idx": idx, "topk_weights": w}),
            (TypeError, (x, q[0], q4[1]), {"logits": logits, "top_k": 2}), (TypeError, (x.float(), *q), {"logits": logits, "top_k": 2}),
            (ValueError, (x[:, :56], *q), {"logits": logits, "top_k": 2}), (ValueError, (x, q[0][:, :32], q[1]), {"logits": logits, "top_k": 2}),
            (ValueError, (x, *q), {"logits": logits[:2], "top_k": 2}), (TypeError, (x, *q), {"topk_idx": idx.long(), "topk_weights": w}),
            (ValueError, (x, *q), {"topk_idx": idx, "topk_weights": w, "bias": logits[0]}),
            (ValueError, (x, *q), {"topk_idx": idx, "topk_weights": w, "activation": "relu"}),
            (ValueError, (x, *q), {"topk_idx": idx, "topk_weights": w, "y": x[:2]}),
            (ValueError, (x.cpu(), *q), {"topk_idx": idx, "topk_weights": w}),
            (ep.EpError, (x, *q), {"topk_idx": idx, "topk_weights": w, "y": x}),
            (ep.EpError, (x, *q), {"logits": logits, "top_k": 5}),
            (ep.EpError, (torch.cat([x] * 22), *q), {"logits": torch.cat([logits] * 22), "top_k": 2})):
        with pytest.raises(kind):
            ep.moe_tokens(*args, **kw)
