"""The layer for a few tokens at sizes that take each form of its kernels (tests/test_tokens_shape_cpu.py holds them to
that), among them those of large layers: two row tiles a workgroup in the down product, four in the gate and up products,
partial tiles and steps at every end.  Against float64 with the bounds of test_gpu_24_moe_tokens.py."""
import pytest
import torch

from gpu_helpers import dev, say
from test_gpu_24_moe_tokens import check_y, routing, rows

pytestmark = pytest.mark.gpu

# T, E, K, H, I, form on 256 compute units: ((row tiles, groups) of the 4-bit gate and up products, down's row tiles)
SHAPES = [
    # hidden past 4096, by a whole tile, half a tile and (bf16) eight rows
    (1, 6, 2, 4128, 96, ((1, 1), 2)), (5, 6, 3, 4112, 104, ((1, 1), 2)), (16, 4, 2, 4104, 72, ((1, 1), 2)),
    (7, 12, 4, 4128, 544, ((2, 1), 2)), (17, 5, 2, 4128, 160, ((1, 1), 2)), (40, 6, 3, 4104, 136, ((1, 1), 2)),
    (64, 12, 5, 4160, 544, ((2, 1), 2)),
    # four row tiles a workgroup, whose last is partial, with uneven shares of the summed index
    (8, 40, 8, 544, 224, ((2, 2), 1)), (16, 40, 8, 96, 224, ((2, 2), 1)), (20, 40, 8, 544, 224, ((2, 2), 1)),
    (64, 40, 8, 1312, 224, ((2, 2), 1)), (33, 5, 5, 160, 1760, ((2, 2), 1)),
    # both, and an expert that every token chooses
    (3, 64, 8, 4128, 416, ((2, 2), 2)), (50, 3, 3, 4128, 2848, ((2, 2), 2)),
    # two row tiles a wave, one group
    (6, 40, 8, 352, 160, ((2, 1), 1)), (24, 40, 8, 352, 160, ((2, 1), 1)),
]
# T, E, K, H, I of calls from logits
CHOICES = [(1, 64, 8, 4128, 1056, None), (8, 40, 8, 544, 224, None), (4, 100, 8, 160, 160, None), (2, 5, 2, 4128, 64, None),
           (3, 64, 8, 4128, 416, None)]


def weights(E, H, I, four, seed):
    """As the call takes them, and their float64 values."""
    import combine_ep_layout_amd as ep
    g = torch.Generator(device=dev()).manual_seed(seed)
    up, down = ((torch.randn(E, r, c, device=dev(), generator=g) * c ** -0.5).bfloat16() for r, c in ((2 * I, H), (H, I)))
    if not four:
        return (up, down), (up.double(), down.double())
    q = [ep.mxfp4_quantize(w) for w in (up, down)]
    return q, [ep.mxfp4_cast_back(w).double() for w in q]


def forms(cases):
    return [pytest.param(c, four, id="-".join(map(str, (*c[:5], "4bit" if four else "bf16"))))
            for c in cases for four in (False, True) if not four or (c[3] % 32 == 0 and c[4] % 32 == 0)]


@pytest.mark.parametrize("case,four", forms(SHAPES))
def test_given_choice(case, four):
    import combine_ep_layout_amd as ep
    T, E, K, H, I, _ = case
    say(f"[tokens shapes] {case} {'4 bit' if four else 'bf16'}")
    q, (up, down) = weights(E, H, I, four, T)
    x = rows(T, H, T)
    for masked, kind in ((0.0, "silu"), (0.4, "gelu")):
        idx, w = routing(T, E, K, T, masked)
        y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w, activation=kind)[0]
        check_y(y, x, idx, w, up, down, kind)
        assert torch.equal(ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w, activation=kind)[0], y)


@pytest.mark.parametrize("case,four", forms(CHOICES))
def test_choice_from_logits(case, four):
    import combine_ep_layout_amd as ep
    T, E, K, H, I, _ = case
    say(f"[tokens shapes] logits {case} {'4 bit' if four else 'bf16'}")
    q, (up, down) = weights(E, H, I, four, T + 1)
    x, logits = rows(T, H, T), torch.randn(T, E, device=dev(), generator=torch.Generator(device=dev()).manual_seed(E))
    y, idx, w = ep.moe_tokens(x, *q, logits=logits, top_k=K, score="sigmoid", scale=2.5)
    assert torch.equal(idx, ep.route(logits, K, score="sigmoid", scale=2.5)[0])
    check_y(y, x, idx, w, up, down, "silu")
