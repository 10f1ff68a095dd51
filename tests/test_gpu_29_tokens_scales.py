"""The layer for a few tokens with 4-bit weights at the ends of the exponent bytes' range, in both products, and beside rows
of NaN and infinity: against float64, with inputs that make the least and the largest powers count in y."""
import pytest
import torch

from gpu_helpers import dev, say
from mxfp4_reference import decode
from test_gpu_24_moe_tokens import check_y, routing, rows

pytestmark = pytest.mark.gpu

E, K, H, I = 3, 2, 96, 64


def codes_of(rows_, cols, g, small):
    """Random codes; small: of magnitudes up to 3/2, which 2^127 keeps below 2^128."""
    c = torch.randint(0, 256, (E, rows_, cols // 2), device=dev(), generator=g).to(torch.uint8)
    return c & 0xBB if small else c


def layer(up_bytes, down_bytes, seed):
    """Codes and scales whose bytes are drawn from [lo, hi], and their values in float64."""
    import combine_ep_layout_amd as ep
    g = torch.Generator(device=dev()).manual_seed(seed)
    q = []
    for (lo, hi), r, c in ((up_bytes, 2 * I, H), (down_bytes, H, I)):
        scales = torch.randint(lo, hi + 1, (E, r, c // 32), device=dev(), generator=g).to(torch.uint8)
        q.append(ep.Mxfp4(codes_of(r, c, g, hi == 254), scales))
    return q, values_of(q)


def values_of(q):
    return [torch.from_numpy(decode(w.codes.cpu().numpy(), w.scales.cpu().numpy())).to(dev()) for w in q]


@pytest.mark.parametrize("T", [2, 20])
@pytest.mark.parametrize("name,up_bytes,down_bytes,power", [
    # 2^-127 to 2^-125 times x of 2^122; 2^127 and 2^126 times x of 2^-125: g and u of one to some hundred
    ("least, gate and up", (0, 2), (124, 126), 122), ("largest, gate and up", (253, 254), (124, 126), -125),
    # a of some 2^120; a of some 2^-95
    ("least, down", (124, 126), (0, 2), 56), ("largest, down", (124, 126), (253, 254), -51)])
def test_ends_of_the_range(name, up_bytes, down_bytes, power, T):
    import combine_ep_layout_amd as ep
    say(f"[tokens scales] {name} {T}")
    q, (up, down) = layer(up_bytes, down_bytes, T)
    g = torch.Generator(device=dev()).manual_seed(T + 1)
    # magnitudes of 1 to 4: no x is subnormal
    x = (1 + 3 * torch.rand(T, H, device=dev(), generator=g)) * torch.where(torch.rand(T, H, device=dev(), generator=g) < 0.5, -1.0, 1.0)
    x = torch.ldexp(x, torch.tensor(power, device=dev())).bfloat16()
    idx, w = routing(T, E, K, T)
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    assert bool(torch.isfinite(y).all()) and float(y.float().abs().max()) > 1e-3
    check_y(y, x, idx, w, up, down, "silu")
    # the same as the bf16 weights that the codes stand for, all of them exact in bf16
    back = [ep.mxfp4_cast_back(t) for t in q]
    assert torch.equal(back[0].double(), up) and torch.equal(back[1].double(), down)
    check_y(ep.moe_tokens(x, *back, topk_idx=idx, topk_weights=w)[0], x, idx, w, up, down, "silu")


@pytest.mark.parametrize("T", [2, 20])
@pytest.mark.parametrize("row", [5, I + 5])
def test_nan_bytes_in_gate_and_up(row, T):
    """One block of one expert: its tokens' rows are NaN, the others as they were."""
    import combine_ep_layout_amd as ep
    q, _ = layer((124, 126), (124, 126), 3)
    x, (idx, w) = rows(T, H, T), routing(T, E, K, T)
    idx[0] = torch.tensor([0, 2], device=dev())
    idx[1] = torch.tensor([1, 0], device=dev())
    clean = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    q[0].scales[1, row, 1] = 255
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    hit = (idx == 1).any(1)
    assert bool(torch.isnan(y[hit]).all()) and torch.equal(y[~hit], clean[~hit])


def test_past_the_largest_value():
    """A code of 6 under byte 254 is 2^128 and more: infinity, as in the cast back."""
    import combine_ep_layout_amd as ep
    q, (up, down) = layer((124, 126), (124, 126), 4)
    x, idx = rows(3, H, 4), torch.tensor([[1], [0], [1]], dtype=torch.int32, device=dev())
    w = torch.ones(3, 1, device=dev())
    clean = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    q[1].codes[1, 7] = 0
    q[1].codes[1, 7, 3], q[1].scales[1, 7, 0] = 7, 254
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    other = ep.moe_tokens(x, *[ep.mxfp4_cast_back(t) for t in q], topk_idx=idx, topk_weights=w)[0]
    assert bool(torch.isinf(y[[0, 2], 7]).all()) and torch.equal(y[[0, 2], 7], other[[0, 2], 7])
    keep = torch.arange(H, device=dev()) != 7
    assert torch.equal(y[:, keep], clean[:, keep]) and torch.equal(y[1], clean[1])


@pytest.mark.parametrize("T", [5, 18, 40])
def test_rows_of_nan_and_infinity_stay_apart(T):
    """Padding rows of a batch may hold anything, in 4 bits as well."""
    import combine_ep_layout_amd as ep
    q, (up, down) = layer((124, 126), (124, 126), 5)
    wide = torch.full((T, 2 * H), float("nan"), dtype=torch.bfloat16, device=dev())
    x = wide[:, H // 2:H // 2 + H]
    x.copy_(rows(T, H, 5))
    idx, w = routing(T, E, K, 5)
    idx[4] = -1
    clean = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    check_y(clean, x, idx, w, up, down, "silu")
    x[4], x[1], x[3] = float("nan"), float("nan"), float("inf")
    y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
    others = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(y[others], clean[others]) and not y[4].any()
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[3]).any())
