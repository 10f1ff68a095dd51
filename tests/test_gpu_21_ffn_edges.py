"""The experts' feed-forward at the edges of what may be asked of it."""
import pytest
import torch

import test_gpu_16_expert_ffn as base
from gpu_helpers import say, dev

setup = base.setup

pytestmark = pytest.mark.gpu

# Every product in the widest tiles, the activation's gradient among them (which needs two rounds of them in the width of
# inter alone): experts of one partial tile, and of several tiles with a partial last one; odd widths.
#       tokens, top_k, experts, block_m, hidden, inter, routing
WIDE = [
    (2400, 4, 64, 16, 1288, 1320, "uniform"),
    (2400, 4, 64, 100, 1304, 1288, "skewed"),
    (2100, 3, 8, 64, 4360, 4424, "skewed"),
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "-".join(map(str, s)))
def test_widest_tiles(shape, act):
    base.test_forward_and_backward(shape, act)


def test_widest_tiles_meet_every_height():
    """The widest shape has forms of their own for a last tile of at most 64 and at most 128 rows."""
    seen = set()
    for shape in WIDE:
        T, K, E, BM, _, _, kind = shape
        s = setup(T, K, E, BM, 8, 8, kind)
        for _, _, n in s["regions"]:
            left = n % 256
            seen.add((n > 256, "64" if 0 < left <= 64 else "128" if 64 < left <= 128 else "256" if left else "none"))
        s["h"].close()
    assert {(False, h) for h in ("64", "128", "256")} <= seen and {(True, h) for h in ("64", "128", "256")} <= seen, seen


def test_out_over_the_pool_cannot_be_saved():
    """The backward pass reads the pool: saved state beside an overwritten pool would give wrong weight gradients."""
    import combine_ep_layout_amd as ep
    say("[ffn] out over the pool, saved")
    s = setup(40, 2, 4, 16, 64, 32, "uniform")
    h = s["h"]
    before = s["pool"].clone()
    with pytest.raises(ep.EpError) as e:
        h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], out=s["pool"], save=True)
    assert e.value.status == ep.EP_ERR_INVALID_ARGUMENT
    assert torch.equal(s["pool"].view(torch.int16), before.view(torch.int16))
    want, _ = h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], save=True)
    h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], out=s["pool"])       # without the saved state it may
    assert torch.equal(s["pool"][s["real"]], want[s["real"]])
    h.close()


@pytest.mark.parametrize("shape", [(3, 1, 1, 4, 65536, 8192, "uniform"), (5, 1, 1, 4, 8192, 65536, "uniform")],
                         ids=["wide rows", "many rows"])
def test_largest_matrices(shape):
    """One expert of 2^29 values a matrix: gate and up fill 2 GiB, the range of the kernels' offsets inside an expert."""
    import combine_ep_layout_amd as ep
    try:
        base.test_forward_and_backward(shape, "silu")
        T, K, E, BM, H, I, kind = shape
        h = ep.EpHandle(T, K, E, BM)
        e = h.layout(torch.zeros(T, K, dtype=torch.int32, device=dev()), torch.ones(T, K, device=dev()))
        empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev())  # noqa: E731
        I += 8
        with pytest.raises(ep.EpError) as error:                # one step further is refused
            h.expert_ffn(e, empty(h.capacity_rows, H), empty(E, 2 * I, H), empty(E, H, I))
        assert error.value.status == ep.EP_ERR_UNSUPPORTED
        h.close()
    finally:
        torch.cuda.empty_cache()
