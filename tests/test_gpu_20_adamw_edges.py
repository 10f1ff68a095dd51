"""AdamW at the ends of its range: gradients whose square leaves fp32, and the step's number on the device against the
host's."""
import pytest
import torch

from gpu_helpers import say, dev

pytestmark = pytest.mark.gpu

HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05)


def states(n, seed=0):
    """8-bit states of n values: codes of magnitude 1 to 8 (m of either sign), scale 1/64 for each 128 values."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    r = lambda: torch.randn(n, device=dev(), generator=g)
    code = lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)
    scale = lambda: torch.full(((n + 127) // 128,), 1.0 / 64, device=dev())
    m = torch.where(r() < 0, -1.0, 1.0) * (1 + r().abs().clamp(max=7))
    return dict(params=[r()], grads=[r()], exp_avgs=[code(m)], exp_avg_scales=[scale()],
                exp_avg_sqs=[code(1 + r().abs().clamp(max=7))], exp_avg_sq_scales=[scale()])


def decode(s, k):
    n = s[k + "s"][0].numel()
    return s[k + "s"][0].view(torch.float8_e4m3fn).float() * s[k + "_scales"][0].repeat_interleave(128)[:n]


def clone(s):
    return {k: [t.clone() for t in v] for k, v in s.items()}


@pytest.mark.parametrize("n,at", [(300, 140), (300, 299), (128, 0), (129, 128), (5000, 4097)])
def test_a_square_past_fp32_makes_its_block_nan(n, at):
    """A finite gradient of 1e20: its square is infinite, and one scale holds the block.  Nothing in the block may stand
    for infinity, which would freeze the neighbours (m / inf = 0) without a sign of it."""
    import combine_ep_layout_amd as ep
    say(f"[adamw] square past fp32: {n} {at}")
    s = states(n)
    plain = clone(s)
    s["grads"][0][at] = 1e20
    plain["grads"][0][at] = 0.0
    block = torch.zeros(n, dtype=torch.bool, device=dev())
    block[at // 128 * 128:(at // 128 + 1) * 128] = True
    for step in (1, 2):
        ep.adamw(**s, step=step, **HYPER)
        ep.adamw(**plain, step=step, **HYPER)
        root = decode(s, "exp_avg_sq")
        assert bool(root[block].isnan().all())
        assert torch.equal(root[~block], decode(plain, "exp_avg_sq")[~block])
        assert torch.equal(s["params"][0][~block], plain["params"][0][~block])
        if step == 1:
            assert bool(s["params"][0].isfinite().all())        # m / inf = 0: the step itself is defined
            assert bool(decode(s, "exp_avg").isfinite().all())
        s["grads"][0][at] = 0.0
    assert bool(s["params"][0][block].isnan().all())            # and the lost state shows at the next step


def test_largest_square_that_fp32_holds():
    """Just below: v stays finite, and so does every code of the block."""
    import combine_ep_layout_amd as ep
    s = states(256)
    s["grads"][0][7] = 1.8e19           # squared 3.2e38, below 3.4e38
    ep.adamw(**s, step=1, **HYPER)
    root = decode(s, "exp_avg_sq")
    assert bool(root.isfinite().all()) and bool((root > 0).all())
