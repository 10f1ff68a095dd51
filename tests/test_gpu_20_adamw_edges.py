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


@pytest.mark.parametrize("eight", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("lr", [1e-3, 3e-4, 7e-4, 2.5e-3, 1e-2])
def test_the_step_on_the_device_is_the_hosts(lr, eight):
    """Bit for bit: an eager run and the replays of a captured one must not drift apart.  The step's two factors are
    computed in double from the same numbers and rounded once; the two sides' pow differ by a few units in 2^-53 at most,
    which 1 - beta2 = 1e-3 at step 1 magnifies to 2^-42, so a rounding to 2^-24 parts them once in 2^17 numbers."""
    import combine_ep_layout_amd as ep
    s = states(1000, seed=1)
    if not eight:
        g = torch.Generator(device=dev()).manual_seed(2)
        r = lambda: torch.randn(1000, device=dev(), generator=g)
        s.update(exp_avgs=[0.1 * r()], exp_avg_sqs=[r().square()], exp_avg_scales=None, exp_avg_sq_scales=None)
    copy = lambda: {k: None if v is None else [t.clone() for t in v] for k, v in s.items()}
    for beta1 in (0.9, 0.95):
        for step in (1, 2, 3, 7, 100, 1000):
            host, device = copy(), copy()
            how = dict(lr=lr, beta1=beta1, beta2=0.999, eps=1e-8, weight_decay=0.1)
            ep.adamw(**host, step=step, **how)
            ep.adamw(**device, step=torch.tensor([step], device=dev()), **how)
            for k, v in host.items():
                assert v is None or torch.equal(v[0], device[k][0]), (k, beta1, step)
