"""The experts' gated feed-forward and its backward pass on the GPU against
float64, element by element within bounds derived from the roundings
(ffn_reference.py): every launch shape, ragged rows, widths off every tile
size, experts without rows, masked slots, tokens without a slot; rows outside
the regions keep their contents and are never read (they hold NaN)."""
import pytest
import torch

import ffn_reference as ref
from gpu_helpers import say, dev

pytestmark = pytest.mark.gpu

#        tokens, top_k, experts, block_m, hidden, inter, routing
SHAPES = [
    (1, 1, 1, 1, 8, 8, "uniform"),
    (1, 8, 64, 64, 512, 256, "uniform"),
    (2, 1, 4, 16, 64, 32, "uniform"),
    (5, 2, 3, 100, 72, 40, "uniform"),
    (33, 3, 24, 16, 200, 136, "masked"),
    (100, 4, 16, 7, 328, 104, "uniform"),      # 25 rows on average: 64-row tiles
    (64, 2, 2, 128, 136, 264, "uniform"),      # 64 rows: 128-row tiles
    (129, 2, 3, 64, 264, 200, "masked"),
    (300, 1, 1, 128, 520, 264, "uniform"),     # one expert: 256-row tiles, a partial second one
    (257, 4, 4, 1, 256, 512, "uniform"),       # no padding rows at all
    (513, 2, 3, 100, 1032, 296, "skewed"),
    (700, 2, 5, 4096, 128, 128, "skewed"),
    (1000, 1, 1024, 1, 64, 48, "skewed"),      # most experts without a row
    (40, 32, 40, 16, 128, 64, "uniform"),      # every expert of every token
    # two rounds of tiles: the widest shape in every product
    (2400, 4, 64, 16, 1288, 648, "uniform"),
    (2400, 4, 64, 100, 1288, 648, "skewed"),
    # few rows, more tiles than compute units: 64 x 128 tiles
    (1280, 2, 128, 16, 400, 400, "uniform"),
]


def routing(T, K, E, kind, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    score = torch.rand(T, E, device=dev(), generator=g)
    if kind == "skewed":                    # most rows to a few experts
        score += 2.0 / (1 + torch.arange(E, device=dev(), dtype=torch.float32))
    idx = score.topk(K, dim=1).indices.to(torch.int32)
    if kind == "masked":
        idx[torch.rand(T, K, device=dev(), generator=g) < 0.4] = -1
        idx[: T // 4] = -1                  # tokens without any slot
    if kind == "none":
        idx.fill_(-1)
    return idx.contiguous()


def setup(T, K, E, BM, H, I, kind, seed=0):
    import combine_ep_layout_amd as ep
    idx = routing(T, K, E, kind, seed)
    h = ep.EpHandle(T, K, E, BM)
    epoch = h.layout(idx, torch.ones(T, K, device=dev()))
    counts = h.array("expert_counts").cpu().tolist()
    starts = [o * BM for o in h.array("expert_pool_block_offset").cpu().tolist()]
    g = torch.Generator(device=dev()).manual_seed(seed + 1)
    normal = lambda *s, std=1.0: torch.empty(s, device=dev(), dtype=torch.bfloat16).normal_(0, std, generator=g)
    cap = h.capacity_rows
    real = torch.zeros(cap, dtype=torch.bool, device=dev())
    for e in range(E):
        real[starts[e]:starts[e] + counts[e]] = True
    pool = torch.full((cap, H), float("nan"), dtype=torch.bfloat16, device=dev())
    grad = pool.clone()
    n = int(real.sum())
    pool[real] = normal(n, H)
    grad[real] = normal(n, H)
    return dict(h=h, epoch=epoch, regions=[(e, starts[e], counts[e]) for e in range(E)], real=real, pool=pool, grad=grad,
                wgu=normal(E, 2 * I, H, std=H ** -0.5), wd=normal(E, H, I, std=I ** -0.5))


def poisoned(shape, dtype):
    return torch.full(shape, 123.0, dtype=dtype, device=dev())


def check_all(s, kind, outputs, grad=False):
    """outputs: name -> tensor over pool rows or experts."""
    rounds = {torch.bfloat16: ref.H_BF16, torch.float32: 2.0 ** -24}
    for e, a, n in s["regions"]:
        x, gu, d = s["pool"][a:a + n].double(), s["wgu"][e].double(), s["wd"][e].double()
        r = ref.expert(x, gu, d, kind, s["grad"][a:a + n].double() if grad else None)
        for name, got in outputs.items():
            value, bound = r[name]
            if name.startswith("grad_w"):
                bound = bound + rounds[got.dtype] * (value.abs() + bound)
                ref.check(f"{name} of expert {e}", got[e], value, bound)
            else:
                ref.check(f"{name} of expert {e}", got[a:a + n], value, bound)
    for name, got in outputs.items():
        if not name.startswith("grad_w"):
            assert bool((got[~s["real"]] == 123.0).all()), f"{name}: a row outside the regions was written"


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_forward_and_backward(shape, act):
    T, K, E, BM, H, I, kind = shape
    say(f"[ffn] {shape} {act}")
    s = setup(*shape)
    h, cap = s["h"], s["h"].capacity_rows
    bf, f32 = torch.bfloat16, torch.float32
    out, a, gu = poisoned((cap, H), bf), poisoned((cap, I), bf), poisoned((cap, 2 * I), f32)
    h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], act, out=out, act=a, gate_up=gu, save=True)
    check_all(s, act, {"out": out, "act": a, "gate_up": gu})
    plain = poisoned((cap, H), bf)
    h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], act, out=plain)
    assert torch.equal(plain, out)                          # saving changes nothing

    import combine_ep_layout_amd as ep
    gp, dgu = poisoned((cap, H), bf), poisoned((cap, 2 * I), bf)
    args = (s["epoch"], s["grad"], s["pool"], s["wgu"], s["wd"], ep.FfnSaved(a, gu), act)
    _, gw, gd = h.expert_ffn_backward(*args, grad_pool=gp, grad_gate_up=dgu)
    assert gw.dtype == bf and gd.dtype == bf
    check_all(s, act, {"grad_gate_up": dgu, "grad_pool": gp, "grad_w_gate_up": gw, "grad_w_down": gd}, grad=True)
    gw32, gd32 = poisoned((E, 2 * I, H), f32), poisoned((E, H, I), f32)
    h.expert_ffn_backward(*args, grad_w_gate_up=gw32, grad_w_down=gd32)
    check_all(s, act, {"grad_w_gate_up": gw32, "grad_w_down": gd32}, grad=True)
    # the two types come from the same sums
    assert torch.equal(gw32.to(bf), gw) and torch.equal(gd32.to(bf), gd)
    twice_w, twice_d = gw32.clone(), gd32.clone()
    h.expert_ffn_backward(*args, grad_w_gate_up=twice_w, grad_w_down=twice_d, accumulate=True)
    assert torch.equal(twice_w, 2 * gw32) and torch.equal(twice_d, 2 * gd32)
    h.close()


def test_no_tokens_and_all_masked():
    for T, kind in ((0, "uniform"), (9, "none")):
        s = setup(T, 2, 4, 16, 64, 32, kind)
        h, cap = s["h"], s["h"].capacity_rows
        out = poisoned((cap, 64), torch.bfloat16)
        _, saved = h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], out=out, save=True)
        assert bool((out == 123.0).all())
        _, gw, gd = h.expert_ffn_backward(s["epoch"], s["grad"], s["pool"], s["wgu"], s["wd"], saved)
        assert not gw.any() and not gd.any()                # no rows: zero gradients, not what memory held
        h.close()


def test_out_may_be_the_pool():
    s = setup(300, 2, 4, 16, 256, 128, "uniform")
    h = s["h"]
    want = h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], out=torch.full_like(s["pool"], 5.0))
    h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], out=s["pool"])
    assert torch.equal(s["pool"][s["real"]], want[s["real"]]) and bool(s["pool"][~s["real"]].isnan().all())
    h.close()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_pre_activations_far_out(act):
    """Gates of huge magnitude: the activation is 0 or the gate itself, its slope 0 or 1, and nothing is NaN."""
    import combine_ep_layout_amd as ep
    h = ep.EpHandle(4, 1, 1, 4)
    e = h.layout(torch.zeros(4, 1, dtype=torch.int32, device=dev()), torch.ones(4, 1, device=dev()))
    bf = torch.bfloat16
    gates = torch.tensor([1e30, -1e30, 3e4, -3e4], device=dev())
    pool = torch.zeros(h.capacity_rows, 8, dtype=bf, device=dev())
    pool[:4, 0], pool[:4, 1] = gates.to(bf), 1.0
    wgu = torch.zeros(1, 16, 8, dtype=bf, device=dev())
    wgu[0, :8, 0], wgu[0, 8:, 1] = 1.0, 1.0                     # gate = the first channel, up = 1
    wd = torch.eye(8, dtype=bf, device=dev())[None].contiguous()
    out, saved = h.expert_ffn(e, pool, wgu, wd, act, save=True)
    want = torch.where(gates > 0, gates, torch.zeros_like(gates)).to(bf)
    assert torch.equal(out[:4], want[:, None].expand(4, 8))
    d = torch.empty(h.capacity_rows, 16, dtype=bf, device=dev())
    h.expert_ffn_backward(e, torch.ones_like(pool), pool, wgu, wd, saved, act, grad_gate_up=d)
    assert torch.equal(d[:4, :8], (gates > 0).to(bf)[:, None].expand(4, 8))
    assert torch.equal(d[:4, 8:], want[:, None].expand(4, 8))
    h.close()


def test_gradient_against_differences():
    """sum(out * grad) along random directions: central differences of the float64 forward formula."""
    s = setup(60, 2, 3, 16, 64, 40, "uniform")
    h = s["h"]
    _, saved = h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], "gelu", save=True)
    gp, gw, gd = h.expert_ffn_backward(s["epoch"], s["grad"], s["pool"], s["wgu"], s["wd"], saved, "gelu",
                                       grad_w_gate_up=torch.empty(s["wgu"].shape, device=dev()),
                                       grad_w_down=torch.empty(s["wd"].shape, device=dev()))
    g = torch.Generator(device=dev()).manual_seed(5)
    pool, wgu, wd = (t.double() for t in (s["pool"], s["wgu"], s["wd"]))
    dirs = [torch.randn(t.shape, dtype=torch.float64, device=dev(), generator=g) for t in (pool, wgu, wd)]

    def value(eps, which):
        p, w, d = (t + (eps * v if i == which else 0) for i, (t, v) in enumerate(zip((pool, wgu, wd), dirs)))
        return sum((ref.expert(p[a:a + n], w[e], d[e], "gelu")["out"][0] * s["grad"][a:a + n].double()).sum()
                   for e, a, n in s["regions"])

    for which, (grad, where) in enumerate(((gp, s["real"]), (gw, slice(None)), (gd, slice(None)))):
        slope = (value(1e-5, which) - value(-1e-5, which)) / 2e-5
        terms = grad[where].double() * dirs[which][where]
        # each gradient value is within three bf16 roundings of itself on average; the errors are independent
        tol = 3 * 2.0 ** -8 * float(terms.square().sum().sqrt()) * 4
        assert abs(float(terms.sum() - slope)) <= tol, (which, float(terms.sum()), float(slope), tol)
    h.close()
