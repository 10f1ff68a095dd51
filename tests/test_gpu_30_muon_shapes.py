"""Orthogonalisation and its step in the widest tiles (tests/test_muon_shape_cpu.py holds the sizes to that) where matrices
end inside a tile, inside a step of the summed index and off whole 16 bytes.  Against float64 as in
test_gpu_26_muon.py."""
import numpy as np
import pytest
import torch

import muon_reference as ref
from gpu_helpers import dev, say
from test_gpu_26_muon import in_fp32, step_inputs

pytestmark = pytest.mark.gpu

# batch, rows, cols
WIDE = [(90, 765, 803), (90, 803, 765), (170, 499, 1009), (85, 1009, 499)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", WIDE, ids=str)
def test_partial_wide_tiles(shape, dtype):
    import combine_ep_layout_amd as ep
    say(f"[muon shapes] {shape} {dtype}")
    x = ref.matrices("noise", *shape, dev(), shape[1]).to(dtype)
    out = ep.orthogonalize(x)
    ref.check("X", out, x)
    assert torch.equal(ep.orthogonalize(x), out)
    for steps in (1, 2):
        ref.near(in_fp32(x, steps), x, steps)


@pytest.mark.parametrize("kind", ["low rank", "rows"])
@pytest.mark.parametrize("shape", WIDE[:2], ids=str)
def test_spectra(kind, shape):
    import combine_ep_layout_amd as ep
    say(f"[muon shapes] {kind} {shape}")
    x = ref.matrices(kind, *shape, dev(), 3)
    ref.check("X", ep.orthogonalize(x), x)


@pytest.mark.parametrize("shape", WIDE[:2], ids=str)
@pytest.mark.parametrize("p_dtype,g_dtype,copy", [(torch.float32, torch.bfloat16, True), (torch.bfloat16, torch.float32, False)])
def test_step(p_dtype, g_dtype, copy, shape):
    import combine_ep_layout_amd as ep
    say(f"[muon shapes] step {shape} {p_dtype}")
    s = step_inputs([shape], p_dtype, g_dtype, copy, 0)
    lr, mu, wd = 3e-2, 0.9, 0.1
    before, m0 = s["params"][0].double(), s["momenta"][0].double()
    ep.muon(s["params"], s["grads"], s["momenta"], lr=lr, momentum=mu, weight_decay=wd, copies=s["copies"])
    g, m = s["grads"][0].double(), s["momenta"][0].double()
    # two products, a sum, the two factors: half steps of 2^-24 each
    assert bool(((m - (mu * m0 + (1 - mu) * g)).abs() <= 4 * 2.0 ** -24 * (m0.abs() + g.abs())).all())
    u = ((1 - mu) * g + mu * m).float()
    # the parameter's own rounding and four fp32 operations on it
    half = (2.0 ** -24 if p_dtype == torch.float32 else ref.H_BF16) + 4 * 2.0 ** -24
    ref.check("step", s["params"][0], u, factor=-lr * 0.2 * max(shape[1:]) ** 0.5, add=before * (1 - lr * wd), rounding=half)
    if copy:
        assert torch.equal(s["copies"][0], s["params"][0].bfloat16())


def workspace_bytes(*shape):
    import combine_ep_layout_amd as ep
    t = np.zeros(1, ep._MUON_TENSOR)
    t["batch"], t["rows"], t["cols"] = shape
    return int(ep.library().ep_muon_workspace_bytes(t.ctypes.data, 1))


@pytest.mark.parametrize("shape", WIDE, ids=str)
def test_the_workspace_changes_no_result(shape):
    """One matrix, or some, at once take smaller tiles."""
    import combine_ep_layout_amd as ep
    x = ref.matrices("decay", *shape, dev(), 9)
    want = ep.orthogonalize(x)
    one = workspace_bytes(1, *shape[1:])
    for n in (1, 20):
        assert torch.equal(ep.orthogonalize(x, workspace=torch.empty(n * one, dtype=torch.uint8, device=dev())), want), n


@pytest.mark.parametrize("shape", WIDE[:2], ids=str)
def test_what_lies_around_stays(shape):
    """Partial tiles end at the matrices' ends, in the results and in the workspace."""
    import combine_ep_layout_amd as ep
    x = ref.matrices("noise", *shape, dev(), 5).bfloat16()
    want = ep.orthogonalize(x)
    size = workspace_bytes(*shape)
    room = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device=dev())         # NaN wherever it is read first
    out_room = torch.full((x.numel() + 64,), 7.0, dtype=torch.bfloat16, device=dev())
    out = out_room[32:-32].view(shape)
    ep.orthogonalize(x, workspace=room[256:-256], out=out)
    assert torch.equal(out, want)
    assert bool((room[:256] == 0xFF).all()) and bool((room[-256:] == 0xFF).all())
    assert bool((out_room[:32] == 7).all()) and bool((out_room[-32:] == 7).all())


def test_millions_of_tiny_matrices():
    """More than one launch holds, in a list and in one tensor."""
    import combine_ep_layout_amd as ep
    n = 1 << 20
    base = ref.matrices("noise", 64, 1, 1, dev(), 8)
    x = base.repeat(n // 64, 1, 1)
    want = in_fp32(base, 5)
    ref.check("X", want, base, rounding=2.0 ** -24)
    params = [torch.zeros(n, 1, 1, device=dev()) for _ in range(9)]
    ep.muon(params, [x.clone() for _ in params], [torch.zeros_like(x) for _ in params], lr=-1.0, momentum=0.0,
            weight_decay=0.0, nesterov=False, scale=1.0)
    for p in params:
        assert torch.equal(p.view(-1, 64, 1, 1), want.expand(n // 64, 64, 1, 1))
    base = ref.matrices("noise", 64, 3, 5, dev(), 9)
    out = ep.orthogonalize(base.repeat(n // 64, 1, 1))
    assert torch.equal(out.view(-1, 64, 3, 5), ep.orthogonalize(base).expand(n // 64, 64, 3, 5))
