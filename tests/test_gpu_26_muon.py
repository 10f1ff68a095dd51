"""Orthogonalisation by Newton-Schulz products and the optimiser step on it, against float64 with the kernels' own
roundings to fp16 put in (and through that against the definition): odd and one-wide sizes, tall and wide, every tile
shape, spectra from noise to low rank, workspaces that hold one matrix, lists of many shapes, graphs, streams, broken
matrices beside whole ones."""
import pytest
import torch

import muon_reference as ref
from gpu_helpers import dev, say

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (3, 1, 7), (2, 7, 1), (1, 16, 16), (2, 33, 65), (3, 65, 33), (1, 130, 257), (2, 300, 1000), (1, 513, 511),
          (1, 1000, 72), (2, 8, 4096), (260, 100, 40), (260, 20, 130), (20, 520, 600), (1, 1, 5000)]


def in_fp32(x, steps):
    """X unrounded: the step of parameters that are zero."""
    import combine_ep_layout_amd as ep
    p, m = torch.zeros(x.shape, device=dev()), torch.zeros(x.shape, device=dev())
    ep.muon([p], [x], [m], lr=-1.0, momentum=0.0, weight_decay=0.0, nesterov=False, scale=1.0, steps=steps)
    return p


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, dtype):
    import combine_ep_layout_amd as ep
    say(f"[orthogonalize] {shape} {dtype}")
    x = ref.matrices("noise", *shape, dev(), shape[1]).to(dtype)
    out = ep.orthogonalize(x)
    assert out.dtype == torch.bfloat16 and out.shape == x.shape
    ref.check("X", out, x)
    assert torch.equal(ep.orthogonalize(x), out)
    for steps in (1, 2):
        ref.near(in_fp32(x, steps), x, steps)


@pytest.mark.parametrize("kind", ["noise", "low rank", "decay", "rows"])
@pytest.mark.parametrize("shape", [(2, 200, 336), (2, 336, 200), (48, 260, 300), (48, 300, 260), (3, 1024, 1024)], ids=str)
def test_spectra(kind, shape):
    """The last but one take the widest tiles in every product."""
    import combine_ep_layout_amd as ep
    say(f"[orthogonalize] {kind} {shape}")
    x = ref.matrices(kind, *shape, dev(), 3)
    ref.check("X", ep.orthogonalize(x), x)
    for steps in (1, 2):
        ref.near(in_fp32(x, steps), x, steps)


@pytest.mark.parametrize("steps,abc,eps", [(1, (3.4445, -4.775, 2.0315), 1e-7), (2, (1.5, -0.5, 0.0), 0.0), (10, (2.0, -1.5, 0.5), 1e-3),
                                           (3, (1.0, 0.0, 0.0), 0.5)])
def test_steps_and_coefficients(steps, abc, eps):
    import combine_ep_layout_amd as ep
    x = ref.matrices("noise", 2, 70, 90, dev(), steps)
    x /= torch.linalg.matrix_norm(x, keepdim=True)      # where eps counts
    out = ep.orthogonalize(x, steps=steps, coefficients=abc, eps=eps)
    ref.check("X", out, x, steps, abc, eps)


def test_tiny_huge_and_broken_matrices():
    import combine_ep_layout_amd as ep
    x = ref.matrices("noise", 6, 40, 50, dev(), 1)
    x[0] *= 1e-35
    x[1] *= 1e35
    x[2] = 0
    good = ep.orthogonalize(x, eps=0.0)
    ref.check("X", good, x, eps=0.0)
    assert not good[2].any()
    x[3, 5, 5], x[4, 0, 49] = float("nan"), float("inf")
    out = ep.orthogonalize(x, eps=0.0)
    assert torch.equal(out[[0, 1, 2, 5]], good[[0, 1, 2, 5]])
    assert bool(torch.isnan(out[3]).any()) and bool(torch.isnan(out[4]).any())
    # with a larger eps than the matrix the result is small, not orthogonal
    assert float(ep.orthogonalize(x[:1], eps=1.0).float().abs().max()) < 1e-30


@pytest.mark.parametrize("shape", [(7, 90, 130), (5, 257, 64)], ids=str)
def test_workspace_of_one_matrix(shape):
    """Fewer matrices at once, the same results; what lies around the buffers stays."""
    import combine_ep_layout_amd as ep
    x = ref.matrices("decay", *shape, dev(), 2)
    want = ep.orthogonalize(x)
    import numpy as np
    t = np.zeros(1, ep._MUON_TENSOR)
    t["batch"], t["rows"], t["cols"] = 1, *shape[1:]
    one = int(ep.library().ep_muon_workspace_bytes(t.ctypes.data, 1))
    for size in (one, 3 * one + 16):
        room = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device=dev())     # NaN wherever it is read first
        out_room = torch.full((x.numel() + 64,), 7.0, dtype=torch.bfloat16, device=dev())
        out = out_room[32:-32].view(shape)
        ep.orthogonalize(x, workspace=room[256:-256], out=out)
        assert torch.equal(out, want)
        assert bool((room[:256] == 0xFF).all()) and bool((room[-256:] == 0xFF).all())
        assert bool((out_room[:32] == 7).all()) and bool((out_room[-32:] == 7).all())
    with pytest.raises(ep.EpError):
        ep.orthogonalize(x, workspace=room[:one // 16 * 16 - 16])


@pytest.mark.parametrize("shape", [(90, 768, 800), (90, 800, 768)], ids=str)
def test_whole_rounds_and_a_rest(shape):
    """Batches whose products go to wide tiles in whole rounds of 256 compute units and to middle ones for the rest."""
    import combine_ep_layout_amd as ep
    x = ref.matrices("noise", *shape, dev(), 11).bfloat16()
    out = ep.orthogonalize(x)
    ref.check("X", out, x)
    assert torch.equal(ep.orthogonalize(x), out)
    ref.near(in_fp32(x, 2), x, 2)


def test_a_rest_of_two_tensors():
    """The rest of the wide tiles' rounds takes one tensor whole and the last matrix of another."""
    import combine_ep_layout_amd as ep
    shapes = [(86, 768, 800), (2, 530, 520)]
    x = [ref.matrices("noise", *s, dev(), s[1]).bfloat16() for s in shapes]
    p, m = ([torch.zeros(s, device=dev()) for s in shapes] for _ in range(2))
    ep.muon(p, x, m, lr=-1.0, momentum=0.0, weight_decay=0.0, nesterov=False, scale=1.0, steps=2)
    for got, u in zip(p, x):
        ref.near(got, u, 2)


def step_inputs(shapes, p_dtype, g_dtype, copy, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    n = lambda s, std: torch.randn(s, device=dev(), generator=g) * std
    return {"params": [n(s, 0.02).to(p_dtype) for s in shapes], "grads": [n(s, 1e-3).to(g_dtype) for s in shapes],
            "momenta": [n(s, 1e-3) for s in shapes],
            "copies": [torch.full(s, 9.0, dtype=torch.bfloat16, device=dev()) for s in shapes] if copy else None}


LIST = [(2, 40, 72), (72, 40), (1, 1, 9), (3, 300, 129), (0, 5, 5), (2, 2, 64, 64), (1, 129, 300)]


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("p_dtype,g_dtype,copy", [(torch.float32, torch.bfloat16, True), (torch.float32, torch.float32, False),
                                                  (torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, False)])
def test_step(p_dtype, g_dtype, copy, nesterov):
    import combine_ep_layout_amd as ep
    s = step_inputs(LIST, p_dtype, g_dtype, copy, 0)
    lr, mu, wd = 3e-2, 0.9, 0.1
    for scale in (None, 1.0):
        before = {k: [t.clone() for t in s[k]] for k in ("params", "momenta")}
        ep.muon(s["params"], s["grads"], s["momenta"], lr=lr, momentum=mu, weight_decay=wd, nesterov=nesterov, scale=scale,
                copies=s["copies"])
        for i, shape in enumerate(LIST):
            if 0 in shape:
                continue
            g, m0 = s["grads"][i].double(), before["momenta"][i].double()
            m = mu * m0 + (1 - mu) * g
            # two products, a sum, the two factors: half steps of 2^-24 each
            assert bool(((s["momenta"][i].double() - m).abs() <= 4 * 2.0 ** -24 * (m0.abs() + g.abs())).all())
            m = s["momenta"][i].double()
            u = ((1 - mu) * g + mu * m if nesterov else m).float()
            f = lr * (scale or 0.2 * max(shape[-2:]) ** 0.5)
            # the parameter's own rounding and four fp32 operations on it
            half = (2.0 ** -24 if p_dtype == torch.float32 else ref.H_BF16) + 4 * 2.0 ** -24
            ref.check(f"step of {shape}", s["params"][i], u, factor=-f, add=before["params"][i].double() * (1 - lr * wd), rounding=half)
            if copy:
                assert torch.equal(s["copies"][i], s["params"][i].bfloat16())


def test_a_list_is_its_tensors_one_by_one():
    """More shapes than one launch takes, tall and wide; the workspace's size changes nothing."""
    import combine_ep_layout_amd as ep
    shapes = [(1 + i % 3, 8 + 5 * i % 70, 11 + 7 * i % 90) for i in range(95)]
    s, one = (step_inputs(shapes, torch.float32, torch.bfloat16, True, 1) for _ in range(2))
    few = step_inputs(shapes, torch.float32, torch.bfloat16, True, 1)
    ep.muon(s["params"], s["grads"], s["momenta"], copies=s["copies"])
    ep.muon(few["params"], few["grads"], few["momenta"], copies=few["copies"],
            workspace=torch.empty(200000, dtype=torch.uint8, device=dev()))
    for i in range(len(shapes)):
        ep.muon([one["params"][i]], [one["grads"][i]], [one["momenta"][i]], copies=[one["copies"][i]])
    # twice what check() allows either
    noises = {shape: ref.noise((0.05 * g.double() + 0.95 * m.double()).float())[1][0]
              for shape, g, m in zip(shapes, s["grads"], s["momenta"])}
    for k in ("params", "momenta", "copies"):
        for a, b, c, shape in zip(s[k], one[k], few[k], shapes):
            assert torch.equal(a, c), (k, shape)
            # alone, smaller tiles may serve: sums in another order, other roundings of the same number
            if k == "momenta":
                assert torch.equal(a, b)
                continue
            f = 1e-3 * 0.2 * max(shape[1:]) ** 0.5
            off = torch.linalg.matrix_norm(a.double() - b.double())
            limit = 2 * 2 * f * noises[shape] + 2 * (2.0 ** -24 if k == "params" else ref.H_BF16) * torch.linalg.matrix_norm(a.double())
            assert bool((off <= limit).all()), (k, shape)


def test_captured_and_replayed():
    import combine_ep_layout_amd as ep
    shapes = [(2, 64, 200), (3, 130, 64)]
    s, e = (step_inputs(shapes, torch.float32, torch.bfloat16, True, 2) for _ in range(2))
    x = torch.randn(2, 64, 200, device=dev())
    ep.orthogonalize(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.muon(s["params"], s["grads"], s["momenta"], copies=s["copies"])
        out = ep.orthogonalize(x)
    for seed in range(3):
        for a, b in zip(s["grads"], e["grads"]):
            a.copy_(torch.randn(a.shape, device=dev(), generator=torch.Generator(device=dev()).manual_seed(seed)))
            b.copy_(a)
        x.copy_(torch.randn(2, 64, 200, device=dev()))
        graph.replay()
        torch.cuda.synchronize()
        ep.muon(e["params"], e["grads"], e["momenta"], copies=e["copies"])
        assert torch.equal(out, ep.orthogonalize(x))
        for k in ("params", "momenta", "copies"):
            assert all(torch.equal(a, b) for a, b in zip(s[k], e[k]))


def test_another_stream():
    import combine_ep_layout_amd as ep
    x = [torch.randn(2, 100, 60 + i, device=dev()) for i in range(4)]
    want = [ep.orthogonalize(t) for t in x]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [ep.orthogonalize(t, stream=side[i % 2]) for i, t in enumerate(x)]
    for q in side:
        torch.cuda.current_stream().wait_stream(q)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refusals():
    import combine_ep_layout_amd as ep
    x = torch.randn(2, 16, 24, device=dev())
    p, g, m = x.clone(), x.clone(), x.clone()
    for kind, call in ((TypeError, lambda: ep.orthogonalize(x.half())), (ValueError, lambda: ep.orthogonalize(x[0, 0])),
                       (ValueError, lambda: ep.orthogonalize(x.mT)), (ValueError, lambda: ep.orthogonalize(x.cpu())),
                       (TypeError, lambda: ep.orthogonalize(x, out=x.clone())), (ep.EpError, lambda: ep.orthogonalize(x, steps=0)),
                       (ValueError, lambda: ep.orthogonalize(x, out=x[:1].bfloat16())),
                       (ValueError, lambda: ep.muon([p], [g], [m, m])), (ValueError, lambda: ep.muon([p], [g.view(2, 24, 16)], [m])),
                       (TypeError, lambda: ep.muon([p], [g], [m.bfloat16()])), (TypeError, lambda: ep.muon([p], [g.half()], [m])),
                       (ValueError, lambda: ep.muon([p], [g], [m], scale=0.0)), (ep.EpError, lambda: ep.muon([p], [p], [m])),
                       (ValueError, lambda: ep.muon([p[0, 0]], [g[0, 0]], [m[0, 0]])),
                       (ep.EpError, lambda: ep.muon([p], [g], [m], momentum=1.0))):
        with pytest.raises(kind):
            call()
    ep.muon([], [], [])
