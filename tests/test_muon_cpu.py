"""Refusals of ep_muon and ep_orthogonalize (host checks only, nothing is launched), the size of their workspace, their
flags and structures against the header, and what fp16 products cost, on the CPU in float64."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import muon_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x1000000000 * (i + 1) for i in range(12)]       # aligned addresses that nothing follows


@pytest.fixture(scope="module")
def ep():
    import combine_ep_layout_amd
    return combine_ep_layout_amd


def test_structures_match_the_header(ep):
    text = open(os.path.join(ROOT, "include", "ep_layout.h")).read()
    for name in ("EP_MUON_PARAM_BF16", "EP_MUON_GRAD_BF16", "EP_MUON_NESTEROV"):
        assert getattr(ep, name) == 1 << int(re.search(rf"#define {name} +\(1u << (\d+)\)", text).group(1))
    fields = lambda n: re.findall(r"(\w+);", re.search(rf"typedef struct {n} \{{(.*?)\}}", text, re.S).group(1))
    assert fields("ep_muon_tensor") == list(ep._MUON_TENSOR.names) and ep._MUON_TENSOR.itemsize == 48
    assert fields("ep_muon_config") == [n for n, _ in ep._MuonConfig._fields_]


def table(ep, *rows):
    t = np.zeros(len(rows), ep._MUON_TENSOR)
    for row, values in zip(t, rows):
        for k, v in values.items():
            row[k] = v
    return t


def need(ep, *rows):
    t = table(ep, *rows)
    return ep.library().ep_muon_workspace_bytes(t.ctypes.data_as(ctypes.c_void_p), len(t))


def muon(ep, tensors, ws=A[8], size=1 << 30, **kw):
    t = table(ep, *tensors)
    cfg = ep._MuonConfig(lr=1e-3, momentum=0.9, weight_decay=0.0, scale=0.0, eps=1e-7, a=3.0, b=-4.0, c=2.0, steps=5)
    for k, v in kw.items():
        setattr(cfg, k, v)
    return ep.library().ep_muon(t.ctypes.data_as(ctypes.c_void_p), len(t), ctypes.byref(cfg), ws, size, None)


def test_workspace(ep):
    one = need(ep, dict(batch=1, rows=100, cols=60))
    # three fp16 values of X and two of the short side's square, each row a multiple of 8, and partial sums
    assert one == 60 * 104 * 6 + 60 * 64 * 4 + 2 * 8
    assert need(ep, dict(batch=7, rows=60, cols=100)) == 7 * one
    assert need(ep, dict(batch=2, rows=60, cols=100), dict(batch=0, rows=5, cols=5), dict(batch=1, rows=100, cols=60)) == 3 * one
    assert need(ep) == 0 and need(ep, dict(batch=3, rows=0, cols=9)) == 0
    assert need(ep, dict(batch=10000, rows=2048, cols=7168)) == 4 << 30
    assert need(ep, dict(batch=2, rows=16384, cols=32768)) == need(ep, dict(batch=1, rows=16384, cols=32768)) > 4 << 30
    for bad in (dict(batch=-1, rows=4, cols=4), dict(batch=1, rows=1 << 17, cols=4), dict(batch=1, rows=30000, cols=30000)):
        assert need(ep, bad) == -1


def test_muon_refusals(ep):
    INV, UNS = ep.EP_ERR_INVALID_ARGUMENT, ep.EP_ERR_UNSUPPORTED
    ok = dict(param=A[0], grad=A[1], momentum=A[2], batch=2, rows=40, cols=24)
    none = dict(ok, batch=0)
    assert muon(ep, []) == ep.EP_OK and muon(ep, [none, dict(ok, rows=0)], ws=None, size=0) == ep.EP_OK
    assert ep.library().ep_muon(None, 1, None, None, 0, None) == INV
    n = 2 * 40 * 24
    for bad in (dict(batch=-1), dict(rows=-1), dict(param=0), dict(grad=0), dict(momentum=0), dict(param=A[0] + 8),
                dict(grad=A[1] + 4), dict(momentum=A[2] + 4), dict(copy=A[3] + 2), dict(grad=A[0]), dict(copy=A[1]),
                dict(momentum=A[0] + n * 4 - 16), dict(copy=A[8] + 64), dict(grad=A[8])):
        assert muon(ep, [{**ok, **bad}]) == INV, bad
    assert muon(ep, [ok, none, ok]) == INV                          # twice
    assert muon(ep, [ok, {**ok, "param": A[4], "momentum": A[5], "grad": A[2]}]) == INV
    assert muon(ep, [{**ok, "copy": A[3]}], flags=ep.EP_MUON_PARAM_BF16) == UNS
    for bad in (dict(rows=1 << 17), dict(rows=30000, cols=30000), dict(batch=1 << 30)):
        assert muon(ep, [{**ok, **bad}]) == UNS, bad
    for bad in (dict(ws=None), dict(ws=A[8] + 8), dict(size=need(ep, dict(ok, batch=1)) - 1), dict(size=-1)):
        assert muon(ep, [ok], **bad) == INV, bad
    for bad in (dict(momentum=1.0), dict(momentum=-0.1), dict(eps=-1.0), dict(eps=float("inf")), dict(lr=float("nan")),
                dict(weight_decay=float("inf")), dict(scale=-1.0), dict(scale=float("nan")), dict(a=float("nan")),
                dict(c=float("inf")), dict(steps=0), dict(steps=101), dict(flags=1)):
        assert muon(ep, [ok], **bad) == INV, bad


def test_orthogonalize_refusals(ep):
    INV, UNS = ep.EP_ERR_INVALID_ARGUMENT, ep.EP_ERR_UNSUPPORTED
    size = need(ep, dict(batch=2, rows=40, cols=24))
    abc = lambda *v: (ctypes.c_double * 3)(*v)
    ok = dict(x=A[0], batch=2, rows=40, cols=24, steps=5, k=None, eps=0.0, flags=0, ws=A[1], size=size, out=A[2])

    def call(**kw):
        a = {**ok, **kw}
        return ep.library().ep_orthogonalize(a["x"], a["batch"], a["rows"], a["cols"], a["steps"], a["k"], a["eps"], a["flags"],
                                             a["ws"], a["size"], a["out"], None)

    assert call(batch=0) == ep.EP_OK and call(cols=0, ws=None, x=None) == ep.EP_OK
    for bad in (dict(batch=-1), dict(rows=-1), dict(steps=0), dict(steps=101), dict(eps=-1.0), dict(eps=float("nan")),
                dict(k=abc(1, float("nan"), 1)), dict(flags=1), dict(flags=ep.EP_MUON_NESTEROV), dict(x=None), dict(out=None),
                dict(ws=None), dict(x=A[0] + 4), dict(out=A[2] + 2), dict(ws=A[1] + 8), dict(size=size // 2 - 1), dict(out=A[0]),
                dict(out=A[1] + size - 16), dict(x=A[1])):
        assert call(**bad) == INV, bad
    assert call(rows=1 << 17) == UNS and call(rows=1 << 15, cols=1 << 15) == UNS


@pytest.mark.parametrize("kind", ["noise", "low rank", "decay", "rows"])
@pytest.mark.parametrize("rows,cols", [(96, 96), (64, 300), (200, 40), (1, 50)])
def test_what_fp16_products_cost(kind, rows, cols):
    """The rounded form against the definition.  With d = 2^-11 / sqrt(3) the root mean square of a rounding, a step
    moves X by at most (|b| + 2 |c| |G|) (2 d |X| |X|_F + d |G|_F) |X| + 2 d |P|_F |X| in the norm (2-norms where no F
    stands), and every later step multiplies that by at most the polynomial's largest slope."""
    x = ref.matrices(kind, 2, rows, cols, "cpu", rows).double()
    want, got = ref.exact(x), ref.rounded(x)
    a, b, c = ref.ABC
    d, bound = 2.0 ** -11 / 3 ** 0.5, torch.zeros(2, dtype=torch.float64)
    y = x / torch.linalg.matrix_norm(x, keepdim=True)
    y = y if rows <= cols else y.mT.contiguous()
    for _ in range(5):
        s = torch.linalg.svdvals(y)
        top, f = s[:, 0], s.square().sum(1).sqrt()
        p = b * s ** 2 + c * s ** 4
        at = torch.linspace(0, 1, 400, dtype=torch.float64) * (top.max() * 1.01)
        slope = (a + 3 * b * at ** 2 + 5 * c * at ** 4).abs().max()
        g_f, p_f = (s ** 4).sum(1).sqrt(), (p ** 2).sum(1).sqrt()
        bound = bound * slope + (abs(b) + 2 * abs(c) * top ** 2) * (2 * d * top * f + d * g_f) * top + 2 * d * p_f * top
        g = y @ y.mT
        y = a * y + (b * g + c * g @ g) @ y
    off = torch.linalg.matrix_norm(got - want)
    assert bool((off <= bound).all())
    if rows > 1:            # of one row, nothing averages out
        assert bool((off <= 3e-3 * torch.linalg.matrix_norm(want)).all())


def test_the_definition():
    """Singular values go through the polynomial, the vectors stay."""
    x = ref.matrices("noise", 1, 20, 33, "cpu")[0].double()
    u, s, v = torch.linalg.svd(x, full_matrices=False)
    s = s / x.norm()
    for _ in range(3):
        s = ref.ABC[0] * s + ref.ABC[1] * s ** 3 + ref.ABC[2] * s ** 5
    assert torch.allclose(ref.exact(x, 3, eps=0.0), u * s @ v, atol=1e-12)
    assert not ref.exact(torch.zeros(3, 4), eps=0.0).any()
