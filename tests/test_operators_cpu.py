"""Refusals of the calls that need no handle (ep_route, ep_route_backward, ep_adamw): host checks
only, nothing is launched; and the flags of the binding against the header's."""
import ctypes
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x10000000 * (i + 1) for i in range(12)]       # aligned addresses that nothing follows


@pytest.fixture(scope="module")
def ep():
    import combine_ep_layout_amd
    return combine_ep_layout_amd


def test_flags_match_the_header(ep):
    text = open(os.path.join(ROOT, "include", "ep_layout.h")).read()
    bits = {}
    for name, bit in re.findall(r"#define (EP_(?:ROUTE|ADAMW|GRAD)_\w+) +\(1u << (\d+)\)", text):
        assert getattr(ep, name) == 1 << int(bit), name
        bits[name] = int(bit)
    assert len(bits) == 8 and len(set(bits.values())) == 8


def test_route_refusals(ep):
    f, INV, UNS = ep.library().ep_route, ep.EP_ERR_INVALID_ARGUMENT, ep.EP_ERR_UNSUPPORTED
    ok = dict(logits=A[0], ld=8, T=4, E=8, K=2, flags=0, bias=None, scale=1.0, idx=A[1], w=A[2])

    def call(**kw):
        a = {**ok, **kw}
        return f(a["logits"], a["ld"], a["T"], a["E"], a["K"], a["flags"], a["bias"], a["scale"], a["idx"], a["w"], None)

    assert call(T=0) == ep.EP_OK
    for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=9), dict(ld=7), dict(scale=float("nan")), dict(flags=1),
                dict(logits=None), dict(logits=A[0] + 2), dict(flags=ep.EP_ROUTE_BF16, logits=A[0] + 1), dict(idx=None),
                dict(w=None), dict(idx=A[1] + 2), dict(flags=ep.EP_ROUTE_SIGMOID, bias=A[3] + 1)):
        assert call(**bad) == INV, bad
    for bad in (dict(E=1025, ld=1025), dict(E=64, ld=64, K=33), dict(bias=A[3]), dict(T=(1 << 25) + 1)):
        assert call(**bad) == UNS, bad


def test_route_backward_refusals(ep):
    f, INV, UNS = ep.library().ep_route_backward, ep.EP_ERR_INVALID_ARGUMENT, ep.EP_ERR_UNSUPPORTED
    ok = dict(logits=A[0], ld=8, T=4, E=8, K=2, flags=0, scale=1.0, idx=A[1], gw=A[2], out=A[3], grad_ld=8)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["logits"], a["ld"], a["T"], a["E"], a["K"], a["flags"], a["scale"], a["idx"], a["gw"], a["out"],
                 a["grad_ld"], None)

    assert call(T=0) == ep.EP_OK
    for bad in (dict(grad_ld=7), dict(out=None), dict(gw=None), dict(idx=None), dict(out=A[3] + 2), dict(flags=2),
                dict(K=9)):
        assert call(**bad) == INV, bad
    assert call(E=2000, ld=2000, grad_ld=2000) == UNS


def adamw(ep, tensors, flags=0, **kw):
    t = np.zeros(len(tensors), ep._ADAMW_TENSOR)
    for row, values in zip(t, tensors):
        for k, v in values.items():
            row[k] = v
    cfg = ep._AdamwConfig(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, grad_scale=1.0, flags=flags)
    for k, v in kw.items():
        setattr(cfg, k, v)
    return ep.library().ep_adamw(t.ctypes.data_as(ctypes.c_void_p), len(tensors), ctypes.byref(cfg), None)


def test_adamw_refusals(ep):
    INV, UNS = ep.EP_ERR_INVALID_ARGUMENT, ep.EP_ERR_UNSUPPORTED
    ok = dict(param=A[0], grad=A[1], exp_avg=A[2], exp_avg_sq=A[3], n=100)
    none = dict(ok, n=0)
    assert adamw(ep, []) == ep.EP_OK and adamw(ep, [none, none]) == ep.EP_OK
    assert ep.library().ep_adamw(None, 1, None, None) == INV
    for bad in (dict(n=-1), dict(param=0), dict(grad=0), dict(exp_avg=0), dict(exp_avg_sq=0), dict(param=A[0] + 8),
                dict(grad=A[1] + 4), dict(exp_avg=A[2] + 4), dict(copy=A[4] + 2), dict(exp_avg_scale=A[5]),
                dict(grad=A[0]), dict(exp_avg=A[0] + 112), dict(copy=A[3]), dict(exp_avg_sq=A[2])):
        assert adamw(ep, [{**ok, **bad}]) == INV, bad
    assert adamw(ep, [ok, {**ok, "param": A[5], "exp_avg": A[6], "exp_avg_sq": A[0] + 384}]) == INV     # across tensors
    assert adamw(ep, [ok, none, ok]) == INV                                                             # twice
    assert adamw(ep, [{**ok, "copy": A[4]}], ep.EP_ADAMW_PARAM_BF16) == UNS
    assert adamw(ep, [{**ok, "n": 1 << 50}]) == UNS and adamw(ep, [{**ok, "n": (1 << 34) + 1}]) == UNS
    eight = {**ok, "exp_avg_scale": A[4], "exp_avg_sq_scale": A[5]}
    for bad in (dict(exp_avg_scale=0), dict(exp_avg_sq_scale=0), dict(exp_avg_scale=A[4] + 2), dict(exp_avg_scale=A[5])):
        assert adamw(ep, [{**eight, **bad}], ep.EP_ADAMW_STATE_8BIT) == INV, bad
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")), dict(eps=-1.0),
                dict(eps=float("inf")), dict(lr=float("inf")), dict(grad_scale=float("nan")), dict(weight_decay=float("nan")), dict(flags=1),
                dict(step_dev=A[6] + 4), dict(grad_scale_dev=A[6] + 2), dict(step_dev=A[0] + 8)):
        assert adamw(ep, [ok], **bad) == INV, bad


def test_feed_forward_null_handle(ep):
    l = ep.library()
    assert l.ep_expert_ffn(None, 1, A[0], 64, A[1], A[2], 32, 0, A[3], A[4], A[5], None) == ep.EP_ERR_INVALID_ARGUMENT
    assert l.ep_expert_ffn_backward(None, 1, A[0], A[1], 64, A[2], A[3], 32, 0, A[4], A[5], 0, A[6], A[7], A[8], A[9],
                                    None) == ep.EP_ERR_INVALID_ARGUMENT


def test_activation_names_match_the_header(ep):
    text = open(os.path.join(ROOT, "include", "ep_layout.h")).read()
    for name, value in ep.ACTIVATIONS.items():
        assert int(re.search(rf"#define EP_ACT_{name.upper()} (\d+)", text).group(1)) == value
