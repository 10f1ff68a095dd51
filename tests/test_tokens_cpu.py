"""Refusals of ep_moe_tokens and the ep_mxfp4 calls: host checks only, nothing is launched; their flags against the
header's; and the 4-bit reference against values written out by hand."""
import ctypes
import os
import re

import numpy as np
import pytest

from mxfp4_reference import decode, encode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x10000000 * (i + 1) for i in range(12)]       # aligned addresses that nothing follows


@pytest.fixture(scope="module")
def ep():
    import combine_ep_layout_amd
    return combine_ep_layout_amd


def test_flags_and_arguments_match_the_header(ep):
    text = open(os.path.join(ROOT, "include", "ep_layout.h")).read()
    for name in ("EP_MOE_MXFP4", "EP_MXFP4_BF16"):
        assert getattr(ep, name) == 1 << int(re.search(rf"#define {name} \(1u << (\d+)\)", text).group(1))
    body = re.search(r"typedef struct ep_moe_tokens_args \{(.*?)\}", text, re.S).group(1)
    fields = re.findall(r"(\w+);", body)
    assert fields == [n for n, _ in ep._MoeTokensArgs._fields_]
    sizes = {"int64_t": 8, "int32_t": 4, "uint32_t": 4, "float": 4}
    for line, (name, kind) in zip(re.findall(r"\s+(.*?);", body), ep._MoeTokensArgs._fields_):
        want = 8 if "*" in line else sizes[line.split()[0]]
        assert ctypes.sizeof(kind) == want, name


def tokens(ep, **kw):
    a = dict(x=A[0], x_ld=64, num_tokens=4, hidden=64, inter=32, num_experts=8, top_k=2, activation=0, flags=0, scale=1.0,
             logits=A[1], logits_ld=8, bias=None, topk_idx=A[2], topk_weights=A[3], w_gate_up=A[4], gate_up_scales=None,
             w_down=A[5], down_scales=None, act=A[6], y=A[7])
    a.update(kw)
    return ep.library().ep_moe_tokens(ctypes.byref(ep._MoeTokensArgs(**a)), None)


def test_moe_tokens_refusals(ep):
    INV, UNS = ep.EP_ERR_INVALID_ARGUMENT, ep.EP_ERR_UNSUPPORTED
    four = dict(flags=ep.EP_MOE_MXFP4, gate_up_scales=A[8], down_scales=A[9])
    assert ep.library().ep_moe_tokens(None, None) == INV
    assert tokens(ep, num_tokens=0) == ep.EP_OK
    for bad in (dict(num_tokens=-1), dict(num_experts=0), dict(top_k=0), dict(top_k=9), dict(hidden=60), dict(inter=36),
                dict(hidden=0), dict(inter=-8), dict(x_ld=56), dict(x_ld=68), dict(activation=2), dict(flags=1),
                dict(logits_ld=7), dict(scale=float("nan")), dict(logits=None, flags=ep.EP_ROUTE_SIGMOID),
                dict(logits=None, bias=A[8]), dict(logits=A[1] + 2), dict(x=None), dict(x=A[0] + 8), dict(topk_idx=None),
                dict(topk_weights=None), dict(topk_idx=A[2] + 2), dict(w_gate_up=None), dict(w_down=A[5] + 8), dict(act=None),
                dict(y=A[7] + 2), dict(gate_up_scales=A[8]), dict(four, gate_up_scales=None), dict(four, down_scales=None),
                dict(four, gate_up_scales=A[8] + 8), dict(four, down_scales=A[9] + 1),
                dict(four, hidden=72, x_ld=72), dict(four, inter=40)):
        assert tokens(ep, **bad) == INV, bad
    for bad in (dict(num_tokens=65), dict(num_experts=1025, logits_ld=1025), dict(top_k=33, num_experts=64, logits_ld=64),
                dict(hidden=1 << 17, x_ld=1 << 17), dict(hidden=1 << 16, x_ld=1 << 16, inter=1 << 14), dict(x_ld=1 << 24),
                dict(logits=None, top_k=33), dict(bias=A[8])):
        assert tokens(ep, **bad) == UNS, bad


def test_moe_tokens_refuses_shared_memory(ep):
    INV = ep.EP_ERR_INVALID_ARGUMENT
    four = dict(flags=ep.EP_MOE_MXFP4, gate_up_scales=A[8], down_scales=A[9])
    sizes = {"x": 4 * 64 * 2, "logits": 4 * 8 * 4, "w_gate_up": 8 * 64 * 64 * 2, "w_down": 8 * 64 * 32 * 2}
    for out, n in (("topk_idx", 32), ("topk_weights", 32), ("act", 8 * 32 * 2), ("y", 4 * 64 * 2)):
        for name, size in sizes.items():
            at = dict(x=A[0], logits=A[1], w_gate_up=A[4], w_down=A[5])[name]
            assert tokens(ep, **{out: at}) == INV and tokens(ep, **{out: at + size - 16}) == INV, (out, name)
        assert tokens(ep, **{out: A[8] + 8 * 64 * 64 // 32 - 16}, **four) == INV
        assert tokens(ep, **{out: A[9]}, **four) == INV
        assert tokens(ep, **{out: A[10]}, flags=ep.EP_ROUTE_SIGMOID, bias=A[10]) == INV
        for other in {"topk_idx", "topk_weights", "act", "y"} - {out}:
            at = dict(topk_idx=A[2], topk_weights=A[3], act=A[6], y=A[7])[other]
            assert tokens(ep, **{out: at}) == INV, (out, other)


def test_mxfp4_refusals(ep):
    INV, UNS = ep.EP_ERR_INVALID_ARGUMENT, ep.EP_ERR_UNSUPPORTED
    q, back = ep.library().ep_mxfp4_quantize, ep.library().ep_mxfp4_cast_back
    assert q(None, 0, 0, None, None, None) == ep.EP_OK and back(None, None, 0, None, None) == ep.EP_OK
    for v, n, flags, c, s in ((A[0], -32, 0, A[1], A[2]), (A[0], 48, 0, A[1], A[2]), (None, 64, 0, A[1], A[2]),
                              (A[0], 64, 0, None, A[2]), (A[0], 64, 0, A[1], None), (A[0] + 4, 64, 0, A[1], A[2]),
                              (A[0], 64, 0, A[1] + 8, A[2]), (A[0], 64, 2, A[1], A[2]), (A[0], 64, 0, A[0] + 240, A[2]),
                              (A[0], 64, 0, A[1], A[0] + 255), (A[0], 64, 0, A[1], A[1] + 31)):
        assert q(v, n, flags, c, s, None) == INV, (v, n, flags, c, s)
    assert q(A[0], (1 << 38) + 32, 0, A[1], A[2], None) == UNS
    for c, s, n, out in ((A[0], A[1], 33, A[2]), (A[0], A[1], -1, A[2]), (None, A[1], 32, A[2]), (A[0], None, 32, A[2]),
                         (A[0], A[1], 32, None), (A[0] + 1, A[1], 32, A[2]), (A[0], A[1], 32, A[2] + 8), (A[0], A[1], 64, A[0] + 16),
                         (A[0], A[2] + 127, 64, A[2])):
        assert back(c, s, n, out, None) == INV, (c, s, n, out)


def test_the_4_bit_reference():
    x = np.zeros(64, np.float32)
    x[:12] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.2, -6, 4.99, 5.01]
    x[32:35] = [6.01, 1.0, -7]
    codes, scales = encode(x)
    assert scales.tolist() == [127, 128]
    assert decode(codes, scales)[:12].tolist() == [6, 4, 4, 2, 2, 1, 1, 0, 0, -6, 4, 6]
    assert decode(codes, scales)[32:35].tolist() == [6, 1, -8] and codes[0] == 7 | 6 << 4 and codes[4] >> 4 == 15
    x[3], x[40] = np.inf, np.nan
    codes, scales = encode(x)
    assert scales.tolist() == [255, 255] and not codes.any() and np.isnan(decode(codes, scales)).all()
