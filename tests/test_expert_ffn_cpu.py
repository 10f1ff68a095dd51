"""Refusals of the experts' feed-forward calls (host checks only: nothing is launched)."""
import ctypes

import pytest


def lib():
    import combine_ep_layout_amd as ep
    return ep, ep.library()


P = [0x10000000 * (i + 1) for i in range(12)]       # 16-byte aligned addresses, never followed


def test_null_handle():
    ep, l = lib()
    assert l.ep_expert_ffn(None, 1, P[0], 64, P[1], P[2], 32, 0, P[3], P[4], P[5], None) == ep.EP_ERR_INVALID_ARGUMENT
    assert l.ep_expert_ffn_backward(None, 1, P[0], P[1], 64, P[2], P[3], 32, 0, P[4], P[5], 0, P[6], P[7], P[8], P[9],
                                    None) == ep.EP_ERR_INVALID_ARGUMENT


def test_activation_names_match_the_header():
    import os, re
    ep, _ = lib()
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ep_layout.h")).read()
    for name, value in ep.ACTIVATIONS.items():
        assert int(re.search(rf"#define EP_ACT_{name.upper()} (\d+)", text).group(1)) == value
    for name in ("EP_GRAD_F32", "EP_GRAD_ACCUMULATE"):
        bit = int(re.search(rf"#define {name} +\(1u << (\d+)\)", text).group(1))
        assert getattr(ep, name) == 1 << bit
