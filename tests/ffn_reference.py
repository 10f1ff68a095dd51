"""The experts' gated feed-forward and its gradients in float64, with bounds on
what rounding may add, from the operator's definition.  Works on any device.

Bounds, per element.  A rounding to bf16 moves a value by at most h = 2^-8 of
it.  A sum of n products in fp32 is off by at most n * u of the sum of their
magnitudes, with u = 2^-23 (a matrix core may truncate where an IEEE add
rounds: twice the half step 2^-24).  The activations are fp32 formulas of a
handful of operations with hardware exp and reciprocal: within f = 2^-18 of
their factors' magnitudes.
"""
import math

import torch

H_BF16 = 2.0 ** -8
U_SUM = 2.0 ** -23
F_ACT = 2.0 ** -18


def activation(g: torch.Tensor, kind: str):
    """act(g), act'(g)."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def expert(x, w_gate_up, w_down, kind, grad_out=None):
    """One expert's results and their bounds: {name: (value, bound)}; x [n, H] etc. float64."""
    I = w_down.shape[1]
    H = x.shape[1]
    n = x.shape[0]
    gu = x @ w_gate_up.T
    e_gu = H * U_SUM * (x.abs() @ w_gate_up.abs().T)
    g, u, e_g, e_u = gu[:, :I], gu[:, I:], e_gu[:, :I], e_gu[:, I:]
    v, s = activation(g, kind)
    a = v * u
    # |act'| <= 1.13 for both activations, |act''| <= 1.2 and |act(g)| <= |g|
    e_a32 = 1.2 * e_g * (u.abs() + e_u) + v.abs() * e_u + F_ACT * g.abs() * u.abs()
    e_a = e_a32 + H_BF16 * (a.abs() + e_a32)
    out = a @ w_down.T
    e_out = e_a @ w_down.abs().T + I * U_SUM * ((a.abs() + e_a) @ w_down.abs().T)
    r = {"act": (a, e_a), "gate_up": (gu, e_gu), "out": (out, e_out + H_BF16 * (out.abs() + e_out))}
    if grad_out is None:
        return r
    da = grad_out @ w_down
    e_da = H * U_SUM * (grad_out.abs() @ w_down.abs())
    dg, du = da * u * s, da * v
    # the formula of act' has terms as large as 1 + |g| before they cancel
    e_s = 1.3 * e_g + F_ACT * (1 + g.abs())
    e_dg = e_da * u.abs() * (s.abs() + e_s) + (da.abs() + e_da) * (e_u * (s.abs() + e_s) + u.abs() * e_s)
    e_du = e_da * v.abs() + (da.abs() + e_da) * (1.2 * e_g + F_ACT * g.abs())
    d = torch.cat([dg, du], 1)
    e_d = torch.cat([e_dg, e_du], 1)
    e_d = e_d + 4 * 2.0 ** -24 * d.abs()
    e_d = e_d + H_BF16 * (d.abs() + e_d)
    w = w_gate_up.abs()
    gp = d @ w_gate_up
    e_gp = e_d @ w + 2 * I * U_SUM * ((d.abs() + e_d) @ w)
    gw = d.T @ x
    e_gw = e_d.T @ x.abs() + n * U_SUM * ((d.abs() + e_d).T @ x.abs())
    gd = grad_out.T @ a
    e_gd = grad_out.abs().T @ e_a + n * U_SUM * (grad_out.abs().T @ (a.abs() + e_a))
    r["grad_gate_up"] = (d, e_d)
    r["grad_pool"] = (gp, e_gp + H_BF16 * (gp.abs() + e_gp))
    r["grad_w_gate_up"] = (gw, e_gw)        # before the rounding to the result's type
    r["grad_w_down"] = (gd, e_gd)
    return r


def check(name, got, value, bound, least=2.0 ** -130):
    """Every element of got within bound of value (least: subnormals of fp32 and bf16)."""
    off = (got.double() - value).abs()
    bad = ~(off <= bound + least)
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside their bounds, first at {i}: got "
                             f"{float(got[tuple(i)])}, want {float(value[tuple(i)])} within {float(bound[tuple(i)])}")
