"""The router's calls refuse results that share memory with what they read, or with each other: host checks, nothing is
launched (nothing could be: the addresses are made up, and calls that pass the checks are made only without a GPU)."""
import random

import pytest
import torch

A = [0x10000000 * (i + 1) for i in range(5)]
T, E, K = 5, 8, 2


@pytest.fixture(scope="module")
def ep():
    import combine_ep_layout_amd
    return combine_ep_layout_amd


def route(ep, logits=A[0], ld=E, idx=A[1], w=A[2], bias=None, flags=0):
    return ep.library().ep_route(logits, ld, T, E, K, flags, bias, 1.0, idx, w, None)


def backward(ep, logits=A[0], ld=E, idx=A[1], gw=A[2], out=A[3], grad_ld=E, flags=0, tokens=T):
    return ep.library().ep_route_backward(logits, ld, tokens, E, K, flags, 1.0, idx, gw, out, grad_ld, None)


def test_route(ep):
    sigmoid = ep.EP_ROUTE_SIGMOID
    last = A[0] + T * E * 4 - 4
    for bad in (dict(idx=A[0]), dict(w=A[0]), dict(idx=last), dict(w=last), dict(idx=A[0] - T * K * 4 + 4), dict(w=A[1]),
                dict(w=A[1] + T * K * 4 - 4), dict(bias=A[1], flags=sigmoid),
                dict(bias=A[2] + T * K * 4 - 4, flags=sigmoid), dict(bias=A[2] - E * 4 + 4, flags=sigmoid),
                dict(ld=100, idx=A[0] + (4 * 100 + E - 1) * 4),             # the last row's last value
                dict(ld=100, idx=A[0] + 99 * 4),                            # from a gap into the next row
                dict(flags=ep.EP_ROUTE_BF16, idx=A[0] + T * E * 2 - 4)):
        assert route(ep, **bad) == ep.EP_ERR_INVALID_ARGUMENT, bad


def test_route_backward(ep):
    for bad in (dict(out=A[0]), dict(out=A[1]), dict(out=A[2]), dict(out=A[1] + T * K * 4 - 4),
                dict(out=A[0] - T * E * 4 + 4),
                dict(ld=100, grad_ld=100, out=A[0] + 7 * 4),                # the first column on the logits' last
                dict(ld=100, grad_ld=100, out=A[0] + 93 * 4),               # into the next row
                dict(ld=100, grad_ld=33, out=A[0] + 8 * 4),                 # the fourth row, at 107, on 100..107
                dict(grad_ld=100, idx=A[3] + 7 * 4),                        # the choice inside the gradient's rows
                dict(grad_ld=100, gw=A[3] + 97 * 4)):
        assert backward(ep, **bad) == ep.EP_ERR_INVALID_ARGUMENT, bad


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: calls that pass the checks would run")
def test_rows_between_rows(ep):
    """Refused exactly when two rows have a value in common, by enumeration."""
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(4000):
        tokens = rng.randint(1, 6)
        ld = rng.choice([E, E + rng.randint(0, 30)])
        grad_ld = rng.choice([ld, E + rng.randint(0, 30)])
        at = rng.randint(-200, 200)
        cells = lambda start, step: {start + i * step + j for i in range(tokens) for j in range(E)}  # noqa: E731
        meet = bool(cells(0, ld) & cells(at, grad_ld))
        got = backward(ep, ld=ld, grad_ld=grad_ld, out=A[0] + 4 * at, tokens=tokens)
        assert (got == ep.EP_ERR_INVALID_ARGUMENT) == meet, (tokens, ld, grad_ld, at, got)
        seen[meet] += 1
    assert min(seen) > 500
