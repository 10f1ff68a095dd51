"""The few-token layer, the 4-bit conversions and the orthogonalised update at the sizes that the header names as their
limits, and past 32 bits of bytes in every buffer that may be so long."""
import pytest
import torch

import muon_reference as ref
from gpu_helpers import dev, say
from test_gpu_24_moe_tokens import check_y, routing, rows
from test_gpu_26_muon import in_fp32

pytestmark = pytest.mark.gpu


class Doubles:
    """An expert's matrix in float64 when it is asked for."""

    def __init__(self, w):
        self.w = w
        codes = w.codes if isinstance(w, tuple) else w
        self.shape = (*codes.shape[:2], codes.shape[2] * (2 if isinstance(w, tuple) else 1))

    def __getitem__(self, e):
        import combine_ep_layout_amd as ep
        if isinstance(self.w, tuple):
            return ep.mxfp4_cast_back(ep.Mxfp4(self.w.codes[e], self.w.scales[e])).double()
        return self.w[e].double()


def weights(E, H, I, four, seed):
    import combine_ep_layout_amd as ep
    g = torch.Generator(device=dev()).manual_seed(seed)
    out = []
    for r, c in ((2 * I, H), (H, I)):
        if four:
            # codes of all kinds, the values' root mean square about c^-1/2
            codes = torch.randint(0, 256, (E, r, c // 2), device=dev(), generator=g, dtype=torch.uint8)
            power = 125 - (c.bit_length() - 1) // 2
            out.append(ep.Mxfp4(codes, torch.randint(power, power + 2, (E, r, c // 32), device=dev(), generator=g,
                                                     dtype=torch.uint8)))
        else:
            out.append(torch.empty(E, r, c, dtype=torch.bfloat16, device=dev()).normal_(0.0, c ** -0.5, generator=g))
    return out


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("H,I", [(65536, 64), (64, 65536), (65536, 8192), (8192, 65536)])
def test_widest_matrices(H, I, four):
    """hidden and inter of 65536, and 2^29 values of a matrix."""
    import combine_ep_layout_amd as ep
    say(f"[limits] {H} {I} {'4 bit' if four else 'bf16'}")
    q = weights(2, H, I, four, 0)
    for T in (3, 18):
        x, (idx, w) = rows(T, H, T), routing(T, 2, 2, T)
        y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
        check_y(y, x, idx, w, *map(Doubles, q), "silu")


@pytest.mark.parametrize("four,E,H,I", [(False, 80, 4096, 4096), (True, 300, 4096, 4096)])
def test_experts_past_32_bits(four, E, H, I):
    """The last experts' matrices lie more than 2^32 bytes behind the first ones'."""
    import combine_ep_layout_amd as ep
    say(f"[limits] {E} experts {'4 bit' if four else 'bf16'}")
    q = weights(E, H, I, four, 1)
    assert (q[0].codes if four else q[0]).nbytes > 2 ** 32
    for T in (1, 20):
        x, (idx, w) = rows(T, H, T), routing(T, 4, 3, T)
        idx = torch.where(idx < 2, idx, E - 4 + idx).contiguous()           # 0, 1 and the last two
        y = ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0]
        check_y(y, x, idx, w, *map(Doubles, q), "silu")


@pytest.mark.parametrize("four", [False, True])
def test_rows_far_apart(four):
    """64 tokens 2^23 values apart."""
    import combine_ep_layout_amd as ep
    T, E, K, H, I = 64, 5, 2, 96, 64
    q = weights(E, H, I, four, 2)
    wide = torch.full((T, 1 << 23), float("nan"), dtype=torch.bfloat16, device=dev())
    x = wide[:, -H:]
    x.copy_(rows(T, H, 2))
    idx, w = routing(T, E, K, 2)
    check_y(ep.moe_tokens(x, *q, topk_idx=idx, topk_weights=w)[0], x, idx, w, *map(Doubles, q), "silu")


def test_conversions_past_32_bits():
    """2^32 values and a few: the end is what it is by itself."""
    import combine_ep_layout_amd as ep
    n, m = (1 << 32) + 96, 4096
    x = torch.empty(n, dtype=torch.bfloat16, device=dev()).normal_(generator=torch.Generator(device=dev()).manual_seed(3))
    q = ep.mxfp4_quantize(x)
    for part in (slice(0, m), slice(n // 64 * 32, n // 64 * 32 + m), slice(n - m, n)):
        want = ep.mxfp4_quantize(x[part].clone())
        assert torch.equal(q.codes[part.start // 2:part.stop // 2], want.codes)
        assert torch.equal(q.scales[part.start // 32:part.stop // 32], want.scales)
    del x
    back = ep.mxfp4_cast_back(q)
    for part in (slice(0, m), slice(n // 64 * 32, n // 64 * 32 + m), slice(n - m, n)):
        some = ep.Mxfp4(q.codes[part.start // 2:part.stop // 2].clone(), q.scales[part.start // 32:part.stop // 32].clone())
        assert torch.equal(back[part], ep.mxfp4_cast_back(some))


@pytest.mark.parametrize("shape", [(1, 8192, 65536), (1, 65536, 8192)], ids=str)
def test_largest_matrices(shape):
    """2^29 values, in the first step: the definition's further ones multiply what it leaves."""
    say(f"[limits] {shape}")
    x = ref.matrices("noise", *shape, dev(), 4)
    ref.near(in_fp32(x, 1), x, 1)


def short_vectors(m, steps=5, abc=ref.ABC):
    """Largest relative error of a vector of m values along the short side, of noise whose long side is so much longer that
    its singular values are alike: s, 1 / sqrt(m) at first, within 1 %.

    A step makes (a + P) x of a column x, P = b G + c G G, G near g I with g = s^2.  Errors of it are a matrix times x, E, or
    a column's own, r.  With h = 2^-11 the rounding of hi moves x by h, and with it the result by r = h |P| / (a + P) of
    itself.  Those of G and P, h of each entry, move the result by E = h sqrt(m) (|b + 2 c g| g + |P|) / (a + P) at most,
    the norms being those of all entries.  An E from before comes out as q E, where q = s p'(s) / p(s) and p the step's
    polynomial of s; an r stays, and moves G by no more than an E of sqrt(m) r would: |q - 1| sqrt(m) r more of E.  In the
    last two steps the part k of P is not rounded, which is no more."""
    a, b, c = abc
    h, root = 2.0 ** -11, m ** 0.5
    s = [f / root for f in (0.99, 1.0, 1.01)]
    E = r = 0.0
    for _ in range(steps):
        g = [v * v for v in s]
        P = [b * v + c * v * v for v in g]
        q = [(a + 3 * b * v + 5 * c * v * v) / (a + b * v + c * v * v) for v in g]
        new = max(h * root * (abs(b + 2 * c * v) * v + abs(p)) / (a + p) for v, p in zip(g, P))
        E = max(map(abs, q)) * E + max(abs(v - 1) for v in q) * root * r + new
        r += max(h * abs(p) / (a + p) for p in P)
        s = [v * (a + p) for v, p in zip(s, P)]
    return E + r


@pytest.mark.parametrize("shape", [(2, 65536, 3), (2, 3, 65536)], ids=str)
def test_three_long_vectors(shape):
    """The matrices and their long vectors as test_gpu_26_muon.py has them.  Of 65536 vectors of three values each some lie
    where four samples of the noise happen to be small together: the reference's own further samples are up to twice
    the bound that check() makes of those, so these vectors have short_vectors()."""
    import combine_ep_layout_amd as ep
    say(f"[limits] {shape}")
    x = ref.matrices("noise", *shape, dev(), 5)
    e, (whole, rows_, cols) = ref.noise(x)
    d = ep.orthogonalize(x).double() - e
    along, across = (-2, -1) if shape[1] > shape[2] else (-1, -2)
    norm = torch.linalg.vector_norm
    n = norm(d, dim=(-2, -1))
    assert bool((n <= 2 * whole + 3 ** -0.5 * ref.H_BF16 * norm(e, dim=(-2, -1))).all())
    assert bool((norm(d, dim=along) <= 4 * (cols if along == -2 else rows_) + ref.H_BF16 * norm(e, dim=along)).all())
    limit = (short_vectors(3) + ref.H_BF16) * norm(e, dim=across)
    assert bool((norm(d, dim=across) <= limit).all())


@pytest.mark.parametrize("shape", [(1, 1, 65536), (3, 65536, 17)], ids=str)
def test_longest_sides(shape):
    import combine_ep_layout_amd as ep
    say(f"[limits] {shape}")
    x = ref.matrices("noise", *shape, dev(), 5)
    ref.check("X", ep.orthogonalize(x), x)


def test_batches_past_32_bits():
    """More than 2^32 bytes of matrices, which go through the workspace in several parts."""
    import combine_ep_layout_amd as ep
    n = 400
    base = ref.matrices("decay", 100, 256, 264, dev(), 6).bfloat16()
    x = base.repeat(n, 1, 1)
    assert x.nbytes > 2 ** 32
    want = ep.orthogonalize(base)
    ref.check("X", want, base)
    out = ep.orthogonalize(x).view(n, *base.shape)
    for i in range(n):
        assert torch.equal(out[i], want), i
