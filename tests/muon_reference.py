"""Newton-Schulz orthogonalisation in float64: the definition, and the same with the kernels' own roundings to fp16 put
in where they are made (sums stay float64).

After one or two steps the kernels and rounded() agree but for fp32 sums and the few values that those put on the
other side of a rounding: near() allows as much as if one rounding in four had gone there, a whole step of 2^-10
each, in the part that is made of rounded values: sqrt(1/4) 2^-10 = 2^-11 of its norm.

Over more steps such flips multiply: values that are e off flip a share e / 2^-10 of the next roundings, which are
then sqrt(e 2^-10) off in the mean, so that after five steps the kernels' roundings have nothing to do with
rounded()'s any more.  They are as many and as large, though, so both are as far from the definition: the distance of
rounded() from it, for inputs that differ in the seventh digit, gives samples of what the kernels' distance is a
further sample of.  check() allows twice the largest of four in the norm, a sum over all values, and four times the largest of
a row or column, whose few roundings scatter more.

A single row is one number s, the norm, times a vector: nothing averages out.  A step makes s (a + P) of it with
P = b G + c G G from G = s^2, both rounded by at most 2^-11: P is off by (|b G + 2 c G^2| + |P|) 2^-11, at most 3.5 * 2^-11
for G below 1.45, and the result by that over min(a + P) = 0.638 of itself.  Three steps of five see a G that is not
small, with slopes about 1 between them: SINGLE.
"""
import torch

ABC = (3.4445, -4.775, 2.0315)
H_BF16 = 2.0 ** -8
SINGLE = 3 * 3.5 * 2.0 ** -11 / 0.638


def _wide(x):
    return (x, False) if x.shape[-2] <= x.shape[-1] else (x.mT.contiguous(), True)


def _start(x, eps):
    n = torch.linalg.matrix_norm(x, keepdim=True)
    return x * torch.where(n == 0, torch.zeros_like(n), 1 / (n + eps))


def exact(x, steps=5, abc=ABC, eps=1e-7):
    a, b, c = abc
    x, tall = _wide(x.double())
    x = _start(x, eps)
    for _ in range(steps):
        g = x @ x.mT.contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if tall else x


def f16(v, scale=1.0):
    return (v * scale).to(torch.float16).double() / scale


def rounded(x, steps=5, abc=ABC, eps=1e-7):
    a, b, c = abc
    x, tall = _wide(x.double())
    s = 2.0 ** round(0.5 * torch.log2(torch.tensor(float(x.shape[-1]))).item())
    x = _start(x, eps)
    one = torch.eye(x.shape[-2], dtype=torch.float64, device=x.device)
    for i in range(steps):
        hi = f16(x, s)
        x = hi + f16(x - hi, s * 2048)
        g = f16(hi @ hi.mT.contiguous(), 1024.0)
        k = 0.0
        if i + 2 >= steps:              # the last two steps: P + k I
            l = g.diagonal(dim1=-2, dim2=-1).mean(-1).clamp_max(1.0)[..., None, None]
            k = -(b * l + c * l * l)
        p = f16(b * g + c * (g @ g) + k * one, 1024.0)
        x = (a - k) * x + p @ hi
    return x.mT if tall else x


def near(got, x, steps, abc=ABC, eps=1e-7):
    """fp32 results of one or two steps, matrix by matrix."""
    want = rounded(x, steps, abc, eps)
    before = exact(x, steps - 1, abc, eps) if steps > 1 else exact(x, 0, abc, eps)
    l = (torch.linalg.matrix_norm(before).square() / min(x.shape[-2:])).clamp_max(1.0)
    k = (abc[1] * l + abc[2] * l * l).abs()
    made = torch.linalg.matrix_norm(want - abc[0] * before) + k * torch.linalg.matrix_norm(before)
    if steps > 1:               # the first step's flips, too
        made = made + torch.linalg.matrix_norm(want)
    off = torch.linalg.matrix_norm(got.double() - want)
    limit = 2.0 ** -11 * made + 2.0 ** -21 * torch.linalg.matrix_norm(want)
    worst = (off / limit.clamp_min(1e-300)).max().item()
    assert worst <= 1, f"after {steps} steps {worst:.3f} of the bound"


def noise(x, steps=5, abc=ABC, eps=1e-7):
    """The definition, and the largest distances of four rounded forms from it: of each matrix, its rows and columns."""
    e = exact(x, steps, abc, eps)
    g = torch.Generator(device=x.device).manual_seed(7)
    most = [torch.zeros((), dtype=torch.float64, device=x.device)] * 3
    for i in range(4):
        near_x = x.double() * (1 + 1e-7 * i * torch.randn(x.shape, dtype=torch.float64, device=x.device, generator=g))
        d = rounded(near_x, steps, abc, eps) - e
        sizes = (torch.linalg.matrix_norm(d), torch.linalg.vector_norm(d, dim=-1), torch.linalg.vector_norm(d, dim=-2))
        most = [torch.maximum(m, s) for m, s in zip(most, sizes)]
    return e, most


def check(name, got, x, steps=5, abc=ABC, eps=1e-7, rounding=H_BF16, factor=1.0, add=None):
    """add + factor times X of x, rounded to the result's type (no value moves by more than half a step; in the norm of many
    values by the root mean square): by matrix, row and column."""
    e, (whole, rows, cols) = noise(x, steps, abc, eps)
    want = factor * e + (0 if add is None else add)
    d = got.double() - want
    f = abs(factor)
    if min(x.shape[-2:]) == 1:
        whole, rows, cols = (n + SINGLE * norm(e) for n, norm in (
            (whole, torch.linalg.matrix_norm), (rows, lambda t: torch.linalg.vector_norm(t, dim=-1)),
            (cols, lambda t: torch.linalg.vector_norm(t, dim=-2))))
    for what, off, size, limit, share in (
            ("row", torch.linalg.vector_norm(d, dim=-1), torch.linalg.vector_norm(want, dim=-1), 4 * f * rows, 1.0),
            ("column", torch.linalg.vector_norm(d, dim=-2), torch.linalg.vector_norm(want, dim=-2), 4 * f * cols, 1.0),
            ("norm", torch.linalg.matrix_norm(d), torch.linalg.matrix_norm(want), 2 * f * whole,
             3 ** -0.5 if x.shape[-1] * x.shape[-2] >= 256 else 1.0)):
        worst = (off / (limit + (share * rounding + 2.0 ** -21) * size).clamp_min(1e-300)).max().item()
        assert worst <= 1, f"{name}: a {what} is {worst:.3f} of its bound"


def matrices(kind, batch, rows, cols, device, seed=0):
    """Inputs of several spectra."""
    g = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s: torch.randn(s, device=device, generator=g)
    k = min(rows, cols)
    if kind == "noise":
        return n(batch, rows, cols)
    if kind == "low rank":
        r = max(1, k // 8)
        return n(batch, rows, r) @ n(batch, r, cols).contiguous()
    if kind == "decay":
        return (n(batch, rows, k) * torch.arange(1, k + 1, device=device) ** -1.0) @ n(batch, k, cols).contiguous()
    if kind == "rows":         # of very different sizes
        return n(batch, rows, cols) * torch.exp(2 * n(batch, rows, 1))
    raise KeyError(kind)
