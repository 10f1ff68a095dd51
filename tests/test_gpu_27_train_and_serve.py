"""The calls together, as they are used: a layer's training step whose matrices take the orthogonalised update, then the
same layer serving a few tokens, in bf16 and in 4 bits; and two streams that serve from the same weights at once."""
import pytest
import torch

import muon_reference as mref
from gpu_helpers import dev, say
from test_gpu_24_moe_tokens import check_y

pytestmark = pytest.mark.gpu

T, E, K, H, I = 96, 8, 2, 256, 160


def layer(seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    n = lambda *s: torch.randn(s, device=dev(), generator=g)
    return n(E, 2 * I, H) * H ** -0.5, n(E, H, I) * I ** -0.5, n(T, H).bfloat16(), n(T, E), n(T, H).bfloat16()


def test_train_then_serve():
    import combine_ep_layout_amd as ep
    up, down, x, logits, gy = layer(0)
    copies = [up.bfloat16(), down.bfloat16()]
    momenta = [torch.zeros_like(up), torch.zeros_like(down)]
    h = ep.EpHandle(T, K, E, 16)
    for step in range(3):
        say(f"[train and serve] step {step}")
        idx, w = ep.route(logits, K)
        epoch = h.layout(idx, w)
        pool, _ = h.new_pool(H)
        h.dispatch(x, pool)
        out, saved = h.expert_ffn(epoch, pool, *copies, save=True)
        geo, gw = h.combine_backward(epoch, gy, out)
        _, gup, gdown = h.expert_ffn_backward(epoch, geo, pool, *copies, saved)
        before = [up.clone(), down.clone()], [m.clone() for m in momenta]
        # gate and up are matrices of their own
        view = lambda t: t.view(2 * E, I, H)
        ep.muon([view(up), down], [view(gup), gdown], [view(momenta[0]), momenta[1]], lr=0.02, momentum=0.9,
                weight_decay=0.01, copies=[view(copies[0]), copies[1]])
        for p, p0, m0, g, shape in ((up, before[0][0], before[1][0], gup, (2 * E, I, H)),
                                    (down, before[0][1], before[1][1], gdown, (E, H, I))):
            m = 0.9 * m0.double() + 0.1 * g.double()
            u = (0.1 * g.double() + 0.9 * m).float().view(shape)
            f = 0.02 * 0.2 * max(shape[1:]) ** 0.5
            # experts without rows have no gradient, and matrices of zeros no update
            mref.check("parameters", p.view(shape), u, factor=-f, add=p0.double().view(shape) * (1 - 0.02 * 0.01),
                       rounding=5 * 2.0 ** -24)
        assert torch.equal(copies[0], up.bfloat16()) and torch.equal(copies[1], down.bfloat16())
    # the trained layer serves: the few-token call against the definition, and against the pool's path
    few = slice(0, 24)
    y, idx, w = ep.moe_tokens(x[few], *copies, logits=logits[few], top_k=K)
    check_y(y, x[few], idx, w, copies[0].double(), copies[1].double(), "silu")
    epoch = h.layout(*ep.route(logits, K))
    h.dispatch(x, pool)
    other = h.combine(epoch, h.expert_ffn(epoch, pool, *copies))[few]
    assert float((y.double() - other.double()).norm() / other.double().norm()) <= 2.0 ** -8     # three roundings and two
    # in 4 bits, from the masters; long batches go through the cast back
    q = [ep.mxfp4_quantize(t) for t in (up, down)]
    back = [ep.mxfp4_cast_back(t) for t in q]
    y4, idx, w = ep.moe_tokens(x[few], *q, logits=logits[few], top_k=K)
    check_y(y4, x[few], idx, w, back[0].double(), back[1].double(), "silu")
    other = h.combine(epoch, h.expert_ffn(epoch, pool, *back))[few]
    assert float((y4.double() - other.double()).norm() / other.double().norm()) <= 2.0 ** -8
    h.close()


def test_two_streams_serve_from_the_same_weights():
    import combine_ep_layout_amd as ep
    up, down, x, logits, _ = layer(1)
    q = [ep.mxfp4_quantize(t) for t in (up, down)]
    parts = [slice(i, i + n) for i, n in ((0, 1), (1, 5), (6, 40), (46, 50))]
    want = [ep.moe_tokens(x[p], *q, logits=logits[p], top_k=K)[0] for p in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [ep.moe_tokens(x[p], *q, logits=logits[p], top_k=K, stream=streams[i % 2])[0] for i, p in enumerate(parts)]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_and_eager_calls_between():
    """Each capture has workspaces of its own: replays in turn, and eager calls, do not meet in memory."""
    import combine_ep_layout_amd as ep
    up, down, x, logits, _ = layer(2)
    w = [up.bfloat16(), down.bfloat16()]
    u = torch.randn(4, 64, 96, device=dev())
    runs = [lambda: ep.moe_tokens(x[:6], *w, logits=logits[:6], top_k=K)[0], lambda: ep.moe_tokens(x[6:46], *w, logits=logits[6:46], top_k=K)[0],
            lambda: ep.orthogonalize(u)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(r())
    for turn in range(3):
        for o in outs:
            o.zero_()
        for i in (0, 2, 1, 0):
            graphs[i].replay()
            eager = runs[(i + turn) % 3]()
            assert torch.equal(eager, want[(i + turn) % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))
