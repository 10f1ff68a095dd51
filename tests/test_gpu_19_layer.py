"""One layer's training step through every call in order: route, layout, dispatch, the experts' feed-forward,
combine, and back through combine_backward, the feed-forward's backward, dispatch_backward and route_backward to
AdamW; against the same layer in float64 with torch's autograd.  Then the serving side: the step in a HIP graph, on
another stream, with two handles at once, and the calls that must be refused."""
import pytest
import torch

import ffn_reference as ref
from gpu_helpers import say, dev

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def parameters(E, H, I, seed=0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(s, device=dev(), generator=g) * std
    return {"router": n(E, H, std=H ** -0.5), "gate_up": n(E, 2 * I, H, std=H ** -0.5), "down": n(E, H, I, std=I ** -0.5)}, n


def step(h, x, grad_y, p, wgu, wd, K, how):
    """Forward and backward of the layer; returns y and every gradient."""
    import combine_ep_layout_amd as ep
    logits = x.float() @ p["router"].T
    idx, w = ep.route(logits, K, **how)
    epoch = h.layout(idx, w)
    pool, _ = h.new_pool(x.shape[1])
    h.dispatch(x, pool)
    out, saved = h.expert_ffn(epoch, pool, wgu, wd, save=True)
    y = h.combine(epoch, out)
    grad_out, grad_w = h.combine_backward(epoch, grad_y, out)
    grad_pool, grad_gu, grad_d = h.expert_ffn_backward(epoch, grad_out, pool, wgu, wd, saved,
                                                       grad_w_gate_up=torch.empty(wgu.shape, device=dev()),
                                                       grad_w_down=torch.empty(wd.shape, device=dev()))
    grad_x = h.dispatch_backward(epoch, grad_pool)
    grad_logits = ep.route_backward(logits, idx, grad_w, **how)
    return y, idx, dict(x=grad_x.float() + grad_logits @ p["router"], router=grad_logits.T @ x.float(), gate_up=grad_gu,
                        down=grad_d)


def reference(x, grad_y, p, wgu, wd, idx, score, scale):
    x = x.double().requires_grad_()
    r, a, b = (t.double().requires_grad_() for t in (p["router"], wgu, wd))
    I = b.shape[2]
    logits = x @ r.T
    prob = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    w = torch.gather(prob, 1, idx.long())
    w = scale * w / w.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(a.shape[0]):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        gu = x[t] @ a[e].T
        o = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ b[e].T
        y = y.index_add(0, t, w[t, k][:, None] * o)
    y.backward(grad_y.double())
    return y.detach(), dict(x=x.grad, router=r.grad, gate_up=a.grad, down=b.grad)


@pytest.mark.parametrize("score,scale", [("softmax", 1.0), ("sigmoid", 2.5)])
def test_training_step(score, scale):
    import combine_ep_layout_amd as ep
    T, K, E, BM, H, I = 300, 3, 10, 32, 256, 136
    say(f"[layer] {score}")
    p, n = parameters(E, H, I)
    x, grad_y = n(T, H).to(BF16), n(T, H).to(BF16)
    wgu, wd = p["gate_up"].to(BF16), p["down"].to(BF16)
    h = ep.EpHandle(T, K, E, BM)
    y, idx, grads = step(h, x, grad_y, p, wgu, wd, K, {"score": score, "scale": scale})
    want_y, want = reference(x, grad_y, p, wgu, wd, idx, score, scale)
    # In the 2-norm the independent roundings to bf16 on the longest path (act, out, y; in the backward grad rows, act's
    # gradient, pool gradient, x gradient, and out inside the weights' gradient) are at most six, of half a step 2^-8 at most each.
    for name, got, value in [("y", y, want_y)] + [(k, grads[k], want[k]) for k in want]:
        off = float((got.double() - value).norm() / value.norm())
        assert off <= 6 * 2.0 ** -8, (name, off)

    # the optimiser's step on every parameter, states in 8 bits for the experts
    names = ["gate_up", "down"]
    params = [p[k].clone() for k in names]
    m = [torch.zeros(t.numel(), dtype=torch.uint8, device=dev()) for t in params]
    v = [torch.zeros_like(t) for t in m]
    ms = [torch.zeros((t.numel() + 127) // 128, device=dev()) for t in params]
    vs = [torch.zeros_like(t) for t in ms]
    copies = [wgu.clone(), wd.clone()]
    before = [t.clone() for t in params]
    ep.adamw([t.view(-1) for t in params], [grads[k].view(-1) for k in names], m, v, step=1, lr=1e-2, weight_decay=0.0,
             exp_avg_scales=ms, exp_avg_sq_scales=vs, copies=[t.view(-1) for t in copies])
    for old, new, copy, k in zip(before, params, copies, names):
        g = grads[k].double()
        # from zero states the first step is lr * g / (|g| + eps), in a handful of fp32 roundings
        want_p = old.double() - 1e-2 * g / (g.abs() + 1e-8)
        assert bool(((new.double() - want_p).abs() <= 16 * 2.0 ** -24 * (old.double().abs() + 1e-2)).all())
        assert torch.equal(copy, new.to(BF16))
    h.close()


def test_graph_replays_follow_new_inputs():
    import combine_ep_layout_amd as ep
    T, K, E, BM, H, I = 96, 2, 6, 16, 128, 72
    p, n = parameters(E, H, I, seed=3)
    wgu, wd = p["gate_up"].to(BF16), p["down"].to(BF16)
    x, grad_y = n(T, H).to(BF16), n(T, H).to(BF16)
    h, eager = ep.EpHandle(T, K, E, BM), ep.EpHandle(T, K, E, BM)
    logits = torch.empty(T, E, device=dev())
    cap = h.capacity_rows
    b = lambda *s, t=BF16: torch.zeros(s, dtype=t, device=dev())
    pool, out, act, gu, dgu, gp = b(cap, H), b(cap, H), b(cap, I), b(cap, 2 * I, t=F32), b(cap, 2 * I), b(cap, H)
    gw, gd, y = b(E, 2 * I, H), b(E, H, I), b(T, H)

    def run(h):
        idx, w = ep.route(logits, K)
        e = h.layout(idx, w)
        h.dispatch(x, pool)
        h.expert_ffn(e, pool, wgu, wd, out=out, act=act, gate_up=gu, save=True)
        h.combine(e, out, y)
        grad_out, grad_w = h.combine_backward(e, grad_y, out, grad_out_rows)
        h.expert_ffn_backward(e, grad_out, pool, wgu, wd, ep.FfnSaved(act, gu), grad_pool=gp, grad_gate_up=dgu,
                              grad_w_gate_up=gw, grad_w_down=gd)
        return ep.route_backward(logits, idx, grad_w)

    grad_out_rows = b(cap, H)
    logits.normal_()
    run(h)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run(h)
    for i in range(4):
        gen = torch.Generator(device=dev()).manual_seed(50 + i)
        logits.normal_(generator=gen)
        x.normal_(generator=gen)
        grad_y.normal_(generator=gen)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, gw, gd, captured)]
        want_logits = run(eager)
        torch.cuda.synchronize()
        for a, c in zip(got, (y, gw, gd, want_logits)):
            assert torch.equal(a, c), i
    h.close()
    eager.close()


def test_two_handles_on_two_streams():
    """Two layers' calls in flight at once, each on its own stream, workspaces made inside the calls."""
    import combine_ep_layout_amd as ep
    T, K, E, BM, H, I = 400, 2, 4, 64, 512, 256
    layers, alone, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        p, n = parameters(E, H, I, seed=20 + i)
        layers.append((ep.EpHandle(T, K, E, BM), n(T, H).to(BF16), n(T, H).to(BF16), p, p["gate_up"].to(BF16), p["down"].to(BF16)))
    for l in layers:
        alone.append(step(*l, K, {}))
    torch.cuda.synchronize()
    for _ in range(3):
        both = []
        for l, s in zip(layers, streams):
            with torch.cuda.stream(s):
                both.append(step(*l, K, {}))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])
    # a stream handed to the call while another is current
    h, x, gy, p, wgu, wd = layers[0]
    e = h.layout(*ep.route(x.float() @ p["router"].T, K))
    pool, _ = h.new_pool(H)
    h.dispatch(x, pool)
    want = h.expert_ffn(e, pool, wgu, wd, out=torch.zeros_like(pool))
    out = torch.zeros_like(pool)
    torch.cuda.synchronize()
    h.expert_ffn(e, pool, wgu, wd, out=out, stream=streams[1])
    junk = [torch.full((h.capacity_rows, I), 3.0, dtype=BF16, device=dev()) for _ in range(4)]     # would reuse the workspace
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del junk
    for l in layers:
        l[0].close()


def test_refusals():
    import combine_ep_layout_amd as ep
    T, K, E, BM, H, I = 20, 2, 4, 16, 64, 32
    p, n = parameters(E, H, I)
    wgu, wd, x = p["gate_up"].to(BF16), p["down"].to(BF16), n(T, H).to(BF16)
    h = ep.EpHandle(T, K, E, BM)
    pool = torch.zeros(h.capacity_rows, H, dtype=BF16, device=dev())
    with pytest.raises(ep.EpError) as ei:
        h.expert_ffn(1, pool, wgu, wd)                      # no layout yet
    assert ei.value.status == ep.EP_ERR_HANDLE_STATE
    e = h.layout(*ep.route(n(T, E), K))
    out, saved = h.expert_ffn(e, pool, wgu, wd, save=True)

    def status(f, *a, **kw):
        with pytest.raises((ep.EpError, ValueError, TypeError)) as ei:
            f(*a, **kw)
        return getattr(ei.value, "status", None)

    assert status(h.expert_ffn, e + 1, pool, wgu, wd) == ep.EP_ERR_HANDLE_STATE
    assert status(h.expert_ffn_backward, e + 1, out, pool, wgu, wd, saved) == ep.EP_ERR_HANDLE_STATE
    INV = ep.EP_ERR_INVALID_ARGUMENT
    wide = torch.zeros(h.capacity_rows, 2 * I, dtype=F32, device=dev())
    assert status(h.expert_ffn, e, pool, wgu, wd, act=pool.view(-1)[: h.capacity_rows * I].view(-1, I)) == INV
    assert status(h.expert_ffn, e, pool, wgu, wd, out=out, gate_up=wide, act=out.view(-1)[: h.capacity_rows * I].view(-1, I),
                  save=True) == INV
    assert status(h.expert_ffn_backward, e, out, pool, wgu, wd, saved, grad_pool=out) == INV
    assert status(h.expert_ffn_backward, e, out, pool, wgu, wd, saved, grad_w_gate_up=wgu) == INV
    for bad in (dict(activation="relu"), dict(out=out.float()), dict(out=out[:-1]), dict(gate_up=wide),
                dict(act=saved.act[:, :16])):
        status(h.expert_ffn, e, pool, wgu, wd, **bad)
    for a in ((pool[:-1], wgu, wd), (pool, wgu[:-1], wd), (pool, wgu, wd[:, :, :16]), (pool.float(), wgu, wd),
              (pool.cpu(), wgu, wd), (pool, wgu.transpose(1, 2), wd)):
        status(h.expert_ffn, e, *a)
    status(h.expert_ffn_backward, e, out, pool, wgu, wd, saved, accumulate=True)
    status(h.expert_ffn_backward, e, out, pool, wgu, wd, saved, grad_w_gate_up=torch.empty_like(wgu),
           grad_w_down=torch.empty(wd.shape, device=dev()))
    odd = torch.zeros(E, 2 * 12, H, dtype=BF16, device=dev()), torch.zeros(E, H, 12, dtype=BF16, device=dev())
    assert status(h.expert_ffn, e, pool, *odd) == INV       # inter % 8
    h.borrow(x)
    assert status(h.expert_ffn, e, pool, wgu, wd) == ep.EP_ERR_HANDLE_STATE         # a view is out
    h.release()
    h.close()


def test_single_token_serving():
    import combine_ep_layout_amd as ep
    E, K, H, I = 16, 4, 256, 128
    p, n = parameters(E, H, I, seed=8)
    wgu, wd = p["gate_up"].to(BF16), p["down"].to(BF16)
    h = ep.EpHandle(4, K, E, 16)
    for t in (1, 3, 1):
        x = n(t, H).to(BF16)
        idx, w = ep.route(x.float() @ p["router"].T, K)
        pool, _ = h.new_pool(H)
        epoch, _ = h.layout_dispatch(idx, w, x, pool)
        y = h.combine(epoch, h.expert_ffn(epoch, pool, wgu, wd))
        want = torch.zeros(t, H, dtype=torch.float64, device=dev())
        bound = torch.zeros_like(want)
        for i in range(t):
            for k in range(K):
                e = int(idx[i, k])
                o, b = ref.expert(x[i:i + 1].double(), wgu[e].double(), wd[e].double(), "silu")["out"]
                want[i] += float(w[i, k]) * o[0]
                bound[i] += float(w[i, k]) * (b[0] + 4 * 2.0 ** -24 * o[0].abs())
        ref.check("y", y, want, bound + ref.H_BF16 * (want.abs() + bound))
    h.close()
