"""Memory that the calls make for themselves, when they are given another stream than the current one.

Work is still queued on the current stream that uses blocks which are free again for the allocator: a call on another
stream that took one of those would race with it.  Results must be those of the same call made alone, their memory must
not be a block that the current stream may still use, and must not be handed out while the current stream reads them."""
import pytest
import torch

from gpu_helpers import say, dev
from test_gpu_16_expert_ffn import setup

pytestmark = pytest.mark.gpu

T, K, E, BM, H, I = 200, 2, 6, 16, 256, 128


def busy():
    """A few milliseconds of work on the current stream."""
    a = torch.ones(4096, 4096, dtype=torch.bfloat16, device=dev())
    for _ in range(20):
        a = a @ a
    return a


def layer():
    """(handle, {name: call(stream) -> tensors it returns}, names of calls with a hidden workspace and its bytes)"""
    import combine_ep_layout_amd as ep
    s = setup(T, K, E, BM, H, I, "uniform")
    h, e, cap = s["h"], s["epoch"], s["h"].capacity_rows
    pool, grad, wgu, wd = (s[k] for k in ("pool", "grad", "wgu", "wd"))
    for t in (pool, grad):
        t.nan_to_num_()                         # rows outside the regions are compared too
    g = torch.Generator(device=dev()).manual_seed(4)
    logits = torch.randn(T, E, device=dev(), generator=g)
    gw = torch.randn(T, K, device=dev(), generator=g)
    gy = torch.randn(T, H, device=dev(), generator=g).bfloat16()
    idx, _ = ep.route(logits, K)
    _, saved = h.expert_ffn(e, pool, wgu, wd, save=True)
    q = torch.randint(0, 120, (T, H), dtype=torch.uint8, device=dev(), generator=g)
    scales = torch.ones(T, H // 128, device=dev())
    real = s["real"]
    calls = {
        "route": lambda st: ep.route(logits, K, stream=st),
        "route_backward": lambda st: (ep.route_backward(logits, idx, gw, stream=st),),
        "cast_back": lambda st: (ep.cast_back(q, scales, "f32", stream=st),),
        "expert_ffn": lambda st: (h.expert_ffn(e, pool, wgu, wd, stream=st),),
        "expert_ffn saved": lambda st: (lambda r: (r[0], *r[1]))(h.expert_ffn(e, pool, wgu, wd, save=True, stream=st)),
        "expert_ffn_backward": lambda st: h.expert_ffn_backward(e, grad, pool, wgu, wd, saved, stream=st),
        "combine": lambda st: (h.combine(e, pool, stream=st),),
        "combine_backward": lambda st: h.combine_backward(e, gy, pool, stream=st),
        "dispatch_backward": lambda st: (h.dispatch_backward(e, grad, stream=st),),
        "array": lambda st: (h.array("pool_recv_token", stream=st),),
    }
    hidden = {"expert_ffn": [(cap, I, torch.bfloat16)], "expert_ffn_backward": [(cap, 2 * I, torch.bfloat16)]}
    # only the regions of pool-shaped results are written
    part = lambda t: t[real] if t.dim() == 2 and t.shape[0] == cap else t
    return h, calls, hidden, part


NAMES = ["route", "route_backward", "cast_back", "expert_ffn", "expert_ffn saved", "expert_ffn_backward", "combine",
         "combine_backward", "dispatch_backward", "array"]


def span(t):
    return t.untyped_storage().data_ptr(), t.untyped_storage().data_ptr() + t.untyped_storage().nbytes()


@pytest.mark.parametrize("name", NAMES)
def test_blocks_still_in_use_are_not_taken(name):
    say(f"[streams] {name}: blocks in use")
    h, calls, hidden, part = layer()
    call, side = calls[name], torch.cuda.Stream()
    want = [part(t).clone() for t in call(None)]
    shapes = [(*t.shape, t.dtype) for t in call(None)] + hidden.get(name, [])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy()
    blocks = [torch.empty(s[:-1], dtype=s[-1], device=dev()) for s in shapes]
    spans = [span(b) for b in blocks]
    for b in blocks:
        b.view(torch.uint8).fill_(0x7B)         # queued behind the work above, when the blocks are long free again
    del b, blocks
    got = call(side)
    for t in got:
        a, z = span(t)
        assert all(z <= lo or hi <= a for lo, hi in spans), "a block that the current stream still writes"
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, part(b))
    h.close()


@pytest.mark.parametrize("name", NAMES)
def test_results_outlive_their_readers(name):
    """A result that the current stream still reads, and that the program has dropped, is not given to the call's stream."""
    say(f"[streams] {name}: results in use")
    h, calls, _, part = layer()
    call, side = calls[name], torch.cuda.Stream()
    want = [part(t).clone() for t in call(None)]
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    busy()
    seen = [t.clone() for t in got]             # queued behind the work above
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):
        junk = [torch.empty(s, dtype=d, device=dev()) for s, d in shapes]
        for j in junk:
            j.view(torch.uint8).fill_(0x7B)
    torch.cuda.synchronize()
    for a, b in zip(want, seen):
        assert torch.equal(a, part(b))
    h.close()


def test_a_workspace_in_use_is_not_taken():
    """expert_ffn drops its workspace on return while its second product still reads it; the next call, on another
    stream, must not write into it."""
    say("[streams] workspace")
    h, calls, _, part = layer()
    side = torch.cuda.Stream()
    want = part(calls["expert_ffn"](None)[0]).clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy()
    first = calls["expert_ffn"](None)[0]
    second = calls["expert_ffn"](side)[0]
    back = calls["expert_ffn_backward"](side)
    torch.cuda.synchronize()
    assert torch.equal(part(first), want) and torch.equal(part(second), want)
    for a, b in zip(back, calls["expert_ffn_backward"](None)):
        assert torch.equal(part(a), part(b))
    h.close()


def test_a_side_stream_inside_a_capture():
    """Calls on a stream that was forked from the capturing one: their memory is the graph's, and replays follow the inputs."""
    import combine_ep_layout_amd as ep
    say("[streams] side stream in a capture")
    h, calls, _, part = layer()
    names = ["expert_ffn saved", "expert_ffn_backward", "combine_backward"]
    logits = torch.randn(T, E, device=dev())
    run = lambda st: [*ep.route(logits, K, stream=st), *(t for n in names for t in calls[n](st))]  # noqa: E731
    run(None)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = run(side)
        main.wait_stream(side)
        after = [t.clone() for t in got]
    for i in range(4):
        logits.normal_(generator=torch.Generator(device=dev()).manual_seed(i))
        g.replay()
        torch.cuda.synchronize()
        seen = [part(t).clone() for t in after]
        for a, b in zip(seen, run(None)):
            assert torch.equal(a, part(b)), i
        torch.cuda.synchronize()
    h.close()
