"""4-bit codes with exponent bytes: every bf16 value and every code at every exponent against the definition, bit for bit,
float32 values next to ties, zeros, subnormals, infinities, odd lengths and what lies around the buffers."""
import numpy as np
import pytest
import torch

from gpu_helpers import bits_of, dev, say, to_dev_bf16
from mxfp4_reference import decode, encode

pytestmark = pytest.mark.gpu


def quantized(values):
    import combine_ep_layout_amd as ep
    q = ep.mxfp4_quantize(values)
    return q.codes.cpu().numpy(), q.scales.cpu().numpy()


def check(values, got):
    codes, scales = encode(values)
    assert np.array_equal(got[1], scales), np.argwhere(got[1] != scales)[:4]
    assert np.array_equal(got[0], codes), np.argwhere(got[0] != codes)[:4]


def test_every_bf16_value():
    """Each value leads a block of zeros, and lies in a block under every power of two up to 2^4 above it."""
    bits = np.arange(65536, dtype=np.uint16)
    for up in range(-1, 5):
        say(f"[mxfp4] bf16, {up}")
        x = np.zeros((65536, 32), np.uint16)
        x[:, 7] = bits
        if up >= 0:
            exponent = (bits >> 7) & 0xFF
            x[:, 30] = np.minimum(exponent.astype(int) + up, 254).astype(np.uint16) << 7
        values = (x.astype(np.uint32) << 16).view(np.float32)
        check(values, quantized(to_dev_bf16(x)))


def test_float32_next_to_ties_and_far_out():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4096, 32)).astype(np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    near = np.concatenate([np.nextafter(ties, np.float32(0)), ties, np.nextafter(ties, np.float32(9)), -ties])
    for i, e in enumerate(range(-126, 126)):
        x[i] = near[:32] * np.float32(2.0) ** e
        x[256 + i] = x[i]
        x[256 + i][np.abs(near) > 6] = 0
    x[1000:1100] *= np.float32(1e-38)
    x[1100:1200] *= np.float32(1e-42)
    x[1200:1300] *= np.float32(5e37)
    x[1300] = 0
    x[1301] = -0.0
    x[1302, 3], x[1303, 4], x[1304, 31] = np.inf, np.nan, -np.inf
    x[1305, 0], x[1306, 0] = np.finfo(np.float32).max, np.float32(1e-45)
    check(x, quantized(torch.from_numpy(x).to(dev())))


@pytest.mark.parametrize("shape", [(32,), (1, 32), (3, 5, 96), (7, 2080), (0, 64), (2, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shapes(shape, dtype):
    x = torch.randn(shape, device=dev()).to(dtype)
    codes, scales = quantized(x)
    assert codes.shape == (*shape[:-1], shape[-1] // 2) and scales.shape == (*shape[:-1], shape[-1] // 32)
    if x.numel():
        check(x.float().cpu().numpy(), (codes, scales))


def test_every_code_at_every_exponent():
    import combine_ep_layout_amd as ep
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1, 1)).reshape(-1, 16)
    scales = np.repeat(np.arange(256, dtype=np.uint8), 16)[:, None]
    out = ep.mxfp4_cast_back(ep.Mxfp4(torch.from_numpy(codes).to(dev()), torch.from_numpy(scales).to(dev())))
    want = decode(codes, scales)
    got = out.float().cpu().numpy()
    finite = np.abs(want) < 2.0 ** 128
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[finite], want[finite].astype(np.float32)), np.argwhere((got != want) & finite)[:4]
    over = ~finite & ~np.isnan(want)
    assert np.array_equal(got[over], np.sign(want[over]) * np.inf)
    # signs of zero too
    assert np.array_equal(np.signbit(got[finite]), np.signbit(want[finite]))


def test_there_and_back_is_within_half_a_step():
    import combine_ep_layout_amd as ep
    x = torch.randn(64, 4096, device=dev())
    q = ep.mxfp4_quantize(x)
    back = ep.mxfp4_cast_back(q).float()
    # the widest step is 2 (between 4 and 6) at the block's power of two
    scale = torch.ldexp(torch.ones_like(q.scales, dtype=torch.float32), q.scales.int() - 127).repeat_interleave(32, 1)
    assert bool(((back - x).abs() <= scale).all())
    again = ep.mxfp4_quantize(back)
    assert torch.equal(ep.mxfp4_cast_back(again), ep.mxfp4_cast_back(q))


def test_given_results_streams_graphs_and_neighbours():
    import combine_ep_layout_amd as ep
    x = torch.randn(33, 96, device=dev()).bfloat16()
    want = ep.mxfp4_quantize(x)
    room_c, room_s = (torch.full((n + 32,), 0x5A, dtype=torch.uint8, device=dev()) for n in (33 * 48, 33 * 3))
    out = ep.Mxfp4(room_c[16:-16].view(33, 48), room_s[16:-16].view(33, 3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ep.mxfp4_quantize(x, out=out, stream=side)
    back = ep.mxfp4_cast_back(out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
    assert torch.equal(back, ep.mxfp4_cast_back(want))
    for room in (room_c, room_s):
        assert bool((room[:16] == 0x5A).all()) and bool((room[-16:] == 0x5A).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.mxfp4_quantize(x, out=out)
    for seed in range(3):
        x.copy_(torch.randn(33, 96, device=dev()))
        graph.replay()
        torch.cuda.synchronize()
        want = ep.mxfp4_quantize(x)
        assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)


def test_binding_refusals():
    import combine_ep_layout_amd as ep
    x = torch.randn(4, 64, device=dev())
    q = ep.mxfp4_quantize(x)
    for kind, call in ((TypeError, lambda: ep.mxfp4_quantize(x.half())), (ValueError, lambda: ep.mxfp4_quantize(x[:, :48])),
                       (ValueError, lambda: ep.mxfp4_quantize(x[:, :32])), (ValueError, lambda: ep.mxfp4_quantize(x.cpu())),
                       (ValueError, lambda: ep.mxfp4_quantize(x, out=ep.Mxfp4(q.codes[:2], q.scales))),
                       (TypeError, lambda: ep.mxfp4_cast_back(ep.Mxfp4(q.codes.int(), q.scales))),
                       (ValueError, lambda: ep.mxfp4_cast_back(ep.Mxfp4(q.codes, q.scales[:, :1]))),
                       (TypeError, lambda: ep.mxfp4_cast_back(q, out=x)), (ValueError, lambda: ep.mxfp4_cast_back(q, out=x[:2].bfloat16()))):
        with pytest.raises(kind):
            call()
