"""The router's calls on memory that lies close together."""
import pytest
import torch

from gpu_helpers import say, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_between_the_logits_rows(dtype):
    """Columns of one buffer, none shared: the call is served, and the other columns keep their values."""
    import combine_ep_layout_amd as ep
    say(f"[route] gradient between the logits' rows, {dtype}")
    wide = torch.randn(300, 100, device=dev()).to(dtype)
    before = wide.clone()
    logits, grad = wide[:, 10:50], wide[:, 50:90]
    idx, w = ep.route(logits, 4)
    gw = torch.randn_like(w)
    ep.route_backward(logits, idx, gw, grad_logits=grad)
    assert torch.equal(grad, ep.route_backward(logits.contiguous(), idx, gw))
    assert torch.equal(wide[:, :50], before[:, :50]) and torch.equal(wide[:, 90:], before[:, 90:])


def test_gradient_over_an_input_is_refused():
    import combine_ep_layout_amd as ep
    say("[route] gradient over an input")
    wide = torch.randn(300, 100, device=dev())
    before = wide.clone()
    logits = wide[:, 10:50]
    idx, w = ep.route(logits, 4)
    for grad in (logits, wide[:, 49:89], wide[:, :40], wide[:, 60:100].as_strided((300, 40), (90, 1), 60)):
        with pytest.raises(ep.EpError) as e:
            ep.route_backward(logits, idx, w, grad_logits=grad)
        assert e.value.status == ep.EP_ERR_INVALID_ARGUMENT
    flat = torch.zeros(300 * 40, device=dev())
    with pytest.raises(ep.EpError):
        ep.route_backward(logits, idx, flat[5:5 + 1200].view(300, 4), grad_logits=flat.view(300, 40))
    assert torch.equal(wide, before)
