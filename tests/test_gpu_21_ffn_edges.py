"""The experts' feed-forward at the edges of what may be asked of it."""
import pytest
import torch

from gpu_helpers import say, dev
from test_gpu_16_expert_ffn import setup

pytestmark = pytest.mark.gpu


def test_out_over_the_pool_cannot_be_saved():
    """The backward pass reads the pool: saved state beside an overwritten pool would give wrong weight gradients."""
    import combine_ep_layout_amd as ep
    say("[ffn] out over the pool, saved")
    s = setup(40, 2, 4, 16, 64, 32, "uniform")
    h = s["h"]
    before = s["pool"].clone()
    with pytest.raises(ep.EpError) as e:
        h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], out=s["pool"], save=True)
    assert e.value.status == ep.EP_ERR_INVALID_ARGUMENT
    assert torch.equal(s["pool"].view(torch.int16), before.view(torch.int16))
    want, _ = h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], save=True)
    h.expert_ffn(s["epoch"], s["pool"], s["wgu"], s["wd"], out=s["pool"])       # without the saved state it may
    assert torch.equal(s["pool"][s["real"]], want[s["real"]])
    h.close()
