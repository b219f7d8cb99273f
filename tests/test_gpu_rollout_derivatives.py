"""What the token log probabilities and the few-token layer do where a derivative is asked for that they do
not have: an error each time, never a result without it."""
import pytest
import torch
from torch.autograd import forward_ad

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R
from test_gpu_moe_w4a16 import make_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


def test_forward_mode(dev):
    logits, ids = torch.randn(3, 40, device=dev), torch.tensor([1, 2, 3], device=dev)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(logits, torch.ones_like(logits))
        with pytest.raises(R.NVFP4Error):
            R.token_logprobs(dual, ids)
        leaf = forward_ad.make_dual(logits.clone().requires_grad_(), torch.ones_like(logits))
        with pytest.raises(RuntimeError):  # torch's own: the function has no formula for it
            R.token_logprobs(leaf, ids)
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda z: R.token_logprobs(z, ids).logprob, (logits,), (torch.ones_like(logits),))
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda z: R.token_logprobs(z, ids).logprob.sum())(logits)
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda z: R.token_logprobs(z, ids).logprob)(logits.expand(2, 3, 40))


def test_the_layer_has_no_gradient(dev):
    x, logits, pgu, pdn = make_layer(dev, 4, 256, 128, 4, 2, seed=3)
    want = R.moe_w4a16_layer(x, logits, 2, pgu, pdn)[0]
    for a, b in ((x.clone().requires_grad_(), logits), (x, logits.clone().requires_grad_())):
        with pytest.raises(R.NVFP4Error):
            R.moe_w4a16_layer(a, b, 2, pgu, pdn)
        with torch.no_grad():
            assert torch.equal(R.moe_w4a16_layer(a, b, 2, pgu, pdn)[0], want)
