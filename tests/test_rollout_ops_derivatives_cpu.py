"""Derivatives that the few-token layer and the token log probabilities do not have are refused, not dropped:
before a device is touched."""
import pytest
import torch
from torch.autograd import forward_ad

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R


@pytest.fixture(scope="module", autouse=True)
def lib():
    from nvfp4_w4a4_moe_02_b200 import build_lib

    build_lib.build()


def layer(x, logits):
    p = R.Packed(torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8), torch.zeros(4), 4, 256, 256, 256)
    return R.moe_w4a16_layer(x, logits, 2, p, p)


def test_the_layer_refuses_what_asks_for_a_gradient():
    x, logits = torch.zeros(1, 256, dtype=torch.bfloat16), torch.zeros(1, 4)
    for args in ((x.clone().requires_grad_(), logits), (x, logits.clone().requires_grad_())):
        with pytest.raises(R.NVFP4Error, match="no gradient"):
            layer(*args)
        with torch.no_grad(), pytest.raises(R.NVFP4Error, match="CUDA"):  # as without a gradient
            layer(*args)


def test_tangents_are_refused():
    x, logits, ids = torch.zeros(1, 256, dtype=torch.bfloat16), torch.zeros(1, 4), torch.zeros(1, dtype=torch.int64)
    with forward_ad.dual_level():
        dx = forward_ad.make_dual(x, torch.ones_like(x))
        dl = forward_ad.make_dual(logits, torch.ones_like(logits))
        for call in (lambda: layer(dx, logits), lambda: layer(x, dl), lambda: R.token_logprobs(dl, ids)):
            with pytest.raises(R.NVFP4Error, match="tangent"):
                call()
            with torch.no_grad(), pytest.raises(R.NVFP4Error, match="tangent"):
                call()
        with pytest.raises(R.NVFP4Error, match="CUDA"):  # a level without tangents changes nothing
            R.token_logprobs(logits, ids)
