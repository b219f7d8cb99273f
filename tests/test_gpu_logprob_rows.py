"""Token log probabilities and their gradient on rows made so that one element lost, taken twice or written
elsewhere shows: the longest row beside a gradient of another phase."""
import math

import pytest
import torch

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


def test_the_longest_row_into_a_gradient_of_another_phase(dev):
    V = (1 << 31) - 1
    logits = torch.zeros(1, V, dtype=torch.bfloat16, device=dev)
    logits[0, V - 1] = 5.0
    ids = torch.tensor([V - 1], device=dev)
    _, stats = R.token_logprobs_forward(logits, ids)
    buf = torch.full((V + 2,), 7.0, dtype=torch.bfloat16, device=dev)
    grad = buf[1:V + 1].view(1, V)
    R.token_logprobs_backward(logits, ids, stats, 1.0, torch.ones(1, device=dev), out=grad)
    assert buf[0] == 7 and buf[V + 1] == 7
    assert (logits[0, :V - 1] == 0).all() and logits[0, V - 1] == 5
    lse = math.log(V - 1 + math.exp(5.0))
    # half a step of bf16 and a part in 2^16 for 2^y and the sum
    assert abs(grad[0, 0].item() / -math.exp(-lse) - 1.0) <= 2.0 ** -8 + 2.0 ** -16
    assert (grad[0, 1:V - 1] == grad[0, 0]).all()
    assert abs(grad[0, V - 1].item() - (1.0 - math.exp(5.0 - lse))) <= 2.0 ** -8 + 2.0 ** -16


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,off,goff", [(5, 700, 1, 1), (5, 700, 0, 1), (4, 9001, 3, 3), (4, 9001, 1, 0), (1300, 2003, 1, 2)])
def test_padding_rows_of_any_content(dev, T, V, off, goff, dtype):
    # padding rows of NaN, edges and other phases included: zeros
    buf = torch.randn(T, V + off, device=dev).to(dtype)
    logits = buf[:, off:]
    ids = torch.arange(T, device=dev) % V
    logits[::2] = float("nan")
    ids[::2] = -1
    st = R.new_status(dev)
    got, stats = R.token_logprobs_forward(logits, ids, 1.0, 3, status=st)
    grad = torch.full((T, V + goff), 7.0, device=dev).to(dtype)[:, goff:]
    one = torch.ones(T, device=dev)
    R.token_logprobs_backward(logits, ids, stats, 1.0, one, one, out=grad, status=st)
    R.check_status(st)
    assert (got.logprob[::2] == 0).all() and (got.entropy[::2] == 0).all() and (got.top_ids[::2] == -1).all()
    assert (grad[::2] == 0).all() and (grad[1::2] != 0).any(1).all() and grad.isfinite().all()
