"""The gradient's p_v = 2^y_v / s where both are exact in binary32: rows of one value, so that y = 0 and
s = V, a whole number.  What remains is one quotient and two products: 3 roundings of 2^-24, and for bf16 half
a step of it.
"""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(3, 3), (5, 700), (2, 5003), (700, 2999), (3, 50257), (2, 100003), (1, 131071),
                                 (1, 300001), (300, 99991)])
def test_rows_of_one_value(dev, T, V, dtype):
    # ordinary rows, and masked by the type's lowest value all along (the exact form)
    for value in (0.0, torch.finfo(dtype).min):
        logits = torch.full((T, V), value, dtype=dtype, device=dev)
        ids = torch.zeros(T, dtype=torch.int64, device=dev)
        r, stats = R.token_logprobs_forward(logits, ids)
        grad = R.token_logprobs_backward(logits, ids, stats, 1.0, torch.ones(T, device=dev))
        half = 0.0 if dtype == torch.float32 else 2.0 ** -9  # of a step relative to the value
        tol = (3 * 2.0 ** -24 + 2 * half) / V
        assert ((grad[:, 1:].double() + 1.0 / V).abs() <= tol).all()
        assert ((grad[:, 0].double() - (1.0 - 1.0 / V)).abs() <= 2.0 ** -23 + half + 2 * half / V).all()
