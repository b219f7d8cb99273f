"""Every split of K over the warps of a team, with chunks that do not divide by it and half chunks: each case
says the team sizes of gate_up and down on 148 SMs, and takes them."""
import pytest
import torch

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R
import few_split
from test_gpu_moe_w4a16 import check, make_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


CASES = [  # every token in both experts: T, H, I, (S of gate_up, of down)
    (1, 2176, 576, (16, 4)),    # sixteen warps on 17 chunks; four on five, of which the last is a half
    (3, 1280, 1344, (8, 8)),    # eight on ten, and on eleven with a half
    (9, 512, 832, (4, 4)),      # four on four, and on seven with a half
    (64, 1408, 1344, (2, 4)),   # two on eleven
    (64, 128, 32768, (1, 16)),  # one chunk against sixteen warps on 256
    (2, 128, 2240, (1, 16)),    # sixteen on eighteen with a half
    (64, 2432, 832, (4, 2)),    # four on nineteen, two on seven with a half
]


@pytest.mark.parametrize("T,H,I,want", CASES)
def test_team_sizes(dev, T, H, I, want):
    x, logits, pgu, pdn = make_layer(dev, T, H, I, 2, 2, seed=H + I)
    st = R.new_status(dev)
    out, ids, w = R.moe_w4a16_layer(x, logits, 2, pgu, pdn, status=st)
    counts = [int((ids == e).sum()) for e in range(2)]
    assert counts == [T, T]
    if torch.cuda.get_device_properties(dev).multi_processor_count == 148:
        assert few_split.of_call(counts, H, I, 148) == want
    check(x, logits, 2, pgu, pdn, out, ids, w, st)
