"""The few-token layer where the blocks of 32 of h differ by many powers of two inside one chunk of 128, and
the down weights of the large ones are zero: what remains is held to the bound of every other test, at one
or two tokens in an expert, at three or more, and at more than eight.
"""
import pytest
import torch

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R
from test_gpu_moe_w4a16 import check, make_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


def stretch_of(i):
    """Which of its row's blocks of 32 column i of h belongs to: in every 64, 0-15 and 32-47, then the others."""
    return i // 64 * 2 + i % 32 // 16


def spread_layer(dev, T, H, I, levels, seed):
    """A layer with every token in both of its experts whose block s of h is about 2^(-2 levels[s % len]) as
    large as the largest: gate and up rows alike are 2^-level of a normal row."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    i = torch.arange(I, device=dev)
    lv = torch.tensor(levels, device=dev)[stretch_of(i) % len(levels)].float()
    w1 = 0.2 * torch.randn(2, 2, I, H, device=dev, generator=g) * torch.exp2(-lv).view(1, 1, I, 1)
    w2 = 0.05 * torch.randn(2, H, I, device=dev, generator=g)
    x = torch.randn(T, H, device=dev, generator=g).bfloat16()
    pgu, _ = R.pack_weights(w1.view(2, 2 * I, H).bfloat16(), gate_up_interleave=True)
    pdn, _ = R.pack_weights(w2.bfloat16())
    return x, torch.randn(T, 2, device=dev, generator=g), pgu, pdn, lv


def zero_columns(pdn, rows, cols):
    """Clears the codes of the given rows and columns in both experts."""
    H, I = pdn.rows, pdn.cols
    c = pdn.codes.view(2, H, I // 2)
    c[:, rows.nonzero(), (cols[0::2]).nonzero().view(1, -1)] = 0


@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 20])
@pytest.mark.parametrize("I,levels", [
    (128, (0, 13, 13, 13)),      # one block 2^26 above its neighbours
    (256, (13, 13, 0, 13)),
    (128, (0, 7, 14, 7)),        # three magnitudes: 1, 2^-14, 2^-28
    (320, (0, 6, 12, 14)),       # 2^-12 beside the largest, the others below; the last chunk a half
    (256, (0, 14, 14, 14, 5, 0, 12, 5)),
    (192, (0, 40, 14)),          # blocks of nothing but zeros between
])
def test_blocks_far_below_their_neighbours(dev, T, I, levels):
    H = 256
    x, logits, pgu, pdn, lv = spread_layer(dev, T, H, I, levels, seed=I + T)
    row = torch.arange(H, device=dev)
    # a third of the rows loses the weights of the largest blocks, another those of all but the smallest
    zero_columns(pdn, row % 3 == 1, lv == 0)
    zero_columns(pdn, row % 3 == 2, lv < 12)
    st = R.new_status(dev)
    out, ids, w = R.moe_w4a16_layer(x, logits, 2, pgu, pdn, status=st)
    assert (ids >= 0).all()
    check(x, logits, 2, pgu, pdn, out, ids, w, st)
    assert (out != 0).float().mean() > 0.9


def test_ordinary_tokens_beside_wide_ones(dev):
    # the same tokens in the company of one whose blocks lie far apart keep their bits
    x, logits, pgu, pdn = make_layer(dev, 6, 256, 128, 2, 2, seed=41)
    want = R.moe_w4a16_layer(x, logits, 2, pgu, pdn)[0]
    x2 = x.clone()
    x2[2] = (x2[2].float() * 2.0 ** -60).bfloat16()
    x2[4] = 0
    got = R.moe_w4a16_layer(x2, logits, 2, pgu, pdn)[0]
    keep = [0, 1, 3, 5]
    assert torch.equal(got[keep], want[keep]) and (got[4] == 0).all()


@pytest.mark.parametrize("T", [1, 2, 3, 9])
def test_an_infinite_block_beside_finite_ones(dev, T):
    # the first block of every chunk overflows binary32 and meets positive weights only, its neighbours are far
    # below: the sum is an infinity, not NaN
    H, I = 256, 128
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    big = stretch_of(torch.arange(I, device=dev)) % 4 == 0
    w1 = 0.2 * torch.randn(2, 2, I, H, device=dev, generator=g)
    w1 = torch.where(big.view(1, 1, I, 1), w1.abs(), w1 * 2.0 ** -12)
    w2 = 0.05 * torch.randn(2, H, I, device=dev, generator=g)
    w2[:, :, big] = 0.05
    x = (2.0 ** 64 * (1.0 + torch.rand(T, H, device=dev, generator=g))).bfloat16()
    pgu, _ = R.pack_weights(w1.view(2, 2 * I, H).bfloat16(), gate_up_interleave=True)
    pdn, _ = R.pack_weights(w2.bfloat16())
    out, ids, w = R.moe_w4a16_layer(x, torch.randn(T, 2, device=dev, generator=g), 2, pgu, pdn)
    assert (out == float("inf")).all()
