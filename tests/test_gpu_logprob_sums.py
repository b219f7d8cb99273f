"""The sums of the token log probabilities, element by element: no logit is lost or taken twice, wherever the
row is cut into vectors, strides, warps and cluster shares.

Sparse rows: all -inf but for n <= 7 equal logits l = 3.  y = l c - RN(l c) is the rounding of the reference,
at most 2^-22 as l c is below 8; every 2^y is the same number e, off by at most 2 steps of 2^-23, and the sum of
n of them by n 2^-24, so that log2 s - y is log2 n but for (2^-22 + 7 * 2^-24) / ln 2 and log2's own step:
  log prob -ln n and entropy ln n, to 2^-22 + 2^-21 + (2^-22 + 2^-24) ln n;
  the gradient 1[v = id] - 1/n there, to (n + 3) 2^-24 (e / s, a product, a difference), and 0 everywhere else;
  the alternatives are the positions in order.
Dense rows: bounds from the threads that take part, n = V / threads + 64 elements in sequence:
  log prob (n + 16) 2^-24 + (|log2 p| + |log2 s| + 8) 2^-22, entropy (n + 32) 2^-23 (1 + E|y| + log2 s)
as derived for the other tests, which take n = V / 32 + 64 and allow 2^-21.
"""
import math
import random

import pytest
import torch

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R
from test_gpu_logprobs import NINF, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


def team(T, V, sms):
    """Threads of a row and blocks among them, as the launch chooses."""
    if V <= 1024:
        return 32, 1
    if V <= 32768 and T >= 4 * sms:
        return 64, 1
    parts = 1
    while parts < 8 and T * parts < 2 * sms and V >= 8192 * parts:
        parts *= 2
    return 256 * parts, parts


def borders(V, N, threads, parts):
    """Positions next to which an index could be off by one, for rows that start on a 16-byte boundary or up
    to a vector off it."""
    nvec = V // N
    at = {0, 1, V - 1, V - 2}
    for v in {0, 1, nvec - 1, nvec}:
        at |= {N * v + d for d in range(-N, 2 * N + 1)}
    block = threads // parts
    for part in range(1, parts):
        at |= {N * (nvec * part // parts) + d for d in range(-N, N + 1)}
    for step in (block, 3 * block, 4 * block, 8 * block, 12 * block):
        at |= {N * step + d for d in range(-N, N + 1)}
    return sorted(p for p in at if 0 <= p < V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,off", [(1, 9, 0), (6, 77, 1), (40, 515, 3), (5, 1024, 0), (5, 1025, 1), (12, 8191, 0),
                                     (3, 16384, 2), (9, 50257, 1), (2, 65536, 0), (1, 131072, 3), (4, 300001, 5),
                                     (600, 1500, 1), (600, 32768, 0), (300, 40001, 1)])
def test_sparse_rows(dev, T, V, off, dtype):
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    threads, parts = team(T, V, sms)
    N = 16 // dtype.itemsize
    rng = random.Random(V + T)
    edge = borders(V, N, threads, parts)
    buf = torch.empty(T, V + off, dtype=dtype, device=dev)
    logits = buf[:, off:]
    for call in range(-(-len(edge) // (2 * T))):  # two borders a row, until all had their turn
        want = []
        logits.fill_(NINF)
        for t in range(T):
            take = edge[(2 * (call * T + t)) % len(edge):][:2] + [rng.randrange(V) for _ in range(rng.randint(0, 5))]
            want.append(sorted(set(take)))
        rows = torch.tensor([t for t in range(T) for _ in want[t]], device=dev)
        cols = torch.tensor([p for ps in want for p in ps], device=dev)
        logits[rows, cols] = 3.0
        ids = torch.tensor([rng.choice(ps) for ps in want], device=dev)
        n = torch.tensor([len(ps) for ps in want], dtype=torch.float64, device=dev)
        k = min(8, V)
        st = R.new_status(dev)
        got, stats = R.token_logprobs_forward(logits, ids, 1.0, k, status=st)
        R.check_status(st)
        tol = 2.0 ** -22 + 2.0 ** -21 + n.log() * (2.0 ** -22 + 2.0 ** -24)
        assert ((got.logprob.double() + n.log()).abs() <= tol).all()
        assert ((got.entropy.double() - n.log()).abs() <= tol).all()
        tops = got.top_ids.tolist()
        for t in range(T):
            assert tops[t][:len(want[t])] == want[t][:k]
        assert (got.top_logprobs.isfinite().sum(1) == n.clamp_max(k)).all()
        grad = R.token_logprobs_backward(logits, ids, stats, 1.0, torch.ones(T, device=dev))
        ref = torch.zeros(T, V, dtype=torch.float64, device=dev)
        ref[rows, cols] = -1.0 / n[rows]
        ref[torch.arange(T, device=dev), ids] += 1.0
        half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -9
        assert ((grad.double() - ref).abs() <= ref.abs() * half + (ref != 0) * 10 * 2.0 ** -24).all()
        assert (grad.double()[ref == 0] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(7, 900), (2, 5000), (3, 32000), (5, 50257), (1, 131072), (40, 131073), (2, 300001),
                                 (700, 1500), (600, 32768), (320, 9000)])
def test_dense_rows_to_the_bound_of_their_team(dev, T, V, dtype):
    threads, _ = team(T, V, torch.cuda.get_device_properties(dev).multi_processor_count)
    n = V / threads + 64
    for seed in range(3):
        logits, ids = make(dev, T, V, dtype, seed=100 * seed + T + V)
        got = R.token_logprobs(logits, ids, temperature=0.7)
        lp, ent, logp, p, *_ = reference(logits, ids, 0.7)
        ls = -logp.amax(-1) / math.log(2)
        tol = (n + 16) * 2.0 ** -24 + (lp.abs() / math.log(2) + ls + 8) * 2.0 ** -22
        assert ((got.logprob.double() - lp).abs() <= tol).all()
        y = (p * (logp - logp.amax(-1, keepdim=True)).abs()).sum(-1) / math.log(2)
        assert ((got.entropy.double() - ent).abs() <= (n + 32) * 2.0 ** -23 * (1 + y + ls)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(1, 4), (3, 5), (2, 700), (2, 5000), (1, 140001), (650, 3000)])
def test_nan_of_either_sign_has_alternatives(dev, T, V, dtype):
    # every alternative is some index of the row, whatever its NaNs are
    it = torch.int32 if dtype == torch.float32 else torch.int16
    bits = (-(1 << 22), 0x7FC00000, -1) if dtype == torch.float32 else (-(1 << 6), 0x7FC0, -1)
    for b in bits:
        for some in (slice(0, V), slice(0, V, 2), slice(V - 1, V)):
            logits, ids = make(dev, T, V, dtype, seed=V)
            logits.view(it)[:, some] = b
            st = R.new_status(dev)
            for k in {1, min(V, 32)}:
                got = R.token_logprobs(logits, ids, top=k, status=st)
                assert int(st.item()) == 4 and got.logprob.isnan().all()
                top = got.top_ids.sort(-1).values
                assert (top >= 0).all() and (top < V).all() and (top[:, 1:] > top[:, :-1]).all()
                assert got.top_logprobs.isnan().all()
