"""Token log probabilities, entropies, top alternatives and their gradient against 64 bits.

Bounds, for rows of V logits, with y the distances to the row's maximum in units of log2:
  sums run over at most n = V / 32 + 64 elements in sequence: relative error (n + 16) 2^-24;
  a probability: relative error r_p = (n + 16) 2^-24 + (|log2 p| + |log2 s| + 8) 2^-22
  (difference, product with c, its rounding, ex2 and log2, each counted twice);
  log prob: the same absolutely; entropy: r (1 + E|y| + log2 s) with r = (n + 32) 2^-23.
Half a step of the gradient's type is added to its bound.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R

pytestmark = pytest.mark.gpu
NINF = -math.inf


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


def seq(V):
    return V / 32 + 64


def reference(logits, ids, temperature):
    """Float64 log probabilities, entropies and log-softmax of every row (padding rows as NaN)."""
    z = logits.double() / temperature
    m = z.amax(-1, keepdim=True)
    logp = torch.log_softmax(torch.where(m == NINF, torch.zeros_like(z), z), -1)
    p = logp.exp()
    ent = torch.special.entr(p).sum(-1)
    lp = logp.gather(1, ids.long().clamp_min(0).unsqueeze(1)).squeeze(1)
    empty = (m == NINF).squeeze(1)
    lp = torch.where(empty, torch.full_like(lp, NINF), lp)
    ent = torch.where(empty, torch.zeros_like(ent), ent)
    pad = ids < 0
    # past the range of binary32 the nearest binary32 value is -inf
    lp, logp = (torch.where(v < torch.finfo(torch.float32).min, NINF, v) for v in (lp, logp))
    return torch.where(pad, 0.0, lp), torch.where(pad, 0.0, ent), logp, p, m, empty, pad


def check_forward(logits, ids, temperature, got, top):
    V = logits.shape[1]
    lp, ent, logp, p, m, empty, pad = reference(logits, ids, temperature)
    ls = (-(logp.amax(-1))).clamp_min(0) / math.log(2)
    fin = lp.isfinite()
    assert torch.equal(got.logprob.double()[~fin], lp[~fin])
    tol = (seq(V) + 16) * 2.0 ** -24 + (lp.abs() + ls + 8) * 2.0 ** -21
    assert ((got.logprob.double() - lp).abs()[fin] <= tol[fin]).all()
    y = torch.where(p > 0, p * (logp - logp.amax(-1, keepdim=True)).abs(), 0.0).sum(-1)
    tol = (seq(V) + 32) * 2.0 ** -23 * (1 + y + ls)
    assert ((got.entropy.double() - ent).abs() <= tol).all()
    if top:
        order = torch.sort(logits.float(), dim=-1, descending=True, stable=True).indices[:, :top]
        order[pad] = -1
        assert torch.equal(got.top_ids, order.int())
        tl = torch.where(pad.unsqueeze(1), 0.0, logp.gather(1, order.clamp_min(0)))
        tl = torch.where((empty & ~pad).unsqueeze(1), NINF, tl)
        fin = tl.isfinite()
        assert torch.equal(got.top_logprobs.double()[~fin], tl[~fin])
        tol = (seq(V) + 16) * 2.0 ** -24 + (tl.abs() + ls.unsqueeze(1) + 8) * 2.0 ** -21
        assert ((got.top_logprobs.double() - tl).abs()[fin] <= tol[fin]).all()


def check_backward(logits, ids, temperature, g_lp, g_ent, grad):
    V = logits.shape[1]
    lp, ent, logp, p, m, empty, pad = reference(logits, ids, temperature)
    one = torch.zeros_like(p).scatter_(1, ids.long().clamp_min(0).unsqueeze(1), 1.0)
    zero = torch.zeros(logits.shape[0], dtype=torch.float64, device=logits.device)
    a = (zero if g_lp is None else g_lp.double()).unsqueeze(1)
    b = (zero if g_ent is None else g_ent.double()).unsqueeze(1)
    plogp = -torch.special.entr(p)
    ref = (a * (one - p) - b * (plogp + p * ent.unsqueeze(1))) / temperature
    dead = (empty | pad).unsqueeze(1)
    ref = torch.where(dead, 0.0, ref)
    q = torch.where(p > 0, logp.abs(), 0.0) / math.log(2)
    ls = q.amin(-1, keepdim=True)
    r = (seq(V) + 16) * 2.0 ** -24 + (q + ls + 8) * 2.0 ** -22
    r_ent = (seq(V) + 32) * 2.0 ** -23 * (1 + (p * q).sum(-1, keepdim=True) + ls)
    tol = (p * r * (a.abs() + b.abs() * (q + ent.unsqueeze(1) + 1)) + p * b.abs() * (r_ent + (q + 1) * r)) / temperature
    half = torch.finfo(grad.dtype).eps / 2
    tol = tol + ref.abs() * (half + 2.0 ** -21) + (a.abs() + b.abs()) * 2.0 ** -120 / temperature
    tol = tol + one * a.abs() * 2.0 ** -22 / temperature
    err = (grad.double() - ref).abs()
    assert (err <= tol).all(), f"worst {(err / tol.clamp_min(1e-300)).max().item():.2f} of the bound"
    assert (grad[dead.squeeze(1)] == 0).all()


def make(dev, T, V, dtype, pitch=None, off=0, seed=0, scale=3.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    buf = torch.full((T, (pitch or V) + off), 1e4, device=dev).to(dtype)
    logits = buf[:, off:off + V]
    logits.copy_((scale * torch.randn(T, V, device=dev, generator=g)).to(dtype))
    ids = torch.randint(0, V, (T,), device=dev, generator=g)
    return logits, ids


SHAPES = [(1, 1, 1), (3, 2, 2), (2, 7, 7), (5, 31, 5), (9, 128, 32), (33, 515, 4), (16, 1000, 0), (4, 1024, 1),
          (4, 1025, 20), (6, 2049, 8), (300, 333, 3), (3, 8191, 32), (3, 32000, 0), (5, 50257, 8), (1, 131072, 20),
          (40, 131073, 5), (2, 300001, 32), (150, 20011, 0), (320, 9000, 2), (700, 4100, 0), (700, 1025, 32),
          (601, 32768, 3), (1300, 1777, 8)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,top", SHAPES)
def test_forward_and_backward(dev, T, V, top, dtype):
    logits, ids = make(dev, T, V, dtype, seed=T + V)
    temperature = (1.0, 0.7, 1.9)[V % 3]
    st = R.new_status(dev)
    got, stats = R.token_logprobs_forward(logits, ids, temperature, top, status=st)
    check_forward(logits, ids, temperature, got, top)
    g_lp, g_ent = torch.randn(T, device=dev), 0.1 * torch.randn(T, device=dev)
    for a, b in ((g_lp, g_ent), (g_lp, None), (None, g_ent), (None, None)):
        grad = R.token_logprobs_backward(logits, ids, stats, temperature, a, b, status=st)
        check_backward(logits, ids, temperature, a, b, grad)
    R.check_status(st)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,pitch,off", [(515, 515, 1), (515, 521, 3), (4099, 4099, 0), (4099, 4101, 5), (4096, 4103, 0),
                                         (70001, 70004, 7), (16, 24, 1)])
def test_pitches_and_alignments(dev, V, pitch, off, dtype):
    T = 11
    logits, ids = make(dev, T, V, dtype, pitch, off, seed=V)
    got, stats = R.token_logprobs_forward(logits, ids.int(), 1.0, 6)
    check_forward(logits, ids, 1.0, got, 6)
    g = torch.randn(T, device=dev)
    want = R.token_logprobs_backward(logits, ids, stats, 1.0, g, g)
    check_backward(logits, ids, 1.0, g, g, want)
    # a gradient of another pitch and phase; what lies around its rows stays
    for goff in (0, 2, 3):
        buf = torch.full((T + 1, V + 9), 5.0, device=dev).to(dtype)
        out = buf[:T, goff:goff + V]
        R.token_logprobs_backward(logits, ids, stats, 1.0, g, g, out=out)
        assert torch.equal(out, want)
        assert (buf[:, :goff] == 5).all() and (buf[:, goff + V:] == 5).all() and (buf[T] == 5).all()
    # in place
    copy = logits.clone()
    base = torch.empty(T, V + 3, device=dev, dtype=dtype)[:, :V].copy_(copy)
    R.token_logprobs_backward(base, ids, stats, 1.0, g, g, out=base)
    assert torch.equal(base, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 3000, 40000])
def test_masks_and_padding(dev, V, dtype):
    T = 12
    logits, ids = make(dev, T, V, dtype, seed=V)
    low = torch.finfo(dtype).min
    logits[0, V // 2:] = NINF
    logits[1, :] = NINF                      # nothing left
    logits[2, :] = NINF
    logits[2, V - 1] = -5.0                  # one token left
    logits[3, :] = low                       # masked by the lowest value, all of it: uniform
    logits[4, 1:] = low
    logits[5, : V - 3] = NINF
    logits[6, ::2] = low
    logits[6, 1::2] = NINF
    logits[7] = 0.0                          # ties
    logits[8, :] = NINF
    logits[8, :5] = low
    ids[0] = V - 1                           # a masked token
    ids[2] = V - 1
    ids[8] = 2
    ids[9] = -1
    ids[10] = -100
    logits[10] = float("nan")                # a padding row is not read
    for temperature in (1.0, 0.5):
        for top in (0, 9, 32):
            st = R.new_status(dev)
            got, stats = R.token_logprobs_forward(logits, ids, temperature, top, status=st)
            R.check_status(st)
            ref_logits = logits.clone()
            ref_logits[10] = 0.0
            check_forward(ref_logits, ids, temperature, got, top)
        g = torch.randn(T, device=dev)
        grad = R.token_logprobs_backward(logits, ids, stats, temperature, g, g)
        check_backward(ref_logits, ids, temperature, g, g, grad)
    assert got.logprob[1] == NINF and got.entropy[1] == 0 and (grad[1] == 0).all()


@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e15, -1e20, -1e30, -2e30, -1e38])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,temperature", [(700, 1.0), (5000, 0.5), (40000, 1e-6), (5000, 1e6)])
def test_masks_by_large_negative_values(dev, V, temperature, dtype, mask):
    # some threads see nothing but the mask's value, others nothing of it
    logits, ids = make(dev, 5, V, dtype, seed=V)
    logits *= temperature
    logits[0, V // 3:] = mask
    logits[1, 1:] = mask
    logits[2, ::2] = mask
    logits[3, :] = mask
    logits[4, : V - 1] = mask
    ids[1] = 0
    ids[4] = V - 1
    st = R.new_status(dev)
    got, stats = R.token_logprobs_forward(logits, ids, temperature, 3, status=st)
    R.check_status(st)
    check_forward(logits, ids, temperature, got, 3)
    g, h = torch.randn(5, device=dev), torch.randn(5, device=dev)
    check_backward(logits, ids, temperature, g, h, R.token_logprobs_backward(logits, ids, stats, temperature, g, h))


@pytest.mark.parametrize("V", [100, 5000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_not_finite_rows(dev, V, dtype):
    logits, ids = make(dev, 5, V, dtype, seed=V)
    clean, cstats = R.token_logprobs_forward(logits, ids, 1.0, 3)
    bad = logits.clone()
    bad[1, V // 3] = float("nan")
    bad[2, V - 1] = float("inf")
    bad[3, :] = float("nan")
    st = R.new_status(dev)
    got, stats = R.token_logprobs_forward(bad, ids, 1.0, 3, status=st)
    assert int(st.item()) == 4
    assert got.logprob[1:4].isnan().all() and got.entropy[1:4].isnan().all()
    assert ((got.top_ids >= 0) & (got.top_ids < V)).all()
    g = torch.ones(5, device=dev)
    grad = R.token_logprobs_backward(bad, ids, stats, 1.0, g)
    assert grad[1:4].isnan().all()
    for t in (0, 4):
        assert got.logprob[t] == clean.logprob[t] and torch.equal(got.top_ids[t], clean.top_ids[t])
        assert torch.equal(grad[t], R.token_logprobs_backward(logits, ids, cstats, 1.0, g)[t])


def test_ids_past_the_vocabulary(dev):
    logits, ids = make(dev, 4, 300, torch.float32)
    ids[2] = 300
    st = R.new_status(dev)
    got, stats = R.token_logprobs_forward(logits, ids, 1.0, 2, status=st)
    assert int(st.item()) == 1
    assert got.logprob[2] == 0 and (got.top_ids[2] == -1).all()
    st.zero_()
    grad = R.token_logprobs_backward(logits, ids, stats, 1.0, torch.ones(4, device=dev), status=st)
    assert int(st.item()) == 1 and (grad[2] == 0).all() and (grad[1] != 0).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", ["ascending", "descending", "equal", "few values"])
@pytest.mark.parametrize("V,T", [(900, 2), (20000, 2), (140001, 2), (3000, 600)])
def test_top_alternatives_of_ordered_rows(dev, V, T, order, dtype):
    v = torch.linspace(-4, 4, V, device=dev).to(dtype)
    if order == "descending":
        v = v.flip(0)
    elif order == "equal":
        v = torch.full_like(v, -0.0)
        v[7::3] = 0.0
    elif order == "few values":
        v = (torch.randint(0, 4, (V,), device=dev) - 2).to(dtype)
    logits = torch.stack([v.roll(777 * t) for t in range(T)])
    ids = torch.arange(T, device=dev) * (V - 1) % V
    got = R.token_logprobs(logits, ids, top=32)
    check_forward(logits, ids, 1.0, got, 32)


@pytest.mark.parametrize("scale,shift", [(1e4, 0.0), (1e-4, 0.0), (3.0, 5e4), (1e30, 0.0)])
def test_ranges(dev, scale, shift):
    logits, ids = make(dev, 6, 3001, torch.float32, scale=scale)
    logits += shift
    got, stats = R.token_logprobs_forward(logits, ids, 1.0, 4)
    check_forward(logits, ids, 1.0, got, 4)
    g = torch.randn(6, device=dev)
    check_backward(logits, ids, 1.0, g, g, R.token_logprobs_backward(logits, ids, stats, 1.0, g, g))


def test_gradient_against_differences(dev):
    T, V, temperature = 3, 37, 0.8
    logits, ids = make(dev, T, V, torch.float32, seed=4, scale=1.0)
    ids[1] = -1
    a, b = torch.randn(T, device=dev), torch.randn(T, device=dev)
    leaf = logits.clone().requires_grad_()
    r = R.token_logprobs(leaf, ids, temperature=temperature)
    ((a * r.logprob).sum() + (b * r.entropy).sum()).backward()

    def loss(x):  # float64, by the definition
        lp, ent, *_ = reference(x, ids, temperature)
        return (a.double() * lp + b.double() * ent).sum(-1)

    eps = 1e-5
    base = logits.double()
    for t in range(T):
        for v in range(0, V, 5):
            d = torch.zeros_like(base)
            d[t, v] = eps
            num = (loss(base + d) - loss(base - d)) / (2 * eps)
            # the difference quotient: eps^2 / 6 of a third derivative below 10, and 2^-52 / eps
            assert abs(num.item() - leaf.grad[t, v].item()) <= 1e-5


def test_autograd_of_broadcast_and_missing_gradients(dev):
    logits, ids = make(dev, 5, 700, torch.bfloat16, seed=6)
    leaf = logits.clone().requires_grad_()
    r = R.token_logprobs(leaf, ids, top=3)
    assert not r.top_logprobs.requires_grad and not r.top_ids.requires_grad
    r.logprob.sum().backward()  # an expanded gradient
    one = torch.ones(5, device=dev)
    check_backward(logits, ids, 1.0, one, None, leaf.grad)
    leaf.grad = None
    R.token_logprobs(leaf, ids).entropy.mean().backward()
    check_backward(logits, ids, 1.0, None, one / 5, leaf.grad)
    with torch.no_grad():
        assert not R.token_logprobs(leaf, ids).logprob.requires_grad


def test_no_rows(dev):
    logits = torch.empty(0, 100, device=dev)
    ids = torch.empty(0, dtype=torch.int64, device=dev)
    r = R.token_logprobs(logits, ids, top=2)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 2)
    leaf = logits.requires_grad_()
    R.token_logprobs(leaf, ids).logprob.sum().backward()
    assert leaf.grad.shape == (0, 100)


def test_streams_give_the_same_bits(dev):
    logits, ids = make(dev, 64, 50257, torch.bfloat16, seed=8)
    want = R.token_logprobs(logits, ids, top=8)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(6):
        got += [R.token_logprobs(logits, ids, top=8, stream=s1), R.token_logprobs(logits, ids, top=8, stream=s2.cuda_stream)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(g, want))


def test_captured_forward_and_backward(dev):
    logits, ids = make(dev, 16, 5003, torch.bfloat16, seed=9)
    logits2, ids2 = make(dev, 16, 5003, torch.bfloat16, seed=10)
    g = torch.randn(16, device=dev)

    def step(x, i):
        r, stats = R.token_logprobs_forward(x, i, 0.9, 4)
        return r.logprob, R.token_logprobs_backward(x, i, stats, 0.9, g, g)

    want = [[t.clone() for t in step(a, b)] for a, b in ((logits, ids), (logits2, ids2))]
    sx, si = logits.clone(), ids.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(sx, si)
    for (a, b), ref in zip(((logits, ids), (logits2, ids2)), want):
        sx.copy_(a)
        si.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, ref))


def test_captured_autograd(dev):
    logits, ids = make(dev, 6, 3001, torch.float32, seed=12)
    g = torch.randn(6, device=dev)

    def step(x):
        leaf = x.detach().requires_grad_()
        r = R.token_logprobs(leaf, ids, temperature=0.9)
        return torch.autograd.grad([r.logprob, r.entropy], [leaf], [g, g])[0]

    want = step(logits)
    x = logits.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_gradients_follow_the_current_stream(dev):
    logits, ids = make(dev, 6, 3001, torch.float32, seed=13)
    leaf = logits.clone().requires_grad_()
    with pytest.raises(R.NVFP4Error):
        R.token_logprobs(leaf, ids, stream=torch.cuda.Stream())
    R.token_logprobs(leaf, ids).logprob.sum().backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = logits.clone().requires_grad_()
        R.token_logprobs(other, ids).logprob.sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(other.grad, leaf.grad)


def test_no_second_derivative(dev):
    logits, ids = make(dev, 2, 50, torch.float32)
    leaf = logits.clone().requires_grad_()
    (g,) = torch.autograd.grad(R.token_logprobs(leaf, ids).logprob.sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_offsets_past_32_bits(dev):
    # the last rows start past 2^32 elements
    T, V = 70, 1 << 26
    logits = torch.empty(T, V, dtype=torch.bfloat16, device=dev)
    ids = torch.full((T,), -1, dtype=torch.int64, device=dev)
    ids[T - 1] = V - 3
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    logits[T - 1] = (3 * torch.randn(V, device=dev, generator=g)).bfloat16()
    got, stats = R.token_logprobs_forward(logits, ids, 1.0, 5)
    row, rid = logits[T - 1:].clone(), ids[T - 1:]
    check_forward(row, rid, 1.0, R.TokenLogprobs(*(t[T - 1:] for t in got)), 5)
    one = torch.ones(T, device=dev)
    grad = R.token_logprobs_backward(logits, ids, stats, 1.0, one, out=logits)
    check_backward(row, rid, 1.0, one[:1], None, grad[T - 1:])
    assert (grad[T - 2] == 0).all()


def test_the_longest_row(dev):
    # V = 2^31 - 1: uniform but for the last token, e^5 times as likely; every sum below is exact or closed
    V = (1 << 31) - 1
    logits = torch.zeros(1, V, dtype=torch.bfloat16, device=dev)
    logits[0, V - 1] = 5.0
    ids = torch.tensor([V - 1], device=dev)
    got, stats = R.token_logprobs_forward(logits, ids, 1.0, 3)
    lse = math.log(V - 1 + math.exp(5.0))
    assert got.top_ids.tolist() == [[V - 1, 0, 1]]
    # sums of 2^20 equal terms per thread; lse is near 21.5, a step of binary32 there is 2^-19
    assert abs(got.logprob.item() - (5.0 - lse)) <= 1e-5
    assert abs(got.entropy.item() - (lse - 5.0 * math.exp(5.0 - lse))) <= 1e-5
    grad = R.token_logprobs_backward(logits, ids, stats, 1.0, torch.ones(1, device=dev), out=logits)
    assert abs(grad[0, V - 1].item() - (1.0 - math.exp(5.0 - lse))) <= 2.0 ** -8
    for v in (0, 1, V // 2, V - 2):
        assert abs(grad[0, v].item() / -math.exp(-lse) - 1.0) <= 2.0 ** -7


def test_refusals(dev):
    logits, ids = make(dev, 4, 64, torch.float32)
    st = torch.zeros(4, 4, device=dev)
    for args, kw in [((logits.half(), ids), {}), ((logits.t(), ids), {}), ((logits, ids[:3]), {}),
                     ((logits, ids.short()), {}), ((logits, ids), {"temperature": 0.0}),
                     ((logits, ids), {"temperature": -1.0}), ((logits, ids), {"temperature": float("nan")}),
                     ((logits, ids), {"top": 33}), ((logits, ids), {"top": -1}), ((logits[:, :3], ids), {"top": 4}),
                     ((logits[:1].expand(4, 64), ids), {}), ((logits[:, :0], ids), {}), ((logits.cpu(), ids), {})]:
        with pytest.raises(R.NVFP4Error):
            R.token_logprobs(*args, **kw)
    for kw in [{"out": torch.empty(4, 63, device=dev)}, {"out": torch.empty(4, 64, device=dev).bfloat16()},
               {"grad_logprob": torch.ones(3, device=dev)}, {"grad_entropy": torch.ones(4, device=dev).double()}]:
        with pytest.raises(R.NVFP4Error):
            R.token_logprobs_backward(logits, ids, st, **kw)
    with pytest.raises(R.NVFP4Error):
        R.token_logprobs_backward(logits, ids, st[:, :3])
