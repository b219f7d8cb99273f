"""A step of both sides together: the rollout's layer from packed weights (moe_w4a16_layer), a head and
the log probabilities of the sampled tokens (token_logprobs), against the trainer's layer from
fake-quantised weights (weight_qdq) with the gradient of the log probabilities.

The two sides compute one function: the trainer's weights are the packed ones rounded to bf16 (relative
error 2^-8), so the log-prob gap is at most twice the largest error of a logit.
"""
import pytest
import torch

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R
from test_gpu_moe_w4a16 import reference

pytestmark = pytest.mark.gpu

T, H, I, E, K, V = 12, 256, 192, 6, 2, 1500


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def model(dev):
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=g)
    return dict(x=rnd(T, H).bfloat16(), router=rnd(T, E), w1=(0.06 * rnd(E, 2 * I, H)).bfloat16(),
                w2=(0.06 * rnd(E, H, I)).bfloat16(), head=0.1 * rnd(V, H))


def rollout(m, packed):
    out, ids, w = R.moe_w4a16_layer(m["x"], m["router"], K, *packed)
    return out, ids, w, out.float() @ m["head"].t()


def trainer(m, w1, w2, ids, w):
    """The layer with fake-quantised weights, binary32 sums, activations as they are."""
    f1, f2 = R.FakeQuantSTE.apply(w1).float(), R.FakeQuantSTE.apply(w2).float()
    out = torch.zeros(T, H, device=w1.device)
    for j in range(K):
        e = ids[:, j].long()
        y = torch.einsum("tnh,th->tn", f1[e], m["x"].float())
        h = torch.nn.functional.silu(y[:, :I]) * y[:, I:]
        out = out + w[:, j:j + 1] * torch.einsum("thi,ti->th", f2[e], h)
    return out @ m["head"].t()


def pack(m):
    return R.pack_weights(m["w1"], gate_up_interleave=True)[0], R.pack_weights(m["w2"])[0]


def test_log_prob_gap_and_gradient(dev, model):
    packed = pack(model)
    out, ids, w, logits = rollout(model, packed)
    roll = R.token_logprobs(logits, logits.argmax(-1), temperature=0.8, top=4)
    tokens = roll.top_ids[:, 1].long()  # the second likeliest as the sampled token
    roll = R.token_logprobs(logits, tokens, temperature=0.8)
    w1, w2 = model["w1"].clone().requires_grad_(), model["w2"].clone().requires_grad_()
    tl = trainer(model, w1, w2, ids, w)
    train = R.token_logprobs(tl, tokens, temperature=0.8)
    gap = (train.logprob - roll.logprob).abs()
    _, tol = reference(model["x"], ids, w, *packed, weight_err=2.0 ** -8)
    bound = 2 * (tol @ model["head"].double().abs().t()).amax(-1) / 0.8
    assert (gap <= bound).all() and gap.max() > 0
    assert ((train.entropy - roll.entropy).abs() <= bound * (1 + 2 * torch.log(torch.tensor(float(V))))).all()

    # the gradient through the layer equals the one of a float64 log softmax: only dlogits differs, by the
    # roundings of binary32, so that the bf16 gradients differ by a step where they round the other way
    (-train.logprob.sum() + 0.01 * train.entropy.sum()).backward()
    v1, v2 = model["w1"].clone().requires_grad_(), model["w2"].clone().requires_grad_()
    logp = torch.log_softmax(trainer(model, v1, v2, ids, w).double() / 0.8, -1)
    ent = -(logp.exp() * logp).sum(-1)
    (-logp.gather(1, tokens.unsqueeze(1)).sum() + 0.01 * ent.sum()).backward()
    for a, b in ((w1, v1), (w2, v2)):
        assert a.grad.norm() > 0
        assert (a.grad.double() - b.grad.double()).norm() <= 2.0 ** -8 * b.grad.double().norm()


def test_one_graph_of_the_rollout_side(dev, model):
    packed = pack(model)
    tokens = torch.randint(0, V, (T,), device=dev)
    m = dict(model, x=model["x"].clone(), router=model["router"].clone())

    def step():
        out, ids, w, logits = rollout(m, packed)
        return out, R.token_logprobs(logits, tokens, top=3)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lp = step()
    for seed in (3, 4):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        m["x"].copy_(torch.randn(T, H, device=dev, generator=g).bfloat16())
        m["router"].copy_(torch.randn(T, E, device=dev, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want, wlp = step()
        assert torch.equal(out, want)
        assert all(torch.equal(a, b) for a, b in zip(lp, wlp))
