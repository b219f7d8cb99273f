"""The whole MoE layer for a few tokens (moe_w4a16_layer) against the layer in 64 bits.

Routing is compared bit for bit with moe_route_topk.  The bound on the output, per element, with
n = K additions of at most 2^-23 relative each (truncating binary32 accumulation) per sum:
  dg = n_H 2^-23 |G||x|, du likewise; dh = 1.1 |u| dg + |silu(g)| du + |h| (2^-11 + 2^-20)
  (h rounded to 11 significant bits, expf and the quotient a few ulp),
  dout = sum_j w_j (|D| dh_j + n_I 2^-23 |D||h_j|) + 2^-8 |out| (half a bf16 step).
"""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R
import nvfp4_layout as L

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    R.load()
    return torch.device("cuda:0")


def make_layer(dev, T, H, I, E, k, seed=0, scale=0.05):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    w1 = (torch.randn(E, 2 * I, H, device=dev, generator=g) * scale).bfloat16()
    w2 = (torch.randn(E, H, I, device=dev, generator=g) * scale).bfloat16()
    x = torch.randn(T, H, device=dev, generator=g)
    x[:, :: max(1, H // 4)] *= 20.0
    logits = torch.randn(T, E, device=dev, generator=g)
    pgu, _ = R.pack_weights(w1, gate_up_interleave=True)
    pdn, _ = R.pack_weights(w2)
    return x.bfloat16(), logits, pgu, pdn


def values(p, e, dev):
    """Float64 weights of one slab, from the packed bytes by the storage definition."""
    s = p.slab(e)
    codes = L.unpack_codes(s.codes.cpu().numpy(), p.rows, p.rows_padded, p.cols)
    sf = torch.from_numpy(L.unpack_sf(s.sf.cpu().numpy(), p.rows, p.rows_padded, p.cols)).view(torch.float8_e4m3fn)
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    return torch.from_numpy(v).to(dev) * sf.double().repeat_interleave(16, 1).to(dev) * s.s_g.double()


def reference(x, ids, w, pgu, pdn, weight_err=0.0):
    """(out, bound) in float64 for the given routing; the bound allows for a relative error of the weights."""
    dev = x.device
    T, H = x.shape
    I = pdn.cols
    xd = x.double()
    out = torch.zeros(T, H, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    n = torch.arange(2 * I, device=dev)
    gate, up = n[n % 128 < 64], n[n % 128 >= 64]
    gam = lambda K: (K + 32) * 2.0 ** -23 + weight_err
    for e in torch.unique(ids[ids >= 0]).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        W, D = values(pgu, e, dev), values(pdn, e, dev)
        y, ya = xd[t] @ W.T, xd[t].abs() @ W.abs().T
        g, u = y[:, gate], y[:, up]
        dg, du = gam(H) * ya[:, gate], gam(H) * ya[:, up]
        si = g * torch.sigmoid(g)
        h = si * u
        dh = 1.1 * u.abs() * dg + si.abs() * du + dg * du + h.abs() * (2.0 ** -11 + 2.0 ** -20)
        wt = w[t, j].double().unsqueeze(1)
        out.index_add_(0, t, wt * (h @ D.T))
        tol.index_add_(0, t, wt * (dh @ D.abs().T + gam(I) * (h.abs() @ D.abs().T)))
    return out, tol + 2.0 ** -8 * out.abs() + 1e-30


def check(x, logits, k, pgu, pdn, out, ids, w, status=None):
    ids_ref, w_ref = R.moe_route_topk(logits, k)
    assert torch.equal(ids, ids_ref) and torch.equal(w, w_ref)
    ref, tol = reference(x, ids, w, pgu, pdn)
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.2f} of the bound"
    if status is not None:
        R.check_status(status)


@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 128, 64, 1, 1),        # the smallest layer: half a chunk of K in the down projection
    (1, 256, 192, 8, 2),
    (3, 2048, 768, 16, 8),
    (8, 384, 64, 4, 1),
    (9, 384, 448, 2, 2),       # nine tokens in each expert: a second pass of eight columns
    (17, 640, 64, 1024, 32),   # the most experts and choices
    (33, 896, 320, 300, 6),
    (64, 256, 128, 3, 3),      # every token in every expert
    (64, 1152, 576, 40, 8),
])
def test_layer_matches_64_bits(dev, T, H, I, E, k):
    x, logits, pgu, pdn = make_layer(dev, T, H, I, E, k, seed=T + H)
    st = R.new_status(dev)
    out, ids, w = R.moe_w4a16_layer(x, logits, k, pgu, pdn, status=st)
    check(x, logits, k, pgu, pdn, out, ids, w, st)


@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 2048, 64, 4, 2),       # a block's sixteen warps on one unit; the down projection half a chunk
    (1, 1152, 1152, 4, 2),     # eight warps on nine chunks
    (3, 1280, 1344, 4, 2),     # eight on ten, and on eleven of which the last is a half
    (64, 512, 1600, 2, 2),     # two on four in gate_up, eight on thirteen with a half
    (64, 128, 32768, 2, 2),    # one chunk against the longest down projection
])
def test_k_split_over_warps(dev, T, H, I, E, k):
    x, logits, pgu, pdn = make_layer(dev, T, H, I, E, k, seed=I)
    st = R.new_status(dev)
    out, ids, w = R.moe_w4a16_layer(x, logits, k, pgu, pdn, status=st)
    check(x, logits, k, pgu, pdn, out, ids, w, st)


@pytest.mark.parametrize("T", range(2, 24, 3))
def test_token_counts(dev, T):
    x, logits, pgu, pdn = make_layer(dev, T, 256, 192, 5, 2, seed=T)
    check(x, logits, 2, pgu, pdn, *R.moe_w4a16_layer(x, logits, 2, pgu, pdn))


def test_a_skewed_router_sends_every_token_to_one_expert(dev):
    x, logits, pgu, pdn = make_layer(dev, 64, 512, 256, 16, 4, seed=5)
    logits[:, 7] += 50.0
    check(x, logits, 4, pgu, pdn, *R.moe_w4a16_layer(x, logits, 4, pgu, pdn))


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-12, 1e4, 2.0 ** 55])
def test_small_and_large_activations(dev, scale):
    # silu saturates at large magnitudes: the first rows of the gate alone decide its sign
    x, logits, pgu, pdn = make_layer(dev, 6, 256, 128, 4, 2, seed=11)
    xs = (x.float() * scale).bfloat16()
    out, ids, w = R.moe_w4a16_layer(xs, logits, 2, pgu, pdn)
    check(xs, logits, 2, pgu, pdn, out, ids, w)


def test_wide_range_inside_one_chunk(dev):
    # one channel 2^28 above the others of its chunk: the small ones are still exact
    x, logits, pgu, pdn = make_layer(dev, 4, 256, 128, 4, 2, seed=12)
    x = torch.randn(4, 256, device=dev).bfloat16()
    x[:, 5] = 2.0 ** 28
    pgu.codes.view(4, 256, 128)[:, :, 2] &= 0x0F  # column 5 of every gate_up row is zero
    out, ids, w = R.moe_w4a16_layer(x, logits, 2, pgu, pdn)
    xz = x.clone()
    xz[:, 5] = 0
    check(xz, logits, 2, pgu, pdn, out, ids, w)


def test_zero_rows_and_zero_experts(dev):
    x, logits, pgu, pdn = make_layer(dev, 5, 256, 128, 4, 2, seed=13)
    x[1] = 0
    pgu.s_g[2] = 0.0
    out, ids, w = R.moe_w4a16_layer(x, logits, 2, pgu, pdn)
    assert (out[1] == 0).all()
    check(x, logits, 2, pgu, pdn, out, ids, w)


def test_nan_and_infinity_stay_in_their_token(dev):
    x, logits, pgu, pdn = make_layer(dev, 12, 256, 128, 3, 2, seed=14)
    clean = R.moe_w4a16_layer(x, logits, 2, pgu, pdn)[0]
    x2 = x.clone()
    x2[3, 100] = float("nan")
    x2[7, 31] = float("inf")
    out = R.moe_w4a16_layer(x2, logits, 2, pgu, pdn)[0]
    assert out[3].isnan().all() and not out[7].isfinite().all()
    keep = [t for t in range(12) if t not in (3, 7)]
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_logits(dev, bad):
    x, logits, pgu, pdn = make_layer(dev, 6, 256, 128, 4, 2, seed=15)
    clean = R.moe_w4a16_layer(x, logits, 2, pgu, pdn)
    logits[4, 3] = bad
    st = R.new_status(dev)
    out, ids, w = R.moe_w4a16_layer(x, logits, 2, pgu, pdn, status=st)
    assert int(st.item()) == 4
    assert (ids[4] == -1).all() and (w[4] == 0).all() and (out[4] == 0).all()
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(ids[keep], clean[1][keep])


def test_all_logits_non_finite(dev):
    x, logits, pgu, pdn = make_layer(dev, 2, 256, 128, 4, 2, seed=16)
    logits.fill_(float("nan"))
    out, ids, _ = R.moe_w4a16_layer(x, logits, 2, pgu, pdn)
    assert (out == 0).all() and (ids == -1).all()


def test_pitches_and_buffers_around_the_rows(dev):
    T, H = 7, 384
    x, logits, pgu, pdn = make_layer(dev, T, H, 192, 6, 3, seed=17)
    plain = R.moe_w4a16_layer(x, logits, 3, pgu, pdn)[0]
    xb = torch.full((T, H + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    xb[:, :H] = x
    ob = torch.full((T + 1, H + 40), 7.0, dtype=torch.bfloat16, device=dev)
    out, _, _ = R.moe_w4a16_layer(xb[:, :H], logits, 3, pgu, pdn, out=ob[:T, :H])
    assert torch.equal(out, plain)
    assert (ob[:, H:] == 7).all() and (ob[T] == 7).all()


def test_workspace_is_not_written_past_its_size(dev):
    T, k, E, I = 5, 3, 6, 192
    x, logits, pgu, pdn = make_layer(dev, T, 384, I, E, k, seed=18)
    n = R.load().moe_w4a16_workspace_size(T, k, 384, I)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=dev)
    ref = R.moe_w4a16_layer(x, logits, k, pgu, pdn)[0]
    out = R.moe_w4a16_layer(x, logits, k, pgu, pdn, workspace=ws[:n])[0]
    assert torch.equal(out, ref) and (ws[n:] == 0xA5).all()


def test_no_tokens(dev):
    x, logits, pgu, pdn = make_layer(dev, 1, 256, 128, 4, 2)
    out, ids, w = R.moe_w4a16_layer(x[:0], logits[:0], 2, pgu, pdn)
    assert out.shape == (0, 256) and ids.shape == (0, 2) and w.shape == (0, 2)


def test_the_same_bits_every_time_on_two_streams(dev):
    x, logits, pgu, pdn = make_layer(dev, 24, 512, 320, 12, 4, seed=19)
    x2, logits2, _, _ = make_layer(dev, 24, 512, 320, 12, 4, seed=20)
    a, b = R.moe_w4a16_layer(x, logits, 4, pgu, pdn)[0], R.moe_w4a16_layer(x2, logits2, 4, pgu, pdn)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((R.moe_w4a16_layer(x, logits, 4, pgu, pdn, stream=s1)[0],
                    R.moe_w4a16_layer(x2, logits2, 4, pgu, pdn, stream=s2.cuda_stream)[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, a) and torch.equal(q, b) for p, q in got)


def test_captured_and_replayed_with_new_inputs(dev):
    x, logits, pgu, pdn = make_layer(dev, 4, 512, 192, 8, 2, seed=21)
    x2, logits2, _, _ = make_layer(dev, 4, 512, 192, 8, 2, seed=22)
    want = [R.moe_w4a16_layer(a, b, 2, pgu, pdn)[0] for a, b in ((x, logits), (x2, logits2))]
    sx, sl = x.clone(), logits.clone()
    R.moe_w4a16_layer(sx, sl, 2, pgu, pdn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = R.moe_w4a16_layer(sx, sl, 2, pgu, pdn)[0]
    for a, b, ref in ((x, logits, want[0]), (x2, logits2, want[1])):
        sx.copy_(a)
        sl.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_refusals(dev):
    x, logits, pgu, pdn = make_layer(dev, 4, 256, 128, 4, 2)
    call = lambda *a, **kw: R.moe_w4a16_layer(*a, **kw)
    big = torch.zeros(65, 256, dtype=torch.bfloat16, device=dev)
    for args, kw in [((big, torch.zeros(65, 4, device=dev), 2, pgu, pdn), {}),
                     ((x, logits, 5, pgu, pdn), {}), ((x, logits, 0, pgu, pdn), {}),
                     ((x.float(), logits, 2, pgu, pdn), {}), ((x, logits.double(), 2, pgu, pdn), {}),
                     ((x, logits[:3], 2, pgu, pdn), {}), ((x.t(), logits, 2, pgu, pdn), {}),
                     ((x, logits, 2, pdn, pgu), {}),
                     ((x, logits, 2, pgu, pdn), {"workspace": torch.empty(16, dtype=torch.uint8, device=dev)}),
                     ((x, logits, 2, pgu, pdn), {"out": torch.empty(4, 256, device=dev)}),
                     ((x, logits, 2, pgu, pdn), {"ids": torch.empty(4, 3, dtype=torch.int32, device=dev)})]:
        with pytest.raises(R.NVFP4Error):
            call(*args, **kw)
    odd = torch.zeros(4, 260, dtype=torch.bfloat16, device=dev)[:, :256]
    with pytest.raises(R.NVFP4Error):
        call(odd, logits, 2, pgu, pdn)
