"""The mixture-of-experts layer for a few tokens and the token log probabilities, as they are measured.

``listed()`` gives the measured cases, ``draw(rng)`` more of the same ranges, ``prepare`` what a
program holds before the call, ``run`` one pass: the plain form in elementary torch operations, or,
where ``own`` is true, this package's calls.  ``work`` counts what a pass cannot do without and
``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------------ cases
def _moe(name, T, H, I, E, k, skew=0.0):
    return {"name": name, "op": "moe", "T": T, "H": H, "I": I, "E": E, "k": k, "skew": skew}


def _lp(name, T, V, dtype, top, temperature=1.0, pitch=0, masked=0.0, padded=0.0, train=False, entropy_grad=False):
    return {"name": name, "op": "logprobs", "T": T, "V": V, "dtype": dtype, "top": top, "temperature": temperature,
            "pitch": pitch or V, "masked": masked, "padded": padded, "train": train, "entropy_grad": entropy_grad}


def listed():
    return [
        # one token through a small layer: nothing but latency
        _moe("moe_1_small", 1, 256, 192, 8, 2),
        # one token through the layer of the prefill configuration (hidden 2048, 128 experts, top 8)
        _moe("moe_1_h2048", 1, 2048, 768, 128, 8),
        # a small odd batch of requests in the same layer
        _moe("moe_7_h2048", 7, 2048, 768, 128, 8),
        # a fuller batch whose router prefers some experts: more than eight tokens meet in one expert
        _moe("moe_48_h2048_skewed", 48, 2048, 768, 128, 8, skew=2.0),
        # one token through the layer of the decode configuration (hidden 7168, 256 experts, top 8)
        _moe("moe_1_h7168", 1, 7168, 2048, 256, 8),
        # the decode configuration's batch: 64 tokens touch most experts
        _moe("moe_64_h7168", 64, 7168, 2048, 256, 8),
        # one sampled token with its alternatives, logits in 32 bits as a sampler holds them
        _lp("logprobs_1_f32_top20", 1, 131072, "f32", 20),
        # a decode batch's sampled tokens with eight alternatives
        _lp("logprobs_64_bf16_top8", 64, 131072, "bf16", 8, temperature=0.7),
        # scoring of ragged sequences: odd vocabulary and pitch, padded tokens, a masked vocabulary
        _lp("logprobs_1999_bf16_odd", 1999, 50257, "bf16", 0, temperature=1.3, masked=0.3, padded=0.1),
        # a classifier-sized vocabulary, many rows: a row is less than a block's work
        _lp("logprobs_20000_f32_small", 20000, 515, "f32", 4, pitch=520),
        # a policy-gradient step with an entropy bonus in 32 bits
        _lp("logprobs_1023_f32_train", 1023, 32000, "f32", 0, temperature=0.9, padded=0.1, train=True,
            entropy_grad=True),
        # the policy-gradient step of a full batch
        _lp("logprobs_4096_bf16_train", 4096, 131072, "bf16", 0, train=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        k = rng.choice([1, 2, 3, 4, 6, 8])
        E = max(k, _log_int(rng, 4, 256))
        H = 128 * _log_int(rng, 1, 56)
        I = 64 * _log_int(rng, 1, 32)
        c = _moe("", _log_int(rng, 1, 64), H, I, E, k, skew=rng.choice([0.0, 0.0, 1.0, 3.0]))
    else:
        V = _log_int(rng, 40, 131072)
        train = rng.random() < 0.4
        T = _log_int(rng, 1, max(1, min(20000, (1 << 28) // V)))
        top = 0 if train else rng.choice([0, 1, 5, 8, 20, 32])
        # alternatives are asked for where the mask leaves that many tokens
        masked = rng.choice([0.0, 0.0, 0.5]) if 4 * top <= V else 0.0
        c = _lp("", T, V, rng.choice(["f32", "bf16"]), top, temperature=rng.choice([1.0, 0.6, 1.7]),
                pitch=V + rng.choice([0, 0, 1, 8, 24]), masked=masked, padded=rng.choice([0.0, 0.2]), train=train,
                entropy_grad=train and rng.random() < 0.5)
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _to_atoms(sf):
    # row-major scales [rows, cols / 16] -> 512-byte atoms of 128 rows x 64 columns, row 32 i + j of
    # an atom at byte 16 j + 4 i
    rows, c16 = sf.shape
    return sf.view(rows // 128, 4, 32, c16 // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _pack(rows, cols, gen):
    """One expert's weights ~ N(0, 0.02), quantised: codes, scale atoms and the tensor scale."""
    w = torch.randn(rows, cols // 16, 16, device="cuda", generator=gen) * 0.02
    s_g = w.abs().max() / 2688.0
    S = (w.abs().amax(-1, keepdim=True) / (6.0 * s_g)).to(torch.float8_e4m3fn)
    v = w / (S.float() * s_g).clamp_min(1e-30)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(rows, cols // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).view(-1), _to_atoms(S.view(torch.uint8).view(rows, cols // 16)), s_g


def prepare(case, seed):
    g = _gen(seed)
    T = case["T"]
    if case["op"] == "moe":
        H, I, E, k = case["H"], case["I"], case["E"], case["k"]
        st = {"case": case, "k": k}
        # activations behind a norm, with a few channels that run hot
        x = torch.randn(T, H, device="cuda", generator=g)
        hot = torch.randperm(H, device="cuda", generator=g)[:4]
        x[:, hot] *= 20.0
        st["x"] = x.bfloat16()
        bias = case["skew"] * torch.randn(E, device="cuda", generator=g)
        st["logits"] = torch.randn(T, E, device="cuda", generator=g) + bias
        for name, rows, cols in (("gate_up", 2 * I, H), ("down", H, I)):
            codes = torch.empty(E, rows * cols // 2, dtype=torch.uint8, device="cuda")
            sf = torch.empty(E, rows * cols // 16, dtype=torch.uint8, device="cuda")
            s_g = torch.empty(E, device="cuda")
            for e in range(E):
                codes[e], sf[e], s_g[e] = _pack(rows, cols, g)
            st[name] = (codes, sf, s_g, rows, cols)
        if own:
            _packed(st)
        return st
    V, ld = case["V"], case["pitch"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    buf = torch.empty(T, ld, dtype=dt, device="cuda")
    step = max(1, (1 << 27) // ld)
    for r in range(0, T, step):
        buf[r:r + step] = 2.5 * torch.randn(min(step, T - r), ld, device="cuda", generator=g)
    ids = torch.randint(0, V, (T,), device="cuda", generator=g)
    logits = buf[:, :V]
    if case["masked"]:
        # a grammar's vocabulary mask: the same share of the vocabulary is out for every row
        out = torch.rand(V, device="cuda", generator=g) < case["masked"]
        logits.masked_fill_(out, -math.inf)
    # the sampled tokens are mostly likely ones
    rows = torch.arange(T, device="cuda")
    logits[rows, ids] = (8.0 + 3.0 * torch.randn(T, device="cuda", generator=g)).to(dt)
    if case["padded"]:
        ids = torch.where(torch.rand(T, device="cuda", generator=g) < case["padded"], torch.full_like(ids, -1), ids)
    st = {"case": case, "logits": logits, "ids": ids}
    if case["train"]:
        live = (ids >= 0).float()
        st["g_lp"] = torch.randn(T, device="cuda", generator=g) * live
        st["g_ent"] = 0.01 * torch.randn(T, device="cuda", generator=g) * live if case["entropy_grad"] else None
    return st


def _packed(st):
    from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R

    for name in ("gate_up", "down"):
        codes, sf, s_g, rows, cols = st[name]
        st["w_" + name] = R.Packed(codes.view(-1), sf.view(-1), s_g, codes.shape[0], rows, rows, cols)


# ------------------------------------------------------------------------------------ plain forms
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _dequant(w, e):
    """Float32 weights of the experts e [n] -> [n, rows, cols]."""
    codes, sf, s_g, rows, cols = w
    n = e.numel()
    lut = torch.tensor(_E2M1, device="cuda")
    c = codes[e].int()
    v = lut[torch.stack((c & 15, c >> 4), -1)].view(n, rows, cols // 16, 16)
    s = sf[e].view(n, rows // 128, cols // 64, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, rows, cols // 16)
    s = s.contiguous().view(torch.float8_e4m3fn).float() * s_g[e].view(n, 1, 1)
    return (v * s.unsqueeze(-1)).view(n, rows, cols)


def _moe_plain_part(st, x, ids, w):
    T, k = ids.shape
    xp = x.repeat_interleave(k, 0).unsqueeze(-1)
    gu = torch.matmul(_dequant(st["gate_up"], ids.reshape(-1)), xp)  # [T k, 2I, 1], gate and up in chunks of 64
    gu = gu.view(T * k, -1, 2, 64)
    gate, up = gu[:, :, 0].reshape(T * k, -1), gu[:, :, 1].reshape(T * k, -1)
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.matmul(_dequant(st["down"], ids.reshape(-1)), h.unsqueeze(-1)).view(T, k, -1)
    return (w.unsqueeze(-1) * y).sum(1)


def _moe_plain(st):
    x, logits, k = st["x"], st["logits"], st["k"]
    T, H = x.shape
    order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = order.indices[:, :k]
    p = torch.exp(order.values[:, :k] - order.values[:, :1])
    w = p / p.sum(-1, keepdim=True)
    # every (token, expert) pair's weights at once, in as few parts as their memory allows
    n = max(1, (1 << 28) // (k * st["gate_up"][3] * H))
    out = torch.cat([_moe_plain_part(st, x[t:t + n].float(), ids[t:t + n], w[t:t + n]) for t in range(0, T, n)])
    return {"out": out.bfloat16(), "ids": ids.int(), "weights": w}


def _logprobs_plain(st):
    c = st["case"]
    live = st["ids"] >= 0
    safe = st["ids"].clamp_min(0)
    it = 1.0 / c["temperature"]
    z = st["logits"].float() * it
    z = z - z.amax(-1, keepdim=True)
    e = torch.exp(z)
    s = e.sum(-1, keepdim=True)
    logp = z - torch.log(s)
    p = e / s
    zero = torch.zeros((), device="cuda")
    lp = torch.where(live, logp.gather(1, safe.unsqueeze(1)).squeeze(1), zero)
    plogp = torch.where(p > 0, p * logp, zero)
    ent = torch.where(live, -plogp.sum(-1), zero)
    out = {"logprob": lp, "entropy": ent}
    if c["top"]:
        order = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        out["top_ids"] = torch.where(live.unsqueeze(1), order, torch.full_like(order, -1)).int()
        out["top_logprobs"] = torch.where(live.unsqueeze(1), logp.gather(1, order), zero)
    if c["train"]:
        grad = -st["g_lp"].unsqueeze(1) * p
        grad.scatter_add_(1, safe.unsqueeze(1), st["g_lp"].unsqueeze(1))
        if st["g_ent"] is not None:
            grad = grad - st["g_ent"].unsqueeze(1) * (plogp + p * ent.unsqueeze(1))
        grad = torch.where(live.unsqueeze(1), grad * it, zero)
        out["grad"] = grad.to(st["logits"].dtype)
    return out


# -------------------------------------------------------------------------------------------- run
def run(st):
    c = st["case"]
    if not own:
        return _moe_plain(st) if c["op"] == "moe" else _logprobs_plain(st)
    from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R

    if c["op"] == "moe":
        if "w_gate_up" not in st:
            _packed(st)
        out, ids, w = R.moe_w4a16_layer(st["x"], st["logits"], st["k"], st["w_gate_up"], st["w_down"])
        return {"out": out, "ids": ids, "weights": w}
    if not c["train"]:
        r = R.token_logprobs(st["logits"], st["ids"], temperature=c["temperature"], top=c["top"])
        out = {"logprob": r.logprob, "entropy": r.entropy}
        if c["top"]:
            out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
        return out
    leaf = st["logits"].detach().requires_grad_()
    r = R.token_logprobs(leaf, st["ids"], temperature=c["temperature"])
    outs, grads = [r.logprob], [st["g_lp"]]
    if st["g_ent"] is not None:
        outs.append(r.entropy)
        grads.append(st["g_ent"])
    (grad,) = torch.autograd.grad(outs, [leaf], grads)
    return {"logprob": r.logprob.detach(), "entropy": r.entropy.detach(), "grad": grad}


def work(case):
    T = case["T"]
    if case["op"] == "moe":
        H, I, E, k = case["H"], case["I"], case["E"], case["k"]
        # expected number of experts that T tokens touch; a skewed router touches fewer, and its
        # share is taken from the same draw of preferences that any seed gives on average
        p = [k / E] * E
        if case["skew"]:
            import random
            r = random.Random(1)
            hits = [0] * E
            n = 400
            for i in range(n):
                if i % 20 == 0:
                    bias = [case["skew"] * r.gauss(0, 1) for _ in range(E)]
                    seen = []
                row = sorted(range(E), key=lambda e: -(bias[e] + r.gauss(0, 1)))[:k]
                seen.append(row)
                if i % 20 == 19:
                    cnt = [0] * E
                    for s in seen:
                        for e in s:
                            cnt[e] += 1
                    for rank, v in enumerate(sorted(cnt, reverse=True)):
                        hits[rank] += v
            p = [h / n for h in hits]
        touched = sum(1.0 - (1.0 - min(q, 1.0)) ** T for q in p)
        weights = touched * 3 * H * I * 9 // 16
        return {"bytes": weights + T * (2 * H + 2 * H + 4 * E + 8 * k), "flops": 2.0 * T * k * 3 * H * I}
    size = 4 if case["dtype"] == "f32" else 2
    rows = T * (1.0 - case["padded"])
    n = rows * case["V"]
    byts = n * size + T * 16 + T * case["top"] * 8
    flops = 8.0 * n
    if case["train"]:
        byts += T * case["V"] * size  # the gradient is written for every row
        flops += 6.0 * n
    return {"bytes": byts, "flops": flops}


# ------------------------------------------------------------------------------------------ exact
def _exact_weights(w, e):
    codes, sf, s_g, rows, cols = w
    c = codes[e].view(rows, cols // 2)
    nib = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    nib[:, 0::2] = c & 15
    nib[:, 1::2] = c >> 4
    mag = (nib & 7).double()
    mag = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    val = torch.where(nib >= 8, -mag, mag)
    r = torch.arange(rows, device="cuda").unsqueeze(1)
    b = torch.arange(cols // 16, device="cuda").unsqueeze(0)
    at = ((r // 128) * (cols // 64) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    s = sf[e][at].view(torch.float8_e4m3fn).double()
    return (val.view(rows, -1, 16) * s.unsqueeze(-1)).view(rows, cols) * s_g[e].double()


def _moe_exact(st):
    x, logits, k = st["x"].double(), st["logits"].double(), st["k"]
    T, H = x.shape
    I = st["down"][4]
    ids = torch.empty(T, k, dtype=torch.int64, device="cuda")
    left = logits.clone()
    for j in range(k):
        ids[:, j] = left.argmax(-1)
        left.scatter_(1, ids[:, j:j + 1], -math.inf)
    w = torch.softmax(logits.gather(1, ids), -1)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    n = torch.arange(2 * I, device="cuda")
    gate_row, up_row = n[n % 128 < 64], n[n % 128 >= 64]
    for e in torch.unique(ids).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        y = x[t] @ _exact_weights(st["gate_up"], e).T
        gate = y[:, gate_row]
        h = gate * torch.sigmoid(gate) * y[:, up_row]
        out.index_add_(0, t, w[t, j].unsqueeze(1) * (h @ _exact_weights(st["down"], e).T))
    return {"out": out, "ids": ids.int(), "weights": w}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "moe":
        return _moe_exact(st)
    T, V, k = case["T"], case["V"], case["top"]
    lp = torch.zeros(T, dtype=torch.float64, device="cuda")
    ent = torch.zeros_like(lp)
    ret = {"logprob": lp, "entropy": ent}
    if k:
        ret["top_ids"] = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        ret["top_logprobs"] = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    if case["train"]:
        ret["grad"] = torch.zeros(T, V, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // V)
    for r0 in range(0, T, step):
        rows = (r0 + (st["ids"][r0:r0 + step] >= 0).nonzero().squeeze(1))
        if rows.numel() == 0:
            continue
        ids = st["ids"][rows]
        z = st["logits"][rows].double() / case["temperature"]
        logp = torch.log_softmax(z, -1)
        p = logp.exp()
        lp[rows] = logp[torch.arange(rows.numel(), device="cuda"), ids]
        ent[rows] = torch.special.entr(p).sum(-1)
        if k:
            left = st["logits"][rows].double()
            taken = torch.zeros_like(left, dtype=torch.bool)
            for j in range(k):
                best = torch.where(taken, torch.full_like(left, -math.inf), left).amax(-1, keepdim=True)
                i = ((left == best) & ~taken).int().argmax(-1, keepdim=True)
                taken.scatter_(1, i, True)
                ret["top_ids"][rows, j] = i.squeeze(1).int()
                ret["top_logprobs"][rows, j] = logp.gather(1, i).squeeze(1)
        if case["train"]:
            one = torch.zeros_like(p)
            one[torch.arange(rows.numel(), device="cuda"), ids] = 1.0
            d = st["g_lp"][rows].double().unsqueeze(1) * (one - p)
            if st["g_ent"] is not None:
                d = d + st["g_ent"][rows].double().unsqueeze(1) * (torch.special.entr(p) - p * ent[rows].unsqueeze(1))
            ret["grad"][rows] = d / case["temperature"]
    return ret
