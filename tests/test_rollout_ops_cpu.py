"""Host-side refusals of the few-token MoE layer and the token log probabilities: every bad call
stops before a device is touched (the pointers are made up and never read)."""
import ctypes

import pytest

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from nvfp4_w4a4_moe_02_b200 import build_lib, nvfp4rac

    build_lib.build()
    return nvfp4rac.load()


def layer_args(**kw):
    from nvfp4_w4a4_moe_02_b200.nvfp4rac import CTensor

    a = dict(x=16, T=4, ldx=256, logits=16, k=2, E=4, H=256, I=128, ids=16, w=16, out=16, ldo=256, ws=16, ws_bytes=1 << 30,
             gu={}, dn={})
    a.update(kw)
    gu = dict(codes=16, sf=16, s_g=16, slabs=a["E"], rows=2 * a["I"], rows_padded=2 * a["I"], cols=a["H"], sf_layout=0)
    dn = dict(codes=16, sf=16, s_g=16, slabs=a["E"], rows=a["H"], rows_padded=a["H"], cols=a["I"], sf_layout=0)
    gu.update(a["gu"])
    dn.update(a["dn"])
    return (a["x"], a["T"], a["ldx"], a["logits"], a["k"], ctypes.byref(CTensor(**gu)), ctypes.byref(CTensor(**dn)),
            a["ids"], a["w"], a["out"], a["ldo"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=65), SHAPE), (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=5), SHAPE), (dict(k=33, E=64), SHAPE),
    (dict(E=1025), SHAPE), (dict(E=0), SHAPE), (dict(H=192, ldx=192, ldo=192), SHAPE), (dict(I=96), SHAPE),
    (dict(H=32896, ldx=32896, ldo=32896), SHAPE), (dict(I=0), SHAPE),
    (dict(gu=dict(rows=128)), SHAPE), (dict(gu=dict(rows_padded=384)), SHAPE), (dict(dn=dict(slabs=3)), SHAPE),
    (dict(dn=dict(rows=128)), SHAPE), (dict(dn=dict(sf_layout=1)), SHAPE), (dict(dn=dict(codes=0)), INVALID),
    (dict(gu=dict(s_g=0)), INVALID), (dict(gu=dict(codes=24)), ALIGN),
    (dict(x=0), INVALID), (dict(logits=0), INVALID), (dict(ids=0), INVALID), (dict(w=0), INVALID), (dict(out=0), INVALID),
    (dict(x=18), ALIGN), (dict(ldx=248), ALIGN), (dict(ldx=260), ALIGN), (dict(out=24), ALIGN), (dict(ldo=128), ALIGN),
    (dict(ws=0), INVALID), (dict(ws_bytes=64), INVALID), (dict(ws=24), ALIGN),
])
def test_layer_refusals(lib, kw, status):
    assert lib.moe_w4a16_layer(*layer_args(**kw)) == status
    assert lib.nvfp4_last_error_string()


def test_layer_without_tokens_needs_no_device(lib):
    assert lib.moe_w4a16_layer(*layer_args(T=0, x=0, logits=0, out=0, ids=0, w=0, ws=0, ws_bytes=0)) == OK
    assert lib.moe_w4a16_layer(None, 0, 256, None, 2, None, None, None, None, None, 256, None, 0, None, None) == INVALID


def test_layer_workspace_size(lib):
    assert lib.moe_w4a16_workspace_size(0, 2, 256, 128) == 0
    assert lib.moe_w4a16_workspace_size(64, 8, 7168, 2048) >= 512 * 2048 * 2
    assert lib.moe_w4a16_workspace_size(2, 2, 256, 128) < lib.moe_w4a16_workspace_size(3, 2, 256, 128)


def fwd(**kw):
    a = dict(logits=16, dtype=0, T=4, V=100, ldl=100, ids=16, id_bytes=8, it=1.0, top=0, lp=16, ent=16, stats=16, ti=16,
             tl=16)
    a.update(kw)
    return tuple(a.values()) + (None, None)


def bwd(**kw):
    a = dict(logits=16, dtype=0, T=4, V=100, ldl=100, ids=16, id_bytes=8, it=1.0, stats=16, g=16, ge=16, grad=32, ldg=100)
    a.update(kw)
    return tuple(a.values()) + (None, None)


COMMON = [(dict(dtype=2), INVALID), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(V=0), SHAPE),
          (dict(V=1 << 31, ldl=1 << 31), SHAPE), (dict(ldl=99), ALIGN), (dict(logits=0), INVALID), (dict(logits=18), ALIGN),
          (dict(logits=17, dtype=1), ALIGN), (dict(ids=0), INVALID), (dict(ids=20), ALIGN), (dict(id_bytes=2), INVALID),
          (dict(it=0.0), INVALID), (dict(it=-1.0), INVALID), (dict(it=float("nan")), INVALID),
          (dict(it=float("inf")), INVALID), (dict(stats=24), ALIGN)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(top=33), SHAPE), (dict(top=-1), SHAPE), (dict(top=8, V=7), SHAPE), (dict(lp=0), INVALID),
    (dict(top=2, ti=0), INVALID), (dict(top=2, tl=0), INVALID)])
def test_logprob_refusals(lib, kw, status):
    assert lib.token_logprobs(*fwd(**kw)) == status
    assert lib.nvfp4_last_error_string()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(stats=0), INVALID), (dict(grad=0), INVALID), (dict(ldg=99), ALIGN), (dict(grad=34), ALIGN),
    (dict(grad=16, ldg=104), INVALID)])
def test_logprob_backward_refusals(lib, kw, status):
    assert lib.token_logprobs_backward(*bwd(**kw)) == status
    assert lib.nvfp4_last_error_string()


def test_no_rows_need_no_device(lib):
    assert lib.token_logprobs(*fwd(T=0, logits=0, ids=0, lp=0)) == OK
    assert lib.token_logprobs_backward(*bwd(T=0, logits=0, ids=0, stats=0, grad=0)) == OK


def test_binding_refuses_host_tensors(lib):
    import torch

    from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R

    with pytest.raises(R.NVFP4Error):
        R.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))
    p = R.Packed(torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8), torch.zeros(4), 4, 256, 256, 256)
    with pytest.raises(R.NVFP4Error):
        R.moe_w4a16_layer(torch.zeros(1, 256, dtype=torch.bfloat16), torch.zeros(1, 4), 2, p, p)


def test_a_stream_of_another_device_is_refused():
    import types

    import torch
    from nvfp4_w4a4_moe_02_b200 import nvfp4rac as R

    stream = types.SimpleNamespace(cuda_stream=16, device_index=1)
    with pytest.raises(R.NVFP4Error, match="device 1"):
        R._on(torch.device("cuda", 0), stream)
