"""Arguments that the gated block and the vocabulary cross entropy refuse,
before any device work (no GPU needed), and what their Python forms check."""
import contextlib
import ctypes

import numpy as np
import pytest

from decode_dfloat11_b200 import build as lwc_build
from decode_dfloat11_b200 import layers, lwc

P = 0x10000   # an address that is never touched


@pytest.fixture(scope="module", autouse=True)
def built():
    lwc_build.build()
    return lwc.load()


def gated(**change):
    values = dict(elem=0, act=0, tokens=4, features=16, hidden=32, ld_x=32, ld_gate=32, ld_up=32, x=P, gate=P, up=P)
    values.update(change)
    return lwc.lwc_gated(**values)


def xent(**change):
    values = dict(elem=0, reserved=0, tokens=4, vocab=100, hidden=32, ld_x=32, ld_head=32, x=P, head=P, targets=P,
                  ignore_index=-100)
    values.update(change)
    return lwc.lwc_xent(**values)


def refused(status, call, *args):
    with pytest.raises(lwc.LwcError) as e:
        call(*args)
    assert e.value.status == status, e.value


GATED = [
    (lwc.LWC_ERR_UNSUPPORTED, dict(elem=lwc.LWC_ELEM_FP32)), (lwc.LWC_ERR_UNSUPPORTED, dict(elem=9)),
    (lwc.LWC_ERR_INVALID_ARG, dict(act=5)), (lwc.LWC_ERR_INVALID_ARG, dict(features=0)),
    (lwc.LWC_ERR_INVALID_ARG, dict(hidden=0)), (lwc.LWC_ERR_UNSUPPORTED, dict(tokens=1 << 31)),
    (lwc.LWC_ERR_UNSUPPORTED, dict(features=1 << 31)), (lwc.LWC_ERR_UNSUPPORTED, dict(hidden=1 << 31, ld_x=1 << 31)),
    (lwc.LWC_ERR_INVALID_ARG, dict(ld_x=24)), (lwc.LWC_ERR_INVALID_ARG, dict(ld_gate=24)),
    (lwc.LWC_ERR_INVALID_ARG, dict(ld_up=31)), (lwc.LWC_ERR_INVALID_ARG, dict(x=None)),
    (lwc.LWC_ERR_INVALID_ARG, dict(gate=None)), (lwc.LWC_ERR_INVALID_ARG, dict(up=None)),
    (lwc.LWC_ERR_MISALIGNED, dict(ld_x=33)), (lwc.LWC_ERR_MISALIGNED, dict(ld_up=36)),
    (lwc.LWC_ERR_MISALIGNED, dict(x=P + 8)), (lwc.LWC_ERR_MISALIGNED, dict(gate=P + 2)),
]


@pytest.mark.parametrize("status,change", GATED)
def test_gated_problem(status, change):
    g = gated(**change)
    refused(status, lwc.lwc_gated_forward, g, P, 16)
    refused(status, lwc.lwc_gated_backward, g, P, 16, P, P, P, P, 1 << 30)
    assert lwc.lwc_gated_backward_workspace_bytes(g) == 0


def test_gated_calls():
    g = gated()
    refused(lwc.LWC_ERR_INVALID_ARG, lwc.lwc_gated_forward, g, P, 15)
    refused(lwc.LWC_ERR_INVALID_ARG, lwc.lwc_gated_forward, g, None, 16)
    refused(lwc.LWC_ERR_INVALID_ARG, lwc.lwc_gated_forward, g, P + 1, 16)
    refused(lwc.LWC_ERR_MISALIGNED, lwc.lwc_gated_forward, g, P, 16, P + 2)
    back = lwc.lwc_gated_backward
    refused(lwc.LWC_ERR_INVALID_ARG, back, g, P, 15, P, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_INVALID_ARG, back, g, None, 16, P, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, g, P, 16, P + 1, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, g, P, 16, P, P, P, None, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, g, P, 16, P, P, P, P + 128, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, g, P, 16, P, P, P, P, 1 << 30, P + 1)
    with pytest.raises(lwc.LwcError):
        lwc._check(lwc.load().lwc_gated_forward(None, P, 16, None, None))
    # nothing to do: no device is asked for
    lwc.lwc_gated_forward(gated(tokens=0, x=None), None, 16)
    lwc.lwc_gated_backward(g, P, 16, None, None, None, None, 0)
    lwc.lwc_gated_backward(gated(tokens=0), None, 16, P, None, None, None, 0)


def test_gated_product():
    f = lwc.lwc_gated_product
    refused(lwc.LWC_ERR_UNSUPPORTED, f, lwc.LWC_ELEM_FP32, 0, P, P, 4, P)
    refused(lwc.LWC_ERR_INVALID_ARG, f, 0, 7, P, P, 4, P)
    refused(lwc.LWC_ERR_INVALID_ARG, f, 0, 0, None, P, 4, P)
    refused(lwc.LWC_ERR_INVALID_ARG, f, 0, 0, P, P, 4, None)
    refused(lwc.LWC_ERR_MISALIGNED, f, 0, 0, P + 2, P, 4, P)
    refused(lwc.LWC_ERR_MISALIGNED, f, 0, 0, P, P, 4, P + 1)
    f(0, 0, None, None, 0, None)


XENT = [
    (lwc.LWC_ERR_UNSUPPORTED, dict(elem=lwc.LWC_ELEM_FP32)), (lwc.LWC_ERR_INVALID_ARG, dict(vocab=0)),
    (lwc.LWC_ERR_INVALID_ARG, dict(hidden=0)), (lwc.LWC_ERR_UNSUPPORTED, dict(tokens=1 << 31)),
    (lwc.LWC_ERR_UNSUPPORTED, dict(vocab=1 << 31)), (lwc.LWC_ERR_INVALID_ARG, dict(ld_x=24)),
    (lwc.LWC_ERR_INVALID_ARG, dict(ld_head=24)), (lwc.LWC_ERR_INVALID_ARG, dict(x=None)),
    (lwc.LWC_ERR_INVALID_ARG, dict(head=None)), (lwc.LWC_ERR_INVALID_ARG, dict(targets=None)),
    (lwc.LWC_ERR_MISALIGNED, dict(ld_head=33)), (lwc.LWC_ERR_MISALIGNED, dict(head=P + 8)),
    (lwc.LWC_ERR_MISALIGNED, dict(targets=P + 4)),
]


@pytest.mark.parametrize("status,change", XENT)
def test_xent_problem(status, change):
    x = xent(**change)
    refused(status, lwc.lwc_xent_forward, x, P, P, P, P, P, 1 << 30)
    refused(status, lwc.lwc_xent_backward, x, P, P, 0, True, P, P, P, 1 << 30)
    assert lwc.lwc_xent_forward_workspace_bytes(x) == 0
    assert lwc.lwc_xent_backward_workspace_bytes(x) == 0


def test_xent_calls():
    x = xent()
    fwd, back = lwc.lwc_xent_forward, lwc.lwc_xent_backward
    refused(lwc.LWC_ERR_INVALID_ARG, fwd, x, None, P, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_INVALID_ARG, fwd, x, P, None, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, fwd, x, P + 2, P, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, fwd, x, P, P, P + 1, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, fwd, x, P, P, None, P + 2, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, fwd, x, P, P, P, P, None, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, fwd, x, P, P, P, P, P, 1 << 30, P + 3)
    refused(lwc.LWC_ERR_INVALID_ARG, back, x, None, P, 0, True, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_INVALID_ARG, back, x, P, None, 0, True, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, x, P, P, 0, True, P + 1, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, x, P, P, 0, True, P, P, P + 16, 1 << 30)
    back(x, P, P, 0, True, None, None, None, 0)
    fwd(xent(tokens=0, x=None, targets=None), None, None, None, None, None, 0)


def test_structures_match_the_header():
    assert ctypes.sizeof(lwc.lwc_gated) == 8 + 6 * 8 + 3 * 8
    assert ctypes.sizeof(lwc.lwc_xent) == 8 + 5 * 8 + 3 * 8 + 8


def test_python_forms_check_their_arguments():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    t = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        layers.gated_ffn(x, w, w)
    with pytest.raises(ValueError, match="BF16 or FP16"):
        layers.gated_ffn(x.float(), w, w)
    with pytest.raises(ValueError, match="CUDA"):
        layers.linear_cross_entropy(x, w, t)
    with pytest.raises(ValueError, match="BF16 or FP16"):
        layers.linear_cross_entropy(x.double(), w, t)
    with pytest.raises(ValueError, match="activation"):
        layers._act_id("swish2")


def test_a_product_without_a_gradient_refuses_to_drop_one(monkeypatch):
    """TiledWeights.gated has no backward pass: its result would silently end the graph."""
    torch = pytest.importorskip("torch")
    tw = layers.TiledWeights("cpu")
    tw.descs, tw.blobs, tw.shapes = [lwc.lwc_desc(), lwc.lwc_desc()], [torch.zeros(1)] * 2, [(128, 64), (128, 64)]
    x = torch.zeros(2, 64, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        tw.gated(0, 1, x)
    # nothing is asked for: taken
    for name in ("lwc_gemm_dfloat11_batched", "lwc_gated_product"):
        monkeypatch.setattr(lwc, name, lambda *args, **kwargs: None)
    monkeypatch.setattr(layers, "_On", lambda *args: contextlib.nullcontext())
    with torch.no_grad():
        assert tw.gated(0, 1, x).shape == (2, 128)
    assert tw.gated(0, 1, x.detach()).shape == (2, 128)


@pytest.mark.parametrize("codec,params,values,route", [
    ("dfloat11", {}, "spread", "fused"), ("dfloat11", dict(threads_per_block=64), "spread", "decode"),
    ("dfloat11", dict(threads_per_block=64), "one exponent", "fused"), ("codebook", {}, "spread", "fused")])
def test_one_row_of_any_blob_finds_a_route(monkeypatch, codec, params, values, route):
    """The decode-fused linear layer takes DFloat11 blocks of 32 chunks only; "auto" decodes the others."""
    torch = pytest.importorskip("torch")
    w = np.random.default_rng(1).integers(0x3F00, 0x3F80 if values == "one exponent" else 0x4100, 64 * 64).astype(np.uint16)
    model = layers.ResidentModel(codec, "cpu")
    model.add_layer("ffn", layers.encode_many([w, w], codec, **params), [(64, 64)] * 2)
    taken = []
    for name in ("lwc_linear_dfloat11_batched", "lwc_linear_codebook_batched"):
        monkeypatch.setattr(lwc, name, lambda *args, **kwargs: taken.append("fused"))
    for name in ("lwc_decode_dfloat11_batched", "lwc_decode_codebook_batched"):
        monkeypatch.setattr(lwc, name, lambda *args, **kwargs: taken.append("decode"))
    for name in ("lwc_gated_product", "lwc_gated_forward"):
        monkeypatch.setattr(lwc, name, lambda *args, **kwargs: None)
    monkeypatch.setattr(layers, "_On", lambda *args: contextlib.nullcontext())
    monkeypatch.setattr(layers, "_check_matrices", lambda x, **matrices: None)
    model.gated(0, 0, 1, torch.zeros(1, 64, dtype=torch.bfloat16))
    assert taken == [route]


def test_replaced_layers_are_marshalled_again():
    """Launch arguments are bare addresses: those of a blob, or a layer, that was replaced must not be used."""
    torch = pytest.importorskip("torch")

    def layer(seed):
        g = np.random.default_rng(seed)
        return layers.encode_many([g.integers(0, 1 << 16, 64 * 8).astype(np.uint16) for _ in range(2)], "codebook")

    model = layers.ResidentModel("codebook", "cpu")
    model.add_layer("ffn", layer(1), [(64, 8)] * 2)
    first = model._matrices(0, (0, 1))
    assert model._matrices(0, (0, 1)) is first and model._matrices(0, (1,)) is not first
    assert list(first[0].ins) == [b.data_ptr() for b in model.layers[0]["blobs"]]
    # one blob
    desc, blob = layer(2)[1]
    model.layers[0]["descs"][1], model.layers[0]["blobs"][1] = desc, torch.from_numpy(blob)
    assert list(model._matrices(0, (0, 1))[0].ins) == [b.data_ptr() for b in model.layers[0]["blobs"]]
    # the whole layer, in another shape
    model.layers.clear()
    model.add_layer("ffn", layer(3), [(32, 16)] * 2)
    again = model._matrices(0, (0, 1))
    assert list(again[0].ins) == [b.data_ptr() for b in model.layers[0]["blobs"]] and again[2] == [(32, 16)] * 2
    assert list(again[1].blobs) == list(again[0].ins)
    # the same shape put in as another list
    model.layers[0]["shapes"] = [(16, 32), (16, 32)]
    assert model._matrices(0, (0, 1))[2] == [(16, 32)] * 2


def test_xent_backward_from_losses():
    back = lwc.lwc_xent_backward_losses
    for status, change in XENT:
        refused(status, back, xent(**change), P, P, P, 0, True, P, P, P, 1 << 30)
    x = xent()
    refused(lwc.LWC_ERR_INVALID_ARG, back, x, None, P, P, 0, True, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_INVALID_ARG, back, x, P, None, P, 0, True, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_INVALID_ARG, back, x, P, P, None, 0, True, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, x, P, P + 2, P, 0, True, P, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, x, P, P, P, 0, True, P + 1, P, P, 1 << 30)
    refused(lwc.LWC_ERR_MISALIGNED, back, x, P, P, P, 0, True, P, P, P + 16, 1 << 30)
    back(x, P, None, P, 0, True, None, None, None, 0)


def test_forward_mode_is_refused():
    """A dual tensor asks for no gradient, so its tangent would be dropped silently."""
    torch = pytest.importorskip("torch")
    from torch.autograd import forward_ad
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(128, 64, dtype=torch.bfloat16)
    t, f = torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    h = torch.zeros(2, 128, dtype=torch.bfloat16)
    model = layers.ResidentModel("codebook", "cpu")
    model.layers.append(dict(descs=[lwc.lwc_desc()] * 2, blobs=[torch.zeros(1)] * 2, shapes=[(128, 64)] * 2))
    tw = layers.TiledWeights("cpu")
    tw.descs, tw.blobs, tw.shapes = [lwc.lwc_desc(), lwc.lwc_desc()], [torch.zeros(1)] * 2, [(128, 64), (128, 64)]
    with forward_ad.dual_level():
        def dual(v):
            return forward_ad.make_dual(v, torch.ones_like(v))
        for call in (lambda: layers.gated_ffn(dual(x), w, w), lambda: layers.gated_ffn(x, w, dual(w)),
                     lambda: layers.gated_ffn_backward(dual(h), x, w, w),
                     lambda: layers.linear_cross_entropy(dual(x), w, t), lambda: layers.linear_cross_entropy(x, dual(w), t),
                     lambda: layers.linear_cross_entropy_backward(dual(f), f, x, w, t, reduction="none"),
                     lambda: model.gated(0, 0, 1, dual(x)), lambda: model.cross_entropy(0, 0, dual(x), t),
                     lambda: tw.gated(0, 1, dual(x))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        # plain tensors meet their own checks inside a dual level too
        with pytest.raises(ValueError, match="CUDA"):
            layers.gated_ffn(x, w, w)


@pytest.mark.parametrize("codec,one,other", [("codebook", dict(k=12), dict(k=13)),
                                             ("dfloat11", dict(chunk_bytes=20), dict(chunk_bytes=36))])
def test_tiled_matrices_that_one_launch_does_not_take(monkeypatch, codec, one, other):
    torch = pytest.importorskip("torch")
    calls = []
    for name in (f"lwc_gemm_{codec}", f"lwc_gemm_{codec}_batched"):
        monkeypatch.setattr(lwc, name, lambda *args, name=name, **kwargs: calls.append(name))
    monkeypatch.setattr(lwc, "lwc_gated_product", lambda *args: None)
    monkeypatch.setattr(layers, "_On", lambda *args: contextlib.nullcontext())
    tw = layers.TiledWeights("cpu", codec)
    tw.descs = [lwc.lwc_desc(**one), lwc.lwc_desc(**one), lwc.lwc_desc(**other)]
    tw.blobs, tw.shapes = [torch.zeros(1)] * 3, [(128, 64)] * 3
    for up, want in ((1, [f"lwc_gemm_{codec}_batched"]), (2, [f"lwc_gemm_{codec}"] * 2)):
        calls.clear()
        tw.gated(0, up, torch.zeros(2, 64, dtype=torch.bfloat16))
        assert calls == want
    for rows, together in ((128 * 2048, True), (128 * 2049, False)):
        tw.shapes = [(rows, 64)] * 3
        assert tw._one_launch(0, 1) == together


def test_tiled_matrices_of_another_device_are_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(lwc, "lwc_gemm_dfloat11_batched", lambda *args, **kwargs: pytest.fail("launched"))
    tw = layers.TiledWeights("meta")
    tw.descs, tw.blobs, tw.shapes = [lwc.lwc_desc()] * 2, [torch.zeros(1, device="meta")] * 2, [(128, 64)] * 2
    with pytest.raises(ValueError, match="device"):
        tw.gated(0, 1, torch.zeros(2, 64, dtype=torch.bfloat16))
