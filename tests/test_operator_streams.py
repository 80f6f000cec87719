"""Which stream the operators' own copies run on, and which tensors they record
there, checked with the library's calls replaced by recorders (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from decode_dfloat11_b200 import layers, lwc  # noqa: E402

STREAM = "another stream"


class Recorder:
    """Stands for layers._On: where one is inside it, and what it was given."""
    inside = []
    given = []

    def __init__(self, device, stream=None, used=()):
        self.stream, self.used = stream, used

    def __enter__(self):
        Recorder.inside.append(self.stream)
        Recorder.given.append((self.stream, self.used))
        return self.stream

    def __exit__(self, *error):
        Recorder.inside.pop()


@pytest.fixture
def recorder(monkeypatch):
    Recorder.inside, Recorder.given = [], []
    monkeypatch.setattr(layers, "_On", Recorder)
    copies = []
    plain = torch.Tensor.contiguous

    def contiguous(self, *args, **kwargs):
        if not self.is_contiguous():
            copies.append(list(Recorder.inside))
        return plain(self, *args, **kwargs)

    monkeypatch.setattr(torch.Tensor, "contiguous", contiguous)
    Recorder.copies = copies
    return Recorder


@pytest.fixture
def tiled(monkeypatch):
    """TiledWeights of two 128 x 64 matrices, with calls that do nothing."""
    for name in ("lwc_gemm_dfloat11", "lwc_gemm_dfloat11_batched", "lwc_gated_product", "lwc_linear_dfloat11"):
        monkeypatch.setattr(lwc, name, lambda *args, **kwargs: None)
    tw = layers.TiledWeights("cpu")
    tw.descs, tw.blobs, tw.shapes = [lwc.lwc_desc(), lwc.lwc_desc()], [torch.zeros(1)] * 2, [(128, 64), (128, 64)]
    return tw


@pytest.mark.parametrize("call", ["gated", "gemm", "gemm_batched", "fused_linear"])
def test_a_strided_x_is_copied_on_the_stream_that_reads_it(recorder, tiled, call):
    x = torch.zeros(64, 4, dtype=torch.bfloat16).t()
    if call == "gated":
        tiled.gated(0, 1, x, stream=STREAM)
    elif call == "gemm":
        tiled.gemm(0, x, stream=STREAM)
    elif call == "gemm_batched":
        tiled.gemm_batched([0, 1], [x, x], stream=STREAM)
    else:
        layers.fused_linear(lwc.lwc_desc(), None, (128, 64), x, "dfloat11", stream=STREAM, route="fused")
    assert recorder.copies and all(STREAM in where for where in recorder.copies)
    # and x itself is not given back before the copy was made
    assert any(stream == STREAM and any(t is x for t in used) for stream, used in recorder.given)


@pytest.mark.parametrize("call", ["gated_ffn", "linear_cross_entropy", "resident gated", "resident cross_entropy"])
def test_differentiable_calls_record_what_they_read(recorder, monkeypatch, call):
    """Their owner may free the operands (a loss dropped without a backward pass) before the stream read them."""
    class Function:
        @staticmethod
        def apply(*args):
            return torch.zeros(()), torch.zeros(())

    monkeypatch.setattr(layers, "_functions", lambda: dict.fromkeys(("gated", "xent", "resident_gated", "resident_xent"),
                                                                    Function))
    monkeypatch.setattr(layers, "_check_matrices", lambda x, **matrices: None)
    x = torch.zeros(2, 8, dtype=torch.bfloat16, requires_grad=True)
    w, v = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    t = torch.zeros(2, dtype=torch.int64)
    model = layers.ResidentModel("codebook", "cpu")
    model.layers.append(dict(descs=[lwc.lwc_desc()] * 2, blobs=[torch.zeros(1)] * 2, shapes=[(4, 8)] * 2))
    if call == "gated_ffn":
        read = [x, w, v]
        layers.gated_ffn(x, w, v, stream=STREAM)
    elif call == "linear_cross_entropy":
        read = [x, w, t]
        layers.linear_cross_entropy(x, w, t, stream=STREAM)
    elif call == "resident gated":
        read = [x]
        model.gated(0, 0, 1, x, stream=STREAM)
    else:
        read = [x, t]
        model.cross_entropy(0, 0, x, t, stream=STREAM)
    used = [u for stream, given in recorder.given if stream == STREAM for u in given]
    assert all(any(u is r for u in used) for r in read)


@pytest.mark.parametrize("call", ["tiled gated", "gated_ffn", "resident gated", "gated_ffn_backward",
                                  "linear_cross_entropy", "linear_cross_entropy_backward"])
def test_outputs_and_status_words_are_recorded_too(recorder, tiled, monkeypatch, call):
    """What the stream writes late must not be another tensor's memory by then."""
    for name in ("lwc_gated_forward", "lwc_gated_backward", "lwc_xent_forward", "lwc_xent_backward",
                 "lwc_linear_codebook_batched"):
        monkeypatch.setattr(lwc, name, lambda *args, **kwargs: None)
    for name in ("lwc_gated_backward_workspace_bytes", "lwc_xent_forward_workspace_bytes",
                 "lwc_xent_backward_workspace_bytes"):
        monkeypatch.setattr(lwc, name, lambda *args, **kwargs: 0)
    monkeypatch.setattr(layers, "_check_matrices", lambda x, **matrices: None)
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(128, 64, dtype=torch.bfloat16)
    t, f = torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    out, status = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    if call == "tiled gated":
        tiled.gated(0, 1, x, out=out, stream=STREAM, status=status)
    elif call == "gated_ffn":
        layers.gated_ffn(x, w, w, out=out, stream=STREAM, status=status)
    elif call == "resident gated":
        model = layers.ResidentModel("codebook", "cpu")
        model.layers.append(dict(descs=[lwc.lwc_desc()] * 2, blobs=[torch.zeros(1)] * 2, shapes=[(128, 64)] * 2))
        model.gated(0, 0, 1, x, out=out, stream=STREAM, status=status)
    elif call == "gated_ffn_backward":
        layers.gated_ffn_backward(out, x, w, w, stream=STREAM, status=status)
    elif call == "linear_cross_entropy":
        layers.linear_cross_entropy(x, w, t, stream=STREAM, status=status)
    else:
        layers.linear_cross_entropy_backward(f, f, x, w, t, reduction="none", stream=STREAM, status=status)
    used = [u for stream, given in recorder.given if stream == STREAM for u in given]
    assert any(u is status for u in used)
    assert any(u is out for u in used) or call.startswith("linear")


@pytest.mark.parametrize("codec", layers.CODECS)
def test_a_decoded_buffer_belongs_to_the_stream_that_uses_it(recorder, monkeypatch, codec):
    """fused_linear's route "decode" returns before its buffer has been read."""
    where = []
    plain = torch.empty

    def empty(shape, **kwargs):
        if tuple(shape) == (16, 64):
            where.append(list(Recorder.inside))
        return plain(shape, **kwargs)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "mm", lambda x, w, out_dtype: plain((x.shape[0], w.shape[1]), dtype=out_dtype).zero_())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: layers.contextlib.nullcontext())
    for name in ("lwc_decode_dfloat11_checked", "lwc_decode_codebook_checked"):
        monkeypatch.setattr(lwc, name, lambda *args: None)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    layers.fused_linear(lwc.lwc_desc(), None, (16, 64), x, codec, stream=STREAM, route="decode")
    assert where == [[STREAM]]


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda:1")

    with pytest.raises(ValueError, match="cuda:1"):
        with layers._On(torch.device("cuda:0"), Stream()):
            pytest.fail("entered")
