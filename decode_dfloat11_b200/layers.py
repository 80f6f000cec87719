"""Compressed model weights resident in GPU memory, decoded layer by layer.

This follows the DFloat11 page ("Koniec z kompromisami! DFloat11 ratuje
dokładność modeli AI ...", section "Jak to działa w praktyce? Magia na
poziomie GPU", third pillar): the weights stay compressed in HBM and all the
matrices of one transformer block are decompressed together, in one launch,
right before the block runs. Decoded layers land in a small set of reusable
BF16 buffers (two by default: a ping-pong pair, so layer L+1 can be decoded
while layer L is in use).

Everything here is bookkeeping and argument marshalling around the C ABI
(``lwc_decode_dfloat11_batched`` / ``lwc_decode_codebook_batched``); the
decoding itself runs in liblwc's CUDA kernels.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import os


from . import lwc

CODECS = ("dfloat11", "codebook")


def encode_many(arrays, codec: str = "dfloat11", workers: int | None = None, **params):
    """Encode host BF16 bit-pattern arrays in parallel host threads (the C
    encoder releases the GIL). Returns [(desc, blob), ...] in input order."""
    if codec not in CODECS:
        raise ValueError(f"unknown codec {codec!r}")
    fn = (lambda a: lwc.lwc_encode_dfloat11(a, **params)) if codec == "dfloat11" else lwc.lwc_encode_codebook
    workers = workers or min(len(arrays), os.cpu_count() or 1) or 1
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        return list(ex.map(fn, arrays))


def encode_on_device(tensor, codec: str = "dfloat11", workspace=None, stream=None, **params):
    """Compress a tensor that is already on the GPU into a device blob
    (``lwc_encode_*_device_plan`` + ``lwc_encode_device_write``). BF16 (or any
    16-bit patterns) for both codecs; float32 / float16 tensors with the
    DFloat11 codec use its FP32 / FP16 element types.

    Returns ``(desc, blob)`` with ``blob`` a uint8 CUDA tensor of
    ``desc.total_bytes`` bytes, byte-for-byte what the host encoder would make.
    ``workspace`` (a uint8 CUDA tensor of at least
    ``lwc_encode_device_workspace_bytes(n)`` bytes) may be passed to reuse one
    buffer across tensors; the tensor must not change while this runs."""
    import torch
    if codec not in CODECS:
        raise ValueError(f"unknown codec {codec!r}")
    src = tensor.reshape(-1).contiguous()
    elem = lwc.LWC_ELEM_BF16
    if src.dtype == torch.float32 or src.dtype == torch.int32:
        elem = lwc.LWC_ELEM_FP32
    elif src.dtype == torch.float16:
        elem = lwc.LWC_ELEM_FP16
    elif src.element_size() != 2:
        raise ValueError("expected a 16-bit or 32-bit tensor")
    if elem != lwc.LWC_ELEM_BF16 and codec != "dfloat11":
        raise ValueError("FP32 / FP16 element types are a DFloat11 feature (the codebook takes 16-bit patterns)")
    n = src.numel()
    need = lwc.lwc_encode_device_workspace_bytes(n)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=src.device)
    work_bytes = workspace.numel()
    stream = stream if stream is not None else torch.cuda.current_stream(src.device)
    if codec == "dfloat11":
        desc = lwc.lwc_encode_dfloat11_elements_device_plan(src, n, elem, workspace, work_bytes, stream=stream,
                                                            **params)
    else:
        desc = lwc.lwc_encode_codebook_device_plan(src, n, workspace, work_bytes, stream=stream)
    blob = torch.empty(desc.total_bytes, dtype=torch.uint8, device=src.device)
    desc = lwc.lwc_encode_device_write(src, n, workspace, work_bytes, blob, blob.numel(), stream=stream)
    return desc, blob


# Activation rows from which the DFloat11 decode-fused linear layer is slower
# than decoding the matrix and running the GEMM (Llama-3-8B layer on B200:
# fused 1.43 x faster at M = 1, 0.88 x at M = 4).
DF11_FUSED_MAX_M = 2


def fused_linear(desc, blob, shape, x, codec: str, out=None, stream=None, status=None, route: str = "auto"):
    """y = x W^T with W (``shape`` = (rows, cols), the tensor ``blob``
    decodes to); x: M x cols BF16 on the GPU, M <= 8. Returns ``out`` (M x
    rows FP32, allocated if None).

    route "fused": the decode-fused kernel (W decoded in registers, never
    written); "decode": decode W into a BF16 buffer, then a BF16 x BF16 ->
    FP32 GEMM (torch.mm; its summation order is cuBLAS's, so the bound is
    gamma_cols); "auto": fused, except DFloat11 with more than
    DF11_FUSED_MAX_M rows, where the fused kernel is the slower of the two."""
    import torch
    if codec not in CODECS:
        raise ValueError(f"unknown codec {codec!r}")
    if route not in ("auto", "fused", "decode"):
        raise ValueError(f"unknown route {route!r}")
    if len(shape) != 2:
        raise ValueError("the weight must be a rows x cols matrix")
    rows, cols = int(shape[0]), int(shape[1])
    if x.dim() != 2 or x.shape[1] != cols or x.dtype != torch.bfloat16:
        raise ValueError(f"x must be M x {cols} BF16")
    x = _contiguous_on(x, stream)
    M = int(x.shape[0])
    if out is None:
        out = torch.empty((M, rows), dtype=torch.float32, device=x.device)
    elif tuple(out.shape) != (M, rows) or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {M} x {rows} FP32 tensor")
    if route == "auto":
        route = "decode" if codec == "dfloat11" and M > DF11_FUSED_MAX_M else "fused"
    if route == "decode":
        dec = lwc.lwc_decode_dfloat11_checked if codec == "dfloat11" else lwc.lwc_decode_codebook_checked
        with _On(x.device, stream, (x, out, status)) as s:
            # the buffer belongs to the stream that still uses it when this returns
            w = torch.empty((rows, cols), dtype=torch.bfloat16, device=x.device)
            dec(desc, blob, w, status, s)
            out.copy_(torch.mm(x, w.t(), out_dtype=torch.float32))
        return out
    fn = lwc.lwc_linear_dfloat11 if codec == "dfloat11" else lwc.lwc_linear_codebook
    fn(desc, blob, cols, x, M, out, d_status=status, stream=stream)
    return out


ACTIVATIONS = {"silu": lwc.LWC_ACT_SILU, "gelu": lwc.LWC_ACT_GELU, "gelu_tanh": lwc.LWC_ACT_GELU_TANH,
               "relu": lwc.LWC_ACT_RELU, "sigmoid": lwc.LWC_ACT_SIGMOID}


def _act_id(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r} (known: {', '.join(ACTIVATIONS)})")
    return ACTIVATIONS[act]


def _elem_of(dtype) -> int:
    import torch
    if dtype == torch.bfloat16:
        return lwc.LWC_ELEM_BF16
    if dtype == torch.float16:
        return lwc.LWC_ELEM_FP16
    raise ValueError(f"expected BF16 or FP16 tensors, got {dtype}")


def _check_matrices(x, **matrices):
    """x (... x K) and the matrices (rows x K) that multiply it: one device, one 16-bit type."""
    _elem_of(x.dtype)
    if not x.is_cuda or x.dim() < 1:
        raise ValueError("x must be a CUDA tensor of at least one dimension")
    for name, w in matrices.items():
        if w.dim() != 2 or w.shape[1] != x.shape[-1] or w.shape[0] < 1 or w.shape[1] < 1:
            raise ValueError(f"{name} must be rows x {x.shape[-1]}, got {tuple(w.shape)}")
        if w.dtype != x.dtype or w.device != x.device:
            raise ValueError(f"{name} must have x's type and device ({x.dtype}, {x.device})")


def _refuse_tangents(*tensors):
    """Forward-mode differentiation does not pass through the kernels: a dual
    tensor's tangent would be dropped without a word."""
    import torch
    forward_ad = torch.autograd.forward_ad
    if forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError("the operator has no forward-mode derivative (a dual tensor was given)")


def _rows(t):
    """(t, row stride) of a matrix whose rows the kernels can read where they
    are (16-byte aligned, elements adjacent), else of a copy laid out so."""
    import torch
    rows, cols = t.shape
    if t.data_ptr() % 16 == 0:
        if cols % 8 == 0 and t.is_contiguous():
            return t, cols
        if cols <= 1 or t.stride(1) == 1:
            if rows <= 1:
                return t, -(-cols // 8) * 8
            if t.stride(0) >= cols and t.stride(0) % 8 == 0:
                return t, t.stride(0)
    pad = -(-cols // 8) * 8
    copy = torch.empty((rows, pad), dtype=t.dtype, device=t.device)
    copy[:, :cols].copy_(t)
    return copy, pad


class _On:
    """Work on ``device`` and ``stream`` (None: the device's current stream),
    with allocations that belong to it; gives the raw stream. ``used``: tensors
    that the work reads or writes and that their owner may free before it ran."""
    __slots__ = ("device", "stream", "used", "stack")

    def __init__(self, device, stream=None, used=()):
        self.device, self.stream, self.used, self.stack = device, stream, used, None

    def __enter__(self):
        import torch
        if self.stream is None and torch.cuda.current_device() == self.device.index:
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        if isinstance(self.stream, int):   # a raw handle, as the C calls take
            self.stream = torch.cuda.ExternalStream(self.stream, device=self.device)
        if self.stream is not None and self.stream.device != self.device:
            raise ValueError(f"the stream is of {self.stream.device}, the tensors are on {self.device}")
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(self.device))
        current = torch.cuda.current_stream(self.device)
        if self.stream is None or self.stream == current:
            return current.cuda_stream
        self.stack.enter_context(torch.cuda.stream(self.stream))
        for t in self.used:
            if hasattr(t, "record_stream"):   # a status word or an output may be None, or a plain address
                t.record_stream(self.stream)
        return self.stream.cuda_stream

    def __exit__(self, *error):
        if self.stack is not None:
            return self.stack.__exit__(*error)


def _contiguous_on(x, stream):
    """x with adjacent elements; a copy is made, and belongs, where it is read: on ``stream``."""
    if x.is_contiguous():
        return x
    with _On(x.device, stream, (x,)):
        return x.contiguous()


def _workspace(nbytes, device):
    import torch
    # at least one element, so that the pointer is a real one
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _gated_problem(x2, w_gate, w_up, act):
    """The C problem of a gated block, and what it points to."""
    M, K = x2.shape
    x2, ld_x = _rows(x2)
    w_gate, ld_gate = _rows(w_gate)
    w_up, ld_up = _rows(w_up)
    g = lwc.lwc_gated(_elem_of(x2.dtype), ACTIVATIONS[act], M, w_gate.shape[0], K, ld_x, ld_gate, ld_up, x2.data_ptr(),
                      w_gate.data_ptr(), w_up.data_ptr())
    return g, (x2, w_gate, w_up)


def _check_gated(x, w_gate, w_up, act):
    _act_id(act)
    _refuse_tangents(x, w_gate, w_up)
    _check_matrices(x, w_gate=w_gate)
    if w_up.shape != w_gate.shape:
        raise ValueError(f"w_gate and w_up differ in shape: {tuple(w_gate.shape)}, {tuple(w_up.shape)}")
    if w_up.dtype != x.dtype or w_up.device != x.device:
        raise ValueError(f"w_up must have x's type and device ({x.dtype}, {x.device})")


def _gated_forward(x, w_gate, w_up, act, out, stream, status):
    N = w_gate.shape[0]
    with _On(x.device, stream, (x, w_gate, w_up, out, status)) as s:
        if out is None:
            out = x.new_empty((*x.shape[:-1], N))
        g, keep = _gated_problem(x if x.dim() == 2 else x.reshape(-1, x.shape[-1]), w_gate, w_up, act)
        lwc.lwc_gated_forward(g, out, N, status, s)
    return out


def _gated_backward(dh, x, w_gate, w_up, act, need, stream, status):
    N = w_gate.shape[0]
    with _On(x.device, stream, (dh, x, w_gate, w_up, status)) as s:
        g, keep = _gated_problem(x if x.dim() == 2 else x.reshape(-1, x.shape[-1]), w_gate, w_up, act)
        dh2 = dh if dh.dim() == 2 else dh.reshape(-1, N)
        if not dh2.is_contiguous() and (N > 1 and dh2.stride(1) != 1 or dh2.shape[0] > 1 and dh2.stride(0) < N):
            dh2 = dh2.contiguous()
        dx = x.new_empty(x.shape) if need[0] else None
        dw_gate = w_gate.new_empty(w_gate.shape) if need[1] else None
        dw_up = w_up.new_empty(w_up.shape) if need[2] else None
        work = _workspace(lwc.lwc_gated_backward_workspace_bytes(g, *need), x.device)
        lwc.lwc_gated_backward(g, dh2, max(dh2.stride(0), N), dx, dw_gate, dw_up, work, work.numel(), status, s)
    return dx, dw_gate, dw_up


def gated_ffn_backward(dh, x, w_gate, w_up, act: str = "silu", need=(True, True, True), stream=None, status=None):
    """(dx, dw_gate, dw_up) of ``gated_ffn`` from dh, the gradient of its
    result; ``need`` says which are computed (None for the others). Both
    projections are computed again from x. Makes plain calls on one stream, so
    it can be captured into a CUDA graph."""
    _refuse_tangents(dh)
    _check_gated(x, w_gate, w_up, act)
    if tuple(dh.shape) != (*x.shape[:-1], w_gate.shape[0]) or dh.dtype != x.dtype or dh.device != x.device:
        raise ValueError(f"dh must be {(*x.shape[:-1], w_gate.shape[0])}, of x's type and device")
    return _gated_backward(dh, x, w_gate, w_up, act, need, stream, status)


def gated_ffn(x, w_gate, w_up, act: str = "silu", out=None, stream=None, status=None):
    """h = act(x w_gate^T) * (x w_up^T), the gated half of a feed-forward
    block, in one kernel on the tensor cores.

    x: ... x K, w_gate and w_up: N x K, all BF16 or all FP16 on one GPU (rows
    may be strided); returns ... x N of the same type (``out``: a contiguous
    tensor to fill). act: one of ACTIVATIONS. Sums, activation and product are
    FP32, rounded once. ``stream``: where it runs (the current one if None;
    the caller orders it after what makes the inputs). ``status``: optional
    device status word.

    Differentiable for x, w_gate and w_up (once, in reverse mode); the two
    projections are not kept but computed again in the backward pass, so the
    matrices must still hold the same values there. Matrices decoded into a
    reused buffer do not: use ``ResidentModel.gated``, which decodes them again.
    To capture a backward pass into a CUDA graph, capture ``gated_ffn_backward``:
    autograd's own joins the streams of other graphs of the same leaves that are
    still alive, which a capture forbids."""
    import torch
    _check_gated(x, w_gate, w_up, act)
    if (x.requires_grad or w_gate.requires_grad or w_up.requires_grad) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot be given where gradients are needed")
        with _On(x.device, stream, (x, w_gate, w_up, status)):
            return _functions()["gated"].apply(x, w_gate, w_up, act, status)
    if out is not None:
        _check_out(out, (*x.shape[:-1], w_gate.shape[0]), x)
    return _gated_forward(x, w_gate, w_up, act, out, stream, status)


def _check_out(out, shape, x):
    if tuple(out.shape) != tuple(shape) or out.dtype != x.dtype or out.device != x.device or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {tuple(shape)} tensor of x's type and device")


REDUCTIONS = ("none", "sum", "mean")


def _xent_problem(x2, head, t1, ignore_index):
    """The C problem of a loss, and what it points to."""
    (M, K), V = x2.shape, head.shape[0]
    x2, ld_x = _rows(x2)
    head, ld_head = _rows(head)
    p = lwc.lwc_xent(_elem_of(x2.dtype), 0, M, V, K, ld_x, ld_head, x2.data_ptr(), head.data_ptr(), t1.data_ptr(),
                     ignore_index)
    return p, (x2, head, t1)


def _flat_targets(targets):
    import torch
    if targets.dtype == torch.int64 and targets.is_contiguous():
        return targets   # read as one row of words, whatever its shape
    return targets.reshape(-1).to(torch.int64).contiguous()


def _xent_forward(x, head, targets, ignore_index, reduction, stream, status):
    """(the loss, reduced or per token, the losses per token and the lse per token)."""
    import torch
    with _On(x.device, stream, (x, head, targets, status)) as s:
        p, keep = _xent_problem(x if x.dim() == 2 else x.reshape(-1, x.shape[-1]), head, _flat_targets(targets),
                                ignore_index)
        loss = torch.empty(targets.shape, dtype=torch.float32, device=x.device)
        lse = torch.empty(targets.shape, dtype=torch.float32, device=x.device)
        total = torch.empty((), dtype=torch.float32, device=x.device) if reduction != "none" else None
        work = _workspace(lwc.lwc_xent_forward_workspace_bytes(p), x.device)
        lwc.lwc_xent_forward(p, loss, lse, total if reduction == "sum" else None, total if reduction == "mean" else None,
                             work, work.numel(), status, s)
    return loss if reduction == "none" else total, loss, lse


def _xent_backward(grad, lse, loss, x, w_head, targets, ignore_index, reduction, need, stream, status):
    with _On(x.device, stream, (grad, lse, loss, x, w_head, targets, status)) as s:
        p, keep = _xent_problem(x if x.dim() == 2 else x.reshape(-1, x.shape[-1]), w_head, _flat_targets(targets),
                                ignore_index)
        grad, lse = grad.contiguous(), lse.contiguous()
        dx = x.new_empty(x.shape) if need[0] else None
        dw = w_head.new_empty(w_head.shape) if need[1] else None
        work = _workspace(lwc.lwc_xent_backward_workspace_bytes(p, *need), x.device)
        rest = (grad, 1 if reduction == "none" else 0, reduction == "mean", dx, dw, work, work.numel(), status, s)
        if loss is None:
            lwc.lwc_xent_backward(p, lse, *rest)
        else:
            lwc.lwc_xent_backward_losses(p, lse, loss.contiguous(), *rest)
    return dx, dw


def linear_cross_entropy_backward(grad, lse, x, w_head, targets, ignore_index: int = -100, reduction: str = "mean",
                                  need=(True, True), stream=None, status=None, loss=None):
    """(dx, dw_head) of ``linear_cross_entropy`` from the gradient of its
    result and the lse that it returned; ``need`` says which are computed
    (None for the other). ``loss``: the losses per token (reduction "none"
    returns them), if there are; the result is the same without them, but
    they are computed again, which costs a forward pass. Makes plain calls on
    one stream, so it can be captured into a CUDA graph."""
    import torch
    _refuse_tangents(grad)
    _check_xent(x, w_head, targets, reduction)
    rows = x.shape[:-1] if reduction == "none" else ()
    if tuple(grad.shape) != tuple(rows) or grad.dtype != torch.float32 or grad.device != x.device:
        raise ValueError(f"grad must be a {tuple(rows)} FP32 tensor on {x.device}")
    if tuple(lse.shape) != tuple(x.shape[:-1]) or lse.dtype != torch.float32 or lse.device != x.device:
        raise ValueError(f"lse must be a {tuple(x.shape[:-1])} FP32 tensor on {x.device}")
    if loss is not None and (loss.shape != lse.shape or loss.dtype != torch.float32 or loss.device != x.device):
        raise ValueError(f"loss must be a {tuple(x.shape[:-1])} FP32 tensor on {x.device}")
    return _xent_backward(grad, lse, loss, x, w_head, targets, ignore_index, reduction, need, stream, status)


def _check_xent(x, w_head, targets, reduction):
    _refuse_tangents(x, w_head)
    _check_matrices(x, w_head=w_head)
    _check_targets(x, targets, reduction)


def _check_targets(x, targets, reduction):
    import torch
    if reduction not in REDUCTIONS:
        raise ValueError(f"unknown reduction {reduction!r}")
    if targets.shape != x.shape[:-1] or targets.device != x.device or \
            targets.dtype not in (torch.int64, torch.int32):
        raise ValueError(f"targets must be a {tuple(x.shape[:-1])} tensor of int64 or int32 on {x.device}")


def linear_cross_entropy(x, w_head, targets, ignore_index: int = -100, reduction: str = "mean",
                         return_lse: bool = False, stream=None, status=None):
    """Softmax cross entropy of the logits x w_head^T against ``targets``,
    without ever keeping the logits.

    x: ... x K hidden states, w_head: V x K (BF16 or FP16, rows may be
    strided), targets: ... int64 or int32 word indices. Tokens whose target is
    ``ignore_index`` have loss 0 and pass no gradient, whatever their hidden
    state holds; any other target outside 0 .. V - 1 gives loss NaN, passes no
    gradient and sets LWC_DEVICE_BAD_TARGET in ``status``. Returns FP32: one
    loss per token (reduction "none"), their "sum", or the "mean" over the
    tokens not ignored (0 if there is none); with ``return_lse`` also the log
    of each token's sum of exponentials (not differentiable).

    Differentiable for x and w_head (once, in reverse mode); the backward pass
    computes the logits again, a piece of the vocabulary at a time, so w_head
    must still hold the same values there (``ResidentModel.cross_entropy``
    decodes it again). To capture a backward pass into a CUDA graph, capture
    ``linear_cross_entropy_backward`` (see ``gated_ffn``)."""
    import torch
    _check_xent(x, w_head, targets, reduction)
    if (x.requires_grad or w_head.requires_grad) and torch.is_grad_enabled():
        with _On(x.device, stream, (x, w_head, targets, status)):
            loss, lse = _functions()["xent"].apply(x, w_head, targets, ignore_index, reduction, status)
    else:
        loss, _, lse = _xent_forward(x, w_head, targets, ignore_index, reduction, stream, status)
    return (loss, lse) if return_lse else loss


_FUNCTIONS = {}


def _functions():
    """The autograd functions (made on first use: this module imports torch late)."""
    if _FUNCTIONS:
        return _FUNCTIONS
    import torch

    def once():
        # the backward of a backward would need the kernels' own derivatives
        if torch.is_grad_enabled():
            raise RuntimeError("gated_ffn and linear_cross_entropy are differentiable once (create_graph=True given)")

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w_gate, w_up, act, status):
            ctx.save_for_backward(x, w_gate, w_up)
            ctx.act, ctx.status = act, status
            return _gated_forward(x, w_gate, w_up, act, None, None, status)

        @staticmethod
        def backward(ctx, dh):
            once()
            dx, dw_gate, dw_up = _gated_backward(dh, *ctx.saved_tensors, ctx.act, ctx.needs_input_grad[:3], None,
                                                 ctx.status)
            return dx, dw_gate, dw_up, None, None

    class Xent(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w_head, targets, ignore_index, reduction, status):
            result, loss, lse = _xent_forward(x, w_head, targets, ignore_index, reduction, None, status)
            if reduction == "none":
                result = loss.clone()   # which the caller may change in place
            ctx.save_for_backward(x, w_head, targets, lse, loss)
            ctx.ignore_index, ctx.reduction, ctx.status = ignore_index, reduction, status
            ctx.mark_non_differentiable(lse)
            return result, lse

        @staticmethod
        def backward(ctx, grad, _):
            once()
            x, w_head, targets, lse, loss = ctx.saved_tensors
            dx, dw = _xent_backward(grad, lse, loss, x, w_head, targets, ctx.ignore_index, ctx.reduction,
                                    ctx.needs_input_grad[:2], None, ctx.status)
            return dx, dw, None, None, None, None

    class ResidentGated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, model, layer, gate, up, act, status, route):
            ctx.save_for_backward(x)
            ctx.args = (model, layer, gate, up, act, status)
            return model._gated(layer, gate, up, x, act, None, None, status, route)

        @staticmethod
        def backward(ctx, dh):
            once()
            model, layer, gate, up, act, status = ctx.args
            (x,) = ctx.saved_tensors
            with _On(x.device) as s:
                w_gate, w_up = model._decoded(layer, (gate, up), s, status)
                dx = _gated_backward(dh, x, w_gate, w_up, act, (True, False, False), None, status)[0]
            return dx, None, None, None, None, None, None, None

    class ResidentXent(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, model, layer, index, targets, ignore_index, reduction, status):
            with _On(x.device) as s:
                (w,) = model._decoded(layer, (index,), s, status)
                _check_xent(x, w, targets, reduction)
                result, loss, lse = _xent_forward(x, w, targets, ignore_index, reduction, None, status)
                if reduction == "none":
                    result = loss.clone()
            ctx.save_for_backward(x, targets, lse, loss)
            ctx.args = (model, layer, index, ignore_index, reduction, status)
            return result

        @staticmethod
        def backward(ctx, grad):
            once()
            model, layer, index, ignore_index, reduction, status = ctx.args
            x, targets, lse, loss = ctx.saved_tensors
            with _On(x.device) as s:
                (w,) = model._decoded(layer, (index,), s, status)
                dx = _xent_backward(grad, lse, loss, x, w, targets, ignore_index, reduction, (True, False), None, status)[0]
            return dx, None, None, None, None, None, None, None

    _FUNCTIONS.update(gated=Gated, xent=Xent, resident_gated=ResidentGated, resident_xent=ResidentXent)
    return _FUNCTIONS


# Chunk size of the blobs TiledWeights makes. A 32-chunk block of 20-byte
# chunks holds about 2,000 exponent codes, so the product can run 20 decoder
# warps with about five 8192-weight tiles in flight (36-byte chunks: 12 warps);
# the price is 0.13 bits per weight of chunk gaps and counts. Measured on a
# Llama-3-8B layer (B200), M = 16 / 128 / 256: 20-byte chunks 0.31 / 0.34 /
# 0.42 ms; 24: 0.31 / 0.34 / 0.50; 28: 0.29 / 0.38 / 0.59; 36: 0.32 / 0.41 / 0.67.
GEMM_CHUNK_BYTES = 20


class TiledWeights:
    """Weight matrices held for the tensor-core product (lwc_gemm_dfloat11 /
    lwc_gemm_codebook): each rows x cols BF16 matrix (rows % 128 == 0, cols %
    64 == 0) is put in tile order on the GPU (lwc_tile_order) and compressed
    there by the device encoder of ``codec``. ``gemm`` then computes y = x W^T
    for 1 to 256 activation rows with W decoded straight into the MMA's
    shared-memory operands (the BF16 matrix is never written to device
    memory). A batched call takes matrices of one codec (codebook: one index
    width)."""

    def __init__(self, device, codec: str = "dfloat11"):
        if codec not in CODECS:
            raise ValueError(f"unknown codec {codec!r}")
        self.device = device
        self.codec = codec
        self.descs, self.blobs, self.shapes = [], [], []

    def add(self, w, workspace=None, stream=None, chunk_bytes: int = GEMM_CHUNK_BYTES) -> int:
        """Tile-order and compress one rows x cols BF16 CUDA tensor; returns its index.
        chunk_bytes: DFloat11 chunk size of the blob (see GEMM_CHUNK_BYTES)."""
        import torch
        if w.dim() != 2 or w.element_size() != 2 or not w.is_cuda:
            raise ValueError("expected a rows x cols 16-bit CUDA tensor")
        rows, cols = int(w.shape[0]), int(w.shape[1])
        stream = stream if stream is not None else torch.cuda.current_stream(w.device)
        src = w.contiguous()
        tiled = torch.empty_like(src)
        lwc.lwc_tile_order(src, rows, cols, tiled, stream)
        with torch.cuda.stream(stream):
            params = {"chunk_bytes": chunk_bytes} if self.codec == "dfloat11" else {}
            d, b = encode_on_device(tiled, self.codec, workspace=workspace, stream=stream, **params)
        del tiled
        self.descs.append(d)
        self.blobs.append(b)
        self.shapes.append((rows, cols))
        return len(self.descs) - 1

    @property
    def compressed_bytes(self) -> int:
        return sum(int(d.total_bytes) for d in self.descs)

    def _check_x(self, index: int, x):
        import torch
        rows, cols = self.shapes[index]
        if x.dim() != 2 or x.shape[1] != cols or x.dtype != torch.bfloat16:
            raise ValueError(f"x must be M x {cols} BF16")
        return rows, cols

    def gemm(self, index: int, x, out=None, stream=None, status=None):
        """y = x W^T for matrix ``index``; x: M x cols BF16 (M <= 256). Returns
        ``out`` (M x rows FP32, allocated if None)."""
        import torch
        rows, cols = self._check_x(index, x)
        x = _contiguous_on(x, stream)
        M = int(x.shape[0])
        if out is None:
            out = torch.empty((M, rows), dtype=torch.float32, device=x.device)
        fn = lwc.lwc_gemm_dfloat11 if self.codec == "dfloat11" else lwc.lwc_gemm_codebook
        fn(self.descs[index], self.blobs[index], cols, x, M, out, d_status=status, stream=stream)
        return out

    def gemm_batched(self, indices, xs, outs=None, stream=None, status=None):
        """Several matrices (at most 8), one launch; all x share M."""
        import torch
        pairs = list(zip(indices, xs))
        for i, x in pairs:
            self._check_x(i, x)
        xs = [_contiguous_on(x, stream) for _, x in pairs]
        M = int(xs[0].shape[0])
        if any(int(x.shape[0]) != M for x in xs):
            raise ValueError("all activations of a batched call share M")
        if outs is None:
            outs = [torch.empty((M, self.shapes[i][0]), dtype=torch.float32, device=xs[0].device) for i in indices]
        batch = lwc.LinearBatch([self.descs[i] for i in indices], [self.blobs[i] for i in indices],
                                [self.shapes[i][1] for i in indices], xs, outs, M)
        fn = lwc.lwc_gemm_dfloat11_batched if self.codec == "dfloat11" else lwc.lwc_gemm_codebook_batched
        fn(batch, d_status=status, stream=stream)
        return outs

    def _one_launch(self, a: int, b: int) -> bool:
        """Whether two matrices of one shape fit a batched call: one index width (codebook; two matrices' distinct
        values may lie on either side of a power of two) or chunk size (DFloat11), at most 4096 units of 128 rows."""
        alike = "k" if self.codec == "codebook" else "chunk_bytes"
        return getattr(self.descs[a], alike) == getattr(self.descs[b], alike) and \
            2 * self.shapes[a][0] <= 128 * 4096

    def gated(self, gate: int, up: int, x, act: str = "silu", out=None, stream=None, status=None):
        """h = act(x W_gate^T) * (x W_up^T) for two matrices of one shape, held
        in tile order: both products in one launch where it takes them together
        (x: M x cols BF16, M <= 256), then the activation and the product.
        Returns ``out`` (M x rows BF16, allocated if None). Not differentiable
        (``ResidentModel.gated`` is): an x that asks for a gradient is refused."""
        import torch
        act_id = _act_id(act)
        _refuse_tangents(x)
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError("no gradient passes through TiledWeights.gated (give x.detach(), or use ResidentModel.gated)")
        if self.shapes[gate] != self.shapes[up]:
            raise ValueError(f"matrices differ in shape: {self.shapes[gate]}, {self.shapes[up]}")
        rows, _ = self._check_x(gate, x)
        if any(x.device != self.blobs[i].device for i in (gate, up)):
            raise ValueError("x must be on the matrices' device")
        M = int(x.shape[0])
        if out is not None:
            _check_out(out, (M, rows), x)
        with _On(x.device, stream, (x, out, status)) as s:
            # laid out on the stream that reads it
            x = x.contiguous()
            if x.data_ptr() % 16:
                x = x.clone()
            if out is None:
                out = torch.empty((M, rows), dtype=torch.bfloat16, device=x.device)
            ab = torch.empty((2, M, rows), dtype=torch.float32, device=x.device)
            if self._one_launch(gate, up):
                self.gemm_batched([gate, up], [x, x], [ab[0], ab[1]], stream=s, status=status)
            else:
                for index, y in zip((gate, up), ab):
                    self.gemm(index, x, y, stream=s, status=status)
            lwc.lwc_gated_product(lwc.LWC_ELEM_BF16, act_id, ab[0], ab[1], M * rows, out, s)
        return out


def _can_fuse(codec: str, descs) -> bool:
    """Whether the decode-fused linear layer takes these blobs: every codebook
    blob, and DFloat11 blobs of BF16 elements in blocks of 32 chunks or with a
    single exponent (see lwc_linear_dfloat11)."""
    return codec == "codebook" or all(
        d.elem == lwc.LWC_ELEM_BF16 and (d.threads_per_block == 32 or d.flags & lwc.LWC_FLAG_SINGLE_EXPONENT)
        for d in descs)


def _gated_fused_rows(codec: str, cols: int) -> int:
    """Rows up to which ``ResidentModel.gated`` multiplies in the decode-fused
    linear layers rather than decoding both matrices for the dense kernel. us
    fused / decoded (B200), two matrices of 14336 x 4096: codebook 79 / 132 (1
    row), 109 / 145 (4), 131 / 145 (5), 158 / 145 (8), of 28672 x 8192: 398 / 511
    (4), 767 / 511 (5, where x no longer fits beside the tables); DFloat11 121 /
    131 (1), 148 / 146 (2)."""
    if codec == "dfloat11":
        return 1
    return max(1, min(6, 32768 // cols))


class ResidentModel:
    """Compressed layers in device memory plus reusable BF16 output buffers.

    Usage: ``add_layer`` for every layer (uploads its blobs), ``finalize`` to
    allocate the buffers and marshal the launch arguments once, then
    ``decode(layer, slot, stream)`` per layer; ``views(layer, slot)`` gives
    the decoded matrices (BF16 views into buffer ``slot``).
    """

    def __init__(self, codec: str, device, slots: int = 2):
        import torch
        if codec not in CODECS:
            raise ValueError(f"unknown codec {codec!r}")
        if slots < 2:
            # pipelined() decodes layer L + 1 while layer L is still in use:
            # that needs a second buffer
            raise ValueError(f"ResidentModel needs at least 2 output buffers (got slots={slots})")
        self.codec = codec
        self.device = torch.device(device)
        self.slots = slots
        self.layers: list[dict] = []
        self.buffers = []
        self._batches: list[list] = []

    def add_layer(self, name: str, encoded, shapes) -> None:
        """encoded: [(desc, host blob)] of the layer's matrices, shapes their shapes."""
        import torch
        descs = [d for d, _ in encoded]
        blobs = [torch.from_numpy(b).to(self.device) for _, b in encoded]
        self.layers.append(dict(name=name, descs=descs, blobs=blobs, shapes=[tuple(s) for s in shapes],
                                n=[d.n for d in descs]))

    def add_layer_from_device(self, name: str, tensors, workspace=None, **params) -> None:
        """Compress BF16 tensors that are already on this model's GPU (the
        device encoder) and keep only their blobs."""
        import torch
        encoded = []
        for t in tensors:
            need = lwc.lwc_encode_device_workspace_bytes(t.numel())
            if workspace is None or workspace.numel() < need:
                workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            encoded.append(encode_on_device(t, self.codec, workspace, **params))
        self.layers.append(dict(name=name, descs=[d for d, _ in encoded], blobs=[b for _, b in encoded],
                                shapes=[tuple(t.shape) for t in tensors], n=[d.n for d, _ in encoded]))

    @property
    def compressed_bytes(self) -> int:
        return sum(int(b.numel()) for layer in self.layers for b in layer["blobs"])

    @property
    def weights(self) -> int:
        return sum(sum(layer["n"]) for layer in self.layers)

    def finalize(self) -> None:
        import torch
        biggest = max(sum(layer["n"]) for layer in self.layers)
        # 8 extra elements per matrix keep every view 16-byte aligned
        biggest += 8 * max(len(layer["n"]) for layer in self.layers)
        self.buffers = [torch.empty(biggest, dtype=torch.bfloat16, device=self.device) for _ in range(self.slots)]
        self._batches = []
        for layer in self.layers:
            per_slot = []
            for s in range(self.slots):
                views = self._views(layer, s)
                per_slot.append((lwc.Batch(layer["descs"], layer["blobs"], views), views))
            self._batches.append(per_slot)

    def _views(self, layer, slot):
        out, off = [], 0
        for n, shape in zip(layer["n"], layer["shapes"]):
            out.append(self.buffers[slot][off:off + n].view(shape))
            off += (n + 7) // 8 * 8
        return out

    def views(self, layer: int, slot: int):
        return self._batches[layer][slot][1]

    def decode(self, layer: int, slot: int, stream=None, status=None) -> None:
        batch = self._batches[layer][slot][0]
        if self.codec == "dfloat11":
            lwc.lwc_decode_dfloat11_batched(batch, d_status=status, stream=stream)
        else:
            lwc.lwc_decode_codebook_batched(batch, d_status=status, stream=stream)

    def linear(self, layer: int, index: int, x, out=None, stream=None, status=None, route: str = "auto"):
        """y = x W^T for matrix ``index`` of ``layer``, by default without
        decoding it to memory: the weights are decoded in registers by the
        fused kernel (lwc_linear_dfloat11 / lwc_linear_codebook); see
        fused_linear for ``route``. x: M x cols BF16 on this model's GPU,
        1 <= M <= 8 (token generation); returns (or fills ``out``) the M x rows
        FP32 result."""
        return fused_linear(self.layers[layer]["descs"][index], self.layers[layer]["blobs"][index],
                            self.layers[layer]["shapes"][index], x, self.codec, out=out, stream=stream,
                            status=status, route=route)

    def _matrices(self, layer: int, indices: tuple):
        """Launch arguments of some matrices of ``layer``, their types, and
        whether the decode-fused linear layer takes them: (Batch, LinearBatch,
        shapes, dtypes, fusable). Kept with the layer, and made again once its
        blobs, descriptors or shapes are other ones (the arguments hold bare
        addresses)."""
        import torch
        data = self.layers[layer]
        descs, blobs = [data["descs"][i] for i in indices], [data["blobs"][i] for i in indices]
        of = (*descs, *blobs, *[data["shapes"][i] for i in indices])
        kept = data.setdefault("marshalled", {})
        if indices not in kept or any(a is not b for a, b in zip(kept[indices][0], of)):
            shapes = [tuple(int(v) for v in data["shapes"][i]) for i in indices]
            if any(len(s) != 2 for s in shapes):
                raise ValueError("the weight must be a rows x cols matrix")
            elems = [d.elem if self.codec == "dfloat11" else lwc.LWC_ELEM_BF16 for d in descs]
            if lwc.LWC_ELEM_FP32 in elems:
                raise ValueError("the matrix holds FP32 elements (BF16 and FP16 are taken)")
            none = [None] * len(indices)
            kept[indices] = of, (
                lwc.Batch(descs, blobs, none), lwc.LinearBatch(descs, blobs, [s[1] for s in shapes], none, none, 0),
                shapes, [torch.float16 if e == lwc.LWC_ELEM_FP16 else torch.bfloat16 for e in elems],
                _can_fuse(self.codec, descs))
        return kept[indices][1]

    def _decoded(self, layer: int, indices: tuple, stream, status=None):
        """The matrices ``indices`` of ``layer``, decoded into new buffers."""
        import torch
        batch, _, shapes, dtypes, _ = self._matrices(layer, indices)
        views = [torch.empty(s, dtype=t, device=self.device) for s, t in zip(shapes, dtypes)]
        fn = lwc.lwc_decode_dfloat11_batched if self.codec == "dfloat11" else lwc.lwc_decode_codebook_batched
        fn(batch.into(views), d_status=status, stream=stream)
        return views

    def _gated(self, layer, gate, up, x, act, out, stream, status, route):
        import torch
        _, linear, ((rows, cols), _), _, fusable = self._matrices(layer, (gate, up))
        M = x.numel() // cols
        if route == "auto":
            few = x.dtype == torch.bfloat16 and 1 <= M <= _gated_fused_rows(self.codec, cols)
            route = "fused" if few and fusable else "decode"
        with _On(x.device, stream, (x, out, status)) as s:
            if route == "decode":
                w_gate, w_up = self._decoded(layer, (gate, up), s, status)
                _check_matrices(x, w_gate=w_gate, w_up=w_up)
                return _gated_forward(x, w_gate, w_up, act, out, None, status)
            if x.dtype != torch.bfloat16:
                raise ValueError("the fused route takes BF16 activations")
            x2 = x.reshape(M, cols).contiguous()
            if x2.data_ptr() % 16:
                x2 = x2.clone()
            if out is None:
                out = torch.empty((*x.shape[:-1], rows), dtype=x.dtype, device=x.device)
            ab = torch.empty((2, M, rows), dtype=torch.float32, device=x.device)
            fn = lwc.lwc_linear_dfloat11_batched if self.codec == "dfloat11" else lwc.lwc_linear_codebook_batched
            fn(linear.of((x2, x2), (ab[0], ab[1]), M), d_status=status, stream=s)
            lwc.lwc_gated_product(lwc.LWC_ELEM_BF16, ACTIVATIONS[act], ab[0], ab[1], M * rows, out, s)
        return out

    def gated(self, layer: int, gate: int, up: int, x, act: str = "silu", out=None, stream=None, status=None,
              route: str = "auto"):
        """h = act(x W_gate^T) * (x W_up^T) for two matrices of ``layer`` (one
        shape, rows x cols), which stay compressed; x: ... x cols, returns (or
        fills ``out``) ... x rows of x's type.

        route "fused": both products by the decode-fused linear layer (1 to 8
        rows, BF16), then the activation and the product; "decode": both
        matrices decoded into a temporary buffer, then ``gated_ffn``'s kernel;
        "auto": the faster of the two by codec, rows and columns (the decode
        route for blobs that the fused layer does not take). The fused DFloat11
        layer adds parts of a row atomically, so the last bits of its products
        may vary from run to run; every other route repeats bit for bit.
        Differentiable for x: the backward pass decodes the matrices again
        instead of keeping them."""
        import torch
        if route not in ("auto", "fused", "decode"):
            raise ValueError(f"unknown route {route!r}")
        _act_id(act)
        _refuse_tangents(x)
        (rows, cols), other = self._matrices(layer, (gate, up))[2]
        if (rows, cols) != other:
            raise ValueError(f"expected two matrices of one shape, got {(rows, cols)}, {other}")
        _elem_of(x.dtype)
        if x.dim() < 1 or x.shape[-1] != cols or x.device != self.layers[layer]["blobs"][gate].device:
            raise ValueError(f"x must be a tensor of ... x {cols} on the matrices' device")
        if torch.is_grad_enabled() and x.requires_grad:
            if out is not None:
                raise ValueError("out cannot be given where gradients are needed")
            with _On(x.device, stream, (x, status)):
                return _functions()["resident_gated"].apply(x, self, layer, gate, up, act, status, route)
        if out is not None:
            _check_out(out, (*x.shape[:-1], rows), x)
        return self._gated(layer, gate, up, x, act, out, stream, status, route)

    def cross_entropy(self, layer: int, index: int, x, targets, ignore_index: int = -100, reduction: str = "mean",
                      stream=None, status=None):
        """``linear_cross_entropy`` against matrix ``index`` of ``layer`` (the
        output matrix, vocab x cols), which stays compressed: it is decoded
        into a temporary buffer for the call. Differentiable for x: the
        backward pass decodes it again."""
        import torch
        if x.device != self.layers[layer]["blobs"][index].device:
            raise ValueError("x must be on the matrix's device")
        _check_targets(x, targets, reduction)
        _refuse_tangents(x)
        if x.requires_grad and torch.is_grad_enabled():
            with _On(x.device, stream, (x, targets, status)):
                return _functions()["resident_xent"].apply(x, self, layer, index, targets, ignore_index, reduction,
                                                           status)
        with _On(x.device, stream, (x, targets, status)) as s:
            (w,) = self._decoded(layer, (index,), s, status)
            return linear_cross_entropy(x, w, targets, ignore_index, reduction, status=status)

    def pipelined(self, compute_stream, decode_stream=None):
        """Iterate over the layers with decoding one layer ahead of use.

        Yields ``(layer, views)``; the views are ready for work enqueued on
        ``compute_stream``, and layer + 1 is already being decoded on
        ``decode_stream`` meanwhile (a side stream if None). Enqueue all work
        that reads the yielded views on ``compute_stream`` before advancing
        the generator: a buffer is reused only after an event recorded on
        ``compute_stream`` at that point says its consumer has finished.
        """
        import torch
        ds = decode_stream or torch.cuda.Stream(self.device)
        ready = [torch.cuda.Event() for _ in range(self.slots)]
        free = [torch.cuda.Event() for _ in range(self.slots)]
        used = [False] * self.slots
        ds.wait_stream(compute_stream)   # inputs written before the call are visible
        self.decode(0, 0, ds)
        ready[0].record(ds)
        for i in range(len(self.layers)):
            slot = i % self.slots
            nxt = i + 1
            if nxt < len(self.layers):
                ns = nxt % self.slots
                if used[ns]:
                    ds.wait_event(free[ns])
                self.decode(nxt, ns, ds)
                ready[ns].record(ds)
            compute_stream.wait_event(ready[slot])
            yield i, self.views(i, slot)
            free[slot].record(compute_stream)
            used[slot] = True


class HostPipeline:
    """Compressed tensors held in (pinned) host memory, decoded through the GPU
    back into host memory, with the transfers overlapped: tensor i's upload,
    tensor i-1's decode and tensor i-2's read-back run on three streams, so
    both PCIe directions are busy at once (smallest tensors first, so the
    read-back starts early).

    ``run()`` enqueues one pass on ``stream`` (and two helper streams) and
    returns; work after it on ``stream`` sees the host output complete once
    the stream is synchronised.
    """

    def __init__(self, descs, host_blobs, codec: str, device, host_out=None):
        import torch
        if codec not in CODECS:
            raise ValueError(f"unknown codec {codec!r}")
        self.codec = codec
        self.device = torch.device(device)
        self.descs = list(descs)
        self.pinned_in = [b if isinstance(b, torch.Tensor) and b.is_pinned() else
                          torch.as_tensor(b).pin_memory() for b in host_blobs]
        self.blobs = [torch.empty(b.numel(), dtype=torch.uint8, device=self.device) for b in self.pinned_in]
        ns = [d.n for d in self.descs]
        self.offsets = []            # element offsets, multiples of 8 (16-byte aligned views)
        off = 0
        for n in ns:
            self.offsets.append(off)
            off += (n + 7) // 8 * 8
        self.out = torch.empty(off, dtype=torch.bfloat16, device=self.device)
        self.host_out = host_out if host_out is not None else torch.empty(off, dtype=torch.bfloat16).pin_memory()
        self.views = [self.out[o:o + n] for o, n in zip(self.offsets, ns)]
        self.order = sorted(range(len(ns)), key=lambda i: ns[i])
        self.s_in = torch.cuda.Stream(self.device)
        self.s_out = torch.cuda.Stream(self.device)

    @property
    def h2d_bytes(self) -> int:
        return sum(int(b.numel()) for b in self.pinned_in)

    @property
    def d2h_bytes(self) -> int:
        return 2 * sum(d.n for d in self.descs)

    def run(self, stream) -> None:
        import torch
        decode = lwc.lwc_decode_dfloat11 if self.codec == "dfloat11" else lwc.lwc_decode_codebook
        self.s_in.wait_stream(stream)        # earlier work on `stream` is done with every buffer
        done_in, done_dec = [], []
        for i in self.order:
            with torch.cuda.stream(self.s_in):
                self.blobs[i].copy_(self.pinned_in[i], non_blocking=True)
            ev = torch.cuda.Event()
            ev.record(self.s_in)
            done_in.append(ev)
        for j, i in enumerate(self.order):
            stream.wait_event(done_in[j])
            decode(self.descs[i], self.blobs[i], self.views[i], stream)
            ev = torch.cuda.Event()
            ev.record(stream)
            done_dec.append(ev)
        for j, i in enumerate(self.order):
            self.s_out.wait_event(done_dec[j])
            o, n = self.offsets[i], self.descs[i].n
            with torch.cuda.stream(self.s_out):
                self.host_out[o:o + n].copy_(self.views[i], non_blocking=True)
        stream.wait_stream(self.s_out)
