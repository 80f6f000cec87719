"""The gated feed-forward block (lwc_gated_forward, lwc_gated_backward,
layers.gated_ffn and the compressed forms) against its formulas in 64 bits.

Every element is held to a bound that is added up from the roundings there
are. With u = 2^-23 the unit roundoff the library states for the tensor
cores' sums, gamma = K u / (1 - K u), S_a = sum |x Wg| and S_b = sum |x Wu|:

    |a' - a| <= e_a = gamma S_a,  |b' - b| <= e_b = gamma S_b
    |act(a') - act(a)| <= 1.2 e_a + F |act(a)|        (|act'| <= 1.2)
    |act'(a') - act'(a)| <= 1.2 e_a + F               (|act''| <= 1.2; relu: 1 where |a| <= e_a)

F = 2^-17 covers the activation's own evaluation in FP32: the fast
exponential is off by 2 + 1.16 |v| units in the last place, and |v| <= 20 on
every input here. A rounding to 16 bits is off by at most half a step H
(2^-8 for BF16, 2^-11 for FP16), or, for the smallest FP16 numbers, by 2^-25.
A second product over n terms adds gamma_n of its sum of magnitudes.
"""
import threading

import numpy as np
import pytest
import torch

import synth
from decode_dfloat11_b200 import build as lwc_build
from decode_dfloat11_b200 import layers, lwc

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
F = 2.0 ** -17
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
TYPES = [torch.bfloat16, torch.float16]
ACTS = list(layers.ACTIVATIONS)


@pytest.fixture(scope="module", autouse=True)
def lib(cuda_device):
    lwc_build.build()
    return lwc.load()


def gamma(n):
    return n * U / (1 - n * U)


def act64(name, a):
    """act(a), act'(a) in 64 bits."""
    if name == "silu":
        p = torch.sigmoid(a)
        return a * p, p * (1 + a * torch.sigmoid(-a))
    if name == "gelu":
        p = torch.special.ndtr(a)
        return a * p, p + a * torch.exp(-a * a / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        # (1 + tanh q) / 2 = sigmoid(2 q): the left side has no digit left, in 64 bits either, below q = -18
        q2 = 2 * np.sqrt(2 / np.pi) * (a + 0.044715 * a ** 3)
        p = torch.sigmoid(q2)
        return a * p, p + a * p * torch.sigmoid(-q2) * 2 * np.sqrt(2 / np.pi) * (1 + 0.134145 * a * a)
    if name == "relu":
        return a.clamp(min=0), (a > 0).double()
    p = torch.sigmoid(a)
    return p, p * torch.sigmoid(-a)


class Exact:
    """Values and bounds of one problem."""

    def __init__(self, act, x, wg, wu, dh=None):
        dt = x.dtype
        half, tiny = HALF[dt], TINY[dt]
        K = x.shape[1]
        x, wg, wu = x.double(), wg.double(), wu.double()
        a, b = x @ wg.T, x @ wu.T
        ea, eb = gamma(K) * (x.abs() @ wg.abs().T), gamma(K) * (x.abs() @ wu.abs().T)
        y, s = act64(act, a)
        ey = 1.2 * ea + F * y.abs()
        es = 1.2 * ea + F + ((a.abs() <= ea).double() if act == "relu" else 0)
        self.h = y * b
        eh = ey * (b.abs() + eb) + y.abs() * eb
        self.h_tol = eh + half * (self.h.abs() + eh) + tiny
        if dh is None:
            return
        dh = dh.double()
        da, db = dh * b * s, dh * y
        eda = dh.abs() * (eb * (s.abs() + es) + b.abs() * es) * (1 + 4 * U)
        eda = eda + half * (da.abs() + eda) + tiny
        edb = dh.abs() * ey * (1 + 4 * U)
        edb = edb + half * (db.abs() + edb) + tiny
        M, N = dh.shape

        def product(terms, n):
            value = sum(p @ q for p, _, q in terms)
            mag = sum((p.abs() + e) @ q.abs() for p, e, q in terms)
            err = sum(e @ q.abs() for _, e, q in terms) + gamma(n) * mag
            return value, err + half * (value.abs() + err) + tiny

        self.dx, self.dx_tol = product([(da, eda, wg), (db, edb, wu)], 2 * N)
        self.dwg, self.dwg_tol = product([(da.T, eda.T, x)], M)
        self.dwu, self.dwu_tol = product([(db.T, edb.T, x)], M)


def close(got, want, tol):
    assert got.shape == want.shape
    off = (got.double() - want).abs() - tol
    assert bool((off <= 0).all()), (float(off.max()), int(off.argmax()))


def inputs(M, N, K, dtype, seed=0):
    g = torch.Generator("cuda").manual_seed(1000 * seed + M + 7 * N + 13 * K)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    wg, wu = (torch.randn(N, K, generator=g, device="cuda").mul_(K ** -0.5).to(dtype) for _ in range(2))
    dh = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    return x, wg, wu, dh


SIZES = [(1, 1, 1), (1, 8, 64), (1, 1000, 512), (1, 10_000, 136), (2, 300, 4100), (3, 13, 17), (4, 37, 1000), (5, 37, 1000),
         (4, 9000, 2048), (7, 129, 72), (64, 96, 200), (127, 128, 64),
         (128, 257, 136), (129, 64, 1024), (200, 333, 65), (300, 2048, 320), (513, 1001, 96), (1100, 640, 264)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(M, N, K, dtype):
    x, wg, wu, _ = inputs(M, N, K, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for act in ACTS:
        e = Exact(act, x, wg, wu)
        close(layers.gated_ffn(x, wg, wu, act=act, status=status), e.h, e.h_tol)
    assert int(status) == 0


@pytest.mark.parametrize("M,N,K", [(2560, 1500, 2048), (5000, 2600, 328), (37, 200, 4104)])
def test_gradients_with_an_incomplete_last_wave(M, N, K):
    """More tiles than fit at once, or far fewer, and long contractions: the
    last wave's tiles are split and joined."""
    x, wg, wu, dh = inputs(M, N, K, torch.bfloat16, seed=2)
    e = Exact("silu", x, wg, wu, dh)
    dx, dwg, dwu = layers.gated_ffn_backward(dh, x, wg, wu)
    close(dx, e.dx, e.dx_tol)
    close(dwg, e.dwg, e.dwg_tol)
    close(dwu, e.dwu, e.dwu_tol)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gradients(M, N, K, dtype):
    x, wg, wu, dh = inputs(M, N, K, dtype, seed=1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for act in ACTS:
        e = Exact(act, x, wg, wu, dh)
        dx, dwg, dwu = layers.gated_ffn_backward(dh, x, wg, wu, act=act, status=status)
        close(dx, e.dx, e.dx_tol)
        close(dwg, e.dwg, e.dwg_tol)
        close(dwu, e.dwu, e.dwu_tol)
    assert int(status) == 0


def run_c(x, wg, wu, act="silu", out_ld=None, stream=None):
    """lwc_gated_forward itself, h's rows out_ld apart in a buffer of 7s."""
    (M, K), N = x.shape, wg.shape[0]
    ld = out_ld or N
    out = torch.full((M, ld), 7.0, dtype=x.dtype, device="cuda")
    elem = lwc.LWC_ELEM_BF16 if x.dtype == torch.bfloat16 else lwc.LWC_ELEM_FP16
    g = lwc.lwc_gated(elem, layers.ACTIVATIONS[act], M, N, K, x.stride(0), wg.stride(0), wu.stride(0), x.data_ptr(),
                      wg.data_ptr(), wu.data_ptr())
    lwc.lwc_gated_forward(g, out, ld, None, stream)
    return out


@pytest.mark.parametrize("N,ld", [(40, 40), (40, 48), (37, 41), (130, 200)])
def test_writes_nothing_but_h(N, ld):
    x, wg, wu, _ = inputs(150, N, 72, torch.bfloat16, seed=3)
    e = Exact("silu", x, wg, wu)
    out = run_c(x, wg, wu, out_ld=ld, stream=torch.cuda.current_stream())
    close(out[:, :N], e.h, e.h_tol)
    assert bool((out[:, N:] == 7).all())


def test_strided_rows_and_odd_alignment():
    x, wg, wu, dh = inputs(50, 120, 72, torch.bfloat16, seed=4)
    e = Exact("silu", x, wg, wu, dh)
    want = layers.gated_ffn(x, wg, wu)
    wide = torch.zeros(50, 200, dtype=x.dtype, device="cuda")
    both = torch.zeros(240, 72, dtype=x.dtype, device="cuda")
    both[:120], both[120:] = wg, wu
    for off in (0, 8, 3):   # rows on, and off, 16-byte boundaries
        wide[:, off:off + 72] = x
        assert torch.equal(layers.gated_ffn(wide[:, off:off + 72], both[:120], both[120:]), want)
    # transposed, broadcast and permuted operands
    assert torch.equal(layers.gated_ffn(x.t().contiguous().t(), wg.t().contiguous().t(), wu), want)
    one = x[:1].expand(50, 72)
    assert torch.equal(layers.gated_ffn(one, wg, wu), want[:1].expand(50, 120))
    got = layers.gated_ffn_backward(dh.t().contiguous().t(), wide[:, 3:75], both[:120], both[120:])
    for a, b, tol in zip(got, (e.dx, e.dwg, e.dwu), (e.dx_tol, e.dwg_tol, e.dwu_tol)):
        close(a, b, tol)
    summed = layers.gated_ffn_backward(dh[:1].expand(50, 120), x, wg, wu)
    assert torch.equal(summed[0], layers.gated_ffn_backward(dh[:1].expand(50, 120).contiguous(), x, wg, wu)[0])
    # more dimensions, and an output to fill
    x3 = x.view(5, 10, 72)
    out = torch.empty(5, 10, 120, dtype=x.dtype, device="cuda")
    assert layers.gated_ffn(x3, wg, wu, out=out) is out and torch.equal(out.view(50, 120), want)
    assert layers.gated_ffn_backward(dh.view(5, 10, 120), x3, wg, wu)[0].shape == x3.shape


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
def test_any_choice_of_gradients_is_the_same(need):
    x, wg, wu, dh = inputs(140, 200, 96, torch.bfloat16, seed=5)
    every = layers.gated_ffn_backward(dh, x, wg, wu)
    some = layers.gated_ffn_backward(dh, x, wg, wu, need=need)
    for a, b, n in zip(every, some, need):
        assert (b is None) if not n else torch.equal(a, b)


def test_one_row_without_a_batch():
    x, wg, wu, dh = inputs(1, 24, 16, torch.bfloat16, seed=18)
    assert torch.equal(layers.gated_ffn(x[0], wg, wu), layers.gated_ffn(x, wg, wu)[0])
    got, want = layers.gated_ffn_backward(dh[0], x[0], wg, wu), layers.gated_ffn_backward(dh, x, wg, wu)
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[1])


def test_refusals_on_the_gpu():
    x, wg, wu, dh = inputs(4, 24, 16, torch.bfloat16, seed=19)
    for call in (lambda: layers.gated_ffn(x, wg[:, :8], wu), lambda: layers.gated_ffn(x, wg, wu[:8]),
                 lambda: layers.gated_ffn(x, wg.half(), wu), lambda: layers.gated_ffn(x, wg, wu.cpu()),
                 lambda: layers.gated_ffn(x, wg, wu, act="swish2"), lambda: layers.gated_ffn(x, wg[None], wu),
                 lambda: layers.gated_ffn(x, wg, wu, out=torch.empty(4, 25, device="cuda").bfloat16()),
                 lambda: layers.gated_ffn_backward(dh[:, :8], x, wg, wu),
                 lambda: layers.gated_ffn_backward(dh.float(), x, wg, wu)):
        with pytest.raises(ValueError):
            call()


def test_no_tokens():
    x, wg, wu, _ = inputs(1, 24, 16, torch.bfloat16)
    none = x[:0]
    assert layers.gated_ffn(none, wg, wu).shape == (0, 24)
    dx, dwg, dwu = layers.gated_ffn_backward(none.new_empty(0, 24), none, wg, wu)
    assert dx.shape == (0, 16) and not dwg.any() and not dwu.any() and dwg.shape == wg.shape


def test_infinities_and_nan_stay_in_their_rows():
    x, wg, wu, dh = inputs(300, 64, 64, torch.bfloat16, seed=6)
    want = layers.gated_ffn(x, wg, wu)
    dx = layers.gated_ffn_backward(dh, x, wg, wu, need=(True, False, False))[0]
    bad = x.clone()
    bad[5], bad[130], bad[299] = float("nan"), float("inf"), -float("inf")
    h = layers.gated_ffn(bad, wg, wu)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[5, 130, 299]] = False
    assert torch.equal(h[keep], want[keep]) and bool(h[5].isnan().all())
    got = layers.gated_ffn_backward(dh, bad, wg, wu, need=(True, False, False))[0]
    assert torch.equal(got[keep], dx[keep])


@pytest.mark.parametrize("act", ACTS)
def test_far_arguments_do_not_overflow(act):
    """a of up to +-300 (exp(300) is beyond FP32)."""
    K = 16
    x = torch.linspace(-300, 300, 128, device="cuda").to(torch.bfloat16)[:, None] * torch.eye(1, K, device="cuda").bfloat16()
    wg = torch.eye(8, K, device="cuda").bfloat16()
    wg[:] = wg[0]
    wu = torch.ones(8, K, device="cuda").bfloat16() / 64
    wu[:, 1:] = 0
    h = layers.gated_ffn(x, wg, wu, act=act)
    a = x[:, :1].double()
    want = act64(act, a)[0] * (a / 64)
    assert bool(h.isfinite().all())
    # |act'| <= 1.2 and a is exact; the fast exponential is off by up to 2 + 1.16 |v| units (2^-14 in all here)
    tol = (2.0 ** -14 + 2.0 ** -8) * want.abs() + 1e-30
    close(h, want.expand(128, 8), tol.expand(128, 8))
    dx, dwg, dwu = layers.gated_ffn_backward(torch.ones_like(h), x, wg, wu, act=act)
    assert all(bool(t.isfinite().all()) for t in (dx, dwg, dwu))


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """Directional derivatives by central differences of the 64-bit formula."""
    x, wg, wu, dh = inputs(24, 40, 32, torch.bfloat16, seed=8)
    dx, dwg, dwu = layers.gated_ffn_backward(dh, x, wg, wu, act=act)
    e = Exact(act, x, wg, wu, dh)

    def loss(x, wg, wu):
        return float((act64(act, x @ wg.T)[0] * (x @ wu.T) * dh.double()).sum())

    base = [t.double() for t in (x, wg, wu)]
    g = torch.Generator("cuda").manual_seed(9)
    for i, (grad, tol) in enumerate(((dx, e.dx_tol), (dwg, e.dwg_tol), (dwu, e.dwu_tol))):
        v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4 if act != "relu" else 1e-7   # relu: no argument crosses 0 on the way
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * v, base[i] - h * v
        slope = (loss(*up) - loss(*down)) / (2 * h)
        # the difference's own error: h^2 times a third derivative of order |v|^3 sqrt(n), and cancellation
        mag = float((v.abs() * (grad.double().abs() + tol)).sum())
        assert abs(slope - float((grad.double() * v).sum())) <= float((tol * v.abs()).sum()) + 1e-6 * mag


def test_autograd_is_the_explicit_backward():
    x, wg, wu, dh = inputs(130, 72, 64, torch.float16, seed=10)
    leaves = [t.clone().requires_grad_() for t in (x.view(2, 65, 64), wg, wu)]
    h = layers.gated_ffn(*leaves, act="gelu")
    assert torch.equal(h, layers.gated_ffn(x.view(2, 65, 64), wg, wu, act="gelu"))
    h.backward(dh.view(2, 65, 72))
    want = layers.gated_ffn_backward(dh.view(2, 65, 72), x.view(2, 65, 64), wg, wu, act="gelu")
    assert all(torch.equal(a.grad, b) for a, b in zip(leaves, want))
    # frozen matrices: x alone
    x2 = x.clone().requires_grad_()
    (dx,) = torch.autograd.grad(layers.gated_ffn(x2, wg, wu, act="gelu"), x2, dh)
    assert torch.equal(dx, want[0].view(130, 64))
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(layers.gated_ffn(x2, wg, wu), x2, dh, create_graph=True)
    # one matrix as both, and a broadcast input: their gradients are sums
    w2 = wg.clone().requires_grad_()
    layers.gated_ffn(x, w2, w2, act="gelu").backward(dh)
    _, one, two = layers.gated_ffn_backward(dh, x, wg, wg, act="gelu")
    assert torch.equal(w2.grad, one + two)
    row = x[:1].clone().requires_grad_()
    layers.gated_ffn(row.expand(130, 64), wg, wu, act="gelu").backward(dh)
    dx = layers.gated_ffn_backward(dh, x[:1].expand(130, 64), wg, wu, act="gelu", need=(True, False, False))[0]
    assert torch.equal(row.grad, dx.sum(0, keepdim=True))
    # a sum of two uses
    x3 = x.clone().requires_grad_()
    (layers.gated_ffn(x3, wg, wu) + layers.gated_ffn(x3, wu, wg)).float().sum().backward()
    assert x3.grad.shape == x.shape


def test_streams_and_repeatability():
    x, wg, wu, dh = inputs(700, 512, 256, torch.bfloat16, seed=11)
    want = layers.gated_ffn(x, wg, wu)
    grads = layers.gated_ffn_backward(dh, x, wg, wu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):   # several calls at a time, each with its own workspace
        for s in streams:
            got.append((layers.gated_ffn(x, wg, wu, stream=s), layers.gated_ffn_backward(dh, x, wg, wu, stream=s)))
    torch.cuda.synchronize()
    raw = layers.gated_ffn(x, wg, wu, stream=streams[0].cuda_stream)   # a raw handle
    # the operands may be freed by their owner while another stream still reads them
    x2, wg2, wu2 = x.clone(), wg.clone(), wu.clone()
    streams[1].wait_stream(torch.cuda.current_stream())
    late = layers.gated_ffn(x2, wg2, wu2, stream=streams[1])
    del x2, wg2, wu2
    junk = [torch.full_like(t, 7.0) for t in (x, wg, wu)]
    torch.cuda.synchronize()
    assert torch.equal(raw, want) and torch.equal(late, want) and len(junk) == 3
    for h, g in got:
        assert torch.equal(h, want) and all(torch.equal(a, b) for a, b in zip(g, grads))


def test_host_threads():
    """Calls from host threads that have made no CUDA call before, several at a time."""
    x, wg, wu, _ = inputs(300, 200, 128, torch.bfloat16, seed=17)
    want = layers.gated_ffn(x, wg, wu)
    torch.cuda.synchronize()
    elem, s = lwc.LWC_ELEM_BF16, torch.cuda.current_stream().cuda_stream
    g = lwc.lwc_gated(elem, 0, 300, 200, 128, 128, 128, 128, x.data_ptr(), wg.data_ptr(), wu.data_ptr())
    outs = [torch.empty_like(want) for _ in range(8)]
    failed = []

    def work(out):
        try:
            for _ in range(5):
                lwc.lwc_gated_forward(g, out, 200, None, s)
        except Exception as e:   # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(o,)) for o in outs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and all(torch.equal(o, want) for o in outs)


def test_captured_and_replayed():
    x, wg, wu, dh = inputs(200, 300, 128, torch.bfloat16, seed=12)
    xs, dhs = x.clone(), dh.clone()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        layers.gated_ffn(xs, wg, wu)
        layers.gated_ffn_backward(dhs, xs, wg, wu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = layers.gated_ffn(xs, wg, wu)
        grads = layers.gated_ffn_backward(dhs, xs, wg, wu)
    for seed in (13, 14):
        x2, _, _, dh2 = inputs(200, 300, 128, torch.bfloat16, seed=seed)
        xs.copy_(x2)
        dhs.copy_(dh2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, layers.gated_ffn(x2, wg, wu))
        assert all(torch.equal(a, b) for a, b in zip(grads, layers.gated_ffn_backward(dh2, x2, wg, wu)))


def test_offsets_past_32_bits():
    """h, dA and dB of more than 2^32 bytes: the rows at the end are as right as the first."""
    M, N, K = 160_001, 14_336, 16
    g = torch.Generator("cuda").manual_seed(15)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    wg, wu = (torch.randn(N, K, generator=g, device="cuda").mul_(0.25).bfloat16() for _ in range(2))
    h = layers.gated_ffn(x, wg, wu)
    dh = torch.full((1, 1), 0.5, dtype=x.dtype, device="cuda").expand(M, N).contiguous()
    dx = layers.gated_ffn_backward(dh, x, wg, wu, need=(True, False, False))[0]
    for rows in (slice(0, 130), slice(M // 2, M // 2 + 130), slice(M - 130, M)):
        e = Exact("silu", x[rows], wg, wu, dh[rows])
        close(h[rows], e.h, e.h_tol)
        close(dx[rows], e.dx, e.dx_tol)


# ---- compressed matrices ---------------------------------------------------------


def resident(codec, wg, wu):
    model = layers.ResidentModel(codec, "cuda")
    model.add_layer_from_device("ffn", [wg, wu])
    return model


@pytest.mark.parametrize("codec", layers.CODECS)
@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 130])
def test_resident_model(codec, M):
    N, K = 264, 320
    wg, wu = (synth.normal_bf16((N, K), seed=s, sigma=0.05, outlier_frac=1e-3, device="cuda") for s in (1, 2))
    model = resident(codec, wg, wu)
    g = torch.Generator("cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    dh = torch.randn(M, N, generator=g, device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = Exact("silu", x, wg, wu, dh)   # the fused sums' trees are lower than K terms one by one
    for route in ("auto", "decode") + (("fused",) if M <= 8 else ()):
        h = model.gated(0, 0, 1, x, status=status, route=route)
        close(h, e.h, e.h_tol)
        xg = x.clone().requires_grad_()
        hg = model.gated(0, 0, 1, xg, status=status, route=route)
        close(hg, e.h, e.h_tol)
        hg.backward(dh)
        close(xg.grad, e.dx, e.dx_tol)
    # decoded bit for bit: the same kernel as on the dense matrices
    assert torch.equal(model.gated(0, 0, 1, x, route="decode"), layers.gated_ffn(x, wg, wu))
    out = torch.empty(M, N, dtype=x.dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert model.gated(0, 0, 1, x, out=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, model.gated(0, 0, 1, x))
    assert int(status) == 0


def test_resident_model_fp16_and_empty():
    g = torch.Generator("cuda").manual_seed(1)
    wg, wu = (torch.randn(40, 48, generator=g, device="cuda").mul_(0.1).half() for _ in range(2))
    model = resident("dfloat11", wg, wu)
    x = torch.randn(3, 48, generator=g, device="cuda").half()
    assert torch.equal(model.gated(0, 0, 1, x), layers.gated_ffn(x, wg, wu))
    assert model.gated(0, 0, 1, x[:0]).shape == (0, 40)


@pytest.mark.parametrize("codec", layers.CODECS)
@pytest.mark.parametrize("M", [1, 40, 256])
def test_tiled_weights(codec, M):
    N, K = 256, 192
    wg, wu = (synth.normal_bf16((N, K), seed=s, sigma=0.05, outlier_frac=1e-3, device="cuda") for s in (3, 4))
    tw = layers.TiledWeights("cuda", codec)
    gate, up = tw.add(wg), tw.add(wu)
    x = torch.randn(M, K, generator=torch.Generator("cuda").manual_seed(M), device="cuda").bfloat16()
    for act in ACTS:
        e = Exact(act, x, wg, wu)
        close(tw.gated(gate, up, x, act=act), e.h, e.h_tol)


def test_tiled_weights_on_another_stream():
    """An x that has to be laid out first, on a stream of its own while the current one is busy: the copy is
    made where it is read (unaligned rows too)."""
    N, K, M = 256, 192, 40
    wg, wu = (synth.normal_bf16((N, K), seed=s, sigma=0.05, outlier_frac=1e-3, device="cuda") for s in (3, 4))
    tw = layers.TiledWeights("cuda")
    gate, up = tw.add(wg), tw.add(wu)
    x = torch.randn(M, K, generator=torch.Generator("cuda").manual_seed(20), device="cuda").bfloat16()
    want, a = tw.gated(gate, up, x), tw.gemm(gate, x)
    odd = torch.zeros(M * K + 1, dtype=x.dtype, device="cuda")
    odd[1:] = x.view(-1)
    side = torch.cuda.Stream()
    strided, odd = x.t().contiguous().t(), odd[1:].view(M, K)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)   # some 10 ms on the current stream
        got = [tw.gated(gate, up, strided, stream=stream), tw.gated(gate, up, odd, stream=stream)]
        b = tw.gemm(gate, strided, stream=stream)
        side.synchronize()
        with torch.cuda.stream(side):
            assert all(torch.equal(g, want) for g in got) and torch.equal(a, b)
        torch.cuda.synchronize()


def late(stream, call, *tensors):
    """call(*copies of tensors) on `stream` behind some 100 ms of other work, where the copies are freed, and
    their memory written again, long before the call's kernels run. Once without that work first: loading a
    kernel may wait for the device."""
    for cycles in (1000, 200_000_000):
        copies = [t.clone().requires_grad_(t.requires_grad) for t in tensors]
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(cycles)
        result = call(*copies).detach()
        del copies
        junk = [torch.full_like(t, 7) for t in tensors for _ in range(2)]
        behind = not stream.query()
        torch.cuda.synchronize()
    assert behind, "the work ahead of the call ended too early to show anything"
    return result, junk


@pytest.mark.parametrize("grad", [False, True])
def test_operands_freed_before_the_stream_reads_them(grad):
    x, wg, wu, _ = inputs(300, 512, 256, torch.bfloat16, seed=21)
    t = torch.randint(0, 512, (300,), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    wants = (layers.gated_ffn(x, wg, wu), layers.linear_cross_entropy(x, wg, t, reduction="none"))
    x.requires_grad_(grad)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = late(s, lambda x, wg, wu: layers.gated_ffn(x, wg, wu, stream=s), x, wg, wu)
    assert torch.equal(got, wants[0])
    got, _ = late(s, lambda x, w, t: layers.linear_cross_entropy(x, w, t, reduction="none", stream=s), x, wg, t)
    assert torch.equal(got, wants[1])


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("codec", layers.CODECS)
def test_operands_of_compressed_forms_freed_before_the_stream_reads_them(codec, grad):
    N, K = 264, 320
    wg, wu = (synth.normal_bf16((N, K), seed=s, sigma=0.05, outlier_frac=1e-3, device="cuda") for s in (1, 2))
    model = resident(codec, wg, wu)
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(8, K, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, N, (8,), generator=g, device="cuda")
    s = torch.cuda.Stream()
    for route in ("decode", "fused"):
        want = layers.gated_ffn(x, wg, wu)
        x.requires_grad_(grad)
        got, _ = late(s, lambda x: model.gated(0, 0, 1, x, stream=s, route=route), x)
        x.requires_grad_(False)
        e = Exact("silu", x, wg, wu)
        close(got, e.h, e.h_tol)
        assert route == "fused" or torch.equal(got, want)
    want = model.cross_entropy(0, 0, x, t, reduction="none")
    x.requires_grad_(grad)
    got, _ = late(s, lambda x, t: model.cross_entropy(0, 0, x, t, reduction="none", stream=s), x, t)
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 2])
def test_resident_model_of_other_blocks(M):
    """DFloat11 blobs that the decode-fused linear layer does not take (blocks of 64 chunks)."""
    N, K = 264, 320
    wg, wu = (synth.normal_bf16((N, K), seed=s, sigma=0.05, outlier_frac=1e-3, device="cuda") for s in (1, 2))
    model = layers.ResidentModel("dfloat11", "cuda")
    model.add_layer_from_device("ffn", [wg, wu], threads_per_block=64)
    x = torch.randn(M, K, generator=torch.Generator("cuda").manual_seed(M), device="cuda").bfloat16()
    assert torch.equal(model.gated(0, 0, 1, x), layers.gated_ffn(x, wg, wu))
    xg = x.clone().requires_grad_()
    h = model.gated(0, 0, 1, xg)
    h.backward(torch.ones_like(h))
    assert torch.equal(xg.grad, layers.gated_ffn_backward(torch.ones_like(h), x, wg, wu, need=(True, False, False))[0])
    with pytest.raises(lwc.LwcError, match="blocks of 32 chunks"):
        model.gated(0, 0, 1, x, route="fused")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
def test_arguments_whose_powers_overflow(act):
    """|a| up to 1e38: a^2 and a^3 are beyond FP32, the activation and its slope are not."""
    K = 16
    a = torch.tensor([1e4, 1e7, 1e13, 3e18, 1e20, 1e30, 1e38], device="cuda")
    a = torch.cat([a, -a, a.new_zeros(2)]).bfloat16()
    M = a.numel()
    x = torch.zeros(M, K, device="cuda").bfloat16()
    x[:, 0], x[:, 1] = a, 1.0
    wg, wu = (torch.zeros(8, K, device="cuda").bfloat16() for _ in range(2))
    wg[:, 0], wu[:, 1] = 1.0, 2.0 ** -6     # a and b = 2^-6, exact
    dh = torch.ones(M, 8, device="cuda").bfloat16()
    y, s = act64(act, a.double())
    h = layers.gated_ffn(x, wg, wu, act=act)
    # |v| is 0 or so large that the activation is v, 1 or 0; h is rounded once
    close(h, (y / 64)[:, None].expand(M, 8), (2.0 ** -8 * (y / 64).abs() + 1e-30)[:, None].expand(M, 8))
    dx = layers.gated_ffn_backward(dh, x, wg, wu, act=act, need=(True, False, False))[0]
    want = 8 * s / 64      # eight features alike
    close(dx[:, 0], want, 2 * 2.0 ** -8 * want.abs() + 1e-30)


@pytest.mark.parametrize("codec", layers.CODECS)
def test_tiled_weights_of_unlike_blobs(codec):
    """Two matrices that one launch does not take together: another index width, another chunk size."""
    N, K, M = 256, 192, 40
    wg, wu = (synth.normal_bf16((N, K), seed=s, sigma=0.05, outlier_frac=1e-3, device="cuda") for s in (3, 4))
    if codec == "codebook":
        wu = (wu * 64).round().clamp(-8, 8).div(64).bfloat16()   # a handful of values
    tw = layers.TiledWeights("cuda", codec)
    gate, up = tw.add(wg), tw.add(wu, **({} if codec == "codebook" else {"chunk_bytes": 36}))
    assert (tw.descs[gate].k, tw.descs[gate].chunk_bytes) != (tw.descs[up].k, tw.descs[up].chunk_bytes)
    x = torch.randn(M, K, generator=torch.Generator("cuda").manual_seed(M), device="cuda").bfloat16()
    e = Exact("silu", x, wg, wu)
    close(tw.gated(gate, up, x), e.h, e.h_tol)
    e = Exact("silu", x, wu, wg)
    close(tw.gated(up, gate, x), e.h, e.h_tol)
    e = Exact("silu", x, wg, wg)
    close(tw.gated(gate, gate, x), e.h, e.h_tol)   # one matrix twice
