"""The vocabulary cross entropy (lwc_xent_forward, lwc_xent_backward,
layers.linear_cross_entropy and the compressed form) against its formulas in
64 bits.

Bounds per element, with u = 2^-23 and gamma_n = n u / (1 - n u) as the
library states for the tensor cores' sums, S_iv = sum_k |x_ik W_vk|:

    |z' - z| <= e_z = gamma_K S;   lse and the target's logit are both off by
    at most max_v e_z, plus what FP32 evaluation adds: G (1 + |z|max) with
    G = 2^-19 (sums of at most 2^18 positive terms in pieces of 256, the
    exponent's argument rounded to 2^-24 of at most 2^5, log and exp to a few
    units).
    P: relative e_z + e_lse + G on p, then the rounding to 16 bits, at most
    half a step H (2^-8 BF16, 2^-11 FP16), absolute 2^-25 / 2^14 below FP16's
    normal numbers (P is scaled by 2^14).
"""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from decode_dfloat11_b200 import build as lwc_build
from decode_dfloat11_b200 import layers, lwc

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
G = 2.0 ** -19
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
TYPES = [torch.bfloat16, torch.float16]
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def lib(cuda_device):
    lwc_build.build()
    return lwc.load()


def gamma(n):
    return n * U / (1 - n * U)


class Exact:
    """Values and bounds; c: the gradient of each token's loss."""

    def __init__(self, x, w, t, c=None, ignore=IGNORE):
        dt = x.dtype
        half, tiny = HALF[dt], TINY[dt]
        M, K = x.shape
        V = w.shape[0]
        keep = t != ignore
        x, w = torch.where(keep[:, None], x.double(), 0.0), w.double()
        z = x @ w.T
        ez = gamma(K) * (x.abs() @ w.abs().T)
        lse = torch.logsumexp(z, 1)
        at = torch.where(keep, t, 0)[:, None]
        self.loss = torch.where(keep, lse - z.gather(1, at)[:, 0], 0.0)
        e = ez.amax(1) + G * (1 + z.abs().amax(1))
        self.lse, self.lse_tol = lse, e
        self.loss_tol = torch.where(keep, 2 * e, 0.0)
        self.keep = keep
        if c is None:
            return
        c = torch.where(keep, c.double(), 0.0)[:, None]
        p = torch.exp(z - lse[:, None])
        hot = torch.zeros_like(p).scatter_(1, at, 1.0)
        P = c * (p - hot)
        eP = c.abs() * (p * 1.01 * (ez + e[:, None] + G) + 4 * U)
        # FP16: P / max |c| is scaled by 2^14 (up to another factor of 2) before it is rounded
        eP = eP + half * (P.abs() + eP) + (c != 0) * (tiny * 2.0 ** -13 * c.abs().max() if dt == torch.float16 else tiny)

        def product(p, e, q, n):
            value = p @ q
            err = e @ q.abs() + (gamma(n) + 2.0 ** -18) * ((p.abs() + e) @ q.abs())
            return value, err + half * (value.abs() + err) + tiny

        self.dx, self.dx_tol = product(P, eP, w, V)
        self.dw, self.dw_tol = product(P.T, eP.T, x, M)


def close(got, want, tol):
    assert got.shape == want.shape
    off = (got.double() - want).abs() - tol
    assert bool((off <= 0).all()), (float(off.max()), int(off.argmax()))


def inputs(M, V, K, dtype, seed=0, ignored=0.2):
    g = torch.Generator("cuda").manual_seed(1000 * seed + M + 7 * V + 13 * K)
    w = torch.randn(V, K, generator=g, device="cuda").mul_(K ** -0.5).to(dtype)
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    lean = 10 * torch.rand(M, 1, generator=g, device="cuda")
    x = (torch.randn(M, K, generator=g, device="cuda") + lean * w[t].float()).to(dtype)
    off = torch.rand(M, generator=g, device="cuda") < ignored
    off[0] = False
    return x, w, torch.where(off, IGNORE, t)


def test_gradients_over_several_pieces():
    """P is larger than a piece of the vocabulary (3 pieces here, the last one
    narrower), with tiles to spare in the last wave."""
    M, V, K = 4500, 100_003, 72
    x, w, t = inputs(M, V, K, torch.bfloat16, seed=3)
    grad = torch.tensor(1.3, device="cuda")
    e = Exact(x, w, t, grad.expand(M) / max(1, int((t != IGNORE).sum())))
    loss, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
    close(loss, e.loss, e.loss_tol)
    dx, dw = layers.linear_cross_entropy_backward(grad, lse, x, w, t)
    close(dx, e.dx, e.dx_tol)
    close(dw, e.dw, e.dw_tol)
    # each alone is the same
    assert torch.equal(dx, layers.linear_cross_entropy_backward(grad, lse, x, w, t, need=(True, False))[0])
    assert torch.equal(dw, layers.linear_cross_entropy_backward(grad, lse, x, w, t, need=(False, True))[1])


def test_a_narrow_last_piece_adds_to_the_same_sum():
    """Seven pieces of 1280 words and one of 265: dx's tiles are those of the
    other pieces, whatever suits a contraction that short."""
    M, V, K = 196_000, 9225, 384
    g = torch.Generator("cuda").manual_seed(21)
    w = torch.randn(V, K, generator=g, device="cuda").mul_(K ** -0.5).bfloat16()
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    grad = torch.rand(M, generator=g, device="cuda") + 0.5
    loss, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
    dx, _ = layers.linear_cross_entropy_backward(grad, lse, x, w, t, reduction="none", need=(True, False))
    for rows in (slice(0, 300), slice(98_000, 98_300), slice(M - 300, M)):
        e = Exact(x[rows], w, t[rows], grad[rows])
        close(loss[rows], e.loss, e.loss_tol)
        close(dx[rows], e.dx, e.dx_tol)


SIZES = [(1, 1, 1), (1, 7, 64), (1, 5003, 256), (1, 30_000, 130), (2, 4999, 72), (3, 100, 17), (4, 8, 2000), (5, 100, 17),
         (4, 20_000, 1024), (33, 999, 72), (128, 256, 64), (129, 257, 136),
         (500, 3001, 200), (1000, 512, 1024), (300, 12345, 96)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,V,K", SIZES)
def test_losses(M, V, K, dtype):
    x, w, t = inputs(M, V, K, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = Exact(x, w, t)
    loss, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True, status=status)
    close(loss, e.loss, e.loss_tol)
    close(lse[e.keep], e.lse[e.keep], e.lse_tol[e.keep])
    n = max(1, int(e.keep.sum()))
    for reduction, div in (("sum", 1), ("mean", n)):
        got = layers.linear_cross_entropy(x, w, t, reduction=reduction, status=status)
        # the total is summed in 64 bits and rounded once
        close(got, e.loss.sum() / div, (e.loss_tol.sum() + 2.0 ** -23 * e.loss.abs().sum()) / div)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,V,K", SIZES)
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_gradients(M, V, K, dtype, reduction):
    x, w, t = inputs(M, V, K, dtype, seed=1)
    g = torch.Generator("cuda").manual_seed(5)
    if reduction == "none":
        grad = torch.randn(M, generator=g, device="cuda")
        c = grad
    else:
        grad = torch.tensor(0.7, device="cuda")
        c = grad.expand(M) / (max(1, int((t != IGNORE).sum())) if reduction == "mean" else 1)
    e = Exact(x, w, t, c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, lse = layers.linear_cross_entropy(x, w, t, return_lse=True)
    dx, dw = layers.linear_cross_entropy_backward(grad, lse, x, w, t, reduction=reduction, status=status)
    close(dx, e.dx, e.dx_tol)
    close(dw, e.dw, e.dw_tol)
    assert int(status) == 0


def test_ignored_tokens_bear_nothing_whatever_they_hold():
    x, w, t = inputs(300, 777, 64, torch.bfloat16, seed=4, ignored=0.5)
    loss, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
    grad = torch.ones((), device="cuda")
    dx, dw = layers.linear_cross_entropy_backward(grad, lse, x, w, t)
    bad = x.clone()
    off = t == IGNORE
    bad[off] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()[
        torch.arange(int(off.sum()), device="cuda") % 3][:, None]
    loss2, lse2 = layers.linear_cross_entropy(bad, w, t, reduction="none", return_lse=True)
    assert torch.equal(loss, loss2) and not loss2[off].any()
    dx2, dw2 = layers.linear_cross_entropy_backward(grad, lse2, bad, w, t)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and not dx2[off].any()
    assert torch.equal(layers.linear_cross_entropy(bad, w, t), layers.linear_cross_entropy(x, w, t))


def test_all_tokens_ignored_and_no_tokens():
    x, w, t = inputs(20, 50, 32, torch.bfloat16, seed=5)
    none = torch.full_like(t, IGNORE)
    for reduction in ("mean", "sum"):
        xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
        loss = layers.linear_cross_entropy(xg, wg, none, reduction=reduction)
        assert float(loss.detach()) == 0.0
        loss.backward()
        assert not xg.grad.any() and not wg.grad.any()
        empty = layers.linear_cross_entropy(x[:0], w, t[:0], reduction=reduction)
        assert float(empty) == 0.0
    loss, lse = layers.linear_cross_entropy(x[:0], w, t[:0], reduction="none", return_lse=True)
    assert loss.shape == lse.shape == (0,)
    dx, dw = layers.linear_cross_entropy_backward(torch.ones((), device="cuda"), lse, x[:0], w, t[:0])
    assert dx.shape == (0, 32) and not dw.any()


def test_targets_that_are_no_words():
    x, w, t = inputs(140, 100, 32, torch.bfloat16, seed=6)
    bad = t.clone()
    bad[3], bad[70], bad[139] = 100, -1, 2 ** 40
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = layers.linear_cross_entropy(x, w, bad, reduction="none", return_lse=True, status=status)
    assert int(status) == lwc.LWC_DEVICE_BAD_TARGET
    gone = torch.zeros(140, dtype=torch.bool, device="cuda")
    gone[[3, 70, 139]] = True
    assert bool(loss[gone].isnan().all()) and bool(loss[~gone].isfinite().all())
    dx, dw = layers.linear_cross_entropy_backward(torch.ones((), device="cuda"), lse, x, w, bad, reduction="sum")
    same = torch.where(gone, IGNORE, t)
    dx2, dw2 = layers.linear_cross_entropy_backward(torch.ones((), device="cuda"), lse, x, w, same, reduction="sum")
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_another_ignore_index_and_int32_targets():
    x, w, t = inputs(140, 100, 32, torch.float16, seed=7, ignored=0.0)
    t[5] = 0
    e = Exact(x, w, t, ignore=0)
    got = layers.linear_cross_entropy(x, w, t.to(torch.int32), ignore_index=0, reduction="none")
    close(got, e.loss, e.loss_tol)
    assert float(got[5]) == 0.0


def test_masked_words_and_far_logits():
    """Words whose logits are the type's lowest values (an added mask) have no
    share; logits of +-10000 neither overflow nor vanish."""
    M, V, K = 130, 600, 16
    x, w, t = inputs(M, V, K, torch.bfloat16, seed=8, ignored=0.0)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    w[300:, 0] = torch.finfo(torch.bfloat16).min
    t = t % 300
    e = Exact(x, w, t)
    loss, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
    # the masked words' logits say nothing of the others': bounds from the first 300 alone
    part = Exact(x, w[:300], t)
    close(loss, e.loss, part.loss_tol)
    dx, dw = layers.linear_cross_entropy_backward(torch.ones((), device="cuda"), lse, x, w, t)
    assert not dw[300:].any() and bool(dx[:, 1:].isfinite().all())
    far = torch.zeros(V, K, device="cuda").bfloat16()
    far[:, 0] = torch.linspace(-10000, 10000, V, device="cuda").bfloat16()
    e = Exact(x, far, t)
    loss = layers.linear_cross_entropy(x, far, t, reduction="none")
    close(loss, e.loss, e.loss_tol)


def test_words_of_minus_infinity():
    M, V, K = 40, 300, 16
    x, w, t = inputs(M, V, K, torch.bfloat16, seed=9, ignored=0.0)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    w[100:, 0] = -float("inf")
    t = t % 100
    loss, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
    part = Exact(x, w[:100], t)
    close(loss, part.loss, part.loss_tol)
    # nothing left but -infinity
    w[:, 0] = -float("inf")
    lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)[1]
    assert bool((lse == -float("inf")).all())


def test_strided_rows_and_odd_alignment():
    x, w, t = inputs(70, 333, 72, torch.bfloat16, seed=10)
    loss, lse = layers.linear_cross_entropy(x, w, t, return_lse=True)
    grads = layers.linear_cross_entropy_backward(torch.ones((), device="cuda"), lse, x, w, t)
    wide = torch.zeros(70, 200, dtype=x.dtype, device="cuda")
    for off in (0, 16, 5):
        wide[:, off:off + 72] = x
        xs, ws = wide[:, off:off + 72], w.t().contiguous().t()
        assert torch.equal(layers.linear_cross_entropy(xs, ws, t), loss)
        got = layers.linear_cross_entropy_backward(torch.ones((), device="cuda"), lse, xs, ws, t)
        assert all(torch.equal(a, b) for a, b in zip(got, grads))
    x3, t2 = x.view(7, 10, 72), t.view(7, 10)
    none = layers.linear_cross_entropy(x3, w, t2, reduction="none")
    assert none.shape == (7, 10) and torch.equal(none.view(-1), layers.linear_cross_entropy(x, w, t, reduction="none"))


def test_autograd_is_the_explicit_backward_and_differences():
    M, V, K = 50, 90, 24
    x, w, t = inputs(M, V, K, torch.bfloat16, seed=11)
    for reduction in ("mean", "sum", "none"):
        xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
        loss, lse = layers.linear_cross_entropy(xg, wg, t, reduction=reduction, return_lse=True)
        assert not lse.requires_grad
        up = torch.linspace(0.5, 2, M, device="cuda") if reduction == "none" else torch.tensor(1.5, device="cuda")
        dx, dw = torch.autograd.grad(loss, [xg, wg], up)
        want = layers.linear_cross_entropy_backward(up, lse, x, w, t, reduction=reduction)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        n = max(1, int((t != IGNORE).sum()))
        c = up if reduction == "none" else up.expand(M) / (n if reduction == "mean" else 1)
        e = Exact(x, w, t, c)
        g = torch.Generator("cuda").manual_seed(3)
        for i, (grad, tol) in enumerate(((dx, e.dx_tol), (dw, e.dw_tol))):
            v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
            base, h = [x.double(), w.double()], 1e-5
            up_, down = list(base), list(base)
            up_[i], down[i] = base[i] + h * v, base[i] - h * v

            def total(x, w):
                z = x @ w.T
                at = torch.where(t != IGNORE, t, 0)[:, None]
                return float((c * torch.where(t != IGNORE, torch.logsumexp(z, 1) - z.gather(1, at)[:, 0], 0.0)).sum())

            slope = (total(*up_) - total(*down)) / (2 * h)
            mag = float((v.abs() * (grad.double().abs() + tol)).sum())
            assert abs(slope - float((grad.double() * v).sum())) <= float((tol * v.abs()).sum()) + 1e-6 * mag


def test_one_row_without_a_batch_and_a_loss_changed_in_place():
    x, w, t = inputs(1, 60, 32, torch.bfloat16, seed=18)
    want = layers.linear_cross_entropy(x, w, t)
    assert layers.linear_cross_entropy(x[0], w, t[0], reduction="none").shape == ()
    assert torch.equal(layers.linear_cross_entropy(x[0], w, t[0]), want)
    xg = x[0].clone().requires_grad_()
    loss = layers.linear_cross_entropy(xg, w, t[0])
    loss /= 4   # as gradient accumulation does
    loss.backward()
    x2 = x.clone().requires_grad_()
    (layers.linear_cross_entropy(x2, w, t) / 4).backward()
    assert torch.equal(xg.grad, x2.grad[0])


def test_first_calls_inside_a_capture():
    """A process whose first calls of the library are captured ones."""
    code = """
import torch
from decode_dfloat11_b200 import layers
x = torch.randn(300, 128, device="cuda").bfloat16()
w, v = (torch.randn(500, 128, device="cuda").mul_(0.1).bfloat16() for _ in range(2))
t = torch.randint(0, 500, (300,), device="cuda")
one = torch.ones((), device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    h = layers.gated_ffn(x, w, v)
    d = layers.gated_ffn_backward(h, x, w, v)
    loss, lse = layers.linear_cross_entropy(x, w, t, return_lse=True)
    e = layers.linear_cross_entropy_backward(one, lse, x, w, t)
    one_row = layers.gated_ffn(x[:1], w, v), layers.linear_cross_entropy(x[:1], w, t[:1])
g.replay()
torch.cuda.synchronize()
h2 = layers.gated_ffn(x, w, v)
l2, lse2 = layers.linear_cross_entropy(x, w, t, return_lse=True)
assert torch.equal(h, h2) and torch.equal(loss, l2)
assert all(torch.equal(a, b) for a, b in zip(d, layers.gated_ffn_backward(h2, x, w, v)))
assert all(torch.equal(a, b) for a, b in zip(e, layers.linear_cross_entropy_backward(one, lse2, x, w, t)))
assert torch.equal(one_row[0], layers.gated_ffn(x[:1], w, v))
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_streams_graphs_and_repeatability():
    x, w, t = inputs(500, 3000, 128, torch.bfloat16, seed=12)
    grad = torch.ones((), device="cuda")
    loss, lse = layers.linear_cross_entropy(x, w, t, return_lse=True)
    want = layers.linear_cross_entropy_backward(grad, lse, x, w, t)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)] * 3:
        l2, e2 = layers.linear_cross_entropy(x, w, t, return_lse=True, stream=s)
        got.append((l2, layers.linear_cross_entropy_backward(grad, e2, x, w, t, stream=s)))
    torch.cuda.synchronize()
    for l2, g in got:
        assert torch.equal(l2, loss) and all(torch.equal(a, b) for a, b in zip(g, want))
    xs, ts = x.clone(), t.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l3, e3 = layers.linear_cross_entropy(xs, w, ts, return_lse=True)
        g3 = layers.linear_cross_entropy_backward(grad, e3, xs, w, ts)
    for seed in (13, 14):
        x2, _, t2 = inputs(500, 3000, 128, torch.bfloat16, seed=seed)
        xs.copy_(x2)
        ts.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        l4, e4 = layers.linear_cross_entropy(x2, w, t2, return_lse=True)
        assert torch.equal(l3, l4)
        assert all(torch.equal(a, b) for a, b in zip(g3, layers.linear_cross_entropy_backward(grad, e4, x2, w, t2)))


@pytest.mark.parametrize("codec", layers.CODECS)
def test_resident_model(codec):
    x, w, t = inputs(150, 520, 64, torch.bfloat16, seed=15)
    model = layers.ResidentModel(codec, "cuda")
    model.add_layer_from_device("head", [w])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for reduction in ("none", "mean", "sum"):
        want = layers.linear_cross_entropy(x, w, t, reduction=reduction)
        assert torch.equal(model.cross_entropy(0, 0, x, t, reduction=reduction, status=status), want)
    xg = x.clone().requires_grad_()
    loss = model.cross_entropy(0, 0, xg, t, status=status)
    loss.backward()
    x2 = x.clone().requires_grad_()
    layers.linear_cross_entropy(x2, w, t).backward()
    assert torch.equal(xg.grad, x2.grad) and int(status) == 0


def test_a_block_and_the_loss_together():
    """The operators as a training step uses them: a gated block, its down
    projection, the loss over the vocabulary; gradients of every matrix and of
    the input against 64-bit autograd, in norm: the chain's roundings (h, y,
    their gradients and the operands of the products: at most 8, half a step
    each) add up to at most 8 * 2^-8 of it."""
    M, K, N, V = 200, 96, 256, 1000
    g = torch.Generator("cuda").manual_seed(16)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    wg, wu = (torch.randn(N, K, generator=g, device="cuda").mul_(K ** -0.5).bfloat16() for _ in range(2))
    wd = torch.randn(K, N, generator=g, device="cuda").mul_(N ** -0.5).bfloat16()
    head = torch.randn(V, K, generator=g, device="cuda").mul_(K ** -0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    leaves = [v.clone().requires_grad_() for v in (x, wg, wu, wd, head)]
    h = layers.gated_ffn(leaves[0], leaves[1], leaves[2])
    loss = layers.linear_cross_entropy(leaves[0] + h @ leaves[3].t(), leaves[4], t)
    loss.backward()
    ref = [v.double().requires_grad_() for v in (x, wg, wu, wd, head)]
    a = ref[0] @ ref[1].T
    y = ref[0] + (torch.nn.functional.silu(a) * (ref[0] @ ref[2].T)) @ ref[3].T
    want = torch.nn.functional.cross_entropy(y @ ref[4].T, t)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 8 * 2.0 ** -8 * float(want.detach())
    for v, r in zip(leaves, ref):
        assert float((v.grad.double() - r.grad).norm()) <= 8 * 2.0 ** -8 * float(r.grad.norm())


def confident(M, V, K, dtype, first=0.0):
    """Tokens that are surer and surer of their target: 1 - p from 1e-2 down to below 1e-8 (z_t = `lean` and a
    spread of one; the other words' sum of exponentials is about V e^(1/2))."""
    g = torch.Generator("cuda").manual_seed(23)
    w = torch.randn(V, K, generator=g, device="cuda").mul_(K ** -0.5).to(dtype)
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    lean = torch.linspace(first or 12.0, 28.0, M, device="cuda")[:, None]
    x = (torch.randn(M, K, generator=g, device="cuda") + lean * w[t].float()).to(dtype)
    return x, w, t


def confident_bound(x, w, t, c):
    """dx in 64 bits and its bound, relative to 1 - p. With q_i = 1 - p_i,t and P' the computed P:

    z' - z <= e_z = (gamma_512 + 16 u) S: parts of at most 512 terms, added in FP32. Every word's P is off by at
    most a factor exp(2 e), e = max_v e_z + 2^-22 (1 + |lse|) (the logits' errors, those of the target's logit, the
    lse rounded to FP32); so is the target's own entry -q, which depends on differences of logits alone. Then the
    roundings: P to 16 bits (half a step; FP16's subnormal numbers 2^-25 / 2^14 of the largest c), the FP32 sum
    over V words, the result."""
    half, tiny = HALF[x.dtype], TINY[x.dtype]
    x, w = x.double(), w.double()
    z = x @ w.T
    e = ((gamma(512) + 16 * U) * (x.abs() @ w.abs().T)).amax(1) + 2.0 ** -22 * (1 + torch.logsumexp(z, 1).abs())
    others = z.scatter(1, t[:, None], -float("inf"))
    # log sum over the others less z_t: q / (1 - q) = exp(rest)
    rest = torch.logsumexp(others, 1) - z.gather(1, t[:, None])[:, 0]
    q = torch.sigmoid(rest)
    p = torch.exp(others - z.gather(1, t[:, None])) * torch.sigmoid(-rest)[:, None]
    P = c * p.scatter(1, t[:, None], -q[:, None])
    off = torch.expm1(2 * e)[:, None] + half * torch.exp(2 * e)[:, None]
    eP = P.abs() * off + (c * 2.0 ** -38 if half < 2.0 ** -8 else 0.0)
    dx = P @ w
    err = eP @ w.abs() + (gamma(w.shape[0]) + 2.0 ** -18) * ((P.abs() + eP) @ w.abs())
    return q, dx, err + half * (dx.abs() + err) + tiny


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", [(300, 4096), (100, 4096), (40, 1000)])
def test_gradients_of_confident_tokens(M, K, dtype):
    """The target's entry, p - 1, is right relative to itself however close p is to 1."""
    x, w, t = confident(M, 2000, K, dtype)
    c = 65536.0   # as a loss is scaled for FP16
    q, want, tol = confident_bound(x, w, t, c)
    assert float(q.min()) < 1e-8 and float(q.max()) > 1e-3
    leaf = x.clone().requires_grad_()
    layers.linear_cross_entropy(leaf, w, t, reduction="sum").mul(c).backward()
    # the bound says something: a few hundredths of a row's size, but for the tails of FP16's surest tokens
    sure = q > (1e-6 if dtype == torch.float16 else 0)
    assert bool((tol.norm(dim=1) < 0.05 * want.norm(dim=1))[sure].all())
    close(leaf.grad, want, tol)


@pytest.mark.parametrize("lean", [14.0, 19.5, 23.5, 27.0])
def test_the_gradient_of_one_confident_token(lean):
    """One row: its forward pass runs on the FP32 units, its backward pass on the tensor cores."""
    x, w, t = confident(1, 2000, 4096, torch.bfloat16, first=lean)
    q, want, tol = confident_bound(x, w, t, 1.0)
    leaf = x.clone().requires_grad_()
    layers.linear_cross_entropy(leaf, w, t).backward()
    close(leaf.grad, want, tol)


def test_losses_of_confident_tokens():
    """The loss itself is right relative to itself, down to 1e-8."""
    for M in (300, 100, 2, 1):
        x, w, t = confident(M, 2000, 4096, torch.bfloat16, first=20.0)
        q, _, _ = confident_bound(x, w, t, 1.0)
        z = x.double() @ w.double().T
        e = ((gamma(512) + 16 * U) * (x.double().abs() @ w.double().abs().T)).amax(1) + 2.0 ** -20
        loss = layers.linear_cross_entropy(x, w, t, reduction="none")
        want = -torch.log1p(-q)
        close(loss, want, torch.expm1(2 * e) * want)


def test_gradients_of_far_logits():
    """Logits of thousands: every word's share is as right as the differences of the logits are."""
    M, V, K = 300, 500, 4096
    x, w, t = inputs(M, V, K, torch.bfloat16, seed=24, ignored=0.0)
    x = (x.float() + 2000 * K ** -0.5).bfloat16()   # a direction that all words share
    w = (w.float() + K ** -0.5).bfloat16()
    q, want, tol = confident_bound(x, w, t, 1.0)
    leaf = x.clone().requires_grad_()
    layers.linear_cross_entropy(leaf, w, t, reduction="sum").backward()
    close(leaf.grad, want, tol)


@pytest.mark.parametrize("M", [1, 3, 100, 300])
def test_the_losses_given_or_computed_again_are_the_same(M):
    """The explicit backward pass without the losses per token computes them; autograd keeps them, whatever
    becomes of the result."""
    x, w, t = inputs(M, 900, 200, torch.bfloat16, seed=25)
    losses, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
    for reduction in ("none", "sum", "mean"):
        up = torch.linspace(0.5, 2, M, device="cuda") if reduction == "none" else torch.tensor(1.5, device="cuda")
        want = layers.linear_cross_entropy_backward(up, lse, x, w, t, reduction=reduction)
        strided = torch.stack([losses, losses], 1)[:, 0]
        for loss in (losses, strided):
            got = layers.linear_cross_entropy_backward(up, lse, x, w, t, reduction=reduction, loss=loss)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        leaves = [x.clone().requires_grad_(), w.clone().requires_grad_()]
        result = layers.linear_cross_entropy(*leaves, t, reduction=reduction)
        result.mul_(2)   # in place
        result.backward(up)
        want = layers.linear_cross_entropy_backward(2 * up, lse, x, w, t, reduction=reduction)
        assert all(torch.equal(a.grad, b) for a, b in zip(leaves, want))
    for bad in (losses.double(), losses[:0], losses.cpu()):
        with pytest.raises(ValueError, match="loss must be"):
            layers.linear_cross_entropy_backward(up, lse, x, w, t, loss=bad)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_an_infinite_gradient_stays_in_its_row(bad, dtype):
    x, w, t = inputs(300, 500, 64, dtype, seed=26)
    g = torch.Generator("cuda").manual_seed(2)
    grad = torch.randn(300, generator=g, device="cuda")
    _, lse = layers.linear_cross_entropy(x, w, t, return_lse=True)
    rows = (t != IGNORE).nonzero()[[0, 100], 0]
    zero, spoilt = grad.clone(), grad.clone()
    zero[rows], spoilt[rows] = 0.0, bad
    spoilt[t == IGNORE] = bad   # never looked at
    want, _ = layers.linear_cross_entropy_backward(zero, lse, x, w, t, reduction="none")
    dx, dw = layers.linear_cross_entropy_backward(spoilt, lse, x, w, t, reduction="none")
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(dx[keep], want[keep]) and not dx[t == IGNORE].any()
    assert not bool(dx[rows].isfinite().any()) and not bool(dw.isfinite().all())
    # one value for all tokens: nothing but ignored tokens is left
    for reduction in ("sum", "mean"):
        dx, _ = layers.linear_cross_entropy_backward(torch.tensor(bad, device="cuda"), lse, x, w, t, reduction=reduction)
        assert not dx[t == IGNORE].any() and not bool(dx[t != IGNORE].isfinite().any())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("V", [2, 500])
def test_the_entry_that_weighs_most_is_not_rounded(V, dtype):
    """One token: its target's row of dW is -(1 - p) c x, rounded once: P's scale is its largest entry."""
    K = 256
    g = torch.Generator("cuda").manual_seed(27)
    w = torch.randn(V, K, generator=g, device="cuda").mul_(K ** -0.5).to(dtype)
    for k, lean in enumerate(torch.linspace(0.0, 6.0, 12).tolist()):
        t = torch.tensor([k % V], device="cuda")
        x = (torch.randn(1, K, generator=g, device="cuda") + lean * w[t].float()).to(dtype)
        c = torch.tensor([0.37 + 0.11 * k], device="cuda")
        q, _, _ = confident_bound(x, w, t, float(c))
        # the logits' differences, then expm1, log1p and the scale in FP32
        rel = 2 * (gamma(256) + 16 * U) * float((x.double().abs() @ w.double().abs().T).max()) + 2.0 ** -18
        loss, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
        _, dw = layers.linear_cross_entropy_backward(c, lse, x, w, t, reduction="none", loss=loss)
        want = -q[:, None] * c.double() * x.double()
        close(dw[t], want, (HALF[dtype] * (1 + rel) + rel) * want.abs() + TINY[dtype])


def test_the_scale_of_p_stays_finite():
    """Tokens so sure that no entry of P is left (1 - p below 1e-38), alone and beside another one."""
    x, w, t = inputs(3, 40, 64, torch.bfloat16, seed=28, ignored=0.0)
    t[1] = t[2] = t[0]
    x[0] = x[1] = (200 * w[t[0]].float()).bfloat16()
    for rows in (slice(0, 1), slice(0, 2), slice(0, 3)):
        for dtype in TYPES:
            leaves = [v.detach().clone().to(dtype).requires_grad_() for v in (x[rows], w)]
            loss = layers.linear_cross_entropy(*leaves, t[rows], reduction="sum")
            loss.backward()
            ref = [v.detach().double().requires_grad_() for v in leaves]
            want = torch.nn.functional.cross_entropy(ref[0] @ ref[1].T, t[rows], reduction="sum")
            want.backward()
            for v, r in zip(leaves, ref):
                assert bool(v.grad.isfinite().all())
                # the third token's share is all there is: a chain of three roundings
                assert float((v.grad.double() - r.grad).norm()) <= 3 * HALF[dtype] * float(r.grad.norm()) + 1e-12


def test_no_tokens_and_a_padded_batch_through_autograd():
    x, w, t = inputs(24, 70, 32, torch.bfloat16, seed=29, ignored=0.0)
    for reduction in ("none", "mean", "sum"):
        leaves = [x[:0].clone().requires_grad_(), w.clone().requires_grad_()]
        layers.linear_cross_entropy(*leaves, t[:0], reduction=reduction).sum().backward()
        assert leaves[0].grad.shape == (0, 32) and not leaves[1].grad.any()
    # sequences of 8, 3 and 0 tokens padded to 8: the same as their tokens alone
    keep = torch.arange(8, device="cuda") < torch.tensor([[8], [3], [0]], device="cuda")
    pad = torch.where(keep.view(-1, 1), x, float("nan")).view(3, 8, 32)
    one = [pad.clone().requires_grad_(), w.clone().requires_grad_()]
    two = [x[keep.view(-1)].clone().requires_grad_(), w.clone().requires_grad_()]
    a = layers.linear_cross_entropy(*one, torch.where(keep, t.view(3, 8), IGNORE))
    b = layers.linear_cross_entropy(*two, t[keep.view(-1)])
    assert abs(float(a.detach()) - float(b.detach())) <= 2.0 ** -20 * float(b.detach())
    a.backward()
    b.backward()
    assert not one[0].grad[~keep].any()
    # the same entries, but in another place of the contraction over tokens
    e = Exact(two[0].detach(), w, t[keep.view(-1)], torch.full((11,), 1 / 11, device="cuda"))
    close(one[0].grad[keep], e.dx, e.dx_tol)
    close(one[1].grad, e.dw, e.dw_tol)


def test_two_graphs_replayed_in_turn():
    """Each with its own workspace: a step of one between two of the other changes nothing."""
    graphs, outs, wants = [], [], []
    grad = torch.ones((), device="cuda")
    for seed in (30, 31):
        x, w, t = inputs(300, 600, 128, torch.bfloat16, seed=seed)
        losses, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
        wants.append((losses, *layers.linear_cross_entropy_backward(grad, lse, x, w, t)))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            losses, lse = layers.linear_cross_entropy(x, w, t, reduction="none", return_lse=True)
            given = layers.linear_cross_entropy_backward(grad, lse, x, w, t, loss=losses)
            again = layers.linear_cross_entropy_backward(grad, lse, x, w, t)
        graphs.append((graph, x, w, t))
        outs.append((losses, *given, *again))
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, wants):
            assert torch.equal(got[0], want[0])
            assert all(torch.equal(g, r) for g, r in zip(got[1:], (*want[1:], *want[1:])))
