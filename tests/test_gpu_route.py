"""Routing from logits, its gradient, and the layer with a given routing, against plain float64 forms.

Tolerances. Indices are compared exactly: the library decides from 64-bit keys where 32 bits cannot. Weights: a
score is a few correctly rounded or 1-2 ulp fp32 operations (exp, log1p, divide, sqrt; at most 8 of them), the
softmax argument z - max adds |z - max| 2^-24 with |z - max| < 16 here, and the sum of at most 512 terms in a tree
9 more: below 40 * 2^-24 relative. Gradients are differences of such terms: 64 * 2^-24 of the row's largest
|scale * g * p|, which bounds every factor, plus the rounding of a 16-bit result.
"""
import numpy as np
import pytest
import torch

import routed_expert_ffn_sqrtsoftplus_b200 as moe
from routed_expert_ffn_sqrtsoftplus_b200 import build, synth

import fp4_ref as ref
import parity

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TOL_W = 40 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    build.build()


def _logits(T, E, dtype, seed, off=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((T, E + pad), generator=g) * 1.5
    if off:
        z[:, torch.randperm(E, generator=g)[:off]] = -float("inf")
    return z.to(DT[dtype]).cuda()[:, :E]


def _check(z, k, kind, bias=None, G=1, kept=1, group="top2", renorm=True, scale=1.0):
    idx, w = moe.route(z, k, score=kind, bias=bias, n_groups=G, topk_groups=kept, group_score=group,
                       renormalize=renorm, route_scale=scale)
    ri, rw = ref.route(z.double().cpu().numpy(), k, kind, None if bias is None else bias.cpu().numpy(), G, kept, group,
                       renorm, scale)
    assert np.array_equal(idx.cpu().numpy(), ri)
    err = np.abs(w.cpu().numpy() - rw)
    assert (err <= TOL_W * np.abs(rw)).all(), (err / np.maximum(np.abs(rw), 1e-30)).max()
    return idx, w


@pytest.mark.parametrize("kind", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 2), (7, 32, 32), (33, 128, 3), (65, 130, 8), (32, 384, 6), (9, 512, 16)])
def test_route_plain(kind, dtype, T, E, k):
    for renorm in (True, False):
        _check(_logits(T, E, dtype, T * 7 + E), k, kind, renorm=renorm, scale=1.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("G,kept,E", [(8, 4, 256), (4, 1, 64), (2, 2, 50), (5, 3, 35), (32, 7, 32), (8, 3, 384), (3, 2, 513 // 3 * 3 - 3)])
@pytest.mark.parametrize("group", ["top2", "max"])
def test_route_groups(kind, G, kept, E, group):
    g = torch.Generator().manual_seed(E + G)
    bias = (torch.randn(E, generator=g) * 0.1).cuda()
    k = min(6, kept * (E // G))
    for dtype in ("fp32", "bf16"):
        z = _logits(21, E, dtype, G * 31 + E, off=min(3, E // 8))
        _check(z, k, kind, bias, G, kept, group, scale=2.5)
        _check(z, k, kind, None, G, kept, group, renorm=False)


def test_route_near_ties_are_decided_as_in_64_bits():
    # keys that 32 bits cannot separate: sigmoid(z) + b with b undoing the score up to a few units of 2^-30
    E, T = 64, 40
    g = torch.Generator().manual_seed(5)
    z = torch.randn((T, E), generator=g)
    z[:] = z[0]
    s = torch.sigmoid(z[0].double())
    bias = (0.5 - s).float().cuda()       # every key is 0.5 up to the rounding of the bias
    for kind, G, kept in (("sigmoid", 1, 1), ("sigmoid", 8, 4)):
        _check(z.cuda(), 7, kind, bias, G, kept)


@pytest.mark.parametrize("k", [1, 8, 16, 17, 31, 32])
def test_route_near_tie_at_the_last_slot(k):
    # keys 0.01 apart, but for the last taken and the first left out: those are equal up to the bias' rounding
    E = 48
    g = torch.Generator().manual_seed(k)
    for _ in range(24):
        z = torch.randn((1, E), generator=g)
        want = 1.0 - 0.01 * torch.arange(E).double()
        want[k] = want[k - 1]
        order = torch.randperm(E, generator=g)
        bias = torch.empty(E)
        bias[order] = (want - torch.sigmoid(z[0, order].double())).float()
        _check(z.cuda(), k, "sigmoid", bias.cuda())


def test_route_groups_whose_two_keys_cancel():
    # keys near +-1000: a worth of about 1, of terms that 32 bits round to 2^-14
    g = torch.Generator().manual_seed(11)
    for Eg in (2, 3, 8):
        E = 8 * Eg
        z = 0.3 + 2e-5 * torch.randn((40, E), generator=g)
        bias = torch.full((E,), -2000.0)
        bias[0::Eg], bias[1::Eg] = 1000.0, -1000.0
        _check(z.cuda(), 3, "sigmoid", bias.cuda(), 8, 3)


def test_route_bias_of_the_lowest_value():
    # two lowest values add to -infinity in 32 bits, but their group is not an empty one
    z = torch.randn((5, 24), generator=torch.Generator().manual_seed(12))
    z[:, :8] = -float("inf")
    bias = torch.zeros(24)
    bias[8:16] = torch.finfo(torch.float32).min
    for group in ("top2", "max"):
        idx, _ = _check(z.cuda(), 10, "sigmoid", bias.cuda(), 3, 2, group)
        assert bool((idx[:, 8:].cpu() == torch.tensor([8, 9], dtype=torch.int32)).all())


@pytest.mark.parametrize("E,G", [(200, 8), (100, 4), (480, 5), (512, 8), (64, 2)])
def test_route_rows_that_64_bit_keys_decide(E, G):
    """Every row is full of near ties, next to rows that are not: groups of whole lanes and others."""
    g = torch.Generator().manual_seed(E)
    z = torch.randn((64, E), generator=g)
    z[::2] = z[0]
    bias = (0.5 - torch.sigmoid(z[0].double())).float().cuda()
    for kind in ("sigmoid", "softmax"):
        _check(z.cuda(), 8, kind, bias, G, G // 2)


def test_route_saturated_scores_keep_the_order_of_their_logits():
    # sigmoid is 1 in 64 bits too: every group is worth the same, the logits still decide inside
    z = 40.0 + torch.randperm(64, generator=torch.Generator().manual_seed(13)).float()[None].repeat(3, 1) / 8
    idx, w = moe.route(z.cuda(), 6, score="sigmoid", n_groups=8, topk_groups=4)
    want = torch.argsort(z[0, :32], descending=True)[:6].int()
    assert bool((idx.cpu() == want).all()) and float((w - 1 / 6).abs().max()) <= TOL_W


def test_route_exact_ties_take_the_lower_expert():
    z = torch.zeros((4, 96), device="cuda")
    z[1, 50:] = 1.0
    z[2] = -0.0
    z[3, ::3] = 2.0
    for kind in ("softmax", "sigmoid", "sqrtsoftplus"):
        _check(z, 5, kind)
        _check(z, 5, kind, torch.zeros(96, device="cuda"), 4, 2)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid", "sqrtsoftplus"])
def test_route_extreme_logits(kind):
    low = torch.finfo(torch.float32).min
    z = torch.randn((6, 16), generator=torch.Generator().manual_seed(1))
    z[0] = -float("inf")                        # nothing is left
    z[1] = -float("inf")
    z[1, 9] = -50.0                             # one expert is left, and it is far down
    z[2] = low                                  # the type's lowest value is not an infinity
    z[3, 1:] = -float("inf")
    z[4] -= 300.0                               # scores that underflow before they are renormalised
    z = z.cuda()
    idx, w = moe.route(z, 4, score=kind)
    assert idx[0].tolist() == [-1] * 4 and w[0].tolist() == [0.0] * 4
    assert idx[1].tolist() == [9, -1, -1, -1] and w[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert idx[2].tolist() == [0, 1, 2, 3] and w[2].tolist() == [0.25] * 4
    assert idx[3].tolist() == [0, -1, -1, -1] and w[3].tolist() == [1.0, 0.0, 0.0, 0.0]
    zs = z[4].double().cpu().numpy()
    order = np.argsort(-zs, kind="stable")[:4]
    assert idx[4].tolist() == order.tolist()
    p = np.exp((zs[order] - zs[order].max()) * (0.5 if kind == "sqrtsoftplus" else 1.0))
    assert np.abs(w[4].cpu().numpy() - p / p.sum()).max() <= TOL_W
    _check(z[5:], 4, kind)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_route_rows_that_are_not_finite(bad):
    z = torch.randn((5, 40), generator=torch.Generator().manual_seed(2)).cuda()
    z[3, 17] = bad
    idx, w = moe.route(z, 6, score="sigmoid", bias=torch.zeros(40, device="cuda"), n_groups=4, topk_groups=2)
    assert idx[3].tolist() == [0, 1, 2, 3, 4, 5] and bool(torch.isnan(w[3]).all())
    keep = [0, 1, 2, 4]
    ri, _ = ref.route(z[keep].double().cpu().numpy(), 6, "sigmoid", np.zeros(40), 4, 2)
    assert np.array_equal(idx[keep].cpu().numpy(), ri)
    b = torch.zeros(40, device="cuda")
    b[2] = float("nan")
    idx, w = moe.route(z[:2], 3, score="sigmoid", bias=b)
    assert idx.tolist() == [[0, 1, 2]] * 2 and bool(torch.isnan(w).all())


def test_route_strided_rows_and_given_outputs():
    for dtype in DT:
        z = _logits(11, 60, dtype, 9, pad=7)
        assert z.stride(0) == 67
        i1, w1 = _check(z, 5, "softmax")
        i2, w2 = torch.full((11, 5), 77, dtype=torch.int32, device="cuda"), torch.full((11, 5), 7.0, device="cuda")
        moe.route(z, 5, score="softmax", topk_idx=i2, topk_w=w2)
        assert torch.equal(i1, i2) and torch.equal(w1, w2)
    i, w = moe.route(torch.empty((0, 60), device="cuda"), 5)
    assert i.shape == (0, 5) and w.shape == (0, 5)


def _grad_ref(z, idx, g, kind, renorm, scale):
    """The formula of the gradient in float64, row by row."""
    s = ref.score(z, kind)
    out = np.zeros_like(z)
    for t in range(z.shape[0]):
        sel = [(r, e) for r, e in enumerate(idx[t]) if 0 <= e < z.shape[1]]
        S = sum(s[t, e] for _, e in sel) if renorm else 1.0
        if not sel:
            continue
        gbar = sum(g[t, r] * s[t, e] for r, e in sel) / S if renorm else 0.0
        ds = np.zeros(z.shape[1])
        for r, e in sel:
            ds[e] += scale * (g[t, r] - gbar) / S
        if kind == "softmax":
            out[t] = s[t] * (ds - (ds * s[t]).sum())
        elif kind == "sigmoid":
            out[t] = ds * s[t] * (1 - s[t])
        else:
            with np.errstate(all="ignore"):
                out[t] = np.where(s[t] > 0, ds / (1 + np.exp(-z[t])) / (2 * s[t]), 0.0)
    return out


@pytest.mark.parametrize("kind", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 2), (17, 128, 3), (9, 131, 8), (6, 384, 6), (3, 512, 32)])
def test_route_backward(kind, renorm, dtype, T, E, k):
    z = _logits(T, E, dtype, T + E, off=1 if E > 8 else 0, pad=3)
    idx, _ = moe.route(z, k, score=kind, renormalize=renorm, route_scale=1.5)
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(k)).cuda()
    got = moe.route_backward(g, z, idx, score=kind, renormalize=renorm, route_scale=1.5)
    assert got.dtype == z.dtype and got.shape == (T, E)
    zd, gd = z.double().cpu().numpy(), g.double().cpu().numpy()
    want = _grad_ref(zd, idx.cpu().numpy(), gd, kind, renorm, 1.5)
    step = torch.finfo(z.dtype).eps / 2
    bound = 1.5 * np.abs(gd).sum(1, keepdims=True) * 64 * 2.0 ** -24 + step * np.abs(want) * 1.01
    if dtype == "fp16":
        bound = bound + 2.0 ** -25   # fp16's subnormal step
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound).all(), (err / bound).max()
    # against central differences of the weights (step h: error h^2 from the third derivative, 2^-52 / h from rounding)
    h = 1e-5
    for t in range(min(T, 3)):
        for e in list(idx[t].tolist())[:2] + [E - 1]:
            if e < 0 or np.isneginf(zd[t, e]):
                continue
            d = []
            for sgn in (1, -1):
                zz = zd[t:t + 1].copy()
                zz[0, e] += sgn * h
                d.append((ref.route_weights(zz, idx[t:t + 1].cpu().numpy(), kind, renorm, 1.5) * gd[t:t + 1]).sum())
            assert abs((d[0] - d[1]) / (2 * h) - want[t, e]) <= 1e-8 * (1 + np.abs(gd[t]).sum())


def test_route_backward_odd_selections():
    z = _logits(4, 50, "fp32", 3)
    z[2] = -float("inf")
    idx = torch.tensor([[4, 4, 7], [-1, 3, -1], [-1, -1, -1], [50, 1, -9]], dtype=torch.int32).cuda()
    g = torch.randn((4, 3), generator=torch.Generator().manual_seed(4)).cuda()
    for kind in ("softmax", "sigmoid", "sqrtsoftplus"):
        for renorm in (True, False):
            got = moe.route_backward(g, z, idx, score=kind, renormalize=renorm).double().cpu().numpy()
            zz = z.double().cpu().numpy()
            want = _grad_ref(zz, idx.cpu().numpy(), g.double().cpu().numpy(), kind, renorm, 1.0)
            want[2] = 0.0
            assert np.abs(got - want).max() <= 64 * 2.0 ** -24 * float(g.abs().sum())
            assert (got[2] == 0).all()


def test_route_on_another_stream_and_in_a_graph():
    z = _logits(200, 96, "fp32", 6)
    i0, w0 = moe.route(z, 6, score="sigmoid")
    g = torch.ones_like(w0)
    d0 = moe.route_backward(g, z, i0, score="sigmoid")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    i1, w1 = moe.route(z, 6, score="sigmoid", stream=s)
    d1 = moe.route_backward(g, z, i1, score="sigmoid", stream=s)
    s.synchronize()
    assert torch.equal(i0, i1) and torch.equal(w0, w1) and torch.equal(d0, d1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i2, w2 = moe.route(z, 6, score="sigmoid")
        d2 = moe.route_backward(g, z, i2, score="sigmoid")
    z.copy_(_logits(200, 96, "fp32", 8))
    graph.replay()
    torch.cuda.synchronize()
    i3, w3 = moe.route(z, 6, score="sigmoid")
    assert torch.equal(i2, i3) and torch.equal(w2, w3)
    assert torch.equal(d2, moe.route_backward(g, z, i3, score="sigmoid"))


# ------------------------------------------------------------------ the layer with a given routing
WL = synth.WORKLOADS["tiny"]


@pytest.fixture(scope="module")
def tiny(cuda_device):
    lay = {k: (v.to(cuda_device) if isinstance(v, torch.Tensor) else v)
           for k, v in synth.make_layer(WL.with_tokens(700)).items()}
    layer = moe.MoELayer.from_layer(lay, top_k=WL.k, max_tokens=700)
    yield lay, layer
    layer.close()


@pytest.mark.parametrize("T", [1, 20, 64, 300, 700])
def test_forward_routed_with_the_layers_own_routing(tiny, T):
    lay, layer = tiny
    x = lay["x"][:T].contiguous()
    y, idx, w = layer.forward_with_routing(x)
    assert torch.equal(y, layer.forward_routed(x, idx, w))
    assert layer.status() == moe.MOE_OK


@pytest.mark.parametrize("T", [5, 300])
def test_forward_routed_with_route(tiny, T):
    """route -> the experts' products, as a model with another router runs them: empty slots included."""
    lay, layer = tiny
    x = lay["x"][:T].contiguous()
    z = x.float() @ lay["wg"].float().t()
    z[:, 3] = -float("inf")
    z[2, 2:] = -float("inf")              # this token finds two experts
    z[4] = -float("inf")                  # and this one none
    idx, w = moe.route(z, WL.k, score="sigmoid", bias=torch.linspace(-0.2, 0.2, WL.E, device="cuda"), n_groups=4,
                       topk_groups=3, route_scale=2.5)
    assert idx[2].tolist()[2:] == [-1] * (WL.k - 2) and idx[4].tolist() == [-1] * WL.k
    y = layer.forward_routed(x, idx, w)
    assert layer.status() == moe.MOE_OK
    # expert by expert in float64
    f = lambda w1, w3, w2, v: w2 @ (_silu(np.minimum(w1 @ v, 10.0)) * np.clip(w3 @ v, -10.0, 10.0))  # noqa: E731
    d = {n: parity.f64(lay[n]) for n in ("w1", "w3", "w2", "sh_w1", "sh_w3", "sh_w2")}
    for t in [0, 2, 4, T - 1]:
        v = parity.f64(x[t])
        want = f(d["sh_w1"][0], d["sh_w3"][0], d["sh_w2"][0], v)
        for e, we in zip(idx[t].tolist(), w[t].tolist()):
            if e >= 0:
                want = want + we * f(d["w1"][e], d["w3"][e], d["w2"][e], v)
        err = np.abs(y[t].double().cpu().numpy() - want)
        # parity's bound: h and y rounded to BF16
        assert (err <= parity.TOL_Y * np.sqrt((want ** 2).mean()) + 2.0 ** -8 * np.abs(want)).all()


def _silu(v):
    return v / (1 + np.exp(-v))


def test_forward_routed_bad_indices(tiny):
    lay, layer = tiny
    x = lay["x"][:40].contiguous()
    y0, idx, w = layer.forward_with_routing(x)
    idx[7, 2] = WL.E
    idx[9, 0] = -2
    y = layer.forward_routed(x, idx, w)
    assert layer.status() == moe.MOE_ERR_DEVICE
    assert bool(torch.isnan(y[7]).all()) and bool(torch.isnan(y[9]).all())
    keep = [t for t in range(40) if t not in (7, 9)]
    assert torch.equal(y[keep], y0[keep])
    with pytest.raises(ValueError):
        layer.forward_routed(x, idx[:, :3].contiguous(), w)
    with pytest.raises(ValueError):
        layer.forward_routed(x, idx.long(), w)


def _cancelling_rows(level, T, E, seed):
    """Logits about `level` whose sqrtsoftplus scores a bias takes back to keys of some 1e-5."""
    g = torch.Generator().manual_seed(seed)
    z0 = level * (0.8 + 0.4 * torch.rand(E, generator=g).double())
    bias = (-torch.sqrt(torch.nn.functional.softplus(z0))).float()
    want = -bias.double() + 1e-5 * torch.randn((T, E), generator=g).double()   # the score: key + |bias|
    return torch.log(torch.expm1(want ** 2)).where(want ** 2 < 30, want ** 2).float(), bias


@pytest.mark.parametrize("level", [1.0, 300.0, 1500.0, 1e4])
@pytest.mark.parametrize("E,k", [(8, 2), (16, 3), (64, 1), (64, 8), (200, 12), (512, 32)])
def test_route_sqrtsoftplus_scores_that_a_bias_cancels(level, E, k):
    """A score's 32-bit error goes with the score, not with the small key that the bias leaves of it."""
    z, bias = _cancelling_rows(level, 60 if E > 16 else 400, E, E + k)
    z[1::3] += 0.5 * torch.randn(z[1::3].shape, generator=torch.Generator().manual_seed(k))  # next to ordinary rows
    for G, kept, group in ((1, 1, "max"), (4, 2, "top2"), (4, 2, "max")):
        _check(z.cuda(), k, "sqrtsoftplus", bias.cuda(), G, kept, group)


def test_route_cancelled_scores_by_hand():
    # sqrt(1501.1384) - 38.744522 = 5.6187e-6 against 5.5007e-6, in 32 bits 3.8e-6 against 5.7e-6;
    # sqrt(1036.16) - 32.18944 = -1.888e-6 against -1.875e-6, in 32 bits 0 against -1.85e-6
    for z, b, first in (([1501.1384, 160.7942], [-38.744522, -12.680460], 0), ([1036.16, 0.0], [-32.18944, -0.8325565], 1)):
        idx, _ = _check(torch.tensor([z]).cuda(), 1, "sqrtsoftplus", torch.tensor(b).cuda())
        assert idx.item() == first


@pytest.mark.parametrize("k", [9, 12, 16, 17, 32])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid", "sqrtsoftplus"])
def test_route_many_slots_groups_and_bias(kind, k):
    g = torch.Generator().manual_seed(k)
    for E, G, kept in ((512, 8, 4), (512, 8, 1), (480, 5, 2), (256, 32, 9)):
        bias = (torch.randn(E, generator=g) * 0.1).cuda()
        for dtype in ("fp32", "bf16"):
            _check(_logits(33, E, dtype, E + k, off=5), k, kind, bias, G, kept)


@pytest.mark.parametrize("kind", ["sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_low_logits_without_renormalisation(kind, dtype):
    """Scores that are ordinary 32-bit numbers although e^z is not: sqrt(log(1 + e^z)) is e^-80 at z = -160."""
    z = -torch.linspace(15.0, 80.0 if kind == "sigmoid" else 160.0, 60).repeat(3, 1)
    z[1] = z[1].flip(0)
    z[2, 1::2] = -float("inf")
    z = z.to(DT[dtype]).cuda()
    _check(z, 12, kind, renorm=False, scale=1.5)
    far = z[:, -12:]                 # the lowest ones, as the only experts of their rows
    idx, w = _check(far, 12, kind, renorm=False, scale=1.5)
    g = torch.randn((3, 12), generator=torch.Generator().manual_seed(3)).cuda()
    got = moe.route_backward(g, far, idx, score=kind, renormalize=False, route_scale=1.5).double().cpu().numpy()
    want = _grad_ref(far.double().cpu().numpy(), idx.cpu().numpy(), g.double().cpu().numpy(), kind, False, 1.5)
    # one term an element: the bound is relative to itself
    assert (np.abs(got - want) <= (64 * 2.0 ** -24 + torch.finfo(DT[dtype]).eps / 2) * np.abs(want)).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_weights_carry_the_graph_of_their_logits(kind, renorm, dtype):
    z = _logits(19, 70, dtype, 21, off=2, pad=2).detach().clone().requires_grad_(True)
    bias = torch.linspace(-0.1, 0.1, 70).cuda().requires_grad_(True)
    kw = dict(score=kind, renormalize=renorm, route_scale=2.5)
    idx, w = moe.route(z, 6, bias=bias, n_groups=7, topk_groups=4, **kw)
    i0, w0 = moe.route(z.detach(), 6, bias=bias.detach(), n_groups=7, topk_groups=4, **kw)
    assert torch.equal(idx, i0) and torch.equal(w.detach(), w0) and not idx.requires_grad
    up = torch.randn((19, 6), generator=torch.Generator().manual_seed(5)).cuda()
    (w * up).sum().backward()
    assert torch.equal(z.grad, moe.route_backward(up, z.detach(), idx, **kw)) and bias.grad is None
    # an expanded gradient, and none at all
    z.grad = None
    idx, w = moe.route(z, 6, **kw)
    w.sum().backward()
    assert torch.equal(z.grad, moe.route_backward(torch.ones_like(up), z.detach(), idx, **kw))
    with torch.no_grad():
        assert not moe.route(z, 6, **kw)[1].requires_grad
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    idx, w = moe.route(z, 6, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(torch.autograd.grad(w.sum(), z)[0], z.grad)
    with pytest.raises(ValueError):
        moe.route(z, 6, topk_w=torch.empty((19, 6), device="cuda"), **kw)
    with pytest.raises(RuntimeError):   # its gradient has none of its own
        torch.autograd.grad(torch.autograd.grad(moe.route(z, 6, **kw)[1].sum(), z, create_graph=True)[0].sum(), z)


def test_route_and_its_gradient_in_a_captured_step():
    z = _logits(40, 64, "fp32", 22).detach().clone().requires_grad_(True)
    up = torch.randn((40, 4), generator=torch.Generator().manual_seed(6)).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, w = moe.route(z, 4, score="sigmoid")
        d = torch.autograd.grad(w, z, up)[0]
    with torch.no_grad():
        z.copy_(_logits(40, 64, "fp32", 23))
    graph.replay()
    torch.cuda.synchronize()
    i0, w0 = moe.route(z.detach(), 4, score="sigmoid")
    assert torch.equal(idx, i0) and torch.equal(w.detach(), w0)
    assert torch.equal(d, moe.route_backward(up, z.detach(), i0, score="sigmoid"))


def test_outputs_come_through_the_dispatcher_where_something_listens():
    """A dispatch mode sees the outputs' allocation, and under fake tensors they are fake."""
    from torch.utils._python_dispatch import TorchDispatchMode
    from torch._subclasses.fake_tensor import FakeTensor, FakeTensorMode

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.made = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if "empty" in str(func):
                self.made.append(out.data_ptr())
            return out

    z = _logits(5, 20, "fp32", 1)
    want = moe.route(z, 3)
    with Seen() as seen:
        idx, w = moe.route(z, 3)
    assert {idx.data_ptr(), w.data_ptr()} <= set(seen.made)
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    with FakeTensorMode():
        fake = torch.empty((5, 20), device="cuda")
        assert isinstance(moe._empty(fake, 5, 3, torch.int32), FakeTensor)
    torch.use_deterministic_algorithms(True)
    try:   # memory that nothing writes is filled there
        assert bool(torch.isnan(moe._empty(z, 4, 64, torch.float32)).all())
    finally:
        torch.use_deterministic_algorithms(False)


# ------------------------------------------------------------------ given routings of every kind of layer
@pytest.fixture(scope="module", params=["bf16", "mxfp4", "mxfp8"])
def any_layer(request, cuda_device):
    """(layer, its experts' float64 matrices, whether rows meet them in MXFP8)."""
    from oracle import mx as omx
    lay = synth.make_layer(WL.with_tokens(400), device="cpu")
    q, fmt = None, request.param
    if fmt != "bf16":
        quant = omx.quantize_mxfp4_packed if fmt == "mxfp4" else omx.quantize_mxfp8
        q = {}
        for n, s in (("w1", "s1"), ("w3", "s3"), ("w2", "s2")):
            q[n], q[s] = (torch.from_numpy(np.ascontiguousarray(v)) for v in quant(parity.f64(lay[n])))
    dev = {k: (v.to(cuda_device) if isinstance(v, torch.Tensor) else v) for k, v in lay.items()}
    layer = moe.MoELayer.from_layer(dev, top_k=WL.k, max_tokens=400,
                                    **({} if q is None else {"mx": {n: v.to(cuda_device) for n, v in q.items()}}))
    yield dev["x"], layer, parity.LayerExperts(lay, q)
    layer.close()


def _routed_ref(x, ex, idx, w):
    from oracle import moe as om
    y = np.zeros(x.shape)
    for j in range(ex.n_shared):
        y += om.expert_forward(x, *ex.shared(j), WL.swiglu_limit)[0]
    for e in range(ex.n_routed):
        t, r = np.nonzero(idx == e)
        if len(t):
            o, _ = om.expert_forward(x[t], *ex.routed(e), WL.swiglu_limit, mx_act=ex.routed_is_mx)
            np.add.at(y, t, o * w[t, r][:, None])
    return y


@pytest.mark.parametrize("T", [1, 7, 32, 33, 70, 400])
@pytest.mark.parametrize("how", ["holes", "twice", "one expert", "empty"])
def test_forward_routed_of_every_layer(any_layer, T, how):
    """Empty slots, rows without any expert, experts named twice by a token, every slot the same expert, no expert."""
    xs, layer, ex = any_layer
    x = xs[:T].contiguous()
    g = torch.Generator().manual_seed(T)
    idx = torch.argsort(torch.rand((T, WL.E), generator=g), 1)[:, :WL.k].int()
    w = torch.rand((T, WL.k), generator=g) + 0.1
    if how == "holes":
        idx[torch.rand(idx.shape, generator=g) < 0.4] = -1
        idx[T // 2] = -1
    elif how == "twice":
        idx[::2, 1] = idx[::2, 0]
        idx[T // 3] = 5
    else:
        idx[:] = 3 if how == "one expert" else -1
    y = layer.forward_routed(x, idx.cuda(), w.cuda())
    assert layer.status() == moe.MOE_OK
    want = _routed_ref(parity.f64(x.cpu()), ex, idx.numpy(), w.double().numpy())
    assert parity.output_score(y.double().cpu().numpy(), want) < parity.TOL_Y
