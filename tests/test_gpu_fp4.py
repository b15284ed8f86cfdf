"""Microscaled FP4 quantisation and products against plain float64 forms.

Quantisation is compared bit for bit: the rule decides every code exactly. Products: E2M1 x E2M1 with scales are
exact in the MMA up to its fp32 accumulation, K / 64 steps of at most two units of 2^-24 (it may truncate) of the
running sum, which stays below sum |x w|; then one rounding of the result to its type.
"""
import numpy as np
import pytest
import torch

import routed_expert_ffn_sqrtsoftplus_b200 as moe
from routed_expert_ffn_sqrtsoftplus_b200 import build

import fp4_ref as ref

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FMT = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    build.build()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _x(rows, K, dtype, seed):
    g = _gen(seed)
    x = torch.randn((rows, K), generator=g) * torch.exp(torch.randn((1, K), generator=g))
    if rows > 2:
        x[1] = 0.0
        x[2, :16] = 0.0
    return x.to(DT[dtype])


def _ts(x, fmt):
    return (x.abs().max().float() / 2688.0).reshape(1) if fmt == "nvfp4" else None


def _check_quant(x, fmt, ts=None):
    codes, scales = moe.quantize_fp4(x.cuda(), fmt, None if ts is None else ts.cuda())
    rc, rs, rv = ref.quantize(x.double().numpy(), fmt, None if ts is None else ts.item())
    assert np.array_equal(scales.cpu().numpy(), rs)
    diff = codes.cpu().numpy() != rc
    assert not diff.any(), (np.argwhere(diff)[:4], diff.sum())
    return codes, scales, rv


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (33, 96), (7, 2304), (130, 416)])
def test_quantize(fmt, dtype, rows, K):
    x = _x(rows, K, dtype, rows + K)
    for ts in ((None, _ts(x, fmt)) if fmt == "nvfp4" else (None,)):
        codes, scales, rv = _check_quant(x, fmt, ts)
        for out in DT.values():
            v = moe.dequantize_fp4(codes, scales, fmt, None if ts is None else ts.cuda(), dtype=out)
            want = torch.from_numpy(rv).float()           # e2m1 * d, one rounding to 32 bits
            # two roundings at most (32 bits, then the type); fp16 may be subnormal
            err = (v.cpu().double() - torch.from_numpy(rv)).abs()
            tiny = torch.finfo(out).smallest_normal * torch.finfo(out).eps
            top = torch.finfo(out).max
            ok = err <= want.abs().double() * (torch.finfo(out).eps / 2 + 2.0 ** -24) + tiny
            assert bool((ok | (want.abs() > top)).all())


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_borders(fmt):
    """Values on, and one step beside, every border of both grids."""
    rows = []
    for unit in (1.0, 0.75, 1.125, 2.0 ** -5, 208.0, 3.0 * 2.0 ** -7):
        b = []
        for e in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 3.0):
            v = np.float32(e * unit)
            b += [v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(1e9)), -v]
        b = b[:30] + [6.0 * unit, 0.0]
        rows.append(b)
        b = list(b)
        rows.append([6.0 * unit if i % 16 == 0 else v for i, v in enumerate(b)])
    x = torch.tensor(np.array(rows, dtype=np.float32))
    _check_quant(x, fmt)
    if fmt == "nvfp4":
        for t in (0.3, 1.0 / 3.0, 7e-4):
            ts = torch.tensor([t], dtype=torch.float32)
            _check_quant(x, fmt, ts)
            _check_quant((x * ts).float(), fmt, ts)
        # block maxima at and beside the borders of the scale's grid
        mids = (ref.E4M3[1:] + ref.E4M3[:-1]) / 2 * 6
        y = torch.zeros((len(mids) * 3, 32))
        for i, m in enumerate(mids.astype(np.float32)):
            for j, v in enumerate((m, np.nextafter(m, np.float32(0)), np.nextafter(m, np.float32(1e9)))):
                y[3 * i + j, 3] = float(v)
                y[3 * i + j, 20] = -float(v) / 3
        _check_quant(y, fmt)
        _check_quant(y, fmt, torch.tensor([0.3]))


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_matches_the_weight_quantiser_and_strides(fmt):
    x = _x(9, 128, "bf16", 4).cuda()
    if fmt == "mxfp4":
        c0, s0 = moe.quantize_mxfp4(x)
        c1, s1 = moe.quantize_fp4(x, fmt)
        assert torch.equal(c0, c1) and torch.equal(s0, s1)
    wide = torch.randn((9, 131), generator=_gen(3)).cuda()
    for dtype in DT.values():
        v = wide.to(dtype)[:, 1:129]
        a, b = moe.quantize_fp4(v, fmt), moe.quantize_fp4(v.contiguous(), fmt)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c, s = moe.quantize_fp4(torch.empty((0, 64), device="cuda"), fmt)
    assert c.shape == (0, 32) and moe.dequantize_fp4(c, s, fmt).shape == (0, 64)


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_not_finite_and_extreme(fmt):
    x = torch.randn((3, 96), generator=_gen(8))
    x[0, 5] = float("nan")
    x[1, 40] = -float("inf")
    codes, scales = moe.quantize_fp4(x.cuda(), fmt)
    v = moe.dequantize_fp4(codes, scales, fmt, dtype=torch.float32).cpu()
    bs = ref.BLOCK[fmt]
    bad = torch.zeros((3, 96 // bs), dtype=torch.bool)
    bad[0, 5 // bs] = bad[1, 40 // bs] = True
    assert torch.equal(torch.isnan(v).view(3, -1, bs).all(2), bad) and torch.equal(torch.isnan(v).view(3, -1, bs).any(2), bad)
    big = torch.full((2, 64), torch.finfo(torch.float32).max)
    big[1] = torch.finfo(torch.float32).smallest_normal / 8
    _check_quant(big, fmt)


@pytest.mark.parametrize("ts", [3.0e38, 1.0e38, 2.0 ** 61, 1.7e-18, 1.1e-30, 2.0 ** -118, 1.3e-38, 1e-41, 2.0 ** -149])
def test_quantize_far_tensor_scales(ts):
    # blocks whose scales run from 0 over the subnormal ones to the largest, where the values exist in 32 bits
    g = _gen(17)
    ts = torch.tensor([ts], dtype=torch.float32)
    rows = []
    for e in range(-14, 13):
        amax = ts.double() * 2.0 ** e * (1 + torch.rand(1, generator=g).double())
        rows.append((torch.rand(64, generator=g).double() * 2 - 1) * amax)
    x = torch.stack(rows).clamp(-3.0e38, 3.0e38).float()
    codes, scales = moe.quantize_fp4(x.cuda(), "nvfp4", ts.cuda())
    rc, rs, _ = ref.quantize(x.double().numpy(), "nvfp4", ts.item())
    assert np.array_equal(scales.cpu().numpy(), rs)
    unit = (ref.E4M3[rs].astype(np.float32) * np.float32(ts.item())).repeat(8, 1)
    rc = np.where(unit >= np.finfo(np.float32).tiny, rc, 0)     # a unit below the normal range: zeros
    assert np.array_equal(codes.cpu().numpy(), rc)


# ------------------------------------------------------------------ products
def _weights(E, N, K, fmt, seed):
    w = torch.randn((E * N, K), generator=_gen(seed)) / K ** 0.5
    ts = None
    if fmt == "nvfp4":
        ts = torch.linspace(0.5, 2.0, E).float()
    codes, scales, _ = ref.quantize(w.double().numpy(), fmt)
    return (torch.from_numpy(codes).view(E, N, K // 2).cuda(), torch.from_numpy(scales).view(E, N, -1).cuda(),
            None if ts is None else ts.cuda())


def _bound(xv, wv, want, out):
    K = xv.shape[1]
    mag = np.abs(xv) @ np.abs(wv).T
    eps = torch.finfo(out).eps / 2
    return mag * (K / 64 + 4) * 2 * 2.0 ** -24 + np.abs(want) * eps * 1.01 + (2.0 ** -25 if out == torch.float16 else 0)


def _check_matmul(T, N, K, fmt, out=torch.bfloat16, seed=0):
    x = _x(T, K, "bf16", seed + 1)
    xts = _ts(x, fmt)
    xc, xs, _ = ref.quantize(x.double().numpy(), fmt, None if xts is None else xts.item())
    w, ws, wts = _weights(1, N, K, fmt, seed + 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(x_tensor_scale=None if xts is None else xts.cuda(), w_tensor_scale=wts)
    y = moe.fp4_matmul(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), w[0], ws[0], fmt, out_dtype=out,
                       status=status, **kw)
    xv = ref.values(xc, xs, fmt, None if xts is None else xts.numpy())
    wv = ref.values(w[0].cpu().numpy(), ws[0].cpu().numpy(), fmt, None if wts is None else wts.cpu().numpy()[0])
    want = xv @ wv.T
    assert status.item() == 0
    err = np.abs(y.double().cpu().numpy() - want)
    b = _bound(xv, wv, want, out)
    assert (err <= b).all(), (np.argwhere(err > b)[:5], (err / np.maximum(b, 1e-300)).max())
    z = moe.fp4_linear(x.cuda(), w[0], ws[0], fmt, out=torch.empty_like(y), **kw)
    assert torch.equal(y, z)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 128, 256), (16, 128, 512), (3, 200, 96), (17, 130, 288), (32, 384, 1024),
                                   (5, 4608, 5120), (1, 640, 2304)])
def test_matmul_few_tokens(fmt, T, N, K):
    _check_matmul(T, N, K, fmt)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,N,K", [(33, 256, 256), (64, 100, 320), (96, 1000, 1312), (97, 256, 512), (192, 512, 768),
                                   (193, 300, 800), (500, 700, 2080), (1024, 2304, 512),
                                   (515, 1001, 288), (777, 200, 96)])
def test_matmul_many_tokens(fmt, T, N, K):
    _check_matmul(T, N, K, fmt)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
def test_matmul_output_types(fmt, out):
    for T in (7, 70, 210, 530):
        _check_matmul(T, 333, 544, fmt, out)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,N,K,sizes,pad", [
    (4, 128, 256, [3, 0, 40, 1], 0), (1, 64, 64, [5], 3), (7, 300, 512, [0, 0, 1, 0, 200, 33, 0], 9),
    (64, 130, 288, [i % 5 for i in range(64)], 2), (40, 256, 320, [(7 * i) % 11 * 9 for i in range(40)], 0),
    (3, 512, 256, [0, 0, 0], 4), (512, 32, 64, [1 if i % 3 else 0 for i in range(512)], 1)])
def test_experts(fmt, E, N, K, sizes, pad):
    T = sum(sizes) + pad
    x = _x(T, K, "bf16", E + N)
    xts = _ts(x, fmt)
    w, ws, wts = _weights(E, N, K, fmt, E)
    off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32).cuda()
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.fp4_linear(x.cuda(), w, ws, fmt, x_tensor_scale=None if xts is None else xts.cuda(), w_tensor_scale=wts,
                   offsets=off, out=y)
    _, _, xv = ref.quantize(x.double().numpy(), fmt, None if xts is None else xts.item())
    got = y.double().cpu().numpy()
    assert (got[T - pad:] == 7.0).all()          # rows behind the last expert's stay as they were
    for g in range(E):
        a, b = int(off[g]), int(off[g + 1])
        if a == b:
            continue
        wv = ref.values(w[g].cpu().numpy(), ws[g].cpu().numpy(), fmt, None if wts is None else wts.cpu().numpy()[g])
        want = xv[a:b] @ wv.T
        assert (np.abs(got[a:b] - want) <= _bound(xv[a:b], wv, want, torch.bfloat16)).all(), g


def test_experts_offsets_are_clamped():
    """Offsets out of range or out of order lead nowhere outside x and y: such experts have fewer rows, or none."""
    E, N, K, T = 4, 64, 64, 50
    x = _x(T, K, "bf16", 1).cuda()
    w, ws, _ = _weights(E, N, K, "mxfp4", 2)
    for bad, good in (([0, 20, 10, 30, 50], [0, 20, 20, 30, 50]), ([-5, 7, 9, 1000, 2000], [0, 7, 9, 50, 50]),
                      ([10, 20, 30, 40, 45], [10, 20, 30, 40, 45])):
        ya, yb = (torch.full((T, N), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        moe.fp4_linear(x, w, ws, "mxfp4", offsets=torch.tensor(bad, dtype=torch.int32).cuda(), out=ya)
        moe.fp4_linear(x, w, ws, "mxfp4", offsets=torch.tensor(good, dtype=torch.int32).cuda(), out=yb)
        assert torch.equal(ya, yb)
        assert bool((ya[:good[0]] == 3.0).all()) and bool((ya[good[-1]:] == 3.0).all())


@pytest.mark.parametrize("fmt", FMT)
def test_matmul_nan_stays_in_its_row(fmt):
    x = _x(40, 96, "bf16", 2)
    x[7, 3] = float("nan")
    x[33] = float("inf")
    w, ws, wts = _weights(1, 150, 96, fmt, 3)
    y = moe.fp4_linear(x.cuda(), w[0], ws[0], fmt)
    bad = torch.isnan(y).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 33] and not bool(torch.isnan(y[~bad]).any())


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("K", [96, 288, 512])
@pytest.mark.parametrize("T", [5, 300])
def test_weight_scales_at_any_address(fmt, K, T):
    w, ws, wts = _weights(3, 136, K, fmt, 31)
    x = _x(T, K, "bf16", 32).cuda()
    off = torch.tensor([0, 2, 2, T], dtype=torch.int32).cuda()
    y0 = moe.fp4_linear(x, w, ws, fmt, offsets=off, w_tensor_scale=wts)
    for at in (1, 8):
        buf = torch.empty(ws.numel() + at, dtype=torch.uint8, device="cuda")
        moved = buf[at:].view(ws.shape)
        moved.copy_(ws)
        assert torch.equal(y0, moe.fp4_linear(x, w, moved, fmt, offsets=off, w_tensor_scale=wts))
        c, s = moe.quantize_fp4(x, fmt)
        assert torch.equal(y0, moe.fp4_matmul(c, s, w, moved, fmt, offsets=off, w_tensor_scale=wts))


def test_strided_x_streams_and_graphs():
    x = torch.randn((300, 416), generator=_gen(4)).to(torch.bfloat16).cuda()
    w, ws, wts = _weights(1, 256, 384, "nvfp4", 5)
    ts = torch.tensor([0.01]).cuda()
    for T in (8, 300):
        v = x[:T, 8:392]
        y0 = moe.fp4_linear(v.contiguous(), w[0], ws[0], "nvfp4", x_tensor_scale=ts, w_tensor_scale=wts)
        assert torch.equal(y0, moe.fp4_linear(v, w[0], ws[0], "nvfp4", x_tensor_scale=ts, w_tensor_scale=wts))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ys = [moe.fp4_linear(v, w[0], ws[0], "nvfp4", x_tensor_scale=ts, w_tensor_scale=wts, stream=s) for _ in range(8)]
        s.synchronize()
        assert all(torch.equal(y0, y) for y in ys)
        src = v.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            yg = moe.fp4_linear(src, w[0], ws[0], "nvfp4", x_tensor_scale=ts, w_tensor_scale=wts)
        src.copy_(x[:T, :384])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, moe.fp4_linear(x[:T, :384], w[0], ws[0], "nvfp4", x_tensor_scale=ts, w_tensor_scale=wts))


def test_many_calls_at_once_on_several_streams():
    """Calls on streams that are not ordered with each other, of every tile shape, beside one another."""
    shapes = [(1, 640, 2304), (40, 1024, 1024), (130, 512, 512), (600, 2304, 768), (9, 5120, 2304)]
    cases = []
    for i, (T, N, K) in enumerate(shapes):
        x = torch.randn((T, K), generator=_gen(i)).to(torch.bfloat16).cuda()
        w, ws, _ = _weights(1, N, K, FMT[i % 2], i)
        cases.append((x, w[0], ws[0], FMT[i % 2]))
    want = [moe.fp4_linear(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    got = [[moe.fp4_linear(*c, stream=s) for c, s in zip(cases, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for row in got:
        assert all(torch.equal(a, b) for a, b in zip(row, want))


def test_first_call_of_a_process_may_be_captured():
    import subprocess
    import sys
    code = """
import torch, routed_expert_ffn_sqrtsoftplus_b200 as moe
x = torch.randn(40, 512, device='cuda').to(torch.bfloat16)
big = torch.randn(900, 512, device='cuda').to(torch.bfloat16)
w = torch.randint(0, 256, (384, 256), dtype=torch.uint8, device='cuda')
s = torch.randint(118, 124, (384, 16), dtype=torch.uint8, device='cuda')
z = torch.randn(70, 64, device='cuda')
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = [moe.fp4_linear(x[:1], w, s, 'mxfp4'), moe.fp4_linear(x, w, s, 'mxfp4'), moe.fp4_linear(big, w, s, 'mxfp4')]
    i, v = moe.route(z, 4, score='sigmoid', bias=z[0].contiguous(), n_groups=4, topk_groups=2)
    d = moe.route_backward(v, z, i, score='sigmoid')
g.replay(); torch.cuda.synchronize()
again = [moe.fp4_linear(x[:1], w, s, 'mxfp4'), moe.fp4_linear(x, w, s, 'mxfp4'), moe.fp4_linear(big, w, s, 'mxfp4')]
assert all(torch.equal(a, b) for a, b in zip(outs, again))
j, u = moe.route(z, 4, score='sigmoid', bias=z[0].contiguous(), n_groups=4, topk_groups=2)
assert torch.equal(i, j) and torch.equal(u, v) and torch.equal(d, moe.route_backward(u, z, j, score='sigmoid'))
print('captured')
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert "captured" in r.stdout, r.stderr[-2000:]


def test_two_graphs_of_one_call_do_not_share_their_workspace():
    xs = [torch.randn((300, 512), generator=_gen(i)).to(torch.bfloat16).cuda() for i in range(2)]
    w, ws, _ = _weights(1, 512, 512, "nvfp4", 7)
    graphs, outs = [], []
    for x in xs:
        moe.fp4_linear(x, w[0], ws[0], "nvfp4")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(moe.fp4_linear(x, w[0], ws[0], "nvfp4"))
        graphs.append(g)
    want = [moe.fp4_linear(x, w[0], ws[0], "nvfp4") for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in x (quantisation) and in y (the product): the last rows are right."""
    rows, K = 70000, 32768
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((2, K), generator=_gen(1)).to(torch.bfloat16)
    x[-2:] = tail.cuda()
    codes, scales = moe.quantize_fp4(x, "mxfp4")
    rc, rs, rv = ref.quantize(tail.double().numpy(), "mxfp4")
    assert np.array_equal(codes[-2:].cpu().numpy(), rc) and np.array_equal(scales[-2:].cpu().numpy(), rs)
    assert int(codes[:-2].max()) == 0
    del x
    v = moe.dequantize_fp4(codes, scales, "mxfp4")
    assert np.array_equal(v[-2:].double().cpu().numpy(), rv)
    del v, codes, scales
    T, N, K = 1100000, 2048, 32
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((3, K), generator=_gen(2)).to(torch.bfloat16)
    x[-3:] = tail.cuda()
    w, ws, _ = _weights(1, N, K, "mxfp4", 3)
    y = moe.fp4_linear(x, w[0], ws[0], "mxfp4")
    _, _, xv = ref.quantize(tail.double().numpy(), "mxfp4")
    wv = ref.values(w[0].cpu().numpy(), ws[0].cpu().numpy(), "mxfp4")
    want = xv @ wv.T
    assert (np.abs(y[-3:].double().cpu().numpy() - want) <= _bound(xv, wv, want, torch.bfloat16)).all()
    assert float(y[:-3].abs().max()) == 0.0


def test_route_then_experts():
    """A 4-bit expert layer from the operators: route, sort by expert, gate and up, SwiGLU, down, weighted sum."""
    T, E, H, I, k = 37, 8, 256, 128, 2
    g = _gen(11)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    wg = (torch.randn((E, H), generator=g) / H ** 0.5).cuda()
    w13, s13, _ = _weights(E, 2 * I, H, "mxfp4", 12)
    w2, s2, _ = _weights(E, H, I, "mxfp4", 13)
    idx, w = moe.route(x.float() @ wg.t(), k, score="sigmoid", n_groups=2, topk_groups=1)
    flat = idx.flatten().long()
    order = torch.argsort(flat, stable=True)
    off = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
    gu = moe.fp4_linear(x[order // k], w13, s13, "mxfp4", offsets=off).float()
    h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).to(torch.bfloat16)
    o = moe.fp4_linear(h, w2, s2, "mxfp4", offsets=off, out=torch.empty((T * k, H), device="cuda"))
    y = torch.zeros((T, H), device="cuda").index_add_(0, order // k, o * w.flatten()[order][:, None])
    hn = h.double().cpu().numpy()
    _, _, xv = ref.quantize(x.double().cpu().numpy(), "mxfp4")
    _, _, hv = ref.quantize(hn, "mxfp4")
    want = np.zeros((T, H))
    mag = np.zeros((T, H))
    for r, s in enumerate(order.tolist()):
        e, t = int(flat[s]), s // k
        wv = ref.values(w13[e].cpu().numpy(), s13[e].cpu().numpy(), "mxfp4")
        gv = wv @ xv[t]
        a, b = gv[:I], gv[I:]
        ref_h = a / (1 + np.exp(-a)) * b
        # gate and up are rounded to BF16 (2^-9 each, SiLU's slope at most 1.1), and the product once more
        assert (np.abs(hn[r] - ref_h) <= 2.0 ** -7 * np.abs(b) * (np.abs(a) + 0.3) + 1e-6).all()
        dv = ref.values(w2[e].cpu().numpy(), s2[e].cpu().numpy(), "mxfp4")
        want[t] += float(w.flatten()[s]) * (dv @ hv[r])
        mag[t] += float(w.flatten()[s]) * (np.abs(dv) @ np.abs(hv[r]))
    assert (np.abs(y.double().cpu().numpy() - want) <= mag * 16 * 2.0 ** -24).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,T,N,K", [(1, 1, 2304, 262144), (160, 160, 256, 65536), (1, 600, 512, 65536)],
                         ids=["split", "32 tokens", "arranged"])
def test_waits_that_run_out(fmt, E, T, N, K):
    """A tile takes longer than a limit of a microsecond: the call ends, says so, and spoils neither y nor the next call.

    Each element is right or as it was; the kernels' waits all have limits, and copies in flight are waited for.
    """
    bs = ref.BLOCK[fmt]
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(*((118, 124) if fmt == "mxfp4" else (40, 60)), (E, N, K // bs), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") if E > 1 else None
    if E == 1:
        w, ws = w[0], ws[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = moe.fp4_linear(x, w, ws, fmt, offsets=off, status=status)
    assert status.item() == 0 and bool(torch.isfinite(want).all())
    try:
        moe.fp4_set_wait_timeout(1000)
        for _ in range(3):
            y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
            status.zero_()
            moe.fp4_linear(x, w, ws, fmt, offsets=off, out=y, status=status)
            assert status.item() == 1
            assert bool(((y == want) | (y == 7.0)).all())
    finally:
        moe.fp4_set_wait_timeout(2_000_000_000)
    status.zero_()
    assert torch.equal(want, moe.fp4_linear(x, w, ws, fmt, offsets=off, status=status)) and status.item() == 0


def test_waits_that_run_out_are_told_without_a_status_word():
    T, N, K = 1, 2304, 262144
    w = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    ws = torch.randint(118, 124, (N, K // 32), device="cuda", dtype=torch.uint8)
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    want = moe.fp4_linear(x, w, ws, "mxfp4")
    assert moe.fp4_status() == moe.MOE_OK
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        moe.fp4_set_wait_timeout(1000)
        moe.fp4_linear(x, w, ws, "mxfp4", status=status)
        assert status.item() == 1 and moe.fp4_status() == moe.MOE_OK   # the caller's own word
        moe.fp4_linear(x, w, ws, "mxfp4")
        moe.fp4_matmul(*moe.quantize_fp4(x, "mxfp4"), w, ws, "mxfp4")
    finally:
        moe.fp4_set_wait_timeout(2_000_000_000)
    assert moe.fp4_status() == moe.MOE_ERR_TIMEOUT
    assert moe.fp4_status() == moe.MOE_OK      # reading clears it
    assert torch.equal(want, moe.fp4_linear(x, w, ws, "mxfp4")) and moe.fp4_status() == moe.MOE_OK


@pytest.mark.parametrize("x_ts,w_ts,unit", [
    (1e-22, 1e-20, 2000.0), (3e-38, 1e-3, 2000.0), (1e-30, 1e-13, 2000.0), (2.0 ** -149, 1.0, 2000.0), (1e-3, 1e-41, 2000.0),
    (1e20, 1e20, 2.0 ** -8), (3e38, 2.0, 2.0 ** -8), (3e38, 1e-38, 1.0), (1e-40, 2e38, 1.0)])
@pytest.mark.parametrize("T,K", [(5, 1024), (40, 96), (230, 544)])
def test_matmul_far_tensor_scales(x_ts, w_ts, unit, T, K):
    """Two tensor scales whose product is no ordinary 32-bit number, where the results are ordinary ones."""
    N = 130
    x = torch.randn((T, K), generator=_gen(T)) * unit
    w = torch.randn((N, K), generator=_gen(K)) * unit
    xc, xs, _ = ref.quantize(x.double().numpy(), "nvfp4")
    wc, wsc, _ = ref.quantize(w.double().numpy(), "nvfp4")
    x_ts, w_ts = (torch.tensor([v], dtype=torch.float32) for v in (x_ts, w_ts))
    dev = [torch.from_numpy(a).cuda() for a in (xc, xs, wc, wsc)]
    xv = ref.values(xc, xs, "nvfp4", x_ts.double().numpy())
    wv = ref.values(wc, wsc, "nvfp4", w_ts.double().numpy())
    want = xv @ wv.T
    for out in (torch.float32, torch.bfloat16):
        y = moe.fp4_matmul(*dev, "nvfp4", x_tensor_scale=x_ts.cuda(), w_tensor_scale=w_ts.cuda(), out_dtype=out)
        # below the normal range results have a fixed step: 2^-149 in 32 bits, 2^-133 in bfloat16
        step = 2.0 ** -149 + (2.0 ** -133 if out == torch.bfloat16 else 0.0)
        err = np.abs(y.double().cpu().numpy() - want)
        b = _bound(xv, wv, want, out) + step
        assert (err <= b).all(), (err / b).max()
        assert np.abs(want).max() > 100 * step      # the bound says something


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_tensor_of_zeros_with_the_scale_that_it_calibrates_to(dtype):
    x = torch.zeros((40, 96), dtype=DT[dtype], device="cuda")
    x[1] = -0.0
    ts = (x.abs().max().float() / 2688.0).reshape(1)
    assert ts.item() == 0.0
    codes, scales = moe.quantize_fp4(x, "nvfp4", ts)
    assert not bool(scales.any()) and not bool((codes & 0x77).any())
    assert not bool(moe.dequantize_fp4(codes, scales, "nvfp4", ts, dtype=torch.float32).any())
    w, ws, wts = _weights(1, 64, 96, "nvfp4", 3)
    for T in (3, 40):
        y = moe.fp4_linear(x[:T], w[0], ws[0], "nvfp4", x_tensor_scale=ts, w_tensor_scale=wts)
        assert bool((y == 0).all())


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T", [64, 700])
def test_experts_of_unlike_loads(fmt, T):
    """Most rows, or all of them, on one expert of many: tile shapes go by the mean load."""
    E, N, K = 32, 264, 288
    x = _x(T, K, "bf16", T)
    w, ws, wts = _weights(E, N, K, fmt, 9)
    _, _, xv = ref.quantize(x.double().numpy(), fmt)
    for sizes in ([0] * 7 + [T] + [0] * 24, [1] * 31 + [T - 31], [T - 31] + [1] * 31):
        off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32)
        y = moe.fp4_linear(x.cuda(), w, ws, fmt, w_tensor_scale=wts, offsets=off.cuda()).double().cpu().numpy()
        for g in range(E):
            a, b = int(off[g]), int(off[g + 1])
            if a < b:
                wv = ref.values(w[g].cpu().numpy(), ws[g].cpu().numpy(), fmt, None if wts is None else wts.cpu().numpy()[g])
                want = xv[a:b] @ wv.T
                assert (np.abs(y[a:b] - want) <= _bound(xv[a:b], wv, want, torch.bfloat16)).all(), g
