"""Refusals of the handle-less operators, before any GPU is touched, and the reference forms of their tests."""
import ctypes

import numpy as np
import pytest
import torch

import routed_expert_ffn_sqrtsoftplus_b200 as moe
from routed_expert_ffn_sqrtsoftplus_b200 import build as moe_build

import fp4_ref as ref

FAKE = 0x10000  # 16-byte aligned, never dereferenced: each call is refused first
INV, UNS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


def _cfg(**kw):
    d = dict(n_experts=64, top_k=4, n_groups=4, topk_groups=2, score=1, group_top2=1, renormalize=1, route_scale=1.0)
    d.update(kw)
    return moe._RouteConfig(*[d[n] for n, _ in moe._RouteConfig._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(n_experts=0), INV), (dict(top_k=0), INV), (dict(n_groups=0), INV), (dict(topk_groups=0), INV),
    (dict(topk_groups=5), INV), (dict(n_experts=63), INV), (dict(top_k=33, topk_groups=2), INV),
    (dict(score=3), INV), (dict(score=-1), INV), (dict(route_scale=0.0), INV), (dict(route_scale=float("nan")), INV),
    (dict(route_scale=float("inf")), INV), (dict(n_experts=516), UNS), (dict(top_k=33, topk_groups=4), UNS),
    (dict(n_experts=66, n_groups=33, topk_groups=33), UNS)])
def test_route_refuses_bad_configs(L, kw, want):
    assert L.moe_route(_cfg(**kw), FAKE, 2, 1024, None, 3, FAKE, FAKE, None) == want
    assert L.moe_route_backward(_cfg(**kw), FAKE, FAKE, 2, 1024, FAKE, 3, FAKE, None) == want


def test_route_refuses_bad_arguments(L):
    c = _cfg()
    assert L.moe_route(None, FAKE, 2, 64, None, 3, FAKE, FAKE, None) == INV
    assert L.moe_route(c, None, 2, 64, None, 3, FAKE, FAKE, None) == INV
    assert L.moe_route(c, FAKE, 3, 64, None, 3, FAKE, FAKE, None) == INV
    assert L.moe_route(c, FAKE, 2, 63, None, 3, FAKE, FAKE, None) == INV
    assert L.moe_route(c, FAKE, 2, 64, None, -1, FAKE, FAKE, None) == INV
    assert L.moe_route(c, FAKE + 2, 2, 64, None, 3, FAKE, FAKE, None) == INV
    assert L.moe_route(c, FAKE, 2, 64, FAKE + 1, 3, FAKE, FAKE, None) == INV
    assert L.moe_route(c, FAKE, 2, 64, None, 3, None, FAKE, None) == INV
    assert L.moe_route(c, None, 2, 64, None, 0, None, None, None) == OK
    assert L.moe_route_backward(c, FAKE, FAKE, 2, 64, FAKE, 3, FAKE, None) == INV    # in place
    assert L.moe_route_backward(c, None, FAKE, 2, 64, FAKE, 3, FAKE + 64, None) == INV
    assert L.moe_route_backward(c, None, None, 2, 64, None, 0, None, None) == OK
    assert L.moe_forward_routed(None, FAKE, FAKE, FAKE, 1, FAKE, None) == INV


def test_fp4_refuses_bad_arguments(L):
    q, d = L.moe_quantize_fp4, L.moe_dequantize_fp4
    assert q(2, FAKE, 0, 4, 64, 64, None, FAKE, FAKE, 4, None) == INV
    assert q(0, FAKE, 5, 4, 64, 64, None, FAKE, FAKE, 4, None) == INV
    assert q(0, FAKE, 0, 4, 48, 48, None, FAKE, FAKE, 4, None) == INV
    assert q(0, FAKE, 0, 4, 64, 63, None, FAKE, FAKE, 4, None) == INV
    assert q(0, FAKE, 0, 4, 64, 64, None, FAKE, FAKE, 1, None) == INV
    assert q(1, FAKE, 0, 4, 64, 64, None, FAKE, FAKE, 3, None) == INV
    assert q(0, FAKE, 0, 4, 64, 64, FAKE, FAKE, FAKE, 4, None) == INV     # MXFP4 has no tensor scale
    assert q(0, FAKE + 1, 0, 4, 64, 64, None, FAKE, FAKE, 4, None) == INV
    assert q(0, FAKE, 0, 4, 64, 64, None, FAKE + 8, FAKE, 4, None) == INV
    assert q(0, None, 0, 4, 64, 64, None, FAKE, FAKE, 4, None) == INV
    assert q(0, FAKE, 0, -1, 64, 64, None, FAKE, FAKE, 4, None) == INV
    assert q(0, FAKE, 0, 1 << 40, 64, 64, None, FAKE, FAKE, 4, None) == UNS
    assert q(0, None, 0, 0, 64, 64, None, None, None, 4, None) == OK
    assert d(0, FAKE, FAKE, 4, 64, 1, None, FAKE, 0, None) == INV
    assert d(1, FAKE, FAKE, 4, 40, 4, None, FAKE, 0, None) == INV
    assert d(0, FAKE, FAKE, 4, 64, 2, FAKE, FAKE, 0, None) == INV
    assert d(0, None, None, 0, 64, 2, None, None, 0, None) == OK
    p = L.moe_fp4_pad_scales
    assert p(FAKE, 4, 20, FAKE, 16, None) == INV and p(FAKE, 4, 20, FAKE, 24, None) == INV
    assert p(FAKE, 4, 20, FAKE + 4, 32, None) == INV and p(None, 4, 20, FAKE, 32, None) == INV
    assert p(FAKE, 4, 0, FAKE, 32, None) == INV and p(None, 0, 20, None, 32, None) == OK


def _product(**kw):
    d = dict(format=0, T=4, N=64, K=64, E=1, out_dtype=0, x=FAKE, x_scales=FAKE, x_scale_stride=8, x_tensor_scale=None,
             w=FAKE, w_scales=FAKE, w_scale_stride=8, w_tensor_scale=None, offsets=None, y=FAKE + 64, workspace=None, workspace_bytes=0, status=None)
    d.update(kw)
    return moe._Fp4Product(*[d[n] for n, _ in moe._Fp4Product._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(format=2), INV), (dict(T=-1), INV), (dict(N=0), INV), (dict(K=48), INV), (dict(K=0), INV), (dict(E=0), INV),
    (dict(E=2), INV), (dict(out_dtype=3), INV), (dict(x_scale_stride=1), INV), (dict(format=1), INV), (dict(w_scale_stride=12), INV),
    (dict(K=512), INV), (dict(x_scales=FAKE + 4), INV), (dict(format=1, x_scale_stride=16, w_scale_stride=16, w_scales=FAKE + 8), INV),
    (dict(x_tensor_scale=FAKE), INV), (dict(w_tensor_scale=FAKE), INV), (dict(x=None), INV), (dict(w=FAKE + 8), INV),
    (dict(x=FAKE + 4), INV), (dict(y=FAKE + 1), INV), (dict(y=FAKE), INV), (dict(y=None), INV), (dict(w_scales=None), INV),
    (dict(offsets=FAKE + 2), INV), (dict(T=(1 << 22) + 1), UNS), (dict(E=513, offsets=FAKE), UNS),
    (dict(N=(1 << 18) + 1), UNS), (dict(T=0, x=None, y=None), OK),
    (dict(T=4096, N=4096, K=4096, x_scale_stride=128, w_scale_stride=128), INV),
    (dict(T=4096, N=4096, K=4096, x_scale_stride=128, w_scale_stride=128, workspace=FAKE, workspace_bytes=999), INV),
    (dict(T=4096, workspace=FAKE + 8, workspace_bytes=1 << 40), INV)])
def test_fp4_matmul_refuses_bad_arguments(L, kw, want):
    assert L.moe_fp4_matmul(_product(**kw), None) == want
    if not any(n.startswith("x_scale") for n in kw) and "workspace" not in kw and kw.get("format") != 1:
        # the same with x to be quantised: x's scales are not given, and there is always a workspace
        big = dict(dict(workspace=FAKE, workspace_bytes=1 << 40), **kw)
        if kw.get("x", 0) != FAKE + 4 and kw.get("T") != 4096 and kw.get("w_scale_stride") != 12:   # copied there
            assert L.moe_fp4_linear(_product(**big), 2, 1 << 20, None) == want
    assert L.moe_fp4_matmul(None, None) == INV
    w = L.moe_fp4_workspace_bytes
    assert w(0, 32, 64, 64, 1) == 0 and w(1, 4096, 4096, 4096, 1) > 0 and w(0, 64, 64, 64, 2) == 0 and w(2, 4096, 4096, 4096, 1) == 0
    assert w(0, -1, 64, 64, 1) == 0 and w(0, 4096, 0, 4096, 1) == 0 and w(0, 99, 64, 64, 513) == 0


def test_fp4_linear_refuses_bad_arguments(L):
    w = L.moe_fp4_linear_workspace_bytes
    assert w(0, 4, 64, 256, 1) == 4 * (128 + 16) and w(0, 4, 64, 48, 1) == 0 and w(0, 0, 64, 64, 1) == 0
    assert w(0, 4, 64, 64, 1) == 4 * (32 + 16) + 64 * 16      # aligned rows of w's scales
    assert w(1, 4, 64, 288, 2) == 4 * (144 + 32) + 128 * 32
    f = lambda dt=0, rs=64, **kw: L.moe_fp4_linear(_product(**dict(dict(workspace=FAKE, workspace_bytes=1 << 20), **kw)), dt, rs, None)  # noqa: E731
    assert f(dt=3) == INV and f(rs=63) == INV and f(x=FAKE + 1) == INV and f(x=None) == INV
    assert f(workspace=None) == INV and f(workspace_bytes=4 * 48 - 1) == INV and f(workspace=FAKE + 8) == INV
    assert f(w_scale_stride=12, workspace_bytes=4 * 48 + 64 * 16 - 1) == INV
    assert L.moe_fp4_linear(None, 0, 64, None) == INV and f(T=0) == OK
    # the quantiser counts in 32 bits: 2^33 values a call
    assert f(T=1 << 20, K=1 << 14, w_scale_stride=1 << 10, rs=1 << 14) == UNS
    assert w(0, 1 << 20, 64, 1 << 14, 1) == 0 and w(0, 1 << 19, 64, 1 << 14, 1) > 0


def test_bindings_refuse_bad_tensors(L):
    z = torch.zeros((4, 8))
    for call in (lambda: moe.route(z, 2), lambda: moe.route_backward(z, z, z), lambda: moe.quantize_fp4(z, "mxfp4"),
                 lambda: moe.quantize_fp4(z, "fp5"), lambda: moe.dequantize_fp4(z, z, "mxfp4"),
                 lambda: moe.fp4_linear(z, z, z, "mxfp4"), lambda: moe.fp4_matmul(z, z, z, z, "nvfp4"),
                 lambda: moe.fp4_matmul(z, z, z, z, "e2m1")):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the references themselves
def test_reference_grid_and_codes():
    assert ref.E4M3[126] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3)
    # every half-way point goes to the even code
    for i in range(7):
        mid = (ref.GRID[i] + ref.GRID[i + 1]) / 2
        assert ref.nearest(np.array([mid]), ref.GRID)[0] % 2 == 0
        x = np.zeros((1, 32))
        x[0, 0], x[0, 1] = 6.0, mid
        c, s, v = ref.quantize(x, "mxfp4")
        assert s[0, 0] == 127 and (c[0, 0] >> 4) == ref.nearest(np.array([mid]), ref.GRID)[0]
        assert np.array_equal(ref.values(c, s, "mxfp4"), v)


def test_reference_routing_by_hand():
    z = np.log(np.array([[1.0, 2.0, 3.0, 4.0]]))
    idx, w = ref.route(z, 2, "softmax", renorm=False)
    assert idx.tolist() == [[3, 2]] and np.allclose(w, [[0.4, 0.3]])
    idx, w = ref.route(z, 2, "softmax", bias=np.array([1.0, 0, 0, 0]))
    assert idx.tolist() == [[0, 3]] and np.allclose(w, [[0.2, 0.8]])
    # groups {0, 1} and {2, 3}: 0.1 + 1 + 0.2 against 0.7
    idx, w = ref.route(z, 2, "softmax", bias=np.array([1.0, 0, 0, 0]), G=2, kept=1)
    assert idx.tolist() == [[0, 1]] and np.allclose(w, [[1 / 3, 2 / 3]])
    idx, _ = ref.route(np.full((1, 4), -np.inf), 2, "sigmoid")
    assert idx.tolist() == [[-1, -1]]


def test_structs_match_the_header():
    import os
    import re
    h = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")).read()
    for name, cls in (("moe_route_config", moe._RouteConfig), ("moe_fp4_product", moe._Fp4Product)):
        body = re.search(r"typedef struct \{([^{}]*)\} " + name, h).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [f.strip(" *\n") for line in body.split(";") for f in re.sub(r"^\s*(const )?\w+", "", line).split(",")]
        assert [f for f in fields if f] == [n for n, _ in cls._fields_]


def test_bindings_refuse_sizes_that_32_bits_do_not_hold(L):
    for args in ((8, 0, 1, 1), (8, -1, 1, 1), (8, 9, 1, 1), (8, (1 << 32) + 2, 1, 1), (8, 2, 1 << 32, 1)):
        with pytest.raises(ValueError):
            moe._route_config(*args, "softmax", "max", True, 1.0)
    with pytest.raises(ValueError):
        moe._fp4_workspace_bytes(False, 0, 0, (1 << 32) + 4, 64, 64, 1)
    # CUDA tensors as far as the checks ask, without their memory
    class Rows:
        is_cuda, dtype = True, torch.float32
        def __init__(self, *shape):
            self.shape = shape
        def dim(self):
            return 2
        def stride(self):
            return self.shape[1], 1
    assert moe._rows(Rows(3, 8), "x") == (3, 8, 8, 2)
    for shape in ((1 << 31, 8), ((1 << 32) + 3, 1), (1, 1 << 31)):
        with pytest.raises(ValueError):
            moe._rows(Rows(*shape), "x")


def test_wait_limit_refusals(L):
    assert L.moe_fp4_set_wait_timeout(0) == INV and L.moe_fp4_set_wait_timeout(2_000_000_000) == OK
    for ns in (0, -1, 1 << 64):
        with pytest.raises(ValueError):
            moe.fp4_set_wait_timeout(ns)


def test_workspace_sizes_are_kept_by_the_device_that_they_were_planned_for(monkeypatch):
    """A call under another current device is refused, but may not leave that device's size behind for the tensors' own."""
    current = [0]

    class Library:
        def moe_fp4_workspace_bytes(self, *shape):
            return 100 + current[0]

        moe_fp4_linear_workspace_bytes = moe_fp4_workspace_bytes

    monkeypatch.setattr(moe, "lib", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)

    moe._fp4_workspace_bytes.cache_clear()
    try:
        for dev in (0, 1, 0):
            current[0] = dev
            assert moe._workspace_size(False, 0, 96, 64, 64, 1) == moe._workspace_size(True, 0, 96, 64, 64, 1) == 100 + dev
    finally:
        moe._fp4_workspace_bytes.cache_clear()


def test_group_counts_far_below_zero_are_refused(L):
    # cut to 32 bits they would be 1
    for args in ((1 - (1 << 32), 1), (1, 1 - (1 << 32)), (2 - (1 << 33), 1)):
        with pytest.raises(ValueError):
            moe._route_config(8, 2, *args, "softmax", "max", True, 1.0)
    # and those that fit go to the library, which refuses them
    assert L.moe_route(moe._route_config(8, 2, -1, 1, "softmax", "max", True, 1.0), FAKE, 2, 8, None, 3, FAKE, FAKE, None) == INV
