"""Residual + norm, 8-bit rows and the layer for a few tokens without a GPU: workspace sizes, kernel names and the
refusals that come before any device work (the addresses passed are never followed)."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_fp32_b200 as sm
from sparse_mixture_experts_fp32_b200 import build as smbuild

A = 1 << 20  # an aligned address
BIG = 1 << 40
OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def L():
    smbuild.build()
    return sm.lib()


def few(L, d, k=1, ws=BIG, **over):
    names = ("x", "x_scale", "w_r", "bias", "w_in", "w_in_scale", "w_out", "w_out_scale", "y", "expert", "gate", "slot",
             "counts", "aux", "workspace")
    args = dict.fromkeys(names, A)
    args.update(x_scale=None, bias=None, w_in_scale=None, w_out_scale=None)
    args.update(over)
    return L.switch_layer_fwd_few(None if d is None else ctypes.byref(d), k, *[args[n] for n in names], ws, None)


def fdims(T=4, d=64, F=128, N=4, C=4, dtype=sm.SWITCH_BF16, flags=0):
    return sm.dims(T, d, F, N, C, dtype, flags)


def test_few_refusals(L):
    d = fdims()
    assert few(L, None) == NULL
    for name in ("x", "w_r", "w_in", "w_out", "y", "expert", "gate", "slot", "counts", "aux", "workspace"):
        assert few(L, d, **{name: None}) == NULL, name
        assert few(L, d, **{name: A + 4}) == ALIGN, name
    assert few(L, d, bias=A + 8) == ALIGN
    assert few(L, d, ws=16) == WORKSPACE
    need = sm.switch_few_workspace_size(d, 1)
    assert few(L, d, ws=need - 1) == WORKSPACE
    assert few(L, fdims(T=65, C=65)) == SHAPE
    assert few(L, d, k=0) == SHAPE and few(L, d, k=3) == SHAPE
    assert few(L, fdims(N=1), k=2) == SHAPE
    assert few(L, fdims(d=96)) == SHAPE and few(L, fdims(F=100)) == SHAPE
    assert few(L, fdims(d=96, dtype=sm.SWITCH_E4M3)) == SHAPE
    assert few(L, fdims(N=257)) == SHAPE and few(L, fdims(C=0)) == SHAPE
    assert few(L, fdims(dtype=7)) == DTYPE
    # scales belong to 8-bit experts, which need both
    for name in ("x_scale", "w_in_scale", "w_out_scale"):
        assert few(L, d, **{name: A}) == DTYPE, name
        assert few(L, fdims(dtype=sm.SWITCH_F32), **{name: A}) == DTYPE, name
    e = fdims(dtype=sm.SWITCH_E4M3)
    assert few(L, e) == NULL
    assert few(L, e, w_in_scale=A) == NULL and few(L, e, w_out_scale=A) == NULL
    assert few(L, e, w_in_scale=A, w_out_scale=A + 4) == ALIGN
    for flag in (sm.SWITCH_FLAG_TRAINING, sm.SWITCH_FLAG_ROUTER_STATS, sm.SWITCH_FLAG_GEMM_1CTA):
        assert few(L, fdims(flags=flag)) == UNSUPPORTED


def test_the_8_bit_type_is_refused_by_the_other_calls(L):
    e = fdims(dtype=sm.SWITCH_E4M3)
    b = ctypes.byref(e)
    n = ctypes.c_size_t()
    assert L.switch_workspace_size(b, ctypes.byref(n)) == DTYPE
    assert L.switch_layer_fwd(b, A, A, None, A, A, A, A, A, A, A, A, A, BIG, None) == DTYPE
    assert L.switch_route(b, A, A, None, A, A, A, A, A, A, A, BIG, None) == DTYPE


def test_few_workspace(L):
    for T, k in ((0, 1), (1, 1), (1, 2), (33, 2), (64, 2)):
        d = fdims(T=T, d=1024, F=4096, N=8, C=64)
        got = sm.switch_few_workspace_size(d, k)
        pairs = T * k
        assert got >= pairs * (1024 + 4096) * 4 + T * 8 * 4
        assert got <= (1 << 16) + 512 * (1024 + 4096 + 8) * 4 + T * 8 * 4
    assert L.switch_few_workspace_size(ctypes.byref(fdims()), 1, None) == NULL


def ndims(T=4, d=64, res=sm.SWITCH_BF16, delta=sm.SWITCH_F32, out=sm.SWITCH_BF16, eps=1e-6):
    return sm.SwitchNormDims(T, d, res, delta, out, eps)


def norm(L, n, **over):
    names = ("residual", "delta", "weight", "sum", "out", "scale", "rstd")
    args = dict.fromkeys(names, A)
    args["scale"] = None
    args.update(over)
    return L.switch_norm_fwd(None if n is None else ctypes.byref(n), *[args[k] for k in names], None)


def test_norm_refusals(L):
    n = ndims()
    assert norm(L, None) == NULL
    for name in ("residual", "weight", "out"):
        assert norm(L, n, **{name: None}) == NULL, name
    for name in ("residual", "delta", "weight", "sum", "out", "rstd"):
        assert norm(L, n, **{name: A + 8}) == ALIGN, name
    assert norm(L, n, scale=A) == DTYPE
    assert norm(L, ndims(out=sm.SWITCH_E4M3)) == NULL
    assert norm(L, n, delta=None) == SHAPE  # a sum without a delta
    assert norm(L, ndims(res=sm.SWITCH_E4M3)) == DTYPE and norm(L, ndims(delta=sm.SWITCH_E4M3)) == DTYPE
    assert norm(L, ndims(out=3)) == DTYPE and norm(L, ndims(out=-1)) == DTYPE
    for bad in (ndims(T=-1), ndims(T=1 << 31), ndims(d=0), ndims(d=8193), ndims(eps=-1.0), ndims(eps=float("nan")),
                ndims(eps=float("inf"))):
        assert norm(L, bad) == SHAPE


def norm_bwd(L, n, ws=BIG, **over):
    names = ("sum", "weight", "rstd", "dout", "dsum", "dresidual", "dweight", "workspace")
    args = dict.fromkeys(names, A)
    args.update(over)
    return L.switch_norm_bwd(None if n is None else ctypes.byref(n), *[args[k] for k in names], ws, None)


def test_norm_bwd_refusals(L):
    n = ndims()
    assert norm_bwd(L, None) == NULL
    for name in ("sum", "weight", "rstd", "dout", "dresidual", "dweight", "workspace"):
        assert norm_bwd(L, n, **{name: None}) == NULL, name
    for name in ("sum", "weight", "rstd", "dout", "dsum", "dresidual", "dweight", "workspace"):
        assert norm_bwd(L, n, **{name: A + 4}) == ALIGN, name
    assert norm_bwd(L, n, ws=sm.switch_norm_workspace_size(n) - 1) == WORKSPACE
    assert norm_bwd(L, ndims(res=sm.SWITCH_E4M3)) == DTYPE and norm_bwd(L, ndims(d=8200)) == SHAPE


def test_quantize_refusals(L):
    q = L.switch_quantize_rows
    assert q(4, 8, sm.SWITCH_F32, None, A, A, None) == NULL
    assert q(4, 8, sm.SWITCH_F32, A, None, A, None) == NULL
    assert q(4, 8, sm.SWITCH_F32, A, A, None, None) == NULL
    assert q(4, 8, sm.SWITCH_F32, A + 4, A, A, None) == ALIGN
    assert q(4, 8, sm.SWITCH_E4M3, A, A, A, None) == DTYPE
    assert q(-1, 8, sm.SWITCH_F32, A, A, A, None) == SHAPE
    assert q(4, 0, sm.SWITCH_F32, A, A, A, None) == SHAPE and q(4, 32769, sm.SWITCH_F32, A, A, A, None) == SHAPE


def test_kernel_names(L):
    names = {33: "norm_fwd", 34: "norm_bwd", 35: "norm_dweight", 36: "quantize_rows", 37: "few_router",
             38: "few_experts_simt", 39: "few_experts_tc"}
    for k, v in names.items():
        assert L.switch_kernel_name(k).decode() == v


def test_python_refuses_host_tensors_and_wrong_weights():
    x = torch.zeros(4, 64)
    w = torch.zeros(64)
    with pytest.raises(TypeError):
        sm.norm_fwd(x, w)
    with pytest.raises(TypeError):
        sm.norm_bwd(x, w, torch.zeros(4), x)
    with pytest.raises(TypeError):
        sm.quantize_rows(x)
    w_r, w_in, w_out = torch.zeros(4, 64), torch.zeros(4, 128, 64), torch.zeros(4, 64, 128)
    with pytest.raises(TypeError):
        sm.FewLayer(w_r, w_in, w_out)
    with pytest.raises(ValueError):
        sm.FewLayer(w_r, w_in, w_out, w_in_scale=torch.zeros(4, 128))
    with pytest.raises(ValueError):
        sm.FewLayer(w_r, w_in[0], w_out)
