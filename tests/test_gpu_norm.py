"""Residual + norm, its gradient and 8-bit rows on the GPU against the definitions in 64 bits.

Tolerances, u = 2^-24: a sum of squares adds at most 32 terms in one thread and at most 42 levels after that
(5 in a warp, at most 32 warps), all positive, so it is within 74 u of itself; the mean, eps, the root (which
halves the error) and the reciprocal add 4 u: rstd is within 41 u.  v adds two products: 43 u; scale one division:
44 u.  A rounding to bfloat16 adds 2^-8 of the value, one to e4m3 2^-4 of it, or half of its smallest step, 2^-10,
below the normal range (times scale).
"""
import pytest
import torch

import sparse_mixture_experts_fp32_b200 as sm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return sm.lib()


def rows(T, d, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(T, d, device="cuda").normal_(0, std, generator=g)
    return (x * torch.exp(torch.empty(T, 1, device="cuda").normal_(0, 1, generator=g))).to(dtype)


def check_e4m3(q, scale, v, slack):
    """q, scale against v in 64 bits, where the values that were rounded are within `slack` of v."""
    top = v.abs().amax(1)
    assert ((scale.double() - top / 448).abs() <= (slack + 1) * U * top / 448).all()
    got = q.double() * scale.double()[:, None]
    bound = v.abs() * (2.0 ** -4 + 2 * (slack + 2) * U) + (2.0 ** -10) * (top / 448)[:, None] * 1.001
    assert ((got - v).abs() <= bound).all()
    assert q.double().abs().amax(1).max() <= 448


SIZES = [(1, 1), (1, 1024), (3, 7), (5, 8), (2, 255), (9, 768), (33, 1032), (4, 4099), (1030, 40), (1500, 333),
         (3, 8191), (2, 8192), (1100, 2056), (1027, 8192), (17, 8185), (600, 8189), (3000, 9), (2500, 511)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("res,delta,out", [(F32, None, F32), (F32, F32, BF16), (F32, BF16, E4M3), (BF16, F32, BF16),
                                           (BF16, None, E4M3), (BF16, BF16, F32), (BF16, F32, E4M3)])
def test_norm_fwd(T, d, res, delta, out):
    r = rows(T, d, res, 1, 2.0)
    a = None if delta is None else rows(T, d, delta, 2)
    w = 1 + rows(1, d, F32, 3, 0.3)[0]
    r0 = r.clone()
    got = sm.norm_fwd(r, w, delta=a, eps=1e-5, out_dtype=out)
    assert torch.equal(r, r0)
    s = r
    if a is not None:
        s = (r.float() + a.float()).to(res)  # one rounding of one sum: the same bits
        assert got["sum"].dtype == res and torch.equal(got["sum"], s)
    else:
        assert got["sum"] is None
    s = s.double()
    rstd = 1 / torch.sqrt(s.square().mean(1) + torch.tensor(1e-5, dtype=F32).double().item())
    assert ((got["rstd"].double() - rstd).abs() <= 41 * U * rstd).all()
    v = s * rstd[:, None] * w.double()
    assert got["out"].dtype == out
    if out == E4M3:
        check_e4m3(got["out"], got["scale"], v, 43)
    else:
        assert got["scale"] is None
        half = 0 if out == F32 else 2.0 ** -8
        assert ((got["out"].double() - v).abs() <= v.abs() * (half + 44 * U) + 1e-40).all()


@pytest.mark.parametrize("T,d", SIZES + [(7, 32768), (3, 32765), (1100, 12288), (300, 32767), (40, 8193), (2000, 8185)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_rows(T, d, dtype):
    x = rows(T, d, dtype, 4, 0.1)
    got = sm.quantize_rows(x)
    check_e4m3(got["q"], got["scale"], x.double(), 0)
    # rounding of the quotients, bit for bit
    want = (x.float() / got["scale"][:, None]).clamp(-448, 448).to(E4M3)
    assert torch.equal(got["q"].view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,rows_", [(256, 64), (257, 64), (1024, 16384)])
def test_quantize_rounds_the_quotient_at_middles_small_values_and_zeros(dtype, cols, rows_):
    """Values half way between two e4m3 numbers (and next to it, in float32), below e4m3's normal range, zeros among
    them, at scales of 2^-40 to 2^40: bit for bit the rounding of the divided value."""
    g = torch.Generator(device="cuda").manual_seed(90)
    code = torch.randint(0, 0x7e, (rows_, cols), device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
    lo, hi = code.view(E4M3).float(), (code + 1).view(E4M3).float()
    x = (lo + hi) / 2  # at most 5 significant bits: exact in bfloat16
    if dtype == F32:
        bits = x.view(torch.int32) + torch.randint(-3, 4, x.shape, device="cuda", generator=g, dtype=torch.int32)
        x = torch.where(x > 0, bits.view(F32), x)
    x = x * torch.where(torch.rand(x.shape, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    x = torch.where(torch.rand(x.shape, device="cuda", generator=g) < 0.3, torch.zeros_like(x), x)
    x[:, 0] = 448
    x = (x * 2.0 ** torch.randint(-40, 41, (rows_, 1), device="cuda", generator=g)).to(dtype)
    x[1::4, 0] *= 0.9375  # a scale that is no power of two
    got = sm.quantize_rows(x)
    scale = (x.double().abs().amax(1) / 448).float()  # one rounding of the quotient
    assert torch.equal(got["scale"], scale)
    want = torch.div(x.float(), scale[:, None]).clamp(-448, 448).to(E4M3)
    assert torch.equal(got["q"].view(torch.uint8), want.view(torch.uint8))


def test_quantize_keeps_leading_dimensions():
    x = rows(24, 64, BF16, 5).view(2, 3, 4, 64)
    got = sm.quantize_rows(x)
    assert got["q"].shape == x.shape and got["scale"].shape == (2, 3, 4)
    flat = sm.quantize_rows(x.view(24, 64))
    assert torch.equal(got["q"].view(torch.uint8).view(24, 64), flat["q"].view(torch.uint8))


def plain_grad(s, r, w, g, u):
    d = s.shape[1]
    h = s * r[:, None]
    gw = g * w
    m = (gw * h).sum(1, keepdim=True) / d
    return r[:, None] * (gw - h * m) + u, (g * h).sum(0)


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("res", [F32, BF16])
@pytest.mark.parametrize("with_dsum", [True, False])
def test_norm_bwd(T, d, res, with_dsum):
    s = rows(T, d, res, 6, 2.0)
    w = 1 + rows(1, d, F32, 7, 0.3)[0]
    g = rows(T, d, F32, 8, 0.1)
    u = rows(T, d, F32, 9, 0.1) if with_dsum else None
    r = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    got = sm.norm_bwd(s, w, r, g, dsum=u)
    S, R, W, G = s.double(), r.double(), w.double(), g.double()
    V = u.double() if with_dsum else torch.zeros_like(S)
    want, dw = plain_grad(S, R, W, G, V)
    H, GW = S * R[:, None], G * W
    # m: products of three roundings, at most 32 + 42 additions; then five roundings of the terms of dresidual
    m_abs = (GW * H).abs().sum(1, keepdim=True) / d
    bound = 80 * U * R[:, None] * H.abs() * m_abs + 6 * U * (R[:, None] * (GW.abs() + H.abs() * m_abs) + V.abs())
    assert ((got["dresidual"].double() - want).abs() <= bound + 1e-40).all()
    # dweight: a block adds every 296th row group one by one, then at most 8 groups of its block; float64 after that
    n = T // 296 + 2 + 8 + 2
    assert ((got["dweight"].double() - dw).abs() <= n * U * (G * H).abs().sum(0) + 1e-40).all()


def test_norm_bwd_against_differences():
    """The gradients along random directions against central differences of the forward formula in 64 bits (step
    1e-5: the differences are off by about 1e-10, the kernel's by about 1e-6)."""
    T, d, eps = 6, 40, 1e-3
    res, delta = rows(T, d, F32, 10), rows(T, d, F32, 11)
    w, g, u = 1 + rows(1, d, F32, 12, 0.3)[0], rows(T, d, F32, 13), rows(T, d, F32, 14)
    f = sm.norm_fwd(res, w, delta=delta, eps=eps)
    got = sm.norm_bwd(f["sum"], w, f["rstd"], g, dsum=u)

    def loss(s, wt):
        v = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * wt
        return (v * g.double()).sum() + (s * u.double()).sum()

    S, W = f["sum"].double(), w.double()
    for seed in range(4):
        ds, dw = rows(T, d, F32, 20 + seed).double(), rows(1, d, F32, 30 + seed)[0].double()
        h = 1e-5
        diff = (loss(S + h * ds, W + h * dw) - loss(S - h * ds, W - h * dw)) / (2 * h)
        along = (got["dresidual"].double() * ds).sum() + (got["dweight"].double() * dw).sum()
        size = (got["dresidual"].double() * ds).abs().sum() + (got["dweight"].double() * dw).abs().sum()
        assert abs(diff - along) <= 1e-5 * size


def test_norm_in_place_and_result_reuse():
    r, a, w = rows(5, 768, BF16, 40), rows(5, 768, F32, 41), 1 + rows(1, 768, F32, 42, 0.3)[0]
    want = sm.norm_fwd(r, w, delta=a)
    r2 = r.clone()
    got = sm.norm_fwd(r2, w, delta=a, inplace=True)
    assert got["sum"] is r2 and torch.equal(r2, want["sum"]) and torch.equal(got["out"], want["out"])
    again = sm.norm_fwd(r, w, delta=a, out=want)
    assert again is want and torch.equal(again["sum"], r2)
    with pytest.raises(ValueError):
        sm.norm_fwd(r[:4], w, delta=a[:4], out=want)
    with pytest.raises(ValueError):
        sm.norm_fwd(r, w, delta=a, out=dict(want))
    # the gradient over its own input
    g, u = rows(5, 768, F32, 43), rows(5, 768, F32, 44)
    b = sm.norm_bwd(want["sum"], w, want["rstd"], g, dsum=u)
    dims = sm.SwitchNormDims(5, 768, sm.SWITCH_BF16, 0, 0, 0.0)
    for target in ("dsum", "dout"):
        gg, uu = g.clone(), u.clone()
        over = uu if target == "dsum" else gg
        ws = torch.empty(sm.switch_norm_workspace_size(dims), dtype=torch.uint8, device="cuda")
        dw = torch.empty(768, device="cuda")
        sm.switch_norm_bwd(dims, want["sum"], w, want["rstd"], gg, uu, over, dw, ws)
        assert torch.equal(over, b["dresidual"]) and torch.equal(dw, b["dweight"])


@pytest.mark.parametrize("d", [33, 64])
def test_rows_of_zeros_nan_and_infinity_stay_apart(d):
    x = rows(6, d, F32, 50)
    x[1] = 0
    x[2, 3] = float("nan")
    x[4, 5] = float("inf")
    w = torch.ones(d, device="cuda")
    clean = [0, 1, 3, 5]
    for out in (F32, E4M3):
        f = sm.norm_fwd(x, w, out_dtype=out, eps=0.0 if out == F32 else 1e-6)
        v = f["out"].float()
        assert torch.isfinite(v[[0, 3, 5]]).all()
        assert not torch.isfinite(v[2]).all() and not torch.isfinite(v[4]).all()
        if out == E4M3:
            assert (v[1] == 0).all() and f["scale"][1] == 0
            assert torch.isfinite(f["scale"][clean]).all() and not torch.isfinite(f["scale"][[2, 4]]).any()
    q = sm.quantize_rows(x)
    assert (q["q"][1].float() == 0).all() and q["scale"][1] == 0
    assert torch.isnan(q["scale"][2]) and torch.isinf(q["scale"][4])
    assert torch.isfinite(q["scale"][clean]).all()


def test_no_rows():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    f = sm.norm_fwd(e, w, delta=e, out_dtype=E4M3)
    assert f["out"].shape == (0, 64) and f["scale"].shape == (0,)
    b = sm.norm_bwd(e, w, f["rstd"], e)
    assert (b["dweight"] == 0).all()
    assert sm.quantize_rows(e)["q"].shape == (0, 64)


def test_refusals():
    x, w = rows(4, 64, F32, 60), torch.ones(64, device="cuda")
    with pytest.raises(TypeError):
        sm.norm_fwd(x.half(), w)
    with pytest.raises(TypeError):
        sm.norm_fwd(x, w.bfloat16())
    with pytest.raises(TypeError):
        sm.norm_fwd(x.t().contiguous().t(), w)  # strided
    with pytest.raises(ValueError):
        sm.norm_fwd(x, w, delta=x[:2])
    with pytest.raises(ValueError):
        sm.norm_fwd(x, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        sm.norm_fwd(x, w, out_dtype=torch.float16)
    with pytest.raises(sm.SwitchError):
        sm.norm_fwd(x, w, eps=-1.0)
    with pytest.raises(sm.SwitchError):
        sm.norm_fwd(x.view(-1)[4:4 + 63].view(1, 63), torch.ones(64, device="cuda")[1:])  # misaligned weight
    with pytest.raises(sm.SwitchError):
        sm.quantize_rows(rows(1, 32776, F32, 61))


def test_writes_stay_inside():
    """Outputs in the middle of guarded buffers; an odd width takes the one-element path to the last byte."""
    for d in (33, 64):
        T, pad = 5, 64
        x, a, w = rows(T, d, BF16, 70), rows(T, d, F32, 71), torch.ones(d, device="cuda")
        want = sm.norm_fwd(x, w, delta=a, out_dtype=E4M3)
        bufs = {n: torch.full((want[n].numel() * want[n].element_size() + 2 * pad,), 0xA5, dtype=torch.uint8,
                              device="cuda") for n in ("sum", "out", "scale", "rstd")}
        at = {n: b.data_ptr() + pad for n, b in bufs.items()}
        n = sm.SwitchNormDims(T, d, sm.SWITCH_BF16, sm.SWITCH_F32, sm.SWITCH_E4M3, 1e-6)
        sm.switch_norm_fwd(n, x, a, w, at["sum"], at["out"], at["scale"], at["rstd"],
                           stream=torch.cuda.current_stream())
        for name, b in bufs.items():
            assert (b[:pad] == 0xA5).all() and (b[-pad:] == 0xA5).all(), name
            assert torch.equal(b[pad:-pad], want[name].contiguous().view(-1).view(torch.uint8)), name


def test_streams_and_graphs():
    x, a, w = rows(300, 768, BF16, 80), rows(300, 768, F32, 81), 1 + rows(1, 768, F32, 82, 0.3)[0]
    g = rows(300, 768, F32, 83)
    f0 = sm.norm_fwd(x, w, delta=a, out_dtype=E4M3)
    b0 = sm.norm_bwd(f0["sum"], w, f0["rstd"], g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    f1 = sm.norm_fwd(x, w, delta=a, out_dtype=E4M3, stream=side)
    b1 = sm.norm_bwd(f1["sum"], w, f1["rstd"], g, stream=side.cuda_stream)
    side.synchronize()
    x2, a2 = x.clone(), a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f2 = sm.norm_fwd(x2, w, delta=a2, out_dtype=E4M3)
        b2 = sm.norm_bwd(f2["sum"], w, f2["rstd"], g)
    x2.zero_(), a2.zero_()
    graph.replay()
    x2.copy_(x), a2.copy_(a)
    graph.replay()
    torch.cuda.synchronize()
    for f, b in ((f1, b1), (f2, b2)):
        assert torch.equal(f["out"].view(torch.uint8), f0["out"].view(torch.uint8))
        assert torch.equal(f["sum"], f0["sum"]) and torch.equal(f["scale"], f0["scale"])
        assert torch.equal(b["dresidual"], b0["dresidual"]) and torch.equal(b["dweight"], b0["dweight"])
