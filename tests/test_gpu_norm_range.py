"""Residual + norm and 8-bit rows at the ends of float32's range: rows whose squares are beyond it, rows of zeros
without an eps, beside ordinary rows.  Tolerances as in test_gpu_norm.py: a scaled row has the same roundings."""
import pytest
import torch

import sparse_mixture_experts_fp32_b200 as sm
from test_gpu_norm import BF16, E4M3, F32, U, check_e4m3, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return sm.lib()


def sized(T, d, dtype, seed, powers):
    """Rows of normal values times 2^powers[t % len(powers)], none of which is beyond the type."""
    x = rows(T, d, F32, seed).double()
    x = x / x.abs().amax(1, keepdim=True) * 1.9
    p = torch.tensor([powers[t % len(powers)] for t in range(T)], dtype=torch.float64, device="cuda")
    return (x * torch.exp2(p)[:, None]).to(dtype)


# widths: rows held by a warp (8 to a block), by 64 threads (2 to a block), by 96 and more; multiples of 8 and not
@pytest.mark.parametrize("d", [1, 33, 256, 264, 511, 512, 777, 1024, 8185, 8191, 8192])
@pytest.mark.parametrize("res,out", [(F32, F32), (F32, BF16), (F32, E4M3), (BF16, BF16), (BF16, E4M3)])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_rows_of_every_size(d, res, out, eps):
    T = 21
    # (eps 1e-6 beside values of 2^-120: the output is below the normal range; held to half its step)
    x = sized(T, d, res, 5, [0, 126, 70, -40, 62, -60, -100, 0, 64] + ([-120] if res == F32 else []))
    w = 1 + rows(1, d, F32, 3, 0.3)[0]
    got = sm.norm_fwd(x, w, eps=eps, out_dtype=out)
    s, e = x.double(), torch.tensor(eps, dtype=F32).double().item()
    rstd = 1 / torch.sqrt(s.square().mean(1) + e)
    tiny = 2.0 ** -149
    assert ((got["rstd"].double() - rstd).abs() <= 41 * U * rstd + tiny).all()
    v = s * rstd[:, None] * w.double()
    if out == E4M3:
        ok = v.abs().amax(1) > 2.0 ** -100  # scales below the normal range have fewer bits
        check_e4m3(got["out"][ok], got["scale"][ok], v[ok], 43)
        assert (got["scale"][~ok].double() <= v.abs().amax(1)[~ok]).all() and torch.isfinite(got["out"].float()).all()
    else:
        half = 0 if out == F32 else 2.0 ** -8
        small = 2 * tiny if out == F32 else 2.0 ** -133
        assert ((got["out"].double() - v).abs() <= v.abs() * (half + 44 * U) + small).all()


@pytest.mark.parametrize("d", [8, 33, 264, 300, 1024, 4099])
@pytest.mark.parametrize("out", [F32, BF16, E4M3])
@pytest.mark.parametrize("delta", [False, True])
def test_rows_of_zeros_without_an_eps(d, out, delta):
    x = rows(19, d, F32, 6)
    x[3:12] = 0
    a = torch.zeros_like(x) if delta else None
    w = torch.ones(d, device="cuda")
    got = sm.norm_fwd(x, w, delta=a, eps=0.0, out_dtype=out)
    v = got["out"].float()
    assert (v[3:12] == 0).all() and torch.isinf(got["rstd"][3:12]).all()
    other = [t for t in range(19) if not 3 <= t < 12]
    assert torch.isfinite(v[other]).all() and torch.isfinite(got["rstd"][other]).all()
    if out == E4M3:
        assert (got["scale"][3:12] == 0).all() and (got["scale"][other] > 0).all()


@pytest.mark.parametrize("d", [33, 264, 1024])
def test_a_row_has_the_same_bytes_beside_others(d):
    """Two rows of a block: one whose squares overflow changes nothing in the other."""
    x = rows(8, d, F32, 7)
    w = 1 + rows(1, d, F32, 8, 0.3)[0]
    want = sm.norm_fwd(x, w)
    y = x.clone()
    y[::2] = sized(4, d, F32, 9, [100])
    y[4, 1], y[6, 2] = float("nan"), float("inf")
    got = sm.norm_fwd(y, w)
    assert torch.equal(got["out"][1::2], want["out"][1::2]) and torch.equal(got["rstd"][1::2], want["rstd"][1::2])
    assert torch.isfinite(got["out"][[0, 2]]).all()
    assert not torch.isfinite(got["out"][4]).all() and not torch.isfinite(got["out"][6]).all()


@pytest.mark.parametrize("power", [100, 0, -45])
def test_gradient_of_large_and_small_rows(power):
    """dresidual and dweight behind a forward of such rows, against the formula in 64 bits (test_gpu_norm.py's bounds,
    and rstd's)."""
    T, d = 9, 264
    x = sized(T, d, F32, 10, [power])
    w, g = 1 + rows(1, d, F32, 11, 0.3)[0], rows(T, d, F32, 12, 0.1)
    f = sm.norm_fwd(x, w, eps=0.0)
    got = sm.norm_bwd(x, w, f["rstd"], g)
    S, W, G = x.double(), w.double(), g.double()
    R = 1 / torch.sqrt(S.square().mean(1, keepdim=True))
    H, GW = S * R, G * W
    m = (GW * H).mean(1, keepdim=True)
    size = R * (GW.abs() + H.abs() * (GW * H).abs().mean(1, keepdim=True))
    assert ((got["dresidual"].double() - R * (GW - H * m)).abs() <= 256 * U * size).all()
    assert ((got["dweight"].double() - (G * H).sum(0)).abs() <= (64 + T) * U * (G * H).abs().sum(0)).all()


@pytest.mark.parametrize("cols", [7, 64, 1000, 1024, 4099])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantized_rows_use_the_whole_range(cols, dtype):
    """A row's largest value is 448 scales: it has the code of 448, in every finite row that is not zero."""
    x = rows(40, cols, dtype, 13, 0.1)
    q = sm.quantize_rows(x)["q"].float()
    top = x.float().abs().argmax(1, keepdim=True)
    assert (q.gather(1, top).abs() == 448).all() and (q.gather(1, top).sign() == x.float().gather(1, top).sign()).all()
