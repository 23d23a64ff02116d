"""The layer for a few tokens where values of very different sizes meet within one row of x or of the hidden
activations, and where an expert only passes values through, so that a lost term of a cut operand shows.

Passing through: with one expert the gate is exp(0) / 1 = 1, and with selections for weights every sum has one term,
so y is h as the second product's operand holds it: float32 and three bfloat16 terms hold it exactly, five e4m3 terms
(three hold the 11 bits of a float16, which leaves 2^-11 of the value; two more take 1 / 17 of what is left each; the
rest, kept in 11 bits, is off by 2^-22) within 2^-19, and within 2^-33 of the row's largest value where that is more.
"""
import pytest
import torch

import sparse_mixture_experts_fp32_b200 as sm
from test_gpu_few import BF16, E4M3, F32, U, check, make, plain, run

pytestmark = pytest.mark.gpu

WEIGHTS = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
HELD = {"f32": 0.0, "bf16": 0.0, "e4m3": 2.0 ** -19}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return sm.lib()


def select(rows, cols, pairs, dtype):
    """[1, rows, cols] weights of zeros with ones at `pairs`."""
    w = torch.zeros(1, rows, cols, device="cuda")
    for r, c in pairs:
        w[0, r, c] = 1
    return w.to(dtype)


def through(w, x, F, into, out_of, d, flags=0):
    p = dict(x=x, w_r=torch.zeros(1, d, device="cuda"), logit_bias=None, w_in=select(F, d, into, WEIGHTS[w]),
             w_out=select(d, F, out_of, WEIGHTS[w]))
    if w == "e4m3":
        p["w_in_scale"], p["w_out_scale"] = torch.ones(1, F, device="cuda"), torch.ones(1, d, device="cuda")
    r = run(p, 1, x.shape[0], flags=flags)
    assert (r["gate"] == 1).all()
    return r["y"]


def uniform(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(*shape, device="cuda", generator=g)


@pytest.mark.parametrize("T", [1, 9, 40])
@pytest.mark.parametrize("power", [0, 9, 13, 17, 22, 28])
def test_x_is_held_beside_large_channels(T, power):
    """bfloat16 x in [1, 2) beside channels of 2^power that no weight takes: every bit of it is multiplied."""
    d, F = 128, 64
    x = torch.zeros(T, d, device="cuda")
    x[:, :64] = 1 + uniform(200 + power, T, 64)
    x[:, 70], x[:, 127] = 2.0 ** power, -(2.0 ** power)
    x = x.to(BF16)
    same = [(j, j) for j in range(64)]
    y = through("e4m3", x, F, same, same, d)
    want = x[:, :64].double()
    assert ((y[:, :64].double() - want).abs() <= HELD["e4m3"] * 1.01 * want).all()
    assert (y[:, 64:] == 0).all()


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("power", [8, 12, 15, 18])
@pytest.mark.parametrize("T,d,F,N,k", [(3, 1088, 192, 4, 1), (24, 4096, 128, 2, 2)])
def test_large_channels_within_a_token(T, d, F, N, k, power, zeros):
    """A channel of 2^power among normal ones, its weights as the others' or zeros: within the bounds that tokens
    without one have.  (The router does not look at it: the choices would hang on it alone.)"""
    p = make(T, d, F, N, "e4m3", seed=300 + power)
    at = 77
    p["x"][:, at] = (2.0 ** power * (1 + uniform(301, T))).to(BF16)
    p["w_r"][:, at] = 0
    if zeros:
        p["w_in"].view(torch.uint8)[:, :, at] = 0
    want = plain(p, k, T)
    check(run(p, k), want, k)
    check(run(p, k, flags=sm.SWITCH_FLAG_SIMT_FFN), want, k)


def in_three(v):
    """float32 values as three bfloat16 ones of 8 bits each, all of v's sign, whose sum is v."""
    hi = (v.view(torch.int32) & -65536).view(F32)
    rest = v - hi
    mid = (rest.view(torch.int32) & -65536).view(F32)
    return hi, mid, rest - mid


def hidden(seed, T, w, d, large):
    """x and the selections whose hidden row is v (24 bits, in [1, 2)) at 0..59 and 2^large at 63, and v."""
    v = 1 + uniform(seed, T, 60)
    x = torch.zeros(T, d, device="cuda")
    at = [0, d // 2, d - 64]  # in parts of their own where a row is cut
    into = []
    for a, piece in zip(at, in_three(v)):
        x[:, a:a + 60] = piece
        into += [(j, a + j) for j in range(60)]
    x[:, d - 1] = 2.0 ** large
    into.append((63, d - 1))
    return x.to(F32 if w == "f32" else BF16), into, v.double()


@pytest.mark.parametrize("T", [1, 5, 33])
@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("d,large", [(256, 0), (256, 9), (256, 14), (2112, 0), (2112, 12), (2112, 19)])
def test_hidden_values_are_held_beside_large_ones(T, w, d, large):
    """A hidden value of 2^large that no weight of the second product takes (and its x, which rounds the smallest
    pieces of v to 2^-37 of it)."""
    F = 64
    x, into, v = hidden(400 + large, T, w, d, large)
    y = through(w, x, F, into, [(j, j) for j in range(60)], d)
    floor = (2.0 ** -33 + 3 * 2.0 ** -37) * 2.0 ** large if w == "e4m3" else 0.0
    assert ((y[:, :60].double() - v).abs() <= HELD[w] * 1.01 * v + floor).all()
    assert (y[:, 60:] == 0).all()


@pytest.mark.parametrize("T", [1, 5, 33])
@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("d", [256, 2112])
@pytest.mark.parametrize("large", [10, 24, 60])
def test_what_relu_removes_takes_no_bits(T, w, d, large):
    """A pre-activation of -2^large in the same row."""
    F = 64
    x, into, v = hidden(500 + large, T, w, d, 0)
    x[:, d - 2] = 1
    p_in, p_out = select(F, d, into[:-1], F32), select(d, F, [(j, j) for j in range(60)], WEIGHTS[w])
    p_in[0, 62, d - 2] = -1.0 if w == "e4m3" else -(2.0 ** large)
    p_out[0, :, 62] = 1  # it would show everywhere
    p = dict(x=x, w_r=torch.zeros(1, d, device="cuda"), logit_bias=None, w_in=p_in.to(WEIGHTS[w]), w_out=p_out)
    if w == "e4m3":
        p["w_in_scale"], p["w_out_scale"] = torch.ones(1, F, device="cuda"), torch.ones(1, d, device="cuda")
        p["w_in_scale"][0, 62] = 2.0 ** large
    y = run(p, 1, T)["y"]
    assert ((y[:, :60].double() - v).abs() <= HELD[w] * 1.01 * v).all()
    assert (y[:, 60:] == 0).all()


def test_a_handle_follows_weights_that_move():
    """.data replaced by the same weights elsewhere: read there.  By others of its kind: those."""
    p = make(5, 128, 256, 4, "bf16", seed=70)
    layer = sm.FewLayer(p["w_r"], p["w_in"], p["w_out"], top_k=2)
    want = layer(p["x"])["y"]
    old = p["w_in"].data
    p["w_in"].data = old.clone()
    assert torch.equal(layer(p["x"])["y"], want)
    p["w_in"].data = old * 2
    got = layer(p["x"])["y"]
    assert torch.equal(got, sm.layer_fwd_few(p["x"], p["w_r"], old * 2, p["w_out"], top_k=2)["y"])
    p["w_in"].data = old[:, :128].contiguous()
    with pytest.raises(ValueError):
        layer(p["x"])
    p["w_in"].data = old.float()
    with pytest.raises(TypeError):
        layer(p["x"])
    p["w_in"].data = old
    assert torch.equal(layer(p["x"])["y"], want)
