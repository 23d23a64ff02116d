"""The terms that the layer for a few tokens cuts its operands into, emulated: what they hold, that the tests' bounds
are those, and that a term less would not pass them."""
import pytest
import torch

from test_gpu_few_range import HELD

E4M3, E5M2, F16, F32 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float16, torch.float32


def bfloat16_terms(v, n):
    left, terms = v.float(), []
    for _ in range(n):
        terms.append(left.to(torch.bfloat16).float())
        left = left - terms[-1]
    return sum(t.double() for t in reversed(terms))


def power(v, top):
    """Of two, that brings each row's largest value into [2^top, 2^(top + 1))."""
    return torch.exp2(top - torch.floor(torch.log2(v.abs().amax(-1, keepdim=True).double())))


def e4m3_terms(v, n, carry=True):
    """v >= 0; three terms of its float16, then two of what float16 and they have left."""
    up = power(v, 7)
    s = (v.double() * up).float()
    left = top = s.to(F16)
    terms = []
    for t in range(n):
        if t == 3:
            rest = ((s - top.float()) * 4096).to(F16)
            left = left + rest if carry else rest
        q = left.to(E4M3)
        terms.append(q.double())
        left = (left - q.to(F16)) * 16
    return sum(t / 16.0 ** i for i, t in enumerate(terms)) / up


def e5m2_terms(x, n):
    up = power(x, 14)
    left = (x.double() * up).to(F16)
    terms = []
    for _ in range(n):
        q = left.to(E5M2)
        terms.append(q.double())
        left = (left - q.to(F16)) * 8
    return sum(t / 8.0 ** i for i, t in enumerate(terms)) / up


def values(seed, *shape):
    return 1 + torch.rand(*shape, generator=torch.Generator().manual_seed(seed))


def test_hidden_values_in_bfloat16():
    v = values(1, 64, 60)
    assert torch.equal(bfloat16_terms(v, 3), v.double())
    assert not torch.equal(bfloat16_terms(v, 2), v.double())


@pytest.mark.parametrize("large", [0, 9, 14, 19, 24])
def test_hidden_values_in_e4m3(large):
    v = values(2 + large, 64, 60)
    row = torch.cat([v, torch.full((64, 1), 2.0 ** large)], 1)
    off = lambda *a: (e4m3_terms(row, *a)[:, :60] - v.double()).abs()  # noqa: E731
    # half of the fifth term's smallest step, 2^-10 / 16^4 of a largest value of 2^7 at least, and half of float16's
    # step below 2^-5 where the fourth term begins, 2^-17 / 16^3
    bound = HELD["e4m3"] * v.double() + (2.0 ** -33 + 2.0 ** -36) * 2.0 ** large
    assert (off(5) <= bound).all()
    assert (off(4) > 1.01 * bound).any()
    if large >= 15:
        assert (off(5, False) > 1.01 * bound).any()  # the fourth term without what the third left


@pytest.mark.parametrize("large", [0, 13, 17, 22, 28])
def test_x_in_e5m2(large):
    x = values(30 + large, 64, 60).to(torch.bfloat16)
    row = torch.cat([x.float(), torch.full((64, 1), 2.0 ** large)], 1)
    assert torch.equal(e5m2_terms(row, 3)[:, :60], x.double())
    assert ((e5m2_terms(row, 2)[:, :60] - x.double()).abs() > 1.01 * HELD["e4m3"] * x.double()).any()


@pytest.mark.parametrize("below", [30, 33, 36, 40])
def test_x_below_the_range_of_its_row(below):
    x = (values(60 + below, 64, 60) * 2.0 ** -below).to(torch.bfloat16)
    row = torch.cat([x.float(), torch.full((64, 1), 1.0)], 1)
    # half of the third term's smallest step, 2^-17 / 8^2 of a largest value of 2^14 at least, and of float16's, 2^-25
    assert ((e5m2_terms(row, 3)[:, :60] - x.double()).abs() <= 2.0 ** -37 + 2.0 ** -39).all()
