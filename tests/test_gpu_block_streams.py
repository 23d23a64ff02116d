"""block_fwd and block_bwd on a stream that is not the current one: what they allocate belongs to that stream."""
import pytest
import torch

import sparse_mixture_experts_fp32_b200 as sm
from test_gpu_few import gen, make, normal

pytestmark = pytest.mark.gpu

T, D, F, N = 256, 256, 512, 4


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return sm.lib()


def busy(times=30):
    """A few milliseconds of work on the current stream."""
    big = torch.zeros(1 << 27, device="cuda")

    def work():
        for _ in range(times):
            big.add_(1)
    return work


@pytest.fixture(scope="module")
def case():
    p = make(T, D, F, N, "bf16", seed=60)
    g = gen(61)
    p.update(res=normal(g, T, D), delta=normal(g, T, D), nw=1 + normal(g, D, std=0.2), dy=normal(g, T, D),
             dsum=normal(g, T, D))
    return p


def forward(p, **more):
    return sm.block_fwd(p["res"], p["nw"], p["w_r"], p["w_in"], p["w_out"], delta=p["delta"], capacity=T, **more)


def backward(p, f, **more):
    return sm.block_bwd(f, p["nw"], p["w_r"], p["w_in"], p["w_out"], p["dy"], dsum=p["dsum"], g_aux=0.01, **more)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("top_k", [1, 2])
def test_forward_does_not_take_memory_that_the_current_stream_still_writes(case, top_k, raw):
    want = forward(case, top_k=top_k)["y"]
    side, work = torch.cuda.Stream(), busy()
    torch.cuda.synchronize()
    for _ in range(3):
        work()
        late = [torch.empty(T, D, device="cuda") for _ in range(8)]
        for t in late:
            t.fill_(float("nan"))
        del late, t
        got = forward(case, top_k=top_k, stream=side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        assert torch.equal(got["y"], want)


def test_backward_beside_writes_of_the_current_stream(case):
    f = forward(case, flags=sm.SWITCH_FLAG_TRAINING)
    want = backward(case, f)
    side, work = torch.cuda.Stream(), busy()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            work()
        got = backward(case, f, stream=side)
        over = [torch.empty(T, D, device="cuda").fill_(float("nan")) for _ in range(8)]
        torch.cuda.synchronize()
        del over
        for n in ("dresidual", "dnorm_weight", "dw_in", "dw_out", "dw_r"):
            assert torch.equal(got[n], want[n]), n


def test_a_training_step_on_a_side_stream_and_captured(case):
    want_f = forward(case, flags=sm.SWITCH_FLAG_TRAINING)
    want = backward(case, want_f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f = forward(case, flags=sm.SWITCH_FLAG_TRAINING, stream=side)
    got = backward(case, f, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(f["y"], want_f["y"]) and torch.equal(got["dresidual"], want["dresidual"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = forward(case, flags=sm.SWITCH_FLAG_TRAINING)
        got = backward(case, f)
    for _ in range(2):
        got["dresidual"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f["y"], want_f["y"]) and torch.equal(got["dresidual"], want["dresidual"])
        assert torch.equal(got["dnorm_weight"], want["dnorm_weight"])


def test_a_decoding_step_on_a_side_stream(case):
    p = dict(case)
    few = {n: p[n][:24] for n in ("res", "delta")}
    run = lambda **more: sm.block_fwd(few["res"], p["nw"], p["w_r"], p["w_in"], p["w_out"], delta=few["delta"],  # noqa: E731
                                      capacity=24, top_k=2, **more)
    want = run()["y"]
    side, work = torch.cuda.Stream(), busy()
    torch.cuda.synchronize()
    work()
    late = [torch.empty(24, D, device="cuda") for _ in range(8)]
    for t in late:
        t.fill_(float("nan"))
    del late, t
    got = run(stream=side)["y"]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
