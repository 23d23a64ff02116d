"""The layer for a few tokens on the GPU against the definition in 64 bits, at sizes and routings where it can go
wrong, with float32, bfloat16 and 8-bit experts.

Tolerances.  A product of a weight and an input is exact (8 x 8, 8 x 4 or 4 x 4 significant bits) or rounded once
(float32), and a sum of K of them is, in every kernel here, at most ADDS(K) = 64 + K / 64 additions deep, each off by
at most 2^-23 of the sum of the magnitudes so far (the tensor cores truncate, CUDA cores round).  So
  |h - h_exact| <= ADDS(d) 2^-23 |W_in| |x|,   |o - o_exact| <= (ADDS(F) 2^-23 + 2^-19) |W_out| |h| + |W_out| |dh|
(2^-19 covers the terms that h is cut into, five of 4 bits or three of 8) and y adds a few roundings and the gates'
error.  Logits are within (32 + d / 256) 2^-24 |w_r| |x|; a softmax value moves by twice that, relatively, and by a
few 2^-24 of the exponentials.  Inputs are such that no token's choices are closer than the logits' bound (asserted).
"""
import pytest
import torch

import oracle
import sparse_mixture_experts_fp32_b200 as sm

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return sm.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=F32):
    return torch.empty(*shape, device="cuda").normal_(0, std, generator=g).to(dtype)


def make(T, d, F, N, w="bf16", x=None, seed=0, bias=None):
    g = gen(1000 + seed)
    p = dict(w_r=normal(g, N, d, std=d ** -0.5), logit_bias=bias)
    p["x"] = normal(g, T, d)
    if w == "e4m3":
        for n, r, c in (("w_in", F, d), ("w_out", d, F)):
            # rows of different sizes, so that a scale at the wrong row shows
            t = normal(g, N, r, c, std=c ** -0.5) * torch.exp(normal(g, N, r, 1, std=0.5))
            q = sm.quantize_rows(t)
            p[n], p[n + "_scale"] = q["q"], q["scale"]
        if x == "e4m3":
            q = sm.quantize_rows(p["x"])
            p["x"], p["x_scale"] = q["q"], q["scale"]
        else:
            p["x"] = p["x"].to(BF16)
    else:
        dt = F32 if w == "f32" else BF16
        p["w_in"], p["w_out"] = normal(g, N, F, d, std=d ** -0.5).to(dt), normal(g, N, d, F, std=F ** -0.5).to(dt)
        p["x"] = p["x"].to(dt)
    return p


def run(p, k, C=None, flags=0, **more):
    r = sm.layer_fwd_few(p["x"], p["w_r"], p["w_in"], p["w_out"], top_k=k, capacity=C, logit_bias=p["logit_bias"],
                         x_scale=p.get("x_scale"), w_in_scale=p.get("w_in_scale"), w_out_scale=p.get("w_out_scale"),
                         flags=flags, **more)
    assert sm.switch_check(r["workspace"]) == 0
    return r


def plain(p, k, C):
    """The definition in 64 bits, and the bounds of the module's text."""
    X = p["x"].double()
    if p.get("x_scale") is not None:
        X = X * p["x_scale"].double()[:, None]
    W_r = p["w_r"].double()
    T, d = X.shape
    N, F = p["w_in"].shape[:2]
    h = X @ W_r.T
    if p["logit_bias"] is not None:
        h = h + p["logit_bias"].double()
    size = h.abs().masked_fill(torch.isinf(h), 0)  # a bias of minus infinity takes its expert out, exactly
    slack = ((32 + d / 256) * U * (X.abs() @ W_r.abs().T + size)).amax(1)
    order = torch.sort(h, dim=1, descending=True, stable=True)
    for c in range(min(k, N - 1)):
        gap = order.values[:, c] - order.values[:, c + 1]
        assert ((gap > 2 * slack) | (gap == 0)).all(), "inputs with a near tie"
    expert = order.indices[:, :k]
    prob = torch.softmax(h, 1)
    gate = prob.gather(1, expert)
    ex = expert.tolist()
    seen, slot = [0] * N, [[-1] * k for _ in range(T)]
    for c in range(k):
        for t in range(T):
            e = ex[t][c]
            slot[t][c] = seen[e] if seen[e] < C else -1
            seen[e] += 1
    y, by = torch.zeros(T, d, dtype=torch.float64, device="cuda"), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    adds = lambda K: (64 + K / 64) * 2 * U  # noqa: E731
    grel = 4 * slack + 16 * U
    for e in sorted({e for row in ex for e in row}):
        Wi, Wo = p["w_in"][e].double(), p["w_out"][e].double()
        if p.get("w_in_scale") is not None:
            Wi, Wo = Wi * p["w_in_scale"][e].double()[:, None], Wo * p["w_out_scale"][e].double()[:, None]
        for t in range(T):
            for c in range(k):
                if ex[t][c] != e or slot[t][c] < 0:
                    continue
                z = Wi @ X[t]
                H = z.clamp_min(0)
                bh = adds(d) * (Wi.abs() @ X[t].abs()) + 4 * U * z.abs()
                o, bo = Wo @ H, Wo.abs() @ bh + (adds(F) + 32 * U) * (Wo.abs() @ H)
                y[t] += gate[t, c] * o
                by[t] += gate[t, c] * (bo + (grel[t] + 6 * U) * o.abs())
    first = torch.zeros(N, dtype=torch.float64, device="cuda")
    for row in ex:
        first[row[0]] += 1.0 / T
    aux = N * (first * prob.mean(0)).sum()
    return dict(y=y, by=by, expert=expert.int(), gate=gate, grel=grel[:, None], slot=torch.tensor(slot, device="cuda"),
                counts=torch.tensor(seen, device="cuda"), aux=aux, arel=grel.max())


def check(r, want, k):
    sq = (lambda t: t.squeeze(1)) if k == 1 else (lambda t: t)
    assert torch.equal(r["expert"], sq(want["expert"]))
    assert torch.equal(r["slot"].long(), sq(want["slot"])) and torch.equal(r["counts"].long(), want["counts"])
    assert ((r["gate"].double() - sq(want["gate"])).abs() <= sq(want["gate"] * want["grel"])).all()
    assert abs(r["aux"].double().item() - want["aux"].item()) <= want["aux"].item() * (want["arel"].item() + 4 * U)
    off = (r["y"].double() - want["y"]).abs()
    assert (off <= want["by"]).all(), (off - want["by"]).max()


WX = [("f32", None), ("bf16", None), ("e4m3", None), ("e4m3", "e4m3")]


@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("w,x", WX)
@pytest.mark.parametrize("T,d,F,N", [(1, 64, 64, 2), (1, 512, 1088, 5), (2, 64, 192, 3), (7, 192, 320, 4),
                                     (8, 1024, 256, 16), (9, 256, 1024, 64), (33, 320, 448, 3), (64, 128, 576, 2),
                                     (64, 192, 64, 256), (31, 2112, 64, 8), (32, 1024, 1024, 128)])
def test_few(T, d, F, N, w, x, k):
    p = make(T, d, F, N, w, x, seed=T + d)
    check(run(p, k), plain(p, k, T), k)


@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("T,d,F,N", [(1, 1, 1, 2), (3, 5, 7, 2), (13, 509, 1021, 6), (64, 33, 17, 3), (5, 66, 130, 9),
                                     (17, 1000, 6, 4), (2, 4, 2004, 2)])
def test_few_f32_odd_sizes(T, d, F, N, k):
    p = make(T, d, F, N, "f32", seed=T)
    check(run(p, k), plain(p, k, T), k)


@pytest.mark.parametrize("w,x", WX[1:])
@pytest.mark.parametrize("T", [1, 19])
def test_few_on_cuda_cores(T, w, x):
    """SWITCH_FLAG_SIMT_FFN for 16- and 8-bit experts."""
    p = make(T, 256, 384, 5, w, x, seed=3)
    check(run(p, 2, flags=sm.SWITCH_FLAG_SIMT_FFN), plain(p, 2, T), 2)


@pytest.mark.parametrize("w,x", WX)
@pytest.mark.parametrize("k,C", [(1, 1), (2, 1), (2, 5), (1, 100)])
def test_capacity_drops(w, x, k, C):
    T, N = 40, 4
    bias = torch.tensor([2.0, 0.0, 1.0, -1.0], device="cuda")
    p = make(T, 128, 192, N, w, x, seed=5, bias=bias)
    want = plain(p, k, C)
    r = run(p, k, C)
    check(r, want, k)
    gone = (want["slot"] < 0).all(1)
    assert (r["y"][gone] == 0).all()
    if C == 1:
        assert gone.any()


@pytest.mark.parametrize("w,x", WX)
def test_every_token_to_one_expert(w, x):
    """64 tokens on expert 2 (more than one group), and biases of minus infinity on others."""
    T, N = 64, 6
    bias = torch.tensor([0.0, -float("inf"), 50.0, -float("inf"), -float("inf"), 0.5], device="cuda")
    p = make(T, 128, 192, N, w, x, seed=6, bias=bias)
    r = run(p, 1)
    assert (r["expert"] == 2).all() and torch.equal(r["slot"], torch.arange(T, dtype=torch.int32, device="cuda"))
    check(r, plain(p, 1, T), 1)
    r2 = run(p, 2)
    assert (r2["expert"][:, 0] == 2).all() and ((r2["expert"][:, 1] == 0) | (r2["expert"][:, 1] == 5)).all()


def test_ties_go_to_the_lowest_index():
    p = make(9, 64, 64, 8, "bf16", seed=7)
    p["w_r"][:] = p["w_r"][:1]  # the same logits for every expert, bit for bit
    r = run(p, 2)
    assert (r["expert"][:, 0] == 0).all() and (r["expert"][:, 1] == 1).all()
    assert torch.allclose(r["gate"], torch.full((9, 2), 0.125, device="cuda"), rtol=1e-6, atol=0)
    check(r, plain(p, 2, 9), 2)


@pytest.mark.parametrize("w,x", WX)
def test_large_and_small_inputs(w, x):
    """Tokens of very different sizes, zeros among them, beside one another."""
    p = make(6, 192, 256, 4, w, x, seed=8)
    size = torch.tensor([1e-20, 1.0, 0.0, 1e4, 1e-6, 3e2], device="cuda")
    if x == "e4m3":
        p["x_scale"] = p["x_scale"] * size
    else:
        p["x"] = (p["x"].float() * size[:, None]).to(p["x"].dtype)
    # sizes make the logits differ too much to compare choices of tiny ones: they go by the bias
    p["logit_bias"] = torch.tensor([0.1, 0.3, 0.2, 0.0], device="cuda")
    check(run(p, 1), plain(p, 1, 6), 1)


@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_not_finite_stays_apart(w, bad):
    p = make(12, 128, 192, 4, w, seed=9)
    clean = run(p, 1)
    p["x"][5, 17] = bad
    r = run(p, 1)
    rows = [t for t in range(12) if t != 5]
    assert not torch.isfinite(r["y"][5]).all()
    assert (r["expert"] >= 0).all() and (r["expert"] < 4).all()
    assert torch.equal(r["expert"][rows], clean["expert"][rows])
    assert torch.isfinite(r["y"][rows]).all()
    assert torch.allclose(r["y"][rows], clean["y"][rows], rtol=1e-4, atol=1e-5)


def test_no_tokens():
    p = make(1, 64, 64, 3, "bf16", seed=10)
    p["x"] = p["x"][:0]
    r = run(p, 1)
    assert r["y"].shape == (0, 64) and (r["counts"] == 0).all() and r["aux"].item() == 0


def test_agrees_with_the_layer_and_the_oracle():
    """The same routing outputs as switch_layer_fwd and switch_layer_fwd_top2, and their y up to bfloat16 rounding
    of the hidden activations there (2^-8 of each, as switch_layer_fwd rounds them)."""
    T, d, F, N, C = 48, 256, 512, 8, 9
    p = make(T, d, F, N, "bf16", seed=11, bias=torch.linspace(0.5, -0.5, 8, device="cuda"))
    orc = oracle.Oracle()
    host = lambda t: t.view(torch.int16).cpu().numpy().view("uint16") if t.dtype == BF16 else t.cpu().numpy()  # noqa: E731
    for k, layer in ((1, sm.layer_fwd), (2, sm.layer_fwd_top2)):
        a = run(p, k, C)
        b = layer(p["x"], p["w_r"], p["w_in"], p["w_out"], capacity=C, logit_bias=p["logit_bias"])
        for n in ("expert", "slot", "counts"):
            assert torch.equal(a[n], b[n]), n
        assert torch.allclose(a["gate"], b["gate"], rtol=2e-5, atol=0)
        assert torch.allclose(a["aux"], b["aux"], rtol=2e-5, atol=0)
        rms = a["y"].square().mean().sqrt()
        assert (a["y"] - b["y"]).abs().max() <= 2e-2 * rms
    o = orc.layer_fwd(host(p["x"]), host(p["w_r"]), host(p["w_in"]), host(p["w_out"]), capacity=C,
                      bias=host(p["logit_bias"]), want_probs=True)
    a = run(p, 1, C)
    y = torch.from_numpy(o["y"]).cuda()
    assert ((a["y"].double() - y).abs() <= plain(p, 1, C)["by"] + 1e-12).all()


def test_same_bytes_every_time():
    for w, x in WX:
        p = make(37, 256, 640, 6, w, x, seed=12)
        want = run(p, 2)
        for _ in range(20):
            r = run(p, 2)
            for n in ("y", "gate", "expert", "slot", "counts", "aux"):
                assert torch.equal(r[n], want[n]), (w, n)


def test_handle_results_and_stale_workspaces():
    p = make(5, 128, 256, 4, "bf16", seed=13)
    layer = sm.FewLayer(p["w_r"], p["w_in"], p["w_out"], top_k=2)
    want = layer(p["x"])
    size = layer._dims(5)[2]
    ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")  # needs no initialisation
    r = layer(p["x"], ws=ws)
    assert torch.equal(r["y"], want["y"]) and r["workspace"] is ws
    y0 = want["y"].clone()
    again = layer(p["x"], out=want)
    assert again is want and torch.equal(again["y"], y0)
    with pytest.raises(ValueError):
        layer(p["x"][:3], out=want)
    with pytest.raises(sm.SwitchError) as e:
        layer(p["x"], ws=ws[:256])
    assert e.value.status == 5
    p["w_in"].mul_(2)  # the weights are read at each call
    assert not torch.equal(layer(p["x"])["y"], y0)


def test_refusals():
    p = make(4, 128, 256, 4, "bf16", seed=14)
    layer = sm.FewLayer(p["w_r"], p["w_in"], p["w_out"])
    with pytest.raises(TypeError):
        layer(p["x"].float())
    with pytest.raises(ValueError):
        layer(p["x"][:, :64])
    with pytest.raises(TypeError):
        layer(p["x"].t().contiguous().t())
    with pytest.raises(ValueError):
        layer(p["x"], x_scale=torch.ones(4, device="cuda"))
    with pytest.raises(sm.SwitchError) as e:
        layer(p["x"].repeat(17, 1))  # 68 tokens
    assert e.value.status == 2
    with pytest.raises(sm.SwitchError):
        sm.FewLayer(p["w_r"], p["w_in"], p["w_out"], top_k=3)
    with pytest.raises(sm.SwitchError):
        sm.FewLayer(p["w_r"][:1], p["w_in"][:1], p["w_out"][:1], top_k=2)
    with pytest.raises(ValueError):
        sm.FewLayer(p["w_r"][:3], p["w_in"], p["w_out"])
    with pytest.raises(TypeError):
        sm.FewLayer(p["w_r"].double(), p["w_in"], p["w_out"])
    with pytest.raises(ValueError):
        sm.FewLayer(p["w_r"], p["w_in"].to(E4M3), p["w_out"].to(E4M3))


def test_writes_stay_inside():
    for w, x in WX:
        T, d, F, N, k, pad = 11, 192, 320, 5, 2, 256
        p = make(T, d, F, N, w, x, seed=15)
        want = run(p, k)
        code = {"f32": sm.SWITCH_F32, "bf16": sm.SWITCH_BF16, "e4m3": sm.SWITCH_E4M3}[w]
        dims = sm.dims(T, d, F, N, T, code)
        need = sm.switch_few_workspace_size(dims, k)
        names = ("y", "expert", "gate", "slot", "counts", "aux")
        sizes = {n: want[n].numel() * 4 for n in names}
        sizes["ws"] = need
        bufs = {n: torch.full((s + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda") for n, s in sizes.items()}
        at = {n: b.data_ptr() + pad for n, b in bufs.items()}
        sm.switch_layer_fwd_few(dims, k, p["x"], p.get("x_scale"), p["w_r"], None, p["w_in"], p.get("w_in_scale"),
                                p["w_out"], p.get("w_out_scale"), *[at[n] for n in names],
                                bufs["ws"][pad:pad + need])
        for n, b in bufs.items():
            assert (b[:pad] == 0xA5).all() and (b[pad + sizes[n]:] == 0xA5).all(), n
            if n != "ws":
                assert torch.equal(b[pad:pad + sizes[n]], want[n].contiguous().view(-1).view(torch.uint8)), n


@pytest.mark.parametrize("w,x", WX)
def test_streams_and_graphs(w, x):
    """Calls on two streams at once, and two graphs replayed at once, from one handle."""
    ps = [make(T, 512, 1024, 8, w, x, seed=16 + T) for T in (3, 24)]
    for q in ps[1:]:
        for n in ("w_r", "w_in", "w_out", "w_in_scale", "w_out_scale"):
            if n in ps[0]:
                q[n] = ps[0][n]
    layer = sm.FewLayer(ps[0]["w_r"], ps[0]["w_in"], ps[0]["w_out"], top_k=2, w_in_scale=ps[0].get("w_in_scale"),
                        w_out_scale=ps[0].get("w_out_scale"))
    want = [layer(q["x"], x_scale=q.get("x_scale")) for q in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(10):
        got = [layer(q["x"], x_scale=q.get("x_scale"), stream=s) for q, s in zip(ps, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a["y"], b["y"]) and torch.equal(a["expert"], b["expert"])
            assert sm.switch_check(a["workspace"]) == 0
    graphs, outs = [], []
    for q in ps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(layer(q["x"], x_scale=q.get("x_scale")))
    for _ in range(10):
        for o in outs:
            o["y"].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a["y"], b["y"]) and torch.equal(a["slot"], b["slot"])


def test_captured_behind_a_join_of_streams():
    """A call whose stream has just waited for another one, eagerly and captured: its first kernel may start early
    only behind both."""
    p = make(9, 256, 512, 6, "bf16", seed=17)
    layer = sm.FewLayer(p["w_r"], p["w_in"], p["w_out"], top_k=2)
    want = layer(p["x"])
    x, src, side = torch.zeros_like(p["x"]), p["x"].clone(), torch.cuda.Stream()
    big = torch.zeros(1 << 26, device="cuda")

    def call():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            big.add_(1)  # long enough that x is late
            x.copy_(src)
        main.wait_stream(side)
        return layer(x)

    torch.cuda.synchronize()
    r = call()
    torch.cuda.synchronize()
    assert torch.equal(r["y"], want["y"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call()
    for _ in range(3):
        x.zero_(), r["y"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r["y"], want["y"]) and torch.equal(r["expert"], want["expert"])


def test_calls_on_one_stream_follow_one_another():
    """Calls of different layers and sizes behind one another without a wait, one's y the next one's delta."""
    ps = [make(T, 256, F, N, w, seed=40 + T) for T, F, N, w in ((7, 512, 4, "bf16"), (7, 320, 9, "f32"), (7, 64, 2, "e4m3"))]
    nw = torch.ones(256, device="cuda")
    res = normal(gen(41), 7, 256)

    def chain(wait):
        s, delta, ys = res, None, []
        for q in ps:
            b = sm.block_fwd(s, nw, q["w_r"], q["w_in"], q["w_out"], delta=delta, top_k=2, capacity=7,
                             w_in_scale=q.get("w_in_scale"), w_out_scale=q.get("w_out_scale"))
            s, delta = b["sum"], b["y"]
            ys.append(delta)
            if wait:
                torch.cuda.synchronize()
        return ys

    want = chain(True)
    for _ in range(10):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3"])
def test_block(w):
    """Residual, norm and layer as they are used: a step's block against the definition in 64 bits.  The norm's
    rounding of x (bf16 2^-8, e4m3 2^-4 of a value) is taken from the block itself: its x goes into the definition."""
    T, d, F, N = 20, 256, 384, 6
    p = make(T, d, F, N, w, seed=18)
    g = gen(19)
    res, delta = normal(g, T, d, std=3.0, dtype=BF16), normal(g, T, d)
    nw = 1 + normal(g, d, std=0.2)
    b = sm.block_fwd(res, nw, p["w_r"], p["w_in"], p["w_out"], delta=delta, top_k=2, capacity=T,
                     w_in_scale=p.get("w_in_scale"), w_out_scale=p.get("w_out_scale"))
    assert torch.equal(b["sum"], (res.float() + delta).to(BF16))
    s = b["sum"].double()
    x = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6) * nw.double()
    got = b["x"].double() * (1 if b["x_scale"] is None else b["x_scale"].double()[:, None])
    half = {"f32": 64 * U, "bf16": 2.0 ** -8 * 1.001, "e4m3": 2.0 ** -4 * 1.001}[w]
    floor = x.abs().amax(1, keepdim=True) / 448 * 2.0 ** -10 * 1.001 if w == "e4m3" else 0
    assert ((got - x).abs() <= half * x.abs() + floor).all()
    check(b, plain(dict(p, x=b["x"], x_scale=b["x_scale"]), 2, T), 2)


def test_block_training_step():
    """block_fwd and block_bwd with SWITCH_FLAG_TRAINING against the pieces, and dresidual against differences of
    the norm's formula around the layer's dx."""
    T, d, F, N = 96, 128, 256, 4
    p = make(T, d, F, N, "bf16", seed=20)
    g = gen(21)
    res, delta, nw = normal(g, T, d), normal(g, T, d), 1 + normal(g, d, std=0.2)
    f = sm.block_fwd(res, nw, p["w_r"], p["w_in"], p["w_out"], delta=delta, capacity=T, flags=sm.SWITCH_FLAG_TRAINING)
    dy, dsum = normal(g, T, d), normal(g, T, d)
    got = sm.block_bwd(f, nw, p["w_r"], p["w_in"], p["w_out"], dy, dsum=dsum, g_aux=0.01)
    n = sm.norm_fwd(res, nw, delta=delta, out_dtype=BF16)
    lf = sm.layer_fwd(n["out"], p["w_r"], p["w_in"], p["w_out"], capacity=T, flags=sm.SWITCH_FLAG_TRAINING)
    lb = sm.layer_bwd(lf, n["out"], p["w_r"], p["w_in"], p["w_out"], dy, 0.01)
    nb = sm.norm_bwd(n["sum"], nw, n["rstd"], lb["dx"], dsum=dsum)
    assert torch.equal(f["y"], lf["y"]) and torch.equal(got["dresidual"], nb["dresidual"])
    assert torch.equal(got["dnorm_weight"], nb["dweight"]) and torch.equal(got["dw_in"], lb["dw_in"])
    S, W, dx = n["sum"].double(), nw.double(), lb["dx"].double()
    loss = lambda s: ((s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6) * W) * dx).sum() + (s * dsum.double()).sum()  # noqa: E731
    e = normal(g, T, d).double()
    diff = (loss(S + 1e-5 * e) - loss(S - 1e-5 * e)) / 2e-5
    along = got["dresidual"].double() * e
    assert abs(diff - along.sum()) <= 1e-5 * along.abs().sum()
