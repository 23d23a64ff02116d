"""block_fwd, block_bwd and FewLayer without a GPU: what they refuse, and before any device work."""
import contextlib

import pytest
import torch

import sparse_mixture_experts_fp32_b200 as sm

T, D, F, N = 4, 64, 128, 4


def weights(dtype=torch.bfloat16):
    return torch.zeros(N, D), torch.zeros(N, F, D).to(dtype), torch.zeros(N, D, F).to(dtype)


@pytest.fixture
def no_calls(monkeypatch):
    """Every C function of the library raises."""
    class Library:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")
    monkeypatch.setattr(sm, "lib", lambda: Library())


def test_gradients_of_a_top2_forward_are_refused(no_calls, monkeypatch):
    monkeypatch.setattr(sm, "_current", lambda device: contextlib.nullcontext())
    w_r, w_in, w_out = weights()
    x, dy = torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(T, D)
    two = torch.zeros(T, 2, dtype=torch.int32)
    fwd = dict(expert=two, gate=two.float(), slot=two, counts=torch.zeros(N, dtype=torch.int32), capacity=T,
               workspace=torch.zeros(1 << 16, dtype=torch.uint8), x=x, sum=x, rstd=torch.ones(T))
    for flags in (None, sm.SWITCH_FLAG_TRAINING):
        if flags is not None:
            fwd["flags"] = flags
        with pytest.raises(ValueError, match="one expert per token"):
            sm.layer_bwd(fwd, x, w_r, w_in, w_out, dy)
        with pytest.raises(ValueError, match="one expert per token"):
            sm.block_bwd(fwd, torch.ones(D), w_r, w_in, w_out, dy)


def test_blocks_allocate_on_the_stream_that_they_use(monkeypatch):
    """With stream=, everything within runs with that stream as the current one, and is given none."""
    now, seen = [], []

    class under:
        def __init__(self, stream, device):
            self.stream = stream

        def __enter__(self):
            now.append(self.stream)

        def __exit__(self, *a):
            now.pop()

    def record(name, result):
        def call(*a, stream=None, **k):
            seen.append((name, now[-1] if now else None, stream))
            return dict(result)
        return call

    w_r, w_in, w_out = weights()
    x, rows = torch.zeros(100, D, dtype=torch.bfloat16), torch.zeros(100, D)
    monkeypatch.setattr(sm, "_under", under)
    monkeypatch.setattr(sm, "_current", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(sm, "norm_fwd", record("norm_fwd", dict(out=x, scale=None, sum=rows, rstd=rows[:, 0])))
    monkeypatch.setattr(sm, "norm_bwd", record("norm_bwd", dict(dresidual=rows, dweight=rows[0])))
    monkeypatch.setattr(sm, "layer_bwd", record("layer_bwd", dict(dx=rows)))
    for name in ("layer_fwd", "layer_fwd_top2"):
        monkeypatch.setattr(sm, name, record(name, dict(y=rows)))
    for k, layer in ((1, "layer_fwd"), (2, "layer_fwd_top2")):
        seen.clear()
        f = sm.block_fwd(rows, rows[0], w_r, w_in, w_out, capacity=8, top_k=k, stream="side")
        assert seen == [("norm_fwd", "side", None), (layer, "side", None)]
    seen.clear()
    sm.block_bwd(f, rows[0], w_r, w_in, w_out, rows, stream="side")
    assert seen == [("layer_bwd", "side", None), ("norm_bwd", "side", None)]
    assert not now


def test_a_handle_cannot_be_changed_under_its_plans(monkeypatch):
    """Sizes and addresses are kept per number of tokens: what they come from cannot be set, and weights that have
    other memory are checked again before it is read."""
    checked = sm._want
    monkeypatch.setattr(sm, "_want", lambda name, t, shape, dtypes, device: None if t is None else t.data_ptr())
    w_r, w_in, w_out = weights()
    bias = torch.zeros(N)
    layer = sm.FewLayer(w_r, w_in, w_out, top_k=2, capacity=3, logit_bias=bias)
    assert layer.w_in is w_in and layer.logit_bias is bias and layer.top_k == 2 and layer.capacity == 3
    assert (layer.num_experts, layer.d_ff, layer.d_model, layer.dtype) == (N, F, D, torch.bfloat16)
    for name in ("w_r", "w_in", "w_out", "logit_bias", "w_in_scale", "w_out_scale", "top_k", "capacity",
                 "capacity_factor", "flags", "num_experts", "d_ff", "d_model", "device", "dtype"):
        with pytest.raises(AttributeError):
            setattr(layer, name, None)
    assert layer._dims(7)[0].capacity == 3
    # a call comes to the checks when an address is another one, and stops there
    monkeypatch.setattr(sm, "_want", lambda name, t, *a: checked(name, t, *a) if name == "w_in" else
                        None if t is None else t.data_ptr())
    x = torch.zeros(T, D, dtype=torch.bfloat16)
    w_in.data = torch.zeros(N, F // 2, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="w_in must be"):
        layer(x)
    w_in.data = torch.zeros(N, F, D)
    with pytest.raises(TypeError, match="w_in must be"):
        layer(x)


def test_a_block_refuses_before_it_launches(no_calls):
    """Sizes and options that the layer cannot run with are found before the norm is launched."""
    w_r, w_in, w_out = weights()
    rows, nw = torch.zeros(65, D), torch.ones(D)
    e_in, e_out = w_in.to(torch.float8_e4m3fn), w_out.to(torch.float8_e4m3fn)
    scales = dict(w_in_scale=torch.ones(N, F), w_out_scale=torch.ones(N, D))
    with pytest.raises(ValueError, match="at most 64 tokens, got 65"):
        sm.block_fwd(rows, nw, w_r, e_in, e_out, capacity=8, **scales)
    with pytest.raises(ValueError, match="have w_in_scale and w_out_scale"):
        sm.block_fwd(rows[:8], nw, w_r, e_in, e_out, capacity=8)
    for t in (8, 65):
        with pytest.raises(ValueError, match="give capacity"):
            sm.block_fwd(rows[:t], nw, w_r, w_in, w_out)
        for k in (0, 3):
            with pytest.raises(ValueError, match="top_k must be 1 or 2"):
                sm.block_fwd(rows[:t], nw, w_r, w_in, w_out, capacity=8, top_k=k)


@pytest.fixture
def on_the_host(monkeypatch):
    """The Python of the calls on CPU tensors, up to the launch."""
    launched = []
    monkeypatch.setattr(sm, "_rows", lambda name, t: (t.shape, t.device))
    monkeypatch.setattr(sm, "_want", lambda name, t, *a: None if t is None else t.data_ptr())
    monkeypatch.setattr(sm, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(sm, "_launch", lambda fn, where, *a: launched.append(where))
    return launched


def test_an_input_may_not_be_a_tensor_of_the_result_that_is_overwritten(on_the_host):
    x, w = torch.ones(T, D), torch.ones(D)
    r = sm.norm_fwd(x, w, delta=x.clone())
    sm.norm_fwd(x, w, delta=x, out=r)
    sm.norm_fwd(r["sum"], w, delta=x, out=r)  # sum may be residual
    for bad in (dict(residual=r["out"], delta=x), dict(residual=x, delta=r["out"]), dict(residual=x, delta=r["sum"])):
        with pytest.raises(ValueError, match="result given as out"):
            sm.norm_fwd(weight=w, out=r, **bad)
    g = sm.norm_bwd(x, w, torch.ones(T), x.clone())
    sm.norm_bwd(x, w, torch.ones(T), g["dresidual"], out=g)  # dresidual may be dout or dsum
    sm.norm_bwd(x, w, torch.ones(T), x.clone(), dsum=g["dresidual"], out=g)
    for bad in (dict(sum=g["dresidual"], weight=w), dict(sum=x, weight=g["dweight"])):
        with pytest.raises(ValueError, match="result given as out"):
            sm.norm_bwd(rstd=torch.ones(T), dout=x.clone(), out=g, **bad)
    layer = sm.FewLayer(*weights(torch.float32))
    y = layer(x)
    layer(x, out=y)
    before = len(on_the_host)
    with pytest.raises(ValueError, match="x is a tensor of the result"):
        layer(y["y"], out=y)
    e = torch.float8_e4m3fn
    layer = sm.FewLayer(*weights(e), w_in_scale=torch.ones(N, F), w_out_scale=torch.ones(N, D))
    y = layer(x.to(e), x_scale=torch.ones(T))
    with pytest.raises(ValueError, match="x_scale is a tensor of the result"):
        layer(x.to(e), x_scale=y["gate"], out=y)
    assert len(on_the_host) == before + 1
    empty = sm.norm_fwd(x[:0], w, delta=x[:0])
    sm.norm_fwd(x[:0], w, delta=x[:0], out=empty)


def test_a_stream_of_another_device_is_refused(on_the_host):
    """(Made current, it would change the device, and the call would go to some other stream of its own one.)"""
    class Stream:
        device = torch.device("cuda", 1)

    x, w = torch.ones(T, D), torch.ones(D)
    calls = (lambda s: sm.norm_fwd(x, w, stream=s), lambda s: sm.norm_bwd(x, w, torch.ones(T), x, stream=s),
             lambda s: sm.block_fwd(x, w, *weights(), capacity=T, stream=s),
             lambda s: sm.FewLayer(*weights(torch.float32))(x, stream=s),
             lambda s: sm.layer_fwd_few(x, *weights(torch.float32), stream=s),
             lambda s: sm.block_bwd(dict(expert=x[:, 0]), w, *weights(), x, stream=s))
    for call in calls:
        with pytest.raises(ValueError, match="stream must be on"):
            call(Stream())
    assert not on_the_host


def test_blocks_of_another_device_than_the_current_one(monkeypatch):
    """The layer's calls go by the current device: it is that of the tensors meanwhile."""
    now, seen = [], []

    @contextlib.contextmanager
    def current(device):
        now.append(device)
        yield
        now.pop()

    w_r, w_in, w_out = weights()
    x, rows = torch.zeros(100, D, dtype=torch.bfloat16), torch.zeros(100, D)
    monkeypatch.setattr(sm, "_current", current)
    monkeypatch.setattr(sm, "norm_fwd", lambda *a, **k: dict(out=x, scale=None, sum=rows, rstd=rows[:, 0]))
    monkeypatch.setattr(sm, "norm_bwd", lambda *a, **k: dict(dresidual=rows, dweight=rows[0]))
    monkeypatch.setattr(sm, "layer_bwd", lambda *a, **k: seen.append(list(now)) or dict(dx=rows))
    for name in ("layer_fwd", "layer_fwd_top2"):
        monkeypatch.setattr(sm, name, lambda *a, **k: seen.append(list(now)) or dict(y=rows))
    f = sm.block_fwd(rows, rows[0], w_r, w_in, w_out, capacity=8)
    sm.block_fwd(rows, rows[0], w_r, w_in, w_out, capacity=8, top_k=2)
    sm.block_bwd(f, rows[0], w_r, w_in, w_out, rows)
    assert seen == [[rows.device]] * 3 and not now
