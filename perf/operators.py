"""What the operators around the Switch layer are measured on: the residual's addition with its
root-mean-square norm (16-bit, 32-bit and 8-bit outputs) and that norm's gradient, the rounding of rows
to 8 bits with scales, and the whole layer for a few tokens (top-1 and top-2; float32, bfloat16 and
8-bit experts).

``run`` computes them with elementary torch operations where ``own`` is false and calls
``sparse_mixture_experts_fp32_b200`` where it is true.

A case's "op" is one of
  norm      s = residual + delta;  out = s * rsqrt(mean(s^2) + eps) * weight
  norm_grad the gradients of that with respect to s and weight
  quant     scale = amax(row) / 448;  q = e4m3(row / scale)
  few       router, softmax, top-1 or top-2, capacity slots, the experts' two products with ReLU, and
            the sum of the kept choices' outputs weighted by their gates
"""
import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a decoding step, before a layer with d_model = 1024: latency
        dict(name="norm_one_token", op="norm", T=1, d=1024, res="bf16", delta="f32", out="bf16"),
        # a prompt whose normalised rows go on in 8 bits (16 sequences of 512 tokens), float32 residual stream
        dict(name="norm_prompt_e4m3", op="norm", T=8192, d=768, res="f32", delta="f32", out="e4m3"),
        # a training step's token group of the 128-expert layer, bfloat16 residual stream
        dict(name="norm_train_bf16", op="norm", T=131072, d=1024, res="bf16", delta="f32", out="bf16"),
        # the same group's gradient
        dict(name="norm_grad_train", op="norm_grad", T=131072, d=1024, res="bf16", dsum=True),
        # a short ragged batch with an odd width, nothing arriving on the residual branch
        dict(name="norm_grad_odd", op="norm_grad", T=509, d=333, res="f32", dsum=False),
        # the weights of 32 experts, rounded once when a model is loaded
        dict(name="quant_experts", op="quant", T=131072, d=1024, res="bf16"),
        # a few activation rows of an odd width
        dict(name="quant_rows_odd", op="quant", T=37, d=4099, res="f32"),
        # one token of a decoding step through the 128-expert layer
        dict(name="few_one_token", op="few", T=1, d=1024, F=4096, N=128, k=1, w="bf16", x="bf16", C=0, bias=False),
        # 32 sequences decoded together, two experts for each token
        dict(name="few_top2_batch", op="few", T=32, d=1024, F=4096, N=128, k=2, w="bf16", x="bf16", C=0, bias=False),
        # a small float32 layer of odd sizes, capacity two and popular experts: tokens are dropped
        dict(name="few_f32_odd", op="few", T=13, d=509, F=1021, N=6, k=2, w="f32", x="f32", C=2, bias=True),
        # eight sequences through large experts held in 8 bits
        dict(name="few_large_e4m3", op="few", T=8, d=4096, F=10240, N=64, k=1, w="e4m3", x="bf16", C=0, bias=False),
        # a batch whose rows left the norm in 8 bits, popular experts
        dict(name="few_batch_e4m3", op="few", T=48, d=768, F=2048, N=8, k=2, w="e4m3", x="e4m3", C=0, bias=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_grad", "quant", "few", "few", "few"))
    if op != "few":
        d = _log_int(rng, 1, 8192)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        T = _log_int(rng, 1, min(131072, 131072 * 1024 // d))
        res = rng.choice(("f32", "bf16"))
        if op == "norm":
            return dict(op=op, T=T, d=d, res=res, delta=rng.choice(("none", "f32", "bf16")),
                        out=rng.choice(("f32", "bf16", "e4m3")))
        if op == "norm_grad":
            return dict(op=op, T=T, d=d, res=res, dsum=rng.random() < 0.7)
        return dict(op=op, T=T, d=d, res=res)
    w = rng.choice(("f32", "bf16", "bf16", "e4m3", "e4m3"))
    while True:
        T, k, N = _log_int(rng, 1, 64), rng.choice((1, 2)), _log_int(rng, 2, 256)
        d, F = _log_int(rng, 64, 4096), _log_int(rng, 64, 10240)
        if w != "f32":
            d, F = max(64, d // 64 * 64), max(64, F // 64 * 64)
        active = N * (1 - (1 - 1 / N) ** (T * k))
        if N * 2 * d * F * SIZE[w] <= 6e9 and active * 2 * d * F * SIZE[w] <= 6e8 and T * k * d * F <= 3.4e8:
            break
    x = w if w != "e4m3" else rng.choice(("bf16", "e4m3"))
    C = 0 if rng.random() < 0.6 else rng.randint(1, max(1, T // 2))
    return dict(op=op, T=T, d=d, F=F, N=N, k=k, w=w, x=x, C=C, bias=rng.random() < 0.4)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _to_e4m3(v):
    """Rows of v in 8 bits and their scales (values and distributions as quantised weights have them)."""
    scale = v.abs().amax(-1).float() / E4M3_MAX
    return (v / scale.unsqueeze(-1)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(0.0, std, generator=g)

    T, d = case["T"], case["d"]
    st = dict(case=case)
    if case["op"] in ("norm", "norm_grad"):
        st["eps"] = 1e-6
        st["weight"] = 1.0 + normal(d, std=0.2)
        res = normal(T, d, std=3.0)
        # rows of a residual stream differ in size from token to token, and a few channels are large
        res *= torch.exp(normal(T, 1, std=0.5))
        res[:, :: max(1, d // 3)] *= 8.0
        st["residual"] = res.to(DTYPES[case["res"]])
        if case["op"] == "norm":
            st["delta"] = None if case["delta"] == "none" else normal(T, d, std=0.7).to(DTYPES[case["delta"]])
        else:
            st["dout"] = normal(T, d, std=1e-2)
            st["dsum"] = normal(T, d, std=1e-2) if case["dsum"] else None
            s = st["residual"].float()
            st["rstd"] = torch.rsqrt(s.double().square().mean(-1) + st["eps"]).float()  # kept by the forward pass
    elif case["op"] == "quant":
        v = normal(T, d, std=0.05)
        v *= torch.exp(normal(T, 1, std=0.3))
        st["x"] = v.to(DTYPES[case["res"]])
    else:
        F, N = case["F"], case["N"]
        st["w_r"] = normal(N, d, std=0.1 / math.sqrt(d))
        st["bias"] = None
        if case["bias"]:
            w = torch.arange(1, N + 1, device=dev, dtype=torch.float64) ** -1.0
            st["bias"] = (0.5 * torch.log(w / w.sum())).float()
        x = normal(T, d)
        st["x"], st["x_scale"] = _to_e4m3(x) if case["x"] == "e4m3" else (x.to(DTYPES[case["x"]]), None)
        for name, rows, cols in (("w_in", F, d), ("w_out", d, F)):
            std = 0.1 / math.sqrt(cols)
            if case["w"] == "e4m3":
                q = torch.empty(N, rows, cols, dtype=torch.float8_e4m3fn, device=dev)
                scale = torch.empty(N, rows, device=dev)
                for e in range(N):
                    q[e], scale[e] = _to_e4m3(normal(rows, cols, std=std))
                st[name], st[name + "_scale"] = q, scale
            else:
                st[name], st[name + "_scale"] = normal(N, rows, cols, std=std, dtype=DTYPES[case["w"]]), None
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _norm(st):
    c = st["case"]
    s = st["residual"].float()
    if st["delta"] is not None:
        s = (s + st["delta"].float()).to(st["residual"].dtype)
        stored, s = s, s.float()
    else:
        stored = None
    rstd = 1.0 / torch.sqrt((s * s).sum(-1) / c["d"] + st["eps"])
    v = s * rstd.unsqueeze(-1) * st["weight"]
    if c["out"] != "e4m3":
        return dict(sum=stored, out=v.to(DTYPES[c["out"]]), rstd=rstd)
    scale = v.abs().amax(-1) / E4M3_MAX
    q = (v / scale.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(sum=stored, out=q, scale=scale, rstd=rstd)


def _norm_grad(st):
    d = st["case"]["d"]
    s, r = st["residual"].float(), st["rstd"].unsqueeze(-1)
    hat = s * r
    gw = st["dout"] * st["weight"]
    dres = r * (gw - hat * ((gw * hat).sum(-1, keepdim=True) / d))
    if st["dsum"] is not None:
        dres = dres + st["dsum"]
    return dict(dresidual=dres, dweight=(st["dout"] * hat).sum(0, dtype=torch.float64).float())


def _quant(st):
    v = st["x"].float()
    scale = v.abs().amax(-1) / E4M3_MAX
    return dict(q=(v / scale.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale=scale)


def _few(st):
    c = st["case"]
    T, N, k, d, F = c["T"], c["N"], c["k"], c["d"], c["F"]
    C = c["C"] or T
    x = st["x"].float()
    if st["x_scale"] is not None:
        x = x * st["x_scale"].unsqueeze(-1)
    # logits in 64 bits: experts are chosen by comparing them
    logits = x.double() @ st["w_r"].double().t()
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    ex = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = ex / ex.sum(-1, keepdim=True)
    first = logits.argmax(-1)
    chosen = first.unsqueeze(-1)
    if k == 2:
        second = logits.scatter(-1, chosen, -math.inf).argmax(-1)
        chosen = torch.stack((first, second), -1)
    gate = p.gather(-1, chosen).float()
    # every first choice, in token order, ranks before every second choice
    order = chosen.t().reshape(-1)
    hot = (order.unsqueeze(-1) == torch.arange(N, device=x.device)).long()
    rank = ((hot.cumsum(0) - hot) * hot).sum(-1)
    slot = torch.where(rank < C, rank, torch.full_like(rank, -1)).reshape(k, T).t()
    counts = hot.sum(0)
    aux = N * ((hot[:T].sum(0).double() / T) * p.mean(0)).sum().float().reshape(1)
    # the experts' products, a slice of the (token, choice) pairs at a time (their weights are gathered)
    flat, out = chosen.reshape(-1), torch.empty(T * k, d, device=x.device)
    xs = x.repeat_interleave(k, 0)
    step = max(1, int(4e8 // (d * F)))
    for a in range(0, T * k, step):
        e = flat[a:a + step]
        w_in, w_out = st["w_in"][e].float(), st["w_out"][e].float()
        h = torch.bmm(w_in, xs[a:a + step].unsqueeze(-1)).squeeze(-1)
        if c["w"] == "e4m3":
            h = h * st["w_in_scale"][e]
        o = torch.bmm(w_out, h.clamp_min(0.0).unsqueeze(-1)).squeeze(-1)
        if c["w"] == "e4m3":
            o = o * st["w_out_scale"][e]
        out[a:a + step] = o
    kept = (slot >= 0).unsqueeze(-1)
    y = (torch.where(kept, out.reshape(T, k, d), torch.zeros((), device=x.device)) * gate.unsqueeze(-1)).sum(1)
    if k == 1:
        chosen, gate, slot = chosen.squeeze(-1), gate.squeeze(-1), slot.squeeze(-1)
    return dict(y=y, expert=chosen.int(), gate=gate, slot=slot.int(), counts=counts.int(), aux=aux)


def _run_own(st):
    import sparse_mixture_experts_fp32_b200 as sm

    c = st["case"]
    if c["op"] == "norm":
        r = sm.norm_fwd(st["residual"], st["weight"], delta=st["delta"], eps=st["eps"], out_dtype=DTYPES[c["out"]],
                        out=st.get("out"))
        st["out"] = r
        return {n: r[n] for n in ("sum", "out", "scale", "rstd") if r[n] is not None}
    if c["op"] == "norm_grad":
        r = st["out"] = sm.norm_bwd(st["residual"], st["weight"], st["rstd"], st["dout"], dsum=st["dsum"],
                                    out=st.get("out"))
        return dict(dresidual=r["dresidual"], dweight=r["dweight"])
    if c["op"] == "quant":
        r = st["out"] = sm.quantize_rows(st["x"], out=st.get("out"))
        return dict(q=r["q"], scale=r["scale"])
    if "layer" not in st:  # the handle that a serving program keeps beside its weights
        st["layer"] = sm.FewLayer(st["w_r"], st["w_in"], st["w_out"], top_k=c["k"], capacity=c["C"] or None,
                                  logit_bias=st["bias"], w_in_scale=st["w_in_scale"], w_out_scale=st["w_out_scale"])
    r = st["out"] = st["layer"](st["x"], x_scale=st["x_scale"], out=st.get("out"))
    return {n: r[n] for n in ("y", "expert", "gate", "slot", "counts", "aux")}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        r = _norm(state)
        return {n: v for n, v in r.items() if v is not None}
    return {"norm_grad": _norm_grad, "quant": _quant, "few": _few}[op](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "norm":
        delta = case["delta"]
        per = SIZE[case["res"]] + SIZE[case["out"]]
        per += 0 if delta == "none" else SIZE[delta] + SIZE[case["res"]]
        return dict(bytes=T * d * per + 4 * d + 4 * T * (2 if case["out"] == "e4m3" else 1), flops=6 * T * d)
    if case["op"] == "norm_grad":
        per = SIZE[case["res"]] + 4 + 4 + (4 if case["dsum"] else 0)
        return dict(bytes=T * d * per + 8 * d + 4 * T, flops=10 * T * d)
    if case["op"] == "quant":
        return dict(bytes=T * d * (SIZE[case["res"]] + 1) + 4 * T, flops=3 * T * d)
    F, N, k, C = case["F"], case["N"], case["k"], case["C"] or T
    # the experts that T tokens with k choices reach on average, and the pairs that capacity keeps, for even routing
    active = N * (1 - (1 - 1 / N) ** (T * k))
    pairs = min(T * k, active * C)
    weights = active * 2 * d * F * SIZE[case["w"]]
    if case["w"] == "e4m3":
        weights += active * 4 * (d + F)
    rest = 4 * N * d + T * d * SIZE[case["x"]] + 4 * T * d + 12 * T * k + 4 * N
    return dict(bytes=weights + rest, flops=4 * pairs * d * F + 2 * T * N * d)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_rows_e4m3(v):
    big = torch.max(torch.abs(v), dim=1).values
    scale = big / E4M3_MAX
    q = torch.clamp(v / scale[:, None], -E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), scale


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        q, scale = _exact_rows_e4m3(st["x"].double())
        return dict(q=q, scale=scale)
    if case["op"] == "norm":
        s, stored = st["residual"].double(), None
        if st["delta"] is not None:
            stored = (s + st["delta"].double()).to(DTYPES[case["res"]])
            s = stored.double()
        rms = torch.sqrt(torch.mean(torch.square(s), dim=1) + st["eps"])
        v = s / rms[:, None] * st["weight"].double()
        ans = {} if stored is None else dict(sum=stored)
        if case["out"] == "e4m3":
            q, scale = _exact_rows_e4m3(v)
            return dict(ans, out=q, scale=scale, rstd=1 / rms)
        return dict(ans, out=v, rstd=1 / rms)
    if case["op"] == "norm_grad":
        s, r = st["residual"].double(), st["rstd"].double()
        g, w = st["dout"].double(), st["weight"].double()
        dot = torch.einsum("td,td,d->t", s, g, w)
        grad = torch.einsum("t,td,d->td", r, g, w) - s * (r ** 3 * dot / case["d"])[:, None]
        if st["dsum"] is not None:
            grad += st["dsum"].double()
        return dict(dresidual=grad, dweight=torch.einsum("td,td,t->d", s, g, r))
    T, N, k = case["T"], case["N"], case["k"]
    C = case["C"] or T
    x = st["x"].double()
    if st["x_scale"] is not None:
        x = st["x_scale"].double()[:, None] * x
    h = torch.einsum("td,nd->tn", x, st["w_r"].double())
    if st["bias"] is not None:
        h = h + st["bias"].double()[None]
    p = torch.softmax(h, 1).cpu()
    order = torch.sort(h, dim=1, descending=True, stable=True).indices.cpu()[:, :k].tolist()
    y = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
    seen = [0] * N
    slot = [[-1] * k for _ in range(T)]
    for j in range(k):
        for t in range(T):
            e = order[t][j]
            if seen[e] < C:
                slot[t][j] = seen[e]
            seen[e] += 1
    for e in sorted({e for row in order for e in row}):
        rows = [(t, j) for t in range(T) for j in range(k) if order[t][j] == e and slot[t][j] >= 0]
        if not rows:
            continue
        w_in, w_out = st["w_in"][e].double(), st["w_out"][e].double()
        if case["w"] == "e4m3":
            w_in *= st["w_in_scale"][e].double()[:, None]
            w_out *= st["w_out_scale"][e].double()[:, None]
        o = torch.relu(x[[t for t, _ in rows]] @ w_in.mT) @ w_out.mT
        for i, (t, j) in enumerate(rows):
            y[t] += float(p[t, e]) * o[i]
    f = torch.zeros(N, dtype=torch.float64)
    for row in order:
        f[row[0]] += 1.0 / T
    gate = torch.tensor([[float(p[t, e]) for e in order[t]] for t in range(T)], dtype=torch.float64)
    expert, slots = torch.tensor(order, dtype=torch.int32), torch.tensor(slot, dtype=torch.int32)
    if k == 1:
        gate, expert, slots = gate[:, 0], expert[:, 0], slots[:, 0]
    return dict(y=y, expert=expert, gate=gate, slot=slots, counts=torch.tensor(seen, dtype=torch.int32),
                aux=(N * (f * p.mean(0)).sum()).reshape(1))
