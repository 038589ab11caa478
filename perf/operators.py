"""The operators around the dispatch layout as cases that can be run and timed.

Five operators: the top-k gate with its balance loss (``gate``), quantisation
to e4m3 with a scale for each block of 128 (``rows``: blocks along a row,
``cols``: blocks down a column, transposed), the gated activation between two
expert products (``swiglu``, forward with quantisation; ``swiglu_bwd``), the
expert product over the receive buffer (``product``) and its weight gradient
(``wgrad``).  ``run`` computes them in plain torch operations in 32 bits, or,
where ``own`` is true, with the library's kernels.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 1e-30
DEV = "cuda"

# Work of the largest listed case (multiply-adds of the expert product): bounds what draw() gives.
_MOST_WEIGHTS = 256 * 4096 * 7168
_MOST_MACS = 32768 * 8 * 4096 * 7168


def listed():
    return [
        # One serving step of 64 sequences: the gate of a 256-expert layer; latency is all.
        dict(name="gate-serve", op="gate", tokens=64, experts=256, topk=8, dtype="float32", score="softmax",
             bias=False, masked=0.0, empty=0.0, train=False),
        # The largest training batch (131072 tokens, 384 experts), forward and backward with the balance loss.
        dict(name="gate-train", op="gate", tokens=131072, experts=384, topk=8, dtype="float32", score="softmax",
             bias=False, masked=0.0, empty=0.0, train=True),
        # Ragged batch of bf16 logits with a selection bias, closed experts and padding tokens that route nowhere.
        dict(name="gate-ragged", op="gate", tokens=10007, experts=40, topk=3, dtype="bfloat16", score="sigmoid",
             bias=True, masked=0.05, empty=0.01, train=True),
        # Token rows quantised before an fp8 dispatch of a prefill batch.
        dict(name="rows-prefill", op="rows", rows=32768, cols=7168),
        # Receive rows of one rank's 32 experts quantised down the columns for the weight gradient.
        dict(name="cols-train", op="cols", tokens=4096, topk=8, experts=32, align=128, cols=4096),
        # Activation between the two products: receive buffer of 4096 tokens, top-8, sized for the worst case.
        dict(name="swiglu-fwd", op="swiglu", rows=40000, used=34816, width=2048),
        # Its gradient on an odd number of rows and a width that ends inside a block.
        dict(name="swiglu-bwd", op="swiglu_bwd", rows=10007, used=10007, width=1936),
        # Decoding 16 sequences: about a hundred of 256 experts get one or two rows each; the weights' reading is all.
        dict(name="product-decode", op="product", tokens=16, topk=8, experts=256, align=16, width_in=7168, width_out=4096),
        # Ragged segments and widths that end inside a block.
        dict(name="product-ragged", op="product", tokens=1000, topk=3, experts=40, align=16, width_in=1040, width_out=520),
        # Prefill: 262144 pairs, about 1024 rows an expert.
        dict(name="product-prefill", op="product", tokens=32768, topk=8, experts=256, align=128, width_in=7168,
             width_out=4096),
        # Weight gradient of one rank's 32 experts.
        dict(name="wgrad-train", op="wgrad", tokens=4096, topk=8, experts=32, align=128, width_in=7168, width_out=4096,
             out="bfloat16"),
        # A small one with odd widths, kept in 32 bits.
        dict(name="wgrad-small", op="wgrad", tokens=300, topk=2, experts=8, align=128, width_in=400, width_out=272,
             out="float32"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _width(rng, lo, hi, step):
    v = _log(rng, lo, hi, step)
    return v if v != 3072 else v + step


def draw(rng):
    op = rng.choice(["gate", "gate", "rows", "cols", "swiglu", "swiglu_bwd", "product", "product", "product", "wgrad"])
    if op == "gate":
        experts = _log(rng, 8, 512)
        return dict(op=op, tokens=_log(rng, 1, 100000), experts=experts, topk=rng.randint(1, min(8, experts)),
                    dtype=rng.choice(["float32", "bfloat16"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.1]), empty=rng.choice([0.0, 0.02]),
                    train=rng.random() < 0.7)
    if op == "rows":
        return dict(op=op, rows=_log(rng, 1, 32768), cols=_width(rng, 256, 7168, 16))
    if op in ("swiglu", "swiglu_bwd"):
        rows = _log(rng, 1, 40000)
        return dict(op=op, rows=rows, used=rows - rng.randint(0, rows // 8), width=_width(rng, 128, 4096, 16))
    if op == "cols":
        return dict(op=op, tokens=_log(rng, 1, 4096), topk=rng.randint(1, 4), experts=rng.choice([4, 8, 32]), align=128,
                    cols=_width(rng, 256, 7168, 16))
    if op == "wgrad":
        return dict(op=op, tokens=_log(rng, 16, 8192), topk=rng.randint(1, 4), experts=rng.choice([4, 8, 16, 32]),
                    align=128, width_in=_width(rng, 256, 7168, 16), width_out=_width(rng, 256, 4096, 16),
                    out=rng.choice(["bfloat16", "float32"]))
    while True:
        c = dict(op=op, tokens=_log(rng, 1, 32768), topk=rng.randint(1, 8), experts=rng.choice([1, 8, 32, 64, 256]),
                 align=rng.choice([1, 16, 64, 128]), width_in=_width(rng, 256, 7168, 16),
                 width_out=_width(rng, 256, 7168, 8))
        c["topk"] = min(c["topk"], c["experts"])
        weights = c["experts"] * c["width_in"] * c["width_out"]
        if weights <= _MOST_WEIGHTS and c["tokens"] * c["topk"] * c["width_in"] * c["width_out"] <= _MOST_MACS:
            return c


# ---------------------------------------------------------------- inputs
def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _blocks(n):
    return -(-n // BLOCK)


def _quantize(x):
    """x [..., n] in 32 bits -> e4m3 values and scales [..., blocks of 128 along the last axis]."""
    n, nb = x.shape[-1], _blocks(x.shape[-1])
    if n % BLOCK:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - n))
    v = x.reshape(*x.shape[:-1], nb, BLOCK)
    sf = v.abs().amax(-1).clamp(min=TINY) / E4M3_MAX
    q = (v * (1.0 / sf).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.reshape(x.shape)[..., :n].contiguous(), sf


def _dequantize(q, sf):
    """e4m3 [..., n] and scales [..., blocks] -> 32-bit values."""
    return q.float() * sf.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _routing(case, g):
    """Segments of a random routing: per-expert counts and aligned offsets, the token of each receive row, and where
    each expert's rows are (padded to the longest segment), as a dispatch leaves them."""
    N, K, E, A = case["tokens"], case["topk"], case["experts"], case["align"]
    idx = torch.rand((N, E), generator=g, device=DEV).topk(K, dim=1).indices
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    count = torch.bincount(flat, minlength=E)
    offset = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offset[1:] = torch.cumsum((count + A - 1) // A * A, 0)
    first = torch.cumsum(count, 0) - count
    capacity = N * K + E * (A - 1)
    row = offset[flat[order]] + torch.arange(N * K, device=DEV) - first[flat[order]]
    token = torch.full((capacity,), -1, dtype=torch.int64, device=DEV)
    token[row] = order // K
    active = torch.nonzero(count).reshape(-1)
    longest = int(count.max())
    lane = torch.arange(longest, device=DEV)
    place = torch.where(lane < count[active].unsqueeze(1), offset[active].unsqueeze(1) + lane, capacity)
    return dict(count=count.int(), offset=offset.int(), token=token, active=active, place=place, capacity=capacity)


def _rows_of(values, token):
    """values[token] with zeros in the rows that have no token."""
    return torch.where((token >= 0).unsqueeze(1), values[token.clamp(min=0)], torch.zeros((), dtype=values.dtype, device=DEV))


def _bytes_of(q, index):
    return q.view(torch.uint8)[index].view(torch.float8_e4m3fn)


def _weights(case, g):
    """Random weights [E, out, in] in e4m3 with a scale for each 128x128 block."""
    E, O, I = case["experts"], case["width_out"], case["width_in"]
    q = torch.empty((E, O, I), dtype=torch.float8_e4m3fn, device=DEV)
    per = max(1, min(E, (1 << 30) // (O * I)))
    for e in range(0, E, per):
        part = torch.randn((min(per, E - e), O, I), generator=g, device=DEV)
        q[e:e + per] = (part * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    sf = (torch.rand((E, _blocks(O), _blocks(I)), generator=g, device=DEV) + 0.5) * (0.01 / math.sqrt(I))
    return q, sf


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op == "gate":
        N, E, K = case["tokens"], case["experts"], case["topk"]
        l = torch.randn((N, E), generator=g, device=DEV) * 1.5 + torch.randn((E,), generator=g, device=DEV) * 0.5
        if case["masked"]:
            l = torch.where(torch.rand((N, E), generator=g, device=DEV) < case["masked"], -math.inf, l)
        if case["empty"]:
            l = torch.where(torch.rand((N, 1), generator=g, device=DEV) < case["empty"], -math.inf, l)
        s["logits"] = l.to(getattr(torch, case["dtype"]))
        s["bias"] = _randn(g, E, scale=0.2) if case["bias"] else None
        if case["train"]:
            s["dweights"] = _randn(g, N, K, scale=1.0 / math.sqrt(N))
            s["dloss"] = torch.ones(1, device=DEV)
            s["dlogits"] = torch.zeros_like(s["logits"])
    elif op == "rows":
        R, C = case["rows"], case["cols"]
        s["x"] = _randn(g, R, C, dtype=torch.bfloat16)
        s["q"] = torch.zeros((R, C), dtype=torch.float8_e4m3fn, device=DEV)
        s["sf"] = torch.zeros((R, _blocks(C)), device=DEV)
    elif op in ("swiglu", "swiglu_bwd"):
        R, I = case["rows"], case["width"]
        s["gate_up"] = _randn(g, R, 2 * I, scale=1.2, dtype=torch.bfloat16)
        s["total"] = torch.full((1,), case["used"], dtype=torch.int32, device=DEV)
        if op == "swiglu":
            s["q"] = torch.zeros((R, I), dtype=torch.float8_e4m3fn, device=DEV)
            s["sf"] = torch.zeros((_blocks(I), (R + 3) // 4 * 4), device=DEV)
        else:
            s["dh"] = _randn(g, R, I, scale=0.1, dtype=torch.bfloat16)
            s["dgate_up"] = torch.zeros((R, 2 * I), dtype=torch.bfloat16, device=DEV)
    elif op == "cols":
        r = s["route"] = _routing(case, g)
        s["x"] = _rows_of(_randn(g, case["tokens"], case["cols"], dtype=torch.bfloat16), r["token"])
        nb = _blocks(r["capacity"])
        s["q"] = torch.zeros((case["cols"], nb * BLOCK), dtype=torch.float8_e4m3fn, device=DEV)
        s["sf"] = torch.zeros((nb, case["cols"]), device=DEV)
    elif op == "product":
        r = s["route"] = _routing(case, g)
        q, sf = _quantize(_randn(g, case["tokens"], case["width_in"]))
        at = r["token"].clamp(min=0)
        real = (r["token"] >= 0).unsqueeze(1)
        s["x"] = torch.where(real, q.view(torch.uint8)[at], torch.zeros((), dtype=torch.uint8, device=DEV)).view(
            torch.float8_e4m3fn)
        s["x_sf"] = torch.zeros((sf.shape[1], (r["capacity"] + 3) // 4 * 4), device=DEV)
        s["x_sf"][:, :r["capacity"]] = (sf[at] * real).t()
        s["w"], s["w_sf"] = _weights(case, g)
        s["out"] = torch.zeros((r["capacity"], case["width_out"]), dtype=torch.bfloat16, device=DEV)
    elif op == "wgrad":
        r = s["route"] = _routing(case, g)
        for name, width, scale in (("dy", case["width_out"], 0.05), ("x", case["width_in"], 1.0)):
            rows = _rows_of(_randn(g, case["tokens"], width, scale=scale), r["token"])
            q, sf = _quantize(torch.nn.functional.pad(rows, (0, 0, 0, -rows.shape[0] % BLOCK)).t().contiguous())
            s[name], s[name + "_sf"] = q, sf.t().contiguous()
            del rows, q, sf
        s["dw"] = torch.zeros((case["experts"], case["width_out"], case["width_in"]), dtype=getattr(torch, case["out"]),
                              device=DEV)
    return s


# ---------------------------------------------------------------- one pass
BALANCE_COEF = 0.01
GATE_SCALE = 2.5


def _gate_plain(s):
    c = s["case"]
    E, K = c["experts"], c["topk"]
    l = s["logits"].float()
    key = l if s["bias"] is None else l + s["bias"]
    top = torch.sort(key, dim=1, descending=True, stable=True)
    picked = top.values[:, :K] > -math.inf
    at = top.indices[:, :K]
    idx = torch.where(picked, at, -1)
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-3e38))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    total = p.sum(1, keepdim=True).clamp(min=1e-30)
    chosen = p.gather(1, at) * picked
    D = chosen.sum(1, keepdim=True).clamp(min=1e-30)
    weights = GATE_SCALE * chosen / D
    count = torch.zeros(E + 1, dtype=torch.int32, device=DEV).index_add_(
        0, idx.reshape(-1) + 1, torch.ones(idx.numel(), dtype=torch.int32, device=DEV))[1:]
    routed = (l > -math.inf).any(1).sum().clamp(min=1).float()
    q = p / total
    mean = q.sum(0) / routed
    f = count.float() / (K * routed)
    loss = (BALANCE_COEF * E * (f * mean).sum()).reshape(1)
    out = dict(topk_idx=idx, weights=weights, expert_count=count, prob_mean=mean, loss=loss)
    if c["train"]:
        dw = s["dweights"] * picked
        ds_k = GATE_SCALE / D * (dw - (dw * chosen).sum(1, keepdim=True) / D) * picked
        grad = s["dloss"] * BALANCE_COEF * E * f / routed
        ds = (grad - (q * grad).sum(1, keepdim=True)) / total
        ds = ds.scatter_add(1, at, ds_k)
        if c["score"] == "softmax":
            dl = p * (ds - (p * ds).sum(1, keepdim=True))
        else:
            dl = p * (1.0 - p) * ds
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _swiglu_plain(s):
    I = s["case"]["width"]
    live = (torch.arange(s["case"]["rows"], device=DEV) < s["total"]).unsqueeze(1)
    gate, up = s["gate_up"][:, :I].float(), s["gate_up"][:, I:].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if s["case"]["op"] == "swiglu_bwd":
        dh = s["dh"].float()
        both = torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig], 1)
        return dict(dgate_up=(both * live).to(torch.bfloat16))
    q, sf = _quantize(gate * sig * up)
    q = torch.where(live, q.view(torch.uint8), torch.zeros((), dtype=torch.uint8, device=DEV)).view(torch.float8_e4m3fn)
    sf = torch.nn.functional.pad((sf * live).t(), (0, s["sf"].shape[1] - sf.shape[0]))
    return dict(q=q, sf=sf.contiguous())


def _cols_plain(s):
    r = s["route"]
    x = torch.nn.functional.pad(s["x"].float(), (0, 0, 0, -r["capacity"] % BLOCK))
    q, sf = _quantize(x.t().contiguous())
    live = torch.arange(sf.shape[1], device=DEV) * BLOCK < r["offset"][-1]     # blocks past the last segment stay as they were
    q = torch.where(live.repeat_interleave(BLOCK), q.view(torch.uint8), torch.zeros((), dtype=torch.uint8, device=DEV))
    return dict(q=q.view(torch.float8_e4m3fn), sf=(sf * live).t().contiguous())


def _product_plain(s):
    r, O = s["route"], s["case"]["width_out"]
    at = r["place"].clamp(max=r["capacity"] - 1)
    x = _dequantize(_bytes_of(s["x"], at), s["x_sf"].t()[at])
    w = s["w"].view(torch.uint8)[r["active"]].view(torch.float8_e4m3fn)
    wf = w.float() * s["w_sf"][r["active"]].repeat_interleave(BLOCK, 1)[:, :O].repeat_interleave(BLOCK, 2)[
        :, :, :s["case"]["width_in"]]
    y = torch.bmm(x, wf.transpose(1, 2)).to(torch.bfloat16)
    out = torch.zeros((r["capacity"] + 1, O), dtype=torch.bfloat16, device=DEV)
    out[r["place"].reshape(-1)] = y.reshape(-1, O)
    return dict(out=out[:r["capacity"]])


def _wgrad_plain(s):
    r, c = s["route"], s["case"]
    n = s["dy"].shape[1]
    at = r["place"].clamp(max=n - 1)
    real = (r["place"] < r["capacity"]).unsqueeze(2)
    dy = _dequantize(s["dy"], s["dy_sf"].t()).t()[at] * real
    x = _dequantize(s["x"], s["x_sf"].t()).t()[at] * real
    dw = torch.zeros((c["experts"], c["width_out"], c["width_in"]), dtype=getattr(torch, c["out"]), device=DEV)
    dw[r["active"]] = torch.bmm(dy.transpose(1, 2), x).to(dw.dtype)
    return dict(dw=dw)


def _run_own(s):
    from counting_sort_bucketization_gb300 import binding

    c = s["case"]
    op = c["op"]
    if op == "gate":
        gate = s.get("gate")
        if gate is None:
            desc = binding.LayoutDesc(c["tokens"], c["topk"], c["experts"], 1, 1)
            gate = s["gate"] = binding.Gate(desc, binding.GateConfig(score=c["score"], normalize=True, scale=GATE_SCALE,
                                                                     balance_coef=BALANCE_COEF))
        gate.forward(s["logits"], bias=s["bias"])
        out = dict(topk_idx=gate.topk_idx, weights=gate.weights, expert_count=gate.expert_count,
                   prob_mean=gate.prob_mean, loss=gate.loss)
        if c["train"]:
            gate.backward(s["logits"], s["dlogits"], dweights=s["dweights"], dloss=s["dloss"])
            out["dlogits"] = s["dlogits"]
        return out
    if op == "rows":
        binding.quantize_rows(s["x"], s["q"], s["sf"])
        return dict(q=s["q"], sf=s["sf"])
    if op == "swiglu":
        binding.swiglu_quantize(s["gate_up"], s["q"], s["sf"], total_rows=s["total"])
        return dict(q=s["q"], sf=s["sf"])
    if op == "swiglu_bwd":
        binding.swiglu_backward(s["gate_up"], s["dh"], s["dgate_up"], total_rows=s["total"])
        return dict(dgate_up=s["dgate_up"])
    r = s["route"]
    if "workspace" not in s:
        s["desc"] = binding.LayoutDesc(c["tokens"], c["topk"], c["experts"], 1, c["align"])
        s["workspace"] = binding.new_workspace(s["desc"])
    if op == "cols":
        binding.quantize_cols(s["desc"], s["x"], r["offset"], r["count"], s["q"], s["sf"], s["workspace"])
        return dict(q=s["q"], sf=s["sf"])
    if op == "product":
        binding.expert_gemm(s["desc"], s["x"], s["x_sf"], s["w"], s["w_sf"], r["offset"], r["count"], s["out"],
                            s["workspace"])
        return dict(out=s["out"])
    binding.expert_wgrad(s["desc"], s["dy"], s["dy_sf"], s["x"], s["x_sf"], r["offset"], r["count"], s["dw"],
                         s["workspace"])
    return dict(dw=s["dw"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "gate":
        return _gate_plain(state)
    if op == "rows":
        q, sf = _quantize(state["x"].float())
        return dict(q=q, sf=sf)
    if op in ("swiglu", "swiglu_bwd"):
        return _swiglu_plain(state)
    return dict(cols=_cols_plain, product=_product_plain, wgrad=_wgrad_plain)[op](state)


# ---------------------------------------------------------------- work of one pass
def work(case):
    op = case["op"]
    if op == "gate":
        N, E, K = case["tokens"], case["experts"], case["topk"]
        size = 4 if case["dtype"] == "float32" else 2
        b, f = N * E * size + N * K * 12, 10.0 * N * E
        if case["train"]:
            b, f = b + 2 * N * E * size + N * K * 12, 2 * f
        return dict(bytes=b, flops=f)
    if op == "rows":
        n = case["rows"] * case["cols"]
        return dict(bytes=3 * n + 4 * case["rows"] * _blocks(case["cols"]), flops=3.0 * n)
    if op == "swiglu":
        n = case["used"] * case["width"]
        return dict(bytes=5 * n + 4 * case["used"] * _blocks(case["width"]), flops=10.0 * n)
    if op == "swiglu_bwd":
        n = case["used"] * case["width"]
        return dict(bytes=10 * n, flops=15.0 * n)
    N, K, E, A = case["tokens"], case["topk"], case["experts"], case["align"]
    pairs = N * K
    rows = pairs + E * (A - 1) / 2          # receive rows, gaps among them, in the mean
    active = E * (1 - (1 - K / E) ** N)     # experts with a row, in the mean
    if op == "cols":
        n = rows * case["cols"]
        return dict(bytes=2 * pairs * case["cols"] + n + 4 * n / BLOCK, flops=3.0 * n)
    I, O = case["width_in"], case["width_out"]
    if op == "product":
        b = pairs * (I + 4 * _blocks(I)) + active * (O * I + 4 * _blocks(O) * _blocks(I)) + 2 * rows * O
    else:
        b = rows * (I + O) * (1 + 4 / BLOCK) + (2 if case["out"] == "bfloat16" else 4) * E * O * I
    return dict(bytes=b, flops=2.0 * pairs * I * O)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_gate(case, s):
    import numpy as np

    N, E, K = case["tokens"], case["experts"], case["topk"]
    l32 = s["logits"].float().cpu().numpy()
    key = l32 if s["bias"] is None else l32 + s["bias"].cpu().numpy()      # the selection key is a 32-bit sum
    idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
    picked = np.take_along_axis(key, idx, 1) > -np.inf
    l = l32.astype(np.float64)
    with np.errstate(all="ignore"):
        if case["score"] == "softmax":
            m = np.max(l, axis=1, keepdims=True)
            score = np.exp(l - np.where(np.isfinite(m), m, 0.0))
            score /= np.maximum(score.sum(1, keepdims=True), 1e-300)
        else:
            score = 1.0 / (1.0 + np.exp(-l))
    total = np.maximum(score.sum(1, keepdims=True), 1e-300)
    sel = np.where(picked, np.take_along_axis(score, idx, 1), 0.0)
    den = np.maximum(sel.sum(1, keepdims=True), 1e-300)
    count = np.bincount(idx[picked], minlength=E)
    T = max(1, int(np.isfinite(l).any(1).sum()))
    mean = (score / total).sum(0) / T
    frac = count / (K * T)
    out = dict(topk_idx=None, weights=GATE_SCALE * sel / den, expert_count=None, prob_mean=mean,
               loss=np.array([BALANCE_COEF * E * float(frac @ mean)]))
    if case["train"]:
        dw = np.where(picked, s["dweights"].double().cpu().numpy(), 0.0)
        inner = (dw * sel / den).sum(1, keepdims=True)
        coef = BALANCE_COEF * E * frac / T * float(s["dloss"])
        ds = (coef - ((score / total) @ coef)[:, None]) / total
        rows = np.nonzero(picked)
        np.add.at(ds, (rows[0], idx[rows]), (GATE_SCALE / den * (dw - inner))[rows])
        if case["score"] == "softmax":
            out["dlogits"] = score * (ds - (score * ds).sum(1, keepdims=True))
        else:
            out["dlogits"] = score * (1.0 - score) * ds
    return out


def _exact_blocks(x):
    """x [rows, n] in 64 bits: values over their block's scale, and the scales; what is not rounded is the definition."""
    n, nb = x.shape[1], _blocks(x.shape[1])
    sf = torch.stack([x[:, b * BLOCK:min(n, (b + 1) * BLOCK)].abs().max(1).values for b in range(nb)], 1)
    sf = sf.clamp(min=TINY) / E4M3_MAX
    column = torch.arange(n, device=DEV) // BLOCK
    return x / sf[:, column], sf


def exact(case, seed):
    op = case["op"]
    if op in ("product", "wgrad") and case["tokens"] * case["topk"] * case["width_in"] * case["width_out"] > 2.5e12:
        return None
    s = prepare(case, seed)
    if op == "gate":
        return _exact_gate(case, s)
    if op == "rows":
        q, sf = _exact_blocks(s["x"].double())
        return dict(q=q, sf=sf)
    if op in ("swiglu", "swiglu_bwd"):
        I, used = case["width"], case["used"]
        a, b = s["gate_up"][:used].double().split(I, 1)
        sig = torch.sigmoid(a)
        if op == "swiglu_bwd":
            d = s["dh"][:used].double()
            out = torch.zeros((case["rows"], 2 * I), dtype=torch.float64, device=DEV)
            out[:used, :I] = d * b * (sig + a * sig * (1 - sig))
            out[:used, I:] = d * a * sig
            return dict(dgate_up=out)
        q, sf = _exact_blocks(a * sig * b)
        wide = torch.zeros((case["rows"], I), dtype=torch.float64, device=DEV)
        wide[:used] = q
        scales = torch.zeros(s["sf"].shape, dtype=torch.float64, device=DEV)
        scales[:, :used] = sf.t()
        return dict(q=wide, sf=scales)
    r = s["route"]
    count, offset = r["count"].tolist(), r["offset"].tolist()
    if op == "cols":
        q = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        sf = torch.zeros(s["sf"].shape, dtype=torch.float64, device=DEV)
        for b in range(offset[-1] // BLOCK):
            block = s["x"][b * BLOCK:(b + 1) * BLOCK].double()
            sf[b] = block.abs().max(0).values.clamp(min=TINY) / E4M3_MAX
            q[:, b * BLOCK:(b + 1) * BLOCK] = (block / sf[b]).t()
        return dict(q=q, sf=sf)
    I, O, E = case["width_in"], case["width_out"], case["experts"]
    ib = torch.arange(I, device=DEV) // BLOCK
    ob = torch.arange(O, device=DEV) // BLOCK
    if op == "product":
        out = torch.zeros((r["capacity"], O), dtype=torch.float64, device=DEV)
        for e in range(E):
            if count[e]:
                a, z = offset[e], offset[e] + count[e]
                x = s["x"][a:z].double() * s["x_sf"][:, a:z].double().t()[:, ib]
                w = s["w"][e].double() * s["w_sf"][e].double()[ob][:, ib]
                out[a:z] = x @ w.t()
        return dict(out=out)
    dw = torch.zeros((E, O, I), dtype=torch.float64, device=DEV)
    for e in range(E):
        if count[e]:
            a, z = offset[e], offset[e] + count[e]
            rb = torch.arange(a, z, device=DEV) // BLOCK
            dy = s["dy"][:, a:z].double() * s["dy_sf"].double()[rb].t()
            x = s["x"][:, a:z].double() * s["x_sf"].double()[rb].t()
            dw[e] = dy @ x.t()
    return dict(dw=dw)
