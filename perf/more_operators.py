"""The norm in front of an expert layer, routing by scores and groups, and the combine's gradient as cases.

Four operators that can be run and timed: the residual's addition with a
root-mean-square norm and an output in bf16, e4m3 or both (``norm``), its
gradient (``norm_bwd``), routing by scores with a correction bias and groups of
experts, with the gradient of its weights and balance loss (``route``), and the
gradient of the weighted top-k sum (``combine_bwd``).  ``run`` computes them in
plain torch operations in 32 bits, or, where ``own`` is true, with the library's
kernels.  The plain routing compares its keys in 64 bits: two scores may lie
closer together than 32 bits tell apart, and the choice of experts is a whole
number.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 1e-30
DEV = "cuda"
EPS = 1e-6
ROUTE_SCALE = 2.5
BALANCE_COEF = 0.01

# Work of the largest listed cases: bounds what draw() gives.
_MOST_NORM = 32768 * 7168
_MOST_LOGITS = 131072 * 384
_MOST_COMBINE = 32768 * 8 * 4096


def listed():
    return [
        # One serving step of 64 sequences: residual added, normed rows for the router (bf16) and the dispatch (e4m3).
        dict(name="norm-serve", op="norm", rows=64, used=64, cols=7168, stream="bfloat16", weight="bfloat16", y=True, q=True,
             col_major=False),
        # A prefill batch, the same outputs.
        dict(name="norm-prefill", op="norm", rows=32768, used=32768, cols=7168, stream="bfloat16", weight="bfloat16", y=True,
             q=True, col_major=False),
        # A padded batch with the residual stream in 32 bits, 8-bit rows for a dense product, a width that ends inside a block.
        dict(name="norm-ragged", op="norm", rows=10007, used=9001, cols=1936, stream="float32", weight="float32", y=False,
             q=True, col_major=True),
        # Training: gradient of the norm and its weight, with the residual's own gradient added.
        dict(name="norm-bwd-train", op="norm_bwd", rows=32768, used=32768, cols=4096, stream="bfloat16", weight="bfloat16",
             dresidual=True),
        # A short padded batch with the stream in 32 bits and an odd width.
        dict(name="norm-bwd-ragged", op="norm_bwd", rows=1111, used=1009, cols=1040, stream="float32", weight="float32",
             dresidual=True),
        # Routing of one serving step: 256 experts in 8 groups, 4 of them kept.
        dict(name="route-serve", op="route", tokens=64, experts=256, topk=8, groups=8, topk_groups=4, group_sum=2,
             dtype="float32", score="sigmoid", bias=True, masked=0.0, empty=0.0, train=False),
        # The largest training batch, a group for each of 16 ranks, both directions.
        dict(name="route-train", op="route", tokens=131072, experts=384, topk=8, groups=16, topk_groups=4, group_sum=2,
             dtype="float32", score="sigmoid", bias=True, masked=0.0, empty=0.0, train=True),
        # bf16 logits, softmax, groups by their best expert, closed experts and padding tokens that route nowhere.
        dict(name="route-ragged", op="route", tokens=10007, experts=40, topk=3, groups=4, topk_groups=2, group_sum=1,
             dtype="bfloat16", score="softmax", bias=True, masked=0.05, empty=0.01, train=True),
        # A score bias without groups.
        dict(name="route-flat", op="route", tokens=32768, experts=256, topk=8, groups=1, topk_groups=1, group_sum=1,
             dtype="float32", score="sigmoid", bias=True, masked=0.0, empty=0.0, train=False),
        # Gradient of the combine in training: rows for the expert products' gradients, and the weights' gradient.
        dict(name="combine-bwd-train", op="combine_bwd", tokens=32768, topk=8, experts=384, align=64, cols=4096, masked=0.05,
             dweights=True),
        # A short batch of a wide model.
        dict(name="combine-bwd-few", op="combine_bwd", tokens=48, topk=8, experts=256, align=16, cols=7168, masked=0.0,
             dweights=True),
        # Odd numbers of tokens and slots, some masked.
        dict(name="combine-bwd-ragged", op="combine_bwd", tokens=1001, topk=3, experts=40, align=128, cols=1040, masked=0.1,
             dweights=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "route", "route", "combine_bwd", "combine_bwd"])
    while True:
        if op in ("norm", "norm_bwd"):
            rows = _log(rng, 1, 40000)
            c = dict(op=op, rows=rows, used=rows - rng.choice([0, rng.randint(0, rows // 8)]), cols=_log(rng, 128, 16384, 16),
                     stream=rng.choice(["bfloat16", "bfloat16", "float32"]), weight=rng.choice(["bfloat16", "float32"]))
            if op == "norm":
                c["y"], c["q"] = rng.choice([(True, True), (True, False), (False, True)])
                c["col_major"] = rng.random() < 0.3
                if rng.random() < 0.2:
                    c["stream"] = "none"
            else:
                c["dresidual"] = rng.random() < 0.8
            if c["rows"] * c["cols"] <= _MOST_NORM // (2 if op == "norm_bwd" or c["stream"] == "float32" else 1):
                return c
        elif op == "route":
            groups = rng.choice([1, 2, 4, 8, 16])
            experts = groups * _log(rng, 2, 64)
            kept = rng.randint(1, groups)
            c = dict(op=op, tokens=_log(rng, 1, 131072), experts=experts, topk=rng.randint(1, min(8, kept * experts // groups)),
                     groups=groups, topk_groups=kept, group_sum=rng.choice([1, 2]), dtype=rng.choice(["float32", "bfloat16"]),
                     score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.8, masked=rng.choice([0.0, 0.0, 0.1]),
                     empty=rng.choice([0.0, 0.02]), train=rng.random() < 0.5)
            if c["tokens"] * c["experts"] <= _MOST_LOGITS:
                return c
        else:
            experts = rng.choice([4, 8, 32, 64, 256, 384])
            c = dict(op=op, tokens=_log(rng, 1, 65536), topk=rng.randint(1, min(8, experts)), experts=experts,
                     align=rng.choice([1, 16, 64, 128]), cols=_log(rng, 256, 8192, 8), masked=rng.choice([0.0, 0.05, 0.5]),
                     dweights=rng.random() < 0.85)
            if c["tokens"] * c["topk"] * c["cols"] <= _MOST_COMBINE:
                return c


# ---------------------------------------------------------------- inputs
def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _blocks(n):
    return -(-n // BLOCK)


def _type(name):
    return getattr(torch, name)


def _stream_rows(g, rows, cols, dtype):
    """A residual stream: a few channels far larger than the others, rows of different size."""
    channel = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    row = torch.exp(torch.randn((rows, 1), generator=g, device=DEV) * 0.5)
    return (torch.randn((rows, cols), generator=g, device=DEV) * channel * row).to(dtype)


def _routing(case, g):
    """A random routing as the layout leaves it: slots, counts and aligned offsets."""
    N, K, E, A = case["tokens"], case["topk"], case["experts"], case["align"]
    idx = torch.rand((N, E), generator=g, device=DEV).topk(K, dim=1).indices
    if case["masked"]:
        idx = torch.where(torch.rand((N, K), generator=g, device=DEV) < case["masked"], -1, idx)
    flat = idx.reshape(-1)
    real = flat >= 0
    order = torch.sort(torch.where(real, flat, E), stable=True).indices[:int(real.sum())]
    count = torch.bincount(flat[real], minlength=E)
    offset = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offset[1:] = torch.cumsum((count + A - 1) // A * A, 0)
    first = torch.cumsum(count, 0) - count
    expert = flat[order]
    slot = torch.full((N * K,), -1, dtype=torch.int32, device=DEV)
    slot[order] = (offset[expert] + torch.arange(order.numel(), device=DEV) - first[expert]).int()
    return dict(slot=slot, count=count.int(), offset=offset.int(), capacity=N * K + E * (A - 1))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_bwd"):
        R, C = case["rows"], case["cols"]
        stream = torch.bfloat16 if case["stream"] == "none" else _type(case["stream"])
        s["weight"] = (torch.randn(C, generator=g, device=DEV) * 0.1 + 1.0).to(_type(case["weight"]))
        s["total"] = torch.full((1,), case["used"], dtype=torch.int32, device=DEV) if case["used"] < R else None
        if op == "norm":
            s["x"] = _randn(g, R, C, scale=0.7, dtype=torch.bfloat16)
            if case["stream"] != "none":
                s["residual"] = _stream_rows(g, R, C, stream)
                s["residual_out"] = torch.zeros((R, C), dtype=stream, device=DEV)
            s["y"] = torch.zeros((R, C), dtype=torch.bfloat16, device=DEV) if case["y"] else None
            s["q"] = torch.zeros((R, C), dtype=torch.float8_e4m3fn, device=DEV) if case["q"] else None
            shape = (_blocks(C), (R + 3) // 4 * 4) if case["col_major"] else (R, _blocks(C))
            s["sf"] = torch.zeros(shape, device=DEV) if case["q"] else None
            s["rstd"] = torch.zeros(R, device=DEV)
        else:
            s["z"] = _stream_rows(g, R, C, stream)
            s["rstd"] = torch.empty(R, device=DEV)
            per = max(1, (1 << 27) // C)
            for a in range(0, R, per):
                s["rstd"][a:a + per] = (s["z"][a:a + per].double().square().mean(1) + EPS).rsqrt()
            s["dy"] = _randn(g, R, C, scale=0.05, dtype=torch.bfloat16)
            s["dresidual"] = _randn(g, R, C, scale=0.05, dtype=stream) if case["dresidual"] else None
            s["dz"] = torch.zeros((R, C), dtype=stream, device=DEV)
            s["dx"] = torch.zeros((R, C), dtype=torch.bfloat16, device=DEV) if case["stream"] == "float32" else None
            s["dweight"] = torch.zeros(C, device=DEV)
    elif op == "route":
        N, E, K = case["tokens"], case["experts"], case["topk"]
        l = torch.randn((N, E), generator=g, device=DEV) * 1.5 + torch.randn((E,), generator=g, device=DEV) * 0.5
        if case["masked"]:
            l = torch.where(torch.rand((N, E), generator=g, device=DEV) < case["masked"], -math.inf, l)
        if case["empty"]:
            l = torch.where(torch.rand((N, 1), generator=g, device=DEV) < case["empty"], -math.inf, l)
        s["logits"] = l.to(_type(case["dtype"]))
        scale = 0.05 if case["score"] == "sigmoid" else 0.2 / E
        s["bias"] = _randn(g, E, scale=scale) if case["bias"] else None
        if case["train"]:
            s["dweights"] = _randn(g, N, K, scale=1.0 / math.sqrt(N))
            s["dloss"] = torch.ones(1, device=DEV)
            s["dlogits"] = torch.zeros_like(s["logits"])
    else:
        r = s["route"] = _routing(case, g)
        N, K, C = case["tokens"], case["topk"], case["cols"]
        s["dout"] = _randn(g, N, C, scale=0.1, dtype=torch.bfloat16)
        w = torch.rand((N, K), generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["expert_out"] = torch.empty((r["capacity"], C), dtype=torch.bfloat16, device=DEV)
        per = max(1, (1 << 28) // C)
        for a in range(0, r["capacity"], per):
            s["expert_out"][a:a + per] = _randn(g, min(per, r["capacity"] - a), C, dtype=torch.bfloat16)
        s["dy"] = torch.zeros((r["capacity"], C), dtype=torch.bfloat16, device=DEV)
        s["dweights"] = torch.zeros((N, K), device=DEV) if case["dweights"] else None
    return s


# ---------------------------------------------------------------- one pass
def _quantize(x):
    """x [rows, n] in 32 bits -> e4m3 values and scales [rows, blocks of 128]."""
    n, nb = x.shape[1], _blocks(x.shape[1])
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - n)).view(-1, nb, BLOCK)
    sf = v.abs().amax(-1).clamp(min=TINY) / E4M3_MAX
    q = (v * (1.0 / sf).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(-1, nb * BLOCK)[:, :n].contiguous(), sf


def _norm_plain(s):
    c = s["case"]
    R, n = c["rows"], c["used"]
    out = {}
    z = s["x"][:n].float()
    if c["stream"] != "none":
        z = (z + s["residual"][:n].float()).to(s["residual"].dtype)
        out["residual"] = torch.nn.functional.pad(z, (0, 0, 0, R - n))
        z = z.float()
    r = 1.0 / torch.sqrt((z * z).sum(1, keepdim=True) / c["cols"] + EPS)
    out["rstd"] = torch.nn.functional.pad(r.reshape(-1), (0, R - n))
    y = z * r * s["weight"].float()
    if c["y"]:
        out["y"] = torch.nn.functional.pad(y.to(torch.bfloat16), (0, 0, 0, R - n))
    if c["q"]:
        q, sf = _quantize(y)
        out["q"] = torch.nn.functional.pad(q.view(torch.uint8), (0, 0, 0, R - n)).view(torch.float8_e4m3fn)
        if c["col_major"]:
            out["sf"] = torch.nn.functional.pad(sf.t(), (0, s["sf"].shape[1] - n)).contiguous()
        else:
            out["sf"] = torch.nn.functional.pad(sf, (0, 0, 0, R - n))
    return out


def _norm_bwd_plain(s):
    c = s["case"]
    R, n = c["rows"], c["used"]
    dy, h = s["dy"][:n].float(), s["z"][:n].float() * s["rstd"][:n].unsqueeze(1)
    g = dy * s["weight"].float()
    dz = (g - h * ((g * h).sum(1, keepdim=True) / c["cols"])) * s["rstd"][:n].unsqueeze(1)
    if c["dresidual"]:
        dz = dz + s["dresidual"][:n].float()
    dz = torch.nn.functional.pad(dz, (0, 0, 0, R - n))
    out = dict(dz=dz.to(s["dz"].dtype), dweight=(dy * h).sum(0))
    if s["dx"] is not None:
        out["dx"] = dz.to(torch.bfloat16)
    return out


def _route_plain(s):
    c = s["case"]
    N, E, K, G = c["tokens"], c["experts"], c["topk"], c["groups"]
    l = s["logits"].float()
    open_ = l > -math.inf

    def score(x):
        if c["score"] == "sigmoid":
            return 1.0 / (1.0 + torch.exp(-x))
        p = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-3.4e38))
        return p / p.sum(1, keepdim=True).clamp(min=1e-30)

    # the choice, in 64 bits
    key = score(l.double())
    if s["bias"] is not None:
        key = key + s["bias"].double()
    key = torch.where(open_, key, -math.inf)
    if G > 1:
        best = torch.sort(key.view(N, G, E // G), dim=2, descending=True, stable=True).values[:, :, :c["group_sum"]]
        group = torch.where(best > -math.inf, best, 0.0).sum(2)
        group = torch.where(best[:, :, 0] > -math.inf, group, -math.inf)
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros((N, G), dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        key = torch.where(keep.unsqueeze(2), key.view(N, G, E // G), -math.inf).view(N, E)
    top = torch.sort(key, dim=1, descending=True, stable=True)
    picked = top.values[:, :K] > -math.inf
    at = top.indices[:, :K]
    idx = torch.where(picked, at, -1)

    p = score(l)
    total = p.sum(1, keepdim=True).clamp(min=1e-30)
    chosen = p.gather(1, at) * picked
    D = chosen.sum(1, keepdim=True).clamp(min=1e-30)
    weights = ROUTE_SCALE * chosen / D
    count = torch.zeros(E + 1, dtype=torch.int32, device=DEV).index_add_(
        0, idx.reshape(-1) + 1, torch.ones(idx.numel(), dtype=torch.int32, device=DEV))[1:]
    routed = open_.any(1).sum().clamp(min=1).float()
    q = p / total
    mean = q.sum(0) / routed
    f = count.float() / (K * routed)
    loss = (BALANCE_COEF * E * (f * mean).sum()).reshape(1)
    out = dict(topk_idx=idx, weights=weights, expert_count=count, prob_mean=mean, loss=loss)
    if c["train"]:
        dw = s["dweights"] * picked
        ds_k = ROUTE_SCALE / D * (dw - (dw * chosen).sum(1, keepdim=True) / D) * picked
        grad = s["dloss"] * BALANCE_COEF * E * f / routed
        ds = (grad - (q * grad).sum(1, keepdim=True)) / total
        ds = ds.scatter_add(1, at, ds_k)
        if c["score"] == "softmax":
            dl = p * (ds - (p * ds).sum(1, keepdim=True))
        else:
            dl = p * (1.0 - p) * ds
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _combine_bwd_plain(s):
    c, r = s["case"], s["route"]
    N, K, C = c["tokens"], c["topk"], c["cols"]
    slot = r["slot"].view(N, K).long()
    real = slot >= 0
    dy = torch.zeros((r["capacity"] + 1, C), dtype=torch.bfloat16, device=DEV)
    dweights = torch.zeros((N, K), device=DEV)
    dout = s["dout"].float()
    for k in range(K):
        at = torch.where(real[:, k], slot[:, k], r["capacity"])
        dy[at] = (s["weights"][:, k:k + 1] * dout).to(torch.bfloat16)
        if c["dweights"]:
            y = s["expert_out"][slot[:, k].clamp(min=0)].float()
            dweights[:, k] = torch.where(real[:, k], (y * dout).sum(1), 0.0)
    out = dict(dy=dy[:r["capacity"]])
    if c["dweights"]:
        out["dweights"] = dweights
    return out


def _run_own(s):
    from counting_sort_bucketization_gb300 import binding

    c = s["case"]
    op = c["op"]
    if op == "norm":
        binding.rms_norm(s["x"], s["weight"], y=s["y"], q=s["q"], sf=s["sf"], residual=s.get("residual"),
                         residual_out=s.get("residual_out"), rstd=s["rstd"], eps=EPS, total_rows=s["total"],
                         col_major=c["col_major"])
        out = dict(rstd=s["rstd"])
        if c["stream"] != "none":
            out["residual"] = s["residual_out"]
        if c["y"]:
            out["y"] = s["y"]
        if c["q"]:
            out["q"], out["sf"] = s["q"], s["sf"]
        return out
    if op == "norm_bwd":
        if "workspace" not in s:
            s["workspace"] = binding.new_norm_workspace(c["cols"])
        binding.rms_norm_backward(s["dy"], s["z"], s["rstd"], s["weight"], s["dz"], dresidual=s["dresidual"], dx=s["dx"],
                                  dweight=s["dweight"], workspace=s["workspace"], total_rows=s["total"])
        out = dict(dz=s["dz"], dweight=s["dweight"])
        if s["dx"] is not None:
            out["dx"] = s["dx"]
        return out
    if op == "route":
        gate = s.get("gate")
        if gate is None:
            desc = binding.LayoutDesc(c["tokens"], c["topk"], c["experts"], 1, 1)
            gate = s["gate"] = binding.Gate(desc, binding.GateConfig(
                score=c["score"], normalize=True, scale=ROUTE_SCALE, balance_coef=BALANCE_COEF, bias_on="score",
                num_groups=c["groups"], topk_groups=c["topk_groups"], group_sum=c["group_sum"]))
        gate.forward(s["logits"], bias=s["bias"])
        out = dict(topk_idx=gate.topk_idx, weights=gate.weights, expert_count=gate.expert_count,
                   prob_mean=gate.prob_mean, loss=gate.loss)
        if c["train"]:
            gate.backward(s["logits"], s["dlogits"], dweights=s["dweights"], dloss=s["dloss"])
            out["dlogits"] = s["dlogits"]
        return out
    r = s["route"]
    if "workspace" not in s:
        s["desc"] = binding.LayoutDesc(c["tokens"], c["topk"], c["experts"], 1, c["align"])
        s["workspace"] = binding.new_workspace(s["desc"])
    binding.combine_backward(s["desc"], s["dout"], r["slot"], s["weights"], s["dy"], s["workspace"],
                             expert_out=s["expert_out"] if c["dweights"] else None, dweights=s["dweights"],
                             expert_offset=r["offset"], expert_count=r["count"], zero_pad=True)
    out = dict(dy=s["dy"])
    if c["dweights"]:
        out["dweights"] = s["dweights"]
    return out


def run(state):
    if own:
        return _run_own(state)
    return dict(norm=_norm_plain, norm_bwd=_norm_bwd_plain, route=_route_plain,
                combine_bwd=_combine_bwd_plain)[state["case"]["op"]](state)


# ---------------------------------------------------------------- work of one pass
def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n = case["used"] * case["cols"]
        size = 4 if case["stream"] == "float32" else 2
        if op == "norm":
            b = 2 * n + (0 if case["stream"] == "none" else 2 * size * n) + (2 * n if case["y"] else 0)
            b += n + 4 * case["used"] * _blocks(case["cols"]) if case["q"] else 0
            return dict(bytes=b, flops=6.0 * n)
        b = (2 + 2 * size + (size if case["dresidual"] else 0) + (2 if size == 4 else 0)) * n
        return dict(bytes=b, flops=10.0 * n)
    if op == "route":
        N, E, K = case["tokens"], case["experts"], case["topk"]
        size = 4 if case["dtype"] == "float32" else 2
        b, f = N * E * size + N * K * 12, 12.0 * N * E
        if case["train"]:
            b, f = b + 2 * N * E * size + N * K * 12, 2 * f
        return dict(bytes=b, flops=f)
    N, K, E, A = case["tokens"], case["topk"], case["experts"], case["align"]
    pairs = N * K * (1 - case["masked"])
    gaps = E * (1 - (1 - K * (1 - case["masked"]) / E) ** N) * (A - 1) / 2     # rows, in the mean
    n = case["cols"]
    return dict(bytes=2 * n * (N + pairs + gaps + (pairs if case["dweights"] else 0)) + 8 * N * K,
                flops=(3.0 if case["dweights"] else 1.0) * pairs * n)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_norm(case, s):
    R, C, n = case["rows"], case["cols"], case["used"]
    nb = _blocks(C)
    column = torch.arange(C, device=DEV) // BLOCK
    wide = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)
    out = dict(rstd=wide(R))
    if case["stream"] != "none":
        out["residual"] = wide(R, C)
    if case["y"]:
        out["y"] = wide(R, C)
    if case["q"]:
        out["q"], out["sf"] = wide(R, C), wide(*s["sf"].shape)
    w = s["weight"].double()
    per = max(1, (1 << 26) // C)
    for a in range(0, n, per):
        b = min(n, a + per)
        z = s["x"][a:b].double()
        if case["stream"] != "none":
            z = z + s["residual"][a:b].double()
            out["residual"][a:b] = z
            z = z.to(s["residual"].dtype).double()      # the stream as it is kept is what is normed
        r = torch.rsqrt(torch.einsum("ij,ij->i", z, z) / C + EPS)
        out["rstd"][a:b] = r
        y = torch.einsum("ij,i,j->ij", z, r, w)
        if case["y"]:
            out["y"][a:b] = y
        if case["q"]:
            sf = torch.stack([y[:, i * BLOCK:min(C, (i + 1) * BLOCK)].abs().max(1).values for i in range(nb)], 1)
            sf = sf.clamp(min=TINY) / E4M3_MAX
            out["q"][a:b] = y / sf[:, column]
            if case["col_major"]:
                out["sf"][:, a:b] = sf.t()
            else:
                out["sf"][a:b] = sf
    return out


def _exact_norm_bwd(case, s):
    R, C, n = case["rows"], case["cols"], case["used"]
    dz = torch.zeros((R, C), dtype=torch.float64, device=DEV)
    dweight = torch.zeros(C, dtype=torch.float64, device=DEV)
    w = s["weight"].double()
    per = max(1, (1 << 26) // C)
    for a in range(0, n, per):
        b = min(n, a + per)
        z, dy, r = s["z"][a:b].double(), s["dy"][a:b].double(), s["rstd"][a:b].double()
        dweight += torch.einsum("ij,ij,i->j", dy, z, r)
        inner = torch.einsum("ij,ij,j->i", dy, z, w)
        dz[a:b] = dy * w * r[:, None] - z * (inner * r ** 3 / C)[:, None]
        if case["dresidual"]:
            dz[a:b] += s["dresidual"][a:b].double()
    out = dict(dz=dz, dweight=dweight)
    if s["dx"] is not None:
        out["dx"] = dz
    return out


def _exact_route(case, s):
    import numpy as np

    N, E, K, G = case["tokens"], case["experts"], case["topk"], case["groups"]
    l = s["logits"].double().cpu().numpy()
    closed = np.isneginf(l)
    with np.errstate(all="ignore"):
        if case["score"] == "softmax":
            m = np.max(l, axis=1, keepdims=True)
            score = np.exp(l - np.where(np.isfinite(m), m, 0.0))
            score /= np.maximum(score.sum(1, keepdims=True), 1e-300)
        else:
            score = 1.0 / (1.0 + np.exp(-l))
    key = score + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    key[closed] = -np.inf
    if G > 1:
        by_group = key.reshape(N, G, -1)
        first = by_group.max(2)
        group = first.copy()
        if case["group_sum"] == 2 and E > G:
            second = np.partition(by_group, -2, axis=2)[:, :, -2]
            group += np.where(np.isneginf(second), 0.0, second)
        gone = np.argsort(-group, axis=1, kind="stable")[:, case["topk_groups"]:]
        for j in range(gone.shape[1]):
            by_group[np.arange(N), gone[:, j]] = -np.inf
    idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
    picked = np.take_along_axis(key, idx, 1) > -np.inf
    total = np.maximum(score.sum(1, keepdims=True), 1e-300)
    sel = np.where(picked, np.take_along_axis(score, idx, 1), 0.0)
    den = np.maximum(sel.sum(1, keepdims=True), 1e-300)
    count = np.bincount(idx[picked], minlength=E)
    T = max(1, int((~closed).any(1).sum()))
    mean = (score / total).sum(0) / T
    frac = count / (K * T)
    out = dict(topk_idx=None, weights=ROUTE_SCALE * sel / den, expert_count=None, prob_mean=mean,
               loss=np.array([BALANCE_COEF * E * float(frac @ mean)]))
    if case["train"]:
        dw = np.where(picked, s["dweights"].double().cpu().numpy(), 0.0)
        inner = (dw * sel / den).sum(1, keepdims=True)
        coef = BALANCE_COEF * E * frac / T * float(s["dloss"])
        ds = (coef - ((score / total) @ coef)[:, None]) / total
        rows = np.nonzero(picked)
        np.add.at(ds, (rows[0], idx[rows]), (ROUTE_SCALE / den * (dw - inner))[rows])
        if case["score"] == "softmax":
            out["dlogits"] = score * (ds - (score * ds).sum(1, keepdims=True))
        else:
            out["dlogits"] = score * (1.0 - score) * ds
    return out


def _exact_combine_bwd(case, s):
    r = s["route"]
    N, K, C = case["tokens"], case["topk"], case["cols"]
    dy = torch.zeros((r["capacity"], C), dtype=torch.float64, device=DEV)
    dweights = torch.zeros(N * K, dtype=torch.float64, device=DEV)
    pairs = torch.nonzero(r["slot"] >= 0).reshape(-1)
    per = max(1, (1 << 26) // C)
    for a in range(0, pairs.numel(), per):
        p = pairs[a:a + per]
        at, d = r["slot"][p].long(), s["dout"][p // K].double()
        dy[at] = torch.einsum("i,ij->ij", s["weights"].reshape(-1)[p].double(), d)
        if case["dweights"]:
            dweights[p] = torch.einsum("ij,ij->i", s["expert_out"][at].double(), d)
    out = dict(dy=dy)
    if case["dweights"]:
        out["dweights"] = dweights.view(N, K)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, norm_bwd=_exact_norm_bwd, route=_exact_route,
                combine_bwd=_exact_combine_bwd)[case["op"]](case, s)
