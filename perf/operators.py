"""The operators around a scaled FP8 linear layer, as cases to be measured.

A pre-norm expert block runs layer norm, sorts the tokens by expert (every expert's rows
padded to the multiple of 16 that the FP8 GEMMs need), runs the experts' linears, and adds
the experts' outputs back with the router's weights. Measured here are the parts around the
linears and their gradients:

  ln_fwd        y = (x - mean) rstd gamma + beta, with mean and rstd kept for the backward
  ln_bwd        dx, dgamma, dbeta
  dispatch      sort (slot, source, counts, offsets) and the gather of the tokens' rows
  combine       y[t] = sum_j w[t, j] ys[slot[t, j]]; without weights it is the gradient of
                the dispatch
  combine_bwd   the gradients of the experts' outputs and of the router's weights

``own`` False runs plain torch operations in 32 bits; ``own`` True runs the library's
kernels through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
MULTIPLE = 16          # token rows per expert, as the FP8 GEMMs take them


# ------------------------------------------------------------------------- cases

def _ln(name, op, rows, cols, dtype, params, pad=0):
    return dict(name=name, op=op, rows=rows, cols=cols, dtype=dtype, params=params, pad=pad)


def _moe(name, op, tokens, topk, experts, cols, dtype, drop=0.0, weighted=True, pad=0):
    return dict(name=name, op=op, tokens=tokens, topk=topk, experts=experts, cols=cols,
                dtype=dtype, drop=drop, weighted=weighted, pad=pad)


def listed():
    return [
        # one token of a generation step: latency only
        _ln("ln_fwd_token_4096", "ln_fwd", 1, 4096, "bf16", "same"),
        # a training batch at the MLP workload's tokens and width, parameters in 32 bits
        _ln("ln_fwd_8192x4096", "ln_fwd", 8192, 4096, "bf16", "f32"),
        # a ragged batch of an odd width, cut out of a wider activation
        _ln("ln_fwd_odd_1021x5003", "ln_fwd", 1021, 5003, "f16", "same", pad=13),
        # the smallest linear's tokens and width
        _ln("ln_bwd_64x128", "ln_bwd", 64, 128, "bf16", "same"),
        # the training batch's gradient
        _ln("ln_bwd_8192x4096", "ln_bwd", 8192, 4096, "bf16", "f32"),
        # a wide residual stream kept in 32 bits
        _ln("ln_bwd_4096x14336", "ln_bwd", 4096, 14336, "f32", "f32"),
        # one token of a generation step to two of eight experts
        _moe("dispatch_token", "dispatch", 1, 2, 8, 4096, "bf16"),
        # a training batch to eight of 64 experts, some pairs dropped for capacity
        _moe("dispatch_8192_top8", "dispatch", 8192, 8, 64, 4096, "bf16", drop=0.02),
        # the dispatch's gradient on a small ragged batch of an odd width
        _moe("dispatch_grad_odd", "combine", 77, 3, 10, 1027, "f32", drop=0.1, weighted=False),
        # the training batch's combine
        _moe("combine_8192_top8", "combine", 8192, 8, 64, 4096, "bf16", drop=0.02),
        # a few sequences' tokens of an odd width, cut out of a wider gradient
        _moe("combine_bwd_odd", "combine_bwd", 333, 4, 16, 2049, "f16", drop=0.1, pad=7),
        # a training batch to two of eight experts
        _moe("combine_bwd_8192_top2", "combine_bwd", 8192, 2, 8, 4096, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    """Widths over the range, half of them multiples of 64 as model widths are."""
    c = _log(rng, 64, hi)
    return c if rng.random() < 0.5 else max(64, c // 64 * 64)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "dispatch", "combine", "combine_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    pad = rng.choice([0, 0, rng.randint(1, 64)])
    if op.startswith("ln"):
        cols = _width(rng, 16384)
        rows = _log(rng, 1, min(16384, (1 << 25) // cols))
        params = rng.choice(["same", "f32"])
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, params=params, pad=pad)
    cols = _width(rng, 8192)
    topk = rng.randint(1, 8)
    experts = max(topk, _log(rng, 4, 256))
    tokens = _log(rng, 1, min(16384, (1 << 26) // (cols * topk)))
    drop = rng.choice([0.0, 0.02, 0.1])
    weighted = op != "combine" or rng.random() < 0.5
    return dict(op=op, tokens=tokens, topk=topk, experts=experts, cols=cols, dtype=dtype,
                drop=drop, weighted=weighted, pad=pad)


def _rows(case):
    """Rows of the sorted buffer: every expert's rows rounded up, whatever the routing."""
    n = case["tokens"] * case["topk"]
    return (n + min(case["experts"], n) * (MULTIPLE - 1)) // MULTIPLE * MULTIPLE


def work(case):
    es = SIZES[case["dtype"]]
    if case["op"] in ("ln_fwd", "ln_bwd"):
        rows, cols = case["rows"], case["cols"]
        ps = es if case["params"] == "same" else 4
        if case["op"] == "ln_fwd":
            return dict(bytes=2 * rows * cols * es + 2 * cols * ps + 8 * rows,
                        flops=8 * rows * cols)
        return dict(bytes=3 * rows * cols * es + 3 * cols * ps + 8 * rows, flops=14 * rows * cols)
    t, k, e, cols = case["tokens"], case["topk"], case["experts"], case["cols"]
    n, r = t * k, _rows(case)
    kept = int(n * (1.0 - case["drop"]))
    if case["op"] == "dispatch":
        return dict(bytes=(t + r) * cols * es + 12 * n + 4 * r + 4 * (2 * e + 1), flops=0)
    if case["op"] == "combine":
        return dict(bytes=(t + kept) * cols * es + (8 if case["weighted"] else 4) * n,
                    flops=(2 if case["weighted"] else 1) * kept * cols)
    return dict(bytes=(t + kept + r) * cols * es + 12 * n + 4 * r, flops=3 * kept * cols)


# ------------------------------------------------------------------------- inputs

def _matrix(gen, rows, cols, pad, dtype, std=1.0):
    """[rows, cols] of activations: channels with their own offsets and a few loud ones.
    With ``pad`` the rows are a cut out of a wider tensor."""
    dev = "cuda"
    v = torch.randn((rows, cols + pad), generator=gen, device=dev)
    off = 0.3 * torch.randn(cols + pad, generator=gen, device=dev)
    loud = torch.rand(cols + pad, generator=gen, device=dev) < 0.005
    v = (v * torch.where(loud, 12.0, 1.0) + off) * std
    return v.to(dtype)[:, :cols]


def _route(case, gen):
    """A router's choices: some experts are liked more than others, one gets nothing, and a
    share of the pairs is dropped (index -1)."""
    dev = "cuda"
    t, k, e = case["tokens"], case["topk"], case["experts"]
    logits = torch.randn((t, e), generator=gen, device=dev)
    logits += 0.7 * torch.randn(e, generator=gen, device=dev)
    if e > k:
        logits[:, e // 2] = -1e9
    top, idx = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, dim=1)
    if case["drop"] > 0:
        idx = torch.where(torch.rand((t, k), generator=gen, device=dev) < case["drop"],
                          torch.full_like(idx, -1), idx)
    return idx.contiguous(), w.contiguous()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inputs(case, seed):
    gen = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        rows, cols = case["rows"], case["cols"]
        pt = dt if case["params"] == "same" else torch.float32
        s["x"] = _matrix(gen, rows, cols, case["pad"], dt)
        s["gamma"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(pt)
        if case["op"] == "ln_fwd":
            s["beta"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(pt)
        else:
            s["dy"] = _matrix(gen, rows, cols, case["pad"], dt, std=0.1)
            # what the forward pass kept
            x64 = s["x"].double()
            mean = x64.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x64 - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        return s
    cols = case["cols"]
    s["idx"], s["weights"] = _route(case, gen)
    if case["op"] == "dispatch":
        s["x"] = _matrix(gen, case["tokens"], cols, case["pad"], dt)
        return s
    s["slot"], s["source"], _, _ = _plain_sort(s["idx"], case["experts"], _rows(case))
    s["ys"] = _matrix(gen, _rows(case), cols, case["pad"], dt)
    if case["op"] == "combine_bwd":
        s["dy"] = _matrix(gen, case["tokens"], cols, case["pad"], dt, std=0.1)
    return s


def prepare(case, seed):
    """The inputs; beside them the buffers that a program which runs the operator every step
    keeps for its outputs."""
    s = _inputs(case, seed)
    if not own:
        return s
    dt, dev = DTYPES[case["dtype"]], "cuda"
    if case["op"] in ("ln_fwd", "ln_bwd"):
        rows, cols = case["rows"], case["cols"]
        out = torch.empty((rows, cols), dtype=dt, device=dev)
        if case["op"] == "ln_fwd":
            s["out"] = dict(y=out, mean=torch.empty(rows, device=dev),
                            rstd=torch.empty(rows, device=dev))
        else:
            s["out"] = dict(dx=out, dgamma=torch.empty_like(s["gamma"]),
                            dbeta=torch.empty_like(s["gamma"]))
        return s
    t, k, e, cols, r = case["tokens"], case["topk"], case["experts"], case["cols"], _rows(case)
    i32 = dict(dtype=torch.int32, device=dev)
    if case["op"] == "dispatch":
        s["plan"] = dict(slot=torch.empty((t, k), **i32), source=torch.empty(r, **i32),
                         counts=torch.empty(e, **i32), offsets=torch.empty(e + 1, **i32))
        s["out"] = torch.empty((r, cols), dtype=dt, device=dev)
    elif case["op"] == "combine":
        s["out"] = torch.empty((t, cols), dtype=dt, device=dev)
    else:
        s["out"] = dict(dys=torch.empty((r, cols), dtype=dt, device=dev),
                        dw=torch.empty((t, k), device=dev))
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_sort(idx, experts, rows):
    """Stable sort of the flat (token, choice) pairs by expert. slot: each pair's row of the
    sorted buffer (-1: dropped); source: each row's flat pair (-1: padding)."""
    flat = idx.reshape(-1)
    n = flat.numel()
    dev = flat.device
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=dev)
    counts.index_add_(0, key, torch.ones_like(key))
    padded = (counts[:experts] + MULTIPLE - 1) // MULTIPLE * MULTIPLE
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    offsets = torch.cat([zero, torch.cumsum(padded, 0)])
    starts = torch.cat([zero, torch.cumsum(counts, 0)])
    sk, order = torch.sort(key, stable=True)
    rank = torch.arange(n, device=dev) - starts[sk]
    row = torch.where(sk < experts, offsets[sk] + rank, torch.full_like(sk, -1))
    slot = torch.empty(n, dtype=torch.int64, device=dev)
    slot[order] = row
    source = torch.full((rows + 1,), -1, dtype=torch.int64, device=dev)
    source[torch.where(row >= 0, row, torch.full_like(row, rows))] = order
    return (slot.view(idx.shape).int(), source[:rows].contiguous().int(),
            counts[:experts].int(), offsets.int())


def _plain(s):
    case = s["case"]
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        y = d * rstd * s["gamma"].float() + s["beta"].float()
        return y.to(dt), mean[:, 0], rstd[:, 0]
    if op == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["gamma"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        pt = s["gamma"].dtype
        return dx.to(dt), (dy * xh).sum(0).to(pt), dy.sum(0).to(pt)
    k, rows = case["topk"], _rows(case)
    if op == "dispatch":
        slot, source, counts, offsets = _plain_sort(s["idx"], case["experts"], rows)
        live = source >= 0
        xs = s["x"][torch.where(live, source // k, 0)] * live[:, None]
        return xs, slot, source, counts, offsets
    slot = s["slot"].long()
    kept = slot >= 0
    at = torch.where(kept, slot, 0)
    if op == "combine":
        y = torch.zeros((case["tokens"], case["cols"]), device="cuda")
        for j in range(k):
            v = torch.where(kept[:, j:j + 1], s["ys"][at[:, j]].float(), 0.0)
            y += v * s["weights"][:, j:j + 1] if case["weighted"] else v
        return y.to(dt)
    dy, source = s["dy"].float(), s["source"].long()
    live = source >= 0
    src = torch.where(live, source, 0)
    w = s["weights"].reshape(-1)[src]
    dys = torch.where(live[:, None], dy[src // k] * w[:, None], 0.0).to(dt)
    dw = torch.zeros((case["tokens"], k), device="cuda")
    for j in range(k):
        dot = (dy * s["ys"][at[:, j]].float()).sum(1)
        dw[:, j] = torch.where(kept[:, j], dot, 0.0)
    return dys, dw


# ------------------------------------------------------------------------- the kernels

def _own(s):
    import scaled_fp8_linear_amd as m
    case = s["case"]
    op = case["op"]
    if op == "ln_fwd":
        return m.fp8_layernorm_fwd(s["x"], s["gamma"], s["beta"], eps=EPS, **s["out"])
    if op == "ln_bwd":
        return m.fp8_layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], **s["out"])
    if op == "dispatch":
        slot, source, counts, offsets = m.fp8_moe_sort(s["idx"], case["experts"],
                                                       multiple=MULTIPLE, **s["plan"])
        xs = m.fp8_moe_dispatch(s["x"], slot, source, xs=s["out"])
        return xs, slot, source, counts, offsets
    if op == "combine":
        if not case["weighted"]:
            return m.fp8_moe_dispatch_bwd(s["ys"], s["slot"], dx=s["out"])
        return m.fp8_moe_combine(s["ys"], s["slot"], s["weights"], y=s["out"])
    return m.fp8_moe_combine_bwd(s["dy"], s["ys"], s["slot"], s["source"], s["weights"],
                                 **s["out"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------- 64 bits

def _exact_plan(idx, experts, rows):
    """The sort, pair by pair."""
    pairs = idx.cpu().numpy().reshape(-1)
    bins = [[] for _ in range(experts)]
    for i, e in enumerate(pairs.tolist()):
        if 0 <= e < experts:
            bins[e].append(i)
    slot = np.full(pairs.size, -1, dtype=np.int32)
    source = np.full(rows, -1, dtype=np.int32)
    offsets, at = [0], 0
    for b in bins:
        for r, i in enumerate(b):
            slot[i], source[at + r] = at + r, i
        at += -(-len(b) // MULTIPLE) * MULTIPLE
        offsets.append(at)
    dev = idx.device
    return (torch.from_numpy(slot.reshape(tuple(idx.shape))).to(dev),
            torch.from_numpy(source).to(dev),
            torch.tensor([len(b) for b in bins], dtype=torch.int32, device=dev),
            torch.tensor(offsets, dtype=torch.int32, device=dev))


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "ln_fwd":
        x = s["x"].double()
        mean = x.sum(1) / case["cols"]
        var = (x - mean[:, None]).pow(2).sum(1) / case["cols"]
        rstd = (var + EPS).pow(-0.5)
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None],
                          s["gamma"].double())
        return y, mean, rstd
    if op == "ln_bwd":
        dy, x, rstd = s["dy"].double(), s["x"].double(), s["rstd"].double()[:, None]
        xh = (x - s["mean"].double()[:, None]) * rstd
        g = dy * s["gamma"].double()
        n = case["cols"]
        a, b = g.sum(1, keepdim=True), (g * xh).sum(1, keepdim=True)
        return rstd * (n * g - a - xh * b) / n, (dy * xh).sum(0), dy.sum(0)
    t, k, rows = case["tokens"], case["topk"], _rows(case)
    slot, source, counts, offsets = _exact_plan(s["idx"], case["experts"], rows)
    # the sorted rows as seen from the pairs: row slot[t, j] belongs to token t
    kept = slot >= 0
    tok, choice = torch.nonzero(kept, as_tuple=True)
    row = slot[tok, choice].long()
    if op == "dispatch":
        xs = torch.zeros((rows, case["cols"]), dtype=torch.float64, device="cuda")
        xs[row] = s["x"].double()[tok]
        return xs, slot, source, counts, offsets
    w = s["weights"].double()
    if op == "combine":
        y = torch.zeros((t, case["cols"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            tj = torch.nonzero(kept[:, j])[:, 0]
            v = s["ys"][slot[tj, j].long()].double()
            y[tj] += v * w[tj, j:j + 1] if case["weighted"] else v
        return y
    dy = s["dy"].double()
    dys = torch.zeros((rows, case["cols"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        tj = torch.nonzero(kept[:, j])[:, 0]
        rj = slot[tj, j].long()
        dys[rj] = dy[tj] * w[tj, j:j + 1]
        dw[tj, j] = (dy[tj] * s["ys"][rj].double()).sum(1)
    return dys, dw
