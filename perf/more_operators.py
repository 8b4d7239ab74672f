"""The router, the experts' products and the activation between them, as cases to be measured.

A mixture-of-experts block sends each token to the experts that its router likes best, keeps
the experts evenly used by a balance loss, runs every expert's two linears on its own rows, and
an activation between them. Measured here are these parts and their gradients; the sort, the
dispatch and the combine around them are measured elsewhere:

  route        softmax over the experts, the topk choices (ties to the lowest index) and their
               weights, pairs per expert, the balance loss and the z-loss
  route_bwd    the gradient of the weights and of both losses with respect to the logits
  act          a = act(g) u of h = [g | u] (or act(h)), quantized by tiles of 128 along a row
               for the next product and along the rows for its weight gradient; h kept in
               8 bits for the backward
  act_bwd      the gradient from da and the kept h, quantized both ways, or as it is
  grouped_fwd, grouped_dgrad, grouped_wgrad
               the experts' products of 8-bit codes with a scale for each block of 128

``own`` False runs plain torch operations in 32 bits; ``own`` True runs the library's
kernels through the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
BLOCK = 128            # codes per scale; token rows per expert are a multiple of it
TOP = 448.0            # largest e4m3 value
FLOOR = 1e-12          # a tile of zeros has this amax
GROUPED = ("grouped_fwd", "grouped_dgrad", "grouped_wgrad")


# ------------------------------------------------------------------------- cases

def _route(name, op, tokens, experts, topk, dtype, normalize=True, pad=0, masked=0.0):
    return dict(name=name, op=op, tokens=tokens, experts=experts, topk=topk, dtype=dtype,
                normalize=normalize, pad=pad, masked=masked)


def _act(name, op, rows, cols, act, gated, dtype, valid=None, train=True, plain_out=False):
    return dict(name=name, op=op, rows=rows, valid=rows if valid is None else valid, cols=cols,
                act=act, gated=gated, dtype=dtype, train=train, plain_out=plain_out)


def _grouped(name, op, tokens, experts, topk, n, k):
    return dict(name=name, op=op, tokens=tokens, experts=experts, topk=topk, n=n, k=k)


def listed():
    return [
        # one token of a generation step to two of eight experts: latency only
        _route("route_token", "route", 1, 8, 2, "bf16"),
        # a training batch to eight of 64 experts
        _route("route_8192_top8", "route", 8192, 64, 8, "bf16"),
        # a small ragged batch, probabilities as they are, some experts masked, logits cut
        # out of a wider tensor
        _route("route_bwd_odd", "route_bwd", 333, 60, 3, "f16", normalize=False, pad=5,
               masked=0.1),
        # a long training batch to eight of 256 experts, logits kept in 32 bits
        _route("route_bwd_16384x256", "route_bwd", 16384, 256, 8, "f32"),
        # the activation of one token's two experts in a generation step (nothing is kept)
        _act("act_token", "act", 256, 14336, "silu", True, "bf16", valid=129, train=False),
        # the training batch's activation: both quantized copies and the checkpoint
        _act("act_17408x14336", "act", 17408, 14336, "silu", True, "bf16", valid=17000),
        # a small layer without a gate whose gradient goes on unquantized, in 32 bits
        _act("act_bwd_640x2048", "act_bwd", 640, 2048, "gelu", False, "f32", valid=611,
             plain_out=True),
        # the training batch's gradient
        _act("act_bwd_17408x14336", "act_bwd", 17408, 14336, "silu", True, "bf16", valid=17000),
        # one token of a generation step: two experts' weights are read
        _grouped("grouped_fwd_token", "grouped_fwd", 1, 8, 2, 14336, 4096),
        # the training batch at the MLP workload's tokens and sizes, two of eight experts
        _grouped("grouped_fwd_8192_top2", "grouped_fwd", 8192, 8, 2, 14336, 4096),
        # many small experts with few and uneven rows each
        _grouped("grouped_dgrad_ragged", "grouped_dgrad", 1021, 64, 8, 1408, 2048),
        # the training batch's weight gradients
        _grouped("grouped_wgrad_8192_top2", "grouped_wgrad", 8192, 8, 2, 14336, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _blocks(rng, hi):
    return BLOCK * _log(rng, 1, hi // BLOCK)


def draw(rng):
    op = rng.choice(["route", "route_bwd", "act", "act_bwd", *GROUPED])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("route", "route_bwd"):
        experts = _log(rng, 2, 512)
        topk = min(experts, rng.randint(1, 10))
        tokens = _log(rng, 1, min(32768, (1 << 22) // experts))
        return dict(op=op, tokens=tokens, experts=experts, topk=topk, dtype=dtype,
                    normalize=rng.random() < 0.6, pad=rng.choice([0, 0, rng.randint(1, 64)]),
                    masked=rng.choice([0.0, 0.0, 0.3]))
    if op in ("act", "act_bwd"):
        cols = _blocks(rng, 14336)
        rows = BLOCK * _log(rng, 1, min(136, max(1, (1 << 27) // cols // BLOCK)))
        return dict(op=op, rows=rows, valid=max(0, rows - rng.choice([0, rng.randint(1, 130)])),
                    cols=cols, act=rng.choice(["silu", "gelu", "relu"]),
                    gated=rng.random() < 0.6, dtype=dtype, train=rng.random() < 0.7,
                    plain_out=rng.random() < 0.3)
    n, k = _blocks(rng, 14336), _blocks(rng, 14336)
    experts = _log(rng, 2, max(2, min(128, (1 << 28) // (n * k))))
    topk = min(experts, rng.randint(1, 8))
    tokens = _log(rng, 1, max(1, min(8192, (1 << 39) // (n * k * topk))))
    return dict(op=op, tokens=tokens, experts=experts, topk=topk, n=n, k=k)


def _rows(case):
    """Rows of the sorted buffer: every expert's rows rounded up, whatever the routing."""
    n = case["tokens"] * case["topk"]
    return (n + min(case["experts"], n) * (BLOCK - 1)) // BLOCK * BLOCK


def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        t, e, k, es = case["tokens"], case["experts"], case["topk"], SIZES[case["dtype"]]
        if op == "route":
            return dict(bytes=t * e * es + 8 * t * k + 4 * t + 4 * e + 8, flops=12 * t * e)
        return dict(bytes=2 * t * e * es + 12 * t * k + 4 * t + 4 * e + 8, flops=12 * t * e)
    if op in ("act", "act_bwd"):
        rows, cols, v = case["rows"], case["cols"], case["valid"]
        h, es = cols * (2 if case["gated"] else 1), SIZES[case["dtype"]]
        both = 2 if case["train"] else 1
        tile = 1 + 4 / BLOCK                     # a code and its share of a scale
        if op == "act":
            return dict(bytes=v * h * es + both * rows * cols * tile
                        + (rows * h * tile if case["train"] else 0), flops=20 * v * cols)
        out = rows * h * es if case["plain_out"] else both * rows * h * tile
        return dict(bytes=v * cols * es + v * h * tile + out, flops=30 * v * cols)
    n, k, pairs, rows = case["n"], case["k"], case["tokens"] * case["topk"], _rows(case)
    tile = 1 + 4 / BLOCK
    used = min(case["experts"], pairs)
    if op == "grouped_wgrad":
        moved = pairs * (n + k) * tile + 2 * case["experts"] * n * k
    else:
        i, o = (k, n) if op == "grouped_fwd" else (n, k)
        moved = pairs * i * tile + used * n * k + 2 * rows * o
    return dict(bytes=moved, flops=2 * pairs * n * k)


# ------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _choices(gen, tokens, experts, topk):
    """A router's choices, some experts liked more than others."""
    logits = torch.randn((tokens, experts), generator=gen, device="cuda")
    logits += 0.3 * torch.randn(experts, generator=gen, device="cuda")
    return torch.topk(logits, topk, dim=1).indices


def _codes(gen, shape):
    """Codes of normally distributed values, each tile's largest near the format's."""
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return (v * 120).clamp(-TOP, TOP).to(E4M3)


def _scales(gen, shape, size):
    return size / TOP * torch.exp(0.5 * torch.randn(shape, generator=gen, device="cuda"))


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    s = dict(case=case)
    f32 = dict(device="cuda", dtype=torch.float32)
    if op in ("route", "route_bwd"):
        t, e, k, dt = case["tokens"], case["experts"], case["topk"], DTYPES[case["dtype"]]
        v = torch.randn((t, e + case["pad"]), generator=gen, device="cuda") * 1.5
        v += torch.randn(e + case["pad"], generator=gen, device="cuda") * 0.5
        if case["masked"] > 0:
            gone = torch.rand(e + case["pad"], generator=gen, device="cuda") < case["masked"]
            gone[0] = False
            v = torch.where(gone, -math.inf, v)
        s["logits"] = v.to(dt)[:, :e]
        if op == "route_bwd":
            # what the forward pass kept
            s["idx"], s["weights"], s["lse"], s["counts"], _ = _plain_route(s["logits"], k,
                                                                            case["normalize"])
            s["dweights"] = torch.randn((t, k), generator=gen, **f32)
            s["dlosses"] = torch.tensor([0.01, 0.001], **f32) * (1 + seed % 7)
        return s
    if op in ("act", "act_bwd"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        width = cols * (2 if case["gated"] else 1)
        # the rows that pad the experts are zero: here one in 50
        live = (torch.rand((rows, 1), generator=gen, device="cuda") >= 0.02).to(dt)
        if op == "act":
            s["h"] = torch.randn((rows, width), generator=gen, device="cuda", dtype=dt).mul_(live)
            return s
        s["hq"] = _codes(gen, (rows, width))
        s["hscale"] = _scales(gen, (rows, width // BLOCK), 3.0)
        s["da"] = torch.randn((rows, cols), generator=gen, device="cuda", dtype=dt).mul_(live)
        return s
    t, e, k = case["tokens"], case["experts"], case["topk"]
    rows = _rows(case)
    idx = _choices(gen, t, e, k).reshape(-1)
    counts = torch.zeros(e, dtype=torch.int64, device="cuda")
    counts.index_add_(0, idx, torch.ones_like(idx))
    ends = torch.cumsum((counts + BLOCK - 1) // BLOCK * BLOCK, 0)
    s["offsets"] = torch.cat([ends.new_zeros(1), ends]).int()
    s["counts"] = counts.int()
    # the longest expert's rows: a program that pads its experts to a capacity knows it
    s["capacity"] = int(counts.max())
    row = torch.arange(rows, device="cuda")
    at = torch.searchsorted(ends, row, right=True).clamp(max=e - 1)
    live = (row - s["offsets"].long()[at] < counts[at]) & (row < ends[-1])
    n, kk = case["n"], case["k"]
    if op == "grouped_wgrad":
        for name, width in (("g", n), ("x", kk)):
            q = _codes(gen, (width, rows)).view(torch.uint8) * live.to(torch.uint8)
            s["q" + name] = q.view(E4M3)
            s["s" + name] = _scales(gen, (width, rows // BLOCK), 3.0)
        return s
    i, o = (kk, n) if op == "grouped_fwd" else (n, kk)
    s["qx"] = (_codes(gen, (rows, i)).view(torch.uint8) * live.to(torch.uint8)[:, None]).view(E4M3)
    s["sx"] = _scales(gen, (rows, i // BLOCK), 3.0)
    if op == "grouped_fwd":
        s["qw"] = _codes(gen, (e, o, i))
        s["sw"] = _scales(gen, (e, o // BLOCK, i // BLOCK), 0.1)
    else:
        # the transposed copy of the experts' stacked weights [e n, k], as one quantization of
        # the stack gives it: expert after expert along the columns
        s["qw"] = _codes(gen, (o, e * i)).view(o, e, i).transpose(0, 1)
        s["sw"] = _scales(gen, (o // BLOCK, e * (i // BLOCK)), 0.1) \
            .view(o // BLOCK, e, i // BLOCK).transpose(0, 1)
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_route(logits, topk, normalize):
    x = logits.float()
    t, e = x.shape
    top = x.amax(1, keepdim=True)
    ex = torch.exp(x - top)
    total = ex.sum(1, keepdim=True)
    p = ex / total
    lse = (top + torch.log(total))[:, 0]
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    v, i = v[:, :topk], i[:, :topk]
    kept = v > -math.inf
    w = torch.exp(v - v[:, :1]) if normalize else torch.exp(v - top)
    w = w / (w.sum(1, keepdim=True) if normalize else total)
    idx = torch.where(kept, i, -1)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
    flat = torch.where(kept, i, e).reshape(-1)
    counts.index_add_(0, flat, torch.ones_like(flat))
    counts = counts[:e]
    balance = e / (t * topk) * (counts * p.mean(0)).sum()
    return idx.int(), w, lse, counts.int(), torch.stack([balance, lse.square().mean()])


def _plain_route_bwd(s, case):
    x = s["logits"].float()
    t, e = x.shape
    k = case["topk"]
    p = torch.exp(x - s["lse"][:, None])
    c = s["counts"].float()
    db, dz = s["dlosses"][0], s["dlosses"][1]
    d = db * (e / (t * t * k)) * p * (c - (p * c).sum(1, keepdim=True))
    d += dz * (2.0 / t) * s["lse"][:, None] * p
    kept = s["idx"] >= 0
    w = torch.where(kept, s["weights"], 0.0)
    dw = torch.where(kept, s["dweights"], 0.0)
    dot = (w * dw).sum(1, keepdim=True)
    to = torch.where(kept, s["idx"], 0).long()
    if case["normalize"]:
        d.scatter_add_(1, to, w * (dw - dot))
    else:
        d -= p * dot
        d.scatter_add_(1, to, w * dw)
    return d.to(s["logits"].dtype)


def _tiles(v, dim):
    """v [r, c] quantized by tiles of 128 along `dim`: the codes (transposed for dim 0, so that
    the tiles lie along a row again) and the scales."""
    v = v if dim == 1 else v.t()
    r, c = v.shape
    v = v.reshape(r, c // BLOCK, BLOCK)
    top = v.abs().amax(2).clamp(min=FLOOR)
    q = (v * (TOP / top)[:, :, None]).clamp(-TOP, TOP).to(E4M3)
    return q.reshape(r, c), top / TOP


def _values(q, scale):
    r, c = q.shape
    return (q.float().view(r, c // BLOCK, BLOCK) * scale[:, :, None]).view(r, c)


ROOT = math.sqrt(2.0 / math.pi)


def _act_of(x, act):
    """(act(x), act'(x))."""
    if act == "relu":
        return x.clamp(min=0), (x > 0).to(x.dtype)
    if act == "silu":
        y = torch.sigmoid(x)
        return x * y, y * (1 + x * (1 - y))
    z = ROOT * (x + 0.044715 * x * x * x)        # gelu with the tanh
    th = torch.tanh(z)
    return 0.5 * x * (1 + th), 0.5 * (1 + th) + 0.5 * x * (1 - th * th) * ROOT \
        * (1 + 3 * 0.044715 * x * x)


def _plain_act(s, case):
    cols = case["cols"]
    h = s["h"].float()
    h[case["valid"]:] = 0
    a, _ = _act_of(h[:, :cols], case["act"])
    if case["gated"]:
        a = a * h[:, cols:]
    out = _tiles(a, 1)
    return (*out, *_tiles(a, 0), *_tiles(h, 1)) if case["train"] else out


def _plain_act_bwd(s, case):
    cols = case["cols"]
    h = _values(s["hq"], s["hscale"])
    da = s["da"].float()
    a, d = _act_of(h[:, :cols], case["act"])
    dh = torch.cat([da * h[:, cols:] * d, da * a], 1) if case["gated"] else da * d
    dh[case["valid"]:] = 0
    if case["plain_out"]:
        return dh.to(s["da"].dtype)
    out = _tiles(dh, 1)
    return (*out, *_tiles(dh, 0)) if case["train"] else out


def _members(s, experts):
    """The rows [len(experts), capacity] of some experts, and which of them there are."""
    at = torch.arange(s["capacity"], device="cuda")
    there = at < s["counts"].long()[experts][:, None]
    return torch.where(there, s["offsets"].long()[experts][:, None] + at, 0), there


def _plain_grouped(s, case):
    e, pairs, rows = case["experts"], case["tokens"] * case["topk"], _rows(case)
    if case["op"] == "grouped_wgrad":
        at, there = _members(s, torch.arange(e, device="cuda"))
        g = _values(s["qg"], s["sg"])[:, at.reshape(-1)] * there.reshape(-1)
        x = _values(s["qx"], s["sx"])[:, at.reshape(-1)]
        g = g.view(case["n"], e, -1).transpose(0, 1).contiguous()
        x = x.view(case["k"], e, -1).permute(1, 2, 0).contiguous()
        return torch.bmm(g, x).to(torch.bfloat16)
    qw, sw = s["qw"], s["sw"]
    experts = torch.arange(e, device="cuda")
    if pairs < e:                                # only the experts that were chosen
        experts = torch.sort((s["counts"] > 0).int(), descending=True, stable=True)[1][:pairs]
        qw, sw = qw.view(torch.uint8)[experts].view(E4M3), sw[experts]
    at, there = _members(s, experts)
    x = _values(s["qx"], s["sx"])[at.reshape(-1)].view(*at.shape, -1)
    n, o, i = qw.shape
    w = (qw.float().view(n, o // BLOCK, BLOCK, i // BLOCK, BLOCK)
         * sw[:, :, None, :, None]).view(n, o, i)
    y = torch.bmm(x, w.transpose(1, 2).contiguous()).to(torch.bfloat16)
    out = torch.zeros((rows + 1, o), dtype=torch.bfloat16, device="cuda")
    out[torch.where(there, at, rows).reshape(-1)] = y.view(-1, o)
    return out[:rows]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        return _plain_route(s["logits"], case["topk"], case["normalize"])
    if op == "route_bwd":
        return _plain_route_bwd(s, case)
    if op == "act":
        return _plain_act(s, case)
    if op == "act_bwd":
        return _plain_act_bwd(s, case)
    return _plain_grouped(s, case)


# ------------------------------------------------------------------------- the kernels

def _own(s):
    import scaled_fp8_linear_amd as m
    case = s["case"]
    op = case["op"]
    if op == "route":
        return m.fp8_moe_route(s["logits"], case["topk"], normalize=case["normalize"])
    if op == "route_bwd":
        return m.fp8_moe_route_bwd(s["logits"], s["lse"], s["idx"], s["weights"], s["counts"],
                                   dweights=s["dweights"], dlosses=s["dlosses"],
                                   normalize=case["normalize"])
    if op == "act":
        q, scale, q_t, scale_t, hq, hscale = m.fp8_act_quantize(
            s["h"], act=case["act"], gated=case["gated"], rows_valid=case["valid"],
            want_q_t=case["train"], want_checkpoint=case["train"])
        if not case["train"]:
            return q.view(E4M3), scale
        return q.view(E4M3), scale, q_t.view(E4M3), scale_t, hq.view(E4M3), hscale
    if op == "act_bwd":
        plain = case["plain_out"]
        q, scale, q_t, scale_t, dh = m.fp8_act_quantize_bwd(
            s["da"], s["hq"], s["hscale"], act=case["act"], gated=case["gated"],
            rows_valid=case["valid"], want_q=not plain, want_q_t=case["train"] and not plain,
            want_dh=plain)
        if plain:
            return dh
        if not case["train"]:
            return q.view(E4M3), scale
        return q.view(E4M3), scale, q_t.view(E4M3), scale_t
    if op == "grouped_wgrad":
        return m.fp8_grouped_linear_wgrad(s["qg"], s["qx"], s["sg"], s["sx"], s["offsets"],
                                          s["counts"])
    f = m.fp8_grouped_linear_fwd if op == "grouped_fwd" else m.fp8_grouped_linear_dgrad
    return f(s["qx"], s["qw"], s["sx"], s["sw"], s["offsets"], s["counts"],
             max_rows=case["tokens"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------- 64 bits

def _exact_route(s, case):
    x = s["logits"].double()
    t, e = x.shape
    k = case["topk"]
    p = torch.softmax(x, 1)
    lse = torch.logsumexp(x, 1)
    # lowest index first among equal logits: order by (-logit, index)
    order = torch.argsort(-x, dim=1, stable=True)[:, :k]
    l = torch.gather(x, 1, order)
    kept = torch.isfinite(l)
    w = torch.softmax(l, 1) if case["normalize"] else torch.gather(p, 1, order)
    counts = torch.stack([((order == j) & kept).sum() for j in range(e)])
    balance = e * ((counts / (t * k)) * (p.sum(0) / t)).sum()
    return (torch.where(kept, order, -1).int(), torch.where(kept, w, 0.0), lse, counts.int(),
            torch.stack([balance, (lse * lse).sum() / t]))


def _exact_route_bwd(s, case):
    """By autograd, from the loss that the forward pass defines."""
    x = s["logits"].double().detach().requires_grad_()
    t, e = x.shape
    k = case["topk"]
    logp = torch.log_softmax(x, 1)
    lse = torch.logsumexp(x, 1)
    kept = s["idx"] >= 0
    l = torch.gather(logp, 1, torch.where(kept, s["idx"], 0).long())
    l = torch.where(kept, l, -math.inf)
    w = torch.softmax(l, 1) if case["normalize"] else torch.exp(l)
    dw = s["dweights"].double()
    f = s["counts"].double() / (t * k)
    loss = torch.where(kept, w * dw, 0.0).sum() \
        + s["dlosses"][0].double() * e * (torch.exp(logp).mean(0) * f).sum() \
        + s["dlosses"][1].double() * lse.square().mean()
    g, = torch.autograd.grad(loss, x)
    return torch.where(torch.isinf(x.detach()), 0.0, g)


def _exact_tiles(v, dim):
    v = v if dim == 1 else v.t().contiguous()
    r, c = v.shape
    top = v.view(r, -1, BLOCK).abs().max(2).values
    scale = torch.maximum(top, torch.full_like(top, FLOOR)) / TOP
    return v / scale.repeat_interleave(BLOCK, 1), scale


def _exact_act_of(x, act):
    if act == "relu":
        return torch.relu(x)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def _exact_part(h, case):
    cols = case["cols"]
    a = _exact_act_of(h[:, :cols], case["act"])
    return a * h[:, cols:] if case["gated"] else a


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s, case)
    if op == "route_bwd":
        return _exact_route_bwd(s, case)
    if op == "act":
        h = s["h"].double()
        h[case["valid"]:] = 0
        a = _exact_part(h, case)
        out = _exact_tiles(a, 1)
        return (*out, *_exact_tiles(a, 0), *_exact_tiles(h, 1)) if case["train"] else out
    if op == "act_bwd":
        h = s["hq"].double() * s["hscale"].double().repeat_interleave(BLOCK, 1)
        h.requires_grad_()
        dh, = torch.autograd.grad(_exact_part(h, case), h, s["da"].double())
        dh[case["valid"]:] = 0
        if case["plain_out"]:
            return dh
        out = _exact_tiles(dh, 1)
        return (*out, *_exact_tiles(dh, 0)) if case["train"] else out
    # expert by expert, on the rows that it holds
    first, count = s["offsets"].tolist(), s["counts"].tolist()
    if op == "grouped_wgrad":
        g = s["qg"].double() * s["sg"].double().repeat_interleave(BLOCK, 1)
        x = s["qx"].double() * s["sx"].double().repeat_interleave(BLOCK, 1)
        dw = torch.zeros((case["experts"], case["n"], case["k"]), dtype=torch.float64,
                         device="cuda")
        for j in range(case["experts"]):
            at = slice(first[j], first[j] + count[j])
            dw[j] = g[:, at] @ x[:, at].t().contiguous()
        return dw
    x = s["qx"].double() * s["sx"].double().repeat_interleave(BLOCK, 1)
    y = torch.zeros((_rows(case), s["qw"].shape[1]), dtype=torch.float64, device="cuda")
    for j in range(case["experts"]):
        if count[j]:
            at = slice(first[j], first[j] + count[j])
            w = s["qw"][j].double() * s["sw"][j].double().repeat_interleave(BLOCK, 0) \
                .repeat_interleave(BLOCK, 1)
            y[at] = x[at] @ w.t().contiguous()
    return y
