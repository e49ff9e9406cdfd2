"""The mixture-of-experts operators around the HSTU layer, as they are measured: their cases,
their inputs, their plain forms in elementary torch operations, and their values in 64 bits.

Four operators, each reached through jagged_hstu_attention_02_b200.ops:

  norm     RMS norm of rows with the residual's addition; output in the rows' type or in e4m3
           with scales; mode "train" is the forward and its gradients
  route    (token, choice) pairs sorted by expert, and the tokens' rows moved to their places
  combine  rows brought back to their tokens, weighted and summed; mode "train" with gradients
  proj     the experts' products on sorted rows (jagged in the expert), bf16 or e4m3;
           mode "bwd" gives the gradients of rows and weights
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one scoring step of a small batch: latency
        dict(name="norm-e4m3-decode", op="norm", mode="e4m3", rows=16, width=1024, dtype="bf16",
             group=0, residual=True),
        # long histories' tokens before an 8-bit product, one scale per 128 columns
        dict(name="norm-e4m3-prompt", op="norm", mode="e4m3", rows=16384, width=4096,
             dtype="bf16", group=128, residual=True),
        # the tokens of a MovieLens-shaped batch, 4 heads x 128 wide, forward and gradients
        dict(name="norm-train", op="norm", mode="train", rows=10923, width=512, dtype="bf16",
             group=0, residual=True),
        # candidates of a few users to their experts: latency
        dict(name="route-decode", op="route", tokens=64, choices=4, experts=64, width=1024,
             dtype="e4m3", padding=0.0),
        # a training batch, some of it padding that no expert takes
        dict(name="route-train", op="route", tokens=32768, choices=4, experts=64, width=1024,
             dtype="bf16", padding=0.06),
        # the way back of the small step
        dict(name="combine-decode", op="combine", mode="fwd", tokens=64, choices=4, experts=64,
             width=1024, dtype="bf16", padding=0.0),
        # the way back of the training batch, with the gradients of rows and weights
        dict(name="combine-train", op="combine", mode="train", tokens=32768, choices=4,
             experts=64, width=1024, dtype="bf16", padding=0.06),
        # few rows per expert, bf16: the experts' weights are what is read
        dict(name="proj-decode", op="proj", mode="bf16", rows=256, experts=64, k=1024, n=2048,
             silu=True, padding=0.0),
        # the smallest product: 8-bit weights of a few experts
        dict(name="proj-e4m3-decode", op="proj", mode="e4m3", rows=64, experts=16, k=1024,
             n=1024, silu=True, padding=0.0),
        # two experts for each token of the MovieLens-shaped batch
        dict(name="proj-prompt", op="proj", mode="bf16", rows=21846, experts=8, k=512, n=2048,
             silu=True, padding=0.02),
        # the largest: long histories in 8 bits
        dict(name="proj-e4m3-prompt", op="proj", mode="e4m3", rows=32768, experts=16, k=2048,
             n=4096, silu=True, padding=0.0),
        # gradients of rows and weights behind an activation
        dict(name="proj-train", op="proj", mode="bwd", rows=16384, experts=8, k=1024, n=2048,
             silu=True, padding=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "combine", "proj", "proj"])
    padding = rng.choice([0.0, 0.02, 0.1, 0.5])
    if op == "norm":
        width = _log(rng, 48, 8192)
        width = rng.choice([width, -(-width // 8) * 8, -(-width // 128) * 128])
        rows = _log(rng, 1, max(1, min(32768, (1 << 26) // width)))
        mode = rng.choice(["e4m3", "same", "train"])
        return dict(op=op, mode=mode, rows=rows, width=width, dtype=rng.choice(["bf16", "f32"]),
                    group=rng.choice([0, 32, 64, 128]) if mode == "e4m3" else 0,
                    residual=rng.random() < 0.7)
    if op in ("route", "combine"):
        choices = rng.randint(1, 8)
        experts = max(choices, _log(rng, 2, 256))
        width = _log(rng, 32, 4096)
        width = rng.choice([width, -(-width // 16) * 16, -(-width // 64) * 64])
        tokens = _log(rng, 1, max(1, min(131072, (1 << 27) // (width * choices))))
        c = dict(op=op, tokens=tokens, choices=choices, experts=experts, width=width,
                 padding=padding)
        if op == "route":
            return dict(c, dtype=rng.choice(["bf16", "e4m3", "f32"]))
        return dict(c, mode=rng.choice(["fwd", "train"]), dtype=rng.choice(["bf16", "f32"]))
    mode = rng.choice(["bf16", "e4m3", "bwd"])
    step = rng.choice([16, 64, 128])
    k = -(-_log(rng, 64, 4096) // step) * step
    n = -(-_log(rng, 64, 4096) // step) * step
    experts = _log(rng, 1, max(1, min(128, (1 << 28) // (k * n))))
    rows = _log(rng, 1, max(1, min(32768, (1 << 37) // (k * n))))
    return dict(op=op, mode=mode, rows=rows, experts=experts, k=k, n=n,
                silu=rng.random() < 0.5, padding=padding)


def work(case):
    c = case
    if c["op"] == "norm":
        e, n = _size(c["dtype"]), c["rows"] * c["width"]
        out = 1 if c["mode"] == "e4m3" else e
        b = n * (e * (3 if c["residual"] else 1) + out)        # x, residual, their sum; y
        if c["mode"] == "train":
            b += n * e * 4                                     # dy, dsum, sum; dx
        return {"bytes": b, "flops": n * (16 if c["mode"] == "train" else 6)}
    if c["op"] in ("route", "combine"):
        rows = (1 - c["padding"]) * c["tokens"]
        pairs, e, w = rows * c["choices"], _size(c["dtype"]), c["width"]
        if c["op"] == "route":
            return {"bytes": rows * w * e + pairs * (w * e + 20), "flops": 0}
        b = (pairs + 2 * c["tokens"]) * w * e + pairs * 8      # rows, residual; out
        if c["mode"] == "train":
            b += (2 * pairs + rows) * w * e + pairs * 12       # rows, dout; their gradients
        return {"bytes": b, "flops": pairs * w * (5 if c["mode"] == "train" else 2)}
    s = (1 - c["padding"]) * c["rows"]
    hit = c["experts"] * (1 - math.exp(-s / c["experts"]))     # experts that any row reaches
    if c["mode"] == "bwd":
        b = 2 * (s * (2 * c["k"] + c["n"]) + (hit + c["experts"]) * c["k"] * c["n"])
        return {"bytes": b + (2 * s * c["k"] if c["silu"] else 0), "flops": 4 * s * c["k"] * c["n"]}
    e = 1 if c["mode"] == "e4m3" else 2
    return {"bytes": e * (s * c["k"] + hit * c["k"] * c["n"]) + 2 * s * c["n"],
            "flops": 2 * s * c["k"] * c["n"]}


def _size(dtype):
    return {"bf16": 2, "f32": 4, "e4m3": 1}[dtype]


# ------------------------------------------------------------------ inputs

def _choose(g, tokens, choices, experts, padding):
    """[tokens, choices] distinct experts, some of them more popular, -1 for padding tokens,
    and the weights of the choices."""
    dev = torch.device("cuda")
    score = torch.randn(tokens, experts, generator=g, device=dev)
    score += 0.7 * torch.randn(experts, generator=g, device=dev)
    top, ids = score.topk(choices, dim=1)
    pad = torch.rand(tokens, generator=g, device=dev) < padding
    ids = torch.where(pad[:, None], -1, ids)
    return ids.to(torch.int32).contiguous(), torch.softmax(top, dim=1).contiguous()


def _places(ids, experts):
    """Sorted place of each pair (-1: none) and the experts' offsets."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat >= 0, flat, experts)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    slots = torch.where(flat >= 0, place, -1).to(torch.int32).reshape(ids.shape)
    return slots.contiguous(), order


def _quantised(x, dim):
    """e4m3 values and fp32 scales of x, one scale for each slice along `dim`."""
    scale = x.abs().amax(dim=dim, keepdim=True).clamp_min(1e-20) / 448.0
    return (x / scale).clamp(-448, 448).to(_F8), scale.squeeze(dim).contiguous()


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=c)
    if c["op"] == "norm":
        n, w, dt = c["rows"], c["width"], _DT[c["dtype"]]
        s["x"] = randn(n, w).to(dt)
        # a residual stream: rows of different size, a few columns larger than the others
        s["res"] = (randn(n, w) * (0.5 + 3 * torch.rand(n, 1, generator=g, device=dev)) *
                    (1 + 4 * (torch.rand(w, generator=g, device=dev) < 0.02))
                    ).to(dt) if c["residual"] else None
        s["weight"] = 1 + 0.2 * randn(w)
        if c["mode"] == "train":
            s["dy"], s["dsum"] = randn(n, w).to(dt), randn(n, w).to(dt)
        return s
    if c["op"] == "route":
        t, k, w, e = c["tokens"], c["choices"], c["width"], c["experts"]
        s["ids"], _ = _choose(g, t, k, e, c["padding"])
        x = randn(t, w)
        s["scales"], s["scales_out"] = None, None
        if c["dtype"] == "e4m3":
            s["x"], sc = _quantised(x, 1)
            s["scales"] = sc.reshape(t, 1)
            s["scales_out"] = torch.zeros(t * k, 1, device=dev)
        else:
            s["x"] = x.to(_DT[c["dtype"]])
        # buffers that a serving loop or a training step keeps
        s["xs"] = torch.zeros(t * k, w, dtype=s["x"].dtype, device=dev)
        s["slots"] = torch.zeros(t, k, dtype=torch.int32, device=dev)
        s["offsets"] = torch.zeros(e + 1, dtype=torch.int64, device=dev)
        s["rows"] = torch.zeros(t * k, dtype=torch.int64, device=dev)
        return s
    if c["op"] == "combine":
        t, k, w, dt = c["tokens"], c["choices"], c["width"], _DT[c["dtype"]]
        ids, s["weights"] = _choose(g, t, k, c["experts"], c["padding"])
        s["slots"], _ = _places(ids, c["experts"])
        s["y"] = randn(t * k, w).to(dt)
        s["res"] = randn(t, w).to(dt)
        if c["mode"] == "train":
            s["dout"] = randn(t, w).to(dt)
            s["dy"] = torch.zeros(t * k, w, dtype=dt, device=dev)
            s["dweights"] = torch.zeros(t, k, device=dev)
        return s
    n_rows, e, k, n = c["rows"], c["experts"], c["k"], c["n"]
    live = max(1, int(round(n_rows * (1 - c["padding"]))))
    share = torch.softmax(0.7 * randn(e), 0)
    which = torch.multinomial(share, live, replacement=True, generator=g)
    count = torch.bincount(which, minlength=e)
    s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)])
    s["cap"] = int(count.max())      # what a padded program sizes its buffer by
    w = randn(e, k, n) / math.sqrt(k)
    if c["mode"] == "e4m3":
        s["x"], s["xs"] = _quantised(randn(n_rows, k), 1)
        q, s["ws"] = _quantised(w, 1)
        s["w"] = q.view(torch.uint8).transpose(1, 2).contiguous().view(_F8)      # [e, n, k]
        s["out"] = torch.zeros(n_rows, n, dtype=torch.bfloat16, device=dev)
    else:
        s["w"] = w.to(torch.bfloat16)
        if c["mode"] == "bf16":
            s["x"] = randn(n_rows, k).to(torch.bfloat16)
            s["out"] = torch.zeros(n_rows, n, dtype=torch.bfloat16, device=dev)
        else:
            pre = randn(n_rows, k).to(torch.bfloat16)
            s["pre"] = pre if c["silu"] else None
            s["x"] = (_silu(pre.float()) if c["silu"] else pre.float()).to(torch.bfloat16)
            s["dout"] = randn(n_rows, n).to(torch.bfloat16)
            s["dx"] = torch.zeros(n_rows, k, dtype=torch.bfloat16, device=dev)
            s["dw"] = torch.zeros(e, k, n, dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if own:
        return _OWN[c["op"]](s, c)
    return _PLAIN[c["op"]](s, c)


def _own_norm(s, c):
    from jagged_hstu_attention_02_b200 import ops
    r = ops.rms_norm_rows(s["x"], s["weight"], s["res"], eps=_EPS, e4m3=c["mode"] == "e4m3",
                          group=c["group"], training=c["mode"] == "train")
    if c["mode"] != "train":
        return dict(y=r.y, scales=r.scales, sum=r.sum if c["residual"] else None)
    dx, dw = ops.rms_norm_rows_bwd(s["dy"], r.sum, r.rstd, s["weight"], dsum=s["dsum"])
    return dict(y=r.y, sum=r.sum if c["residual"] else None, rstd=r.rstd, dx=dx, dw=dw)


def _own_route(s, c):
    from jagged_hstu_attention_02_b200 import ops
    r = ops.expert_sort(s["ids"], c["experts"],
                        out=ops.Routing(s["slots"], s["offsets"], s["rows"]))
    ops.expert_dispatch(s["x"], r.slots, scales=s["scales"], out=s["xs"],
                        scales_out=s["scales_out"])
    return dict(slots=r.slots, offsets=r.offsets, rows=r.rows, xs=s["xs"], scales=s["scales_out"])


def _own_combine(s, c):
    from jagged_hstu_attention_02_b200 import ops
    out = ops.expert_combine(s["y"], s["slots"], s["weights"], residual=s["res"])
    if c["mode"] == "fwd":
        return dict(out=out)
    dy, dw = ops.expert_combine_bwd(s["dout"], s["y"], s["slots"], s["weights"],
                                    grads=(s["dy"], s["dweights"]))
    return dict(out=out, dy=dy, dweights=dw)


def _own_proj(s, c):
    from jagged_hstu_attention_02_b200 import ops
    if c["mode"] == "bwd":
        return ops.expert_proj_bwd(s["dout"], s["x"], s["w"], s["offsets"], silu_pre=s["pre"],
                                   grads=(s["dx"], s["dw"]))
    if c["mode"] == "e4m3":
        return ops.expert_proj_e4m3(s["x"], s["xs"], s["w"], s["ws"], s["offsets"],
                                    silu=c["silu"], out=s["out"])
    return ops.expert_proj(s["x"], s["w"], s["offsets"], silu=c["silu"], out=s["out"])


_OWN = dict(norm=_own_norm, route=_own_route, combine=_own_combine, proj=_own_proj)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _silu_slope(x):
    p = 1 / (1 + torch.exp(-x))
    return p * (1 + x * (1 - p))


def _plain_norm(s, c):
    dt = s["x"].dtype
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    total = h.to(dt)
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + _EPS)
    y = h * rstd * s["weight"]
    kept = total if c["residual"] else None
    if c["mode"] == "same":
        return dict(y=y.to(dt), scales=None, sum=kept)
    if c["mode"] == "e4m3":
        rows, width = y.shape
        group = c["group"] or width
        groups = -(-width // group)
        wide = torch.cat([y, y.new_zeros(rows, groups * group - width)], 1)
        wide = wide.reshape(rows, groups, group)
        scale = wide.abs().amax(2) / 448.0
        back = torch.where(scale > 0, 1 / scale, torch.zeros_like(scale))
        q = (wide * back[..., None]).clamp(-448, 448).reshape(rows, groups * group)
        return dict(y=q[:, :width].to(_F8).contiguous(), scales=scale, sum=kept)
    g = s["dy"].float()
    xhat = total.float() * rstd
    gw = g * s["weight"]
    dx = rstd * (gw - xhat * (gw * xhat).mean(1, keepdim=True)) + s["dsum"].float()
    return dict(y=y.to(dt), sum=kept, rstd=rstd.squeeze(1), dx=dx.to(dt), dw=(g * xhat).sum(0))


def _plain_route(s, c):
    t, k, e = c["tokens"], c["choices"], c["experts"]
    slots, order = _places(s["ids"], e)
    flat = s["ids"].reshape(-1)
    count = (flat[None, :] == torch.arange(e, device=flat.device)[:, None]).sum(1)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    live = torch.arange(t * k, device=flat.device) < offsets[-1]
    rows = torch.where(live, torch.div(order, k, rounding_mode="floor"), 0)
    x = s["x"].view(torch.uint8) if s["x"].dtype == _F8 else s["x"]
    xs = torch.where(live[:, None], x[rows], torch.zeros_like(x[:1]))
    xs = xs.view(_F8) if s["x"].dtype == _F8 else xs
    scales = None if s["scales"] is None else torch.where(live[:, None], s["scales"][rows], 0.0)
    return dict(slots=slots, offsets=offsets, rows=rows, xs=xs, scales=scales)


def _plain_combine(s, c):
    dt = s["y"].dtype
    at, live = s["slots"].long().clamp_min(0), (s["slots"] >= 0)
    rows = s["y"].float()[at]                                  # [t, k, w]
    weight = torch.where(live, s["weights"], torch.zeros_like(s["weights"]))
    out = ((weight[..., None] * rows).sum(1) + s["res"].float()).to(dt)
    if c["mode"] == "fwd":
        return dict(out=out)
    g = s["dout"].float()
    dweights = torch.where(live, (g[:, None, :] * rows).sum(2), torch.zeros_like(weight))
    dy = torch.zeros(s["y"].shape[0] + 1, s["y"].shape[1], device=g.device)
    dy[torch.where(live, at, dy.shape[0] - 1)] = weight[..., None] * g[:, None, :]
    return dict(out=out, dy=dy[:-1].to(dt), dweights=dweights)


def _padded(offsets, cap, rows, experts):
    """Row of the [experts * cap] padded buffer that each sorted row takes; the row behind the
    buffer for rows behind the last expert."""
    at = torch.arange(rows, device=offsets.device)
    e = (at[:, None] >= offsets[None, 1:]).sum(1)
    inside = torch.cat([offsets[:-1], offsets[-1:]])[e]
    return torch.where(e < experts, e * cap + at - inside, experts * cap)


def _pad(x, index, experts, cap):
    wide = torch.zeros(experts * cap + 1, x.shape[1], device=x.device)
    wide[index] = x.float()
    return wide[:-1].reshape(experts, cap, x.shape[1])


def _unpad(y, index):
    return torch.cat([y.reshape(-1, y.shape[2]), y.new_zeros(1, y.shape[2])])[index]


def _plain_proj(s, c):
    e, cap = c["experts"], s["cap"]
    index = _padded(s["offsets"], cap, c["rows"], e)
    x = _pad(s["x"], index, e, cap)
    if c["mode"] == "bwd":
        g = _pad(s["dout"], index, e, cap)
        dx = _unpad(torch.bmm(g, s["w"].float().transpose(1, 2)), index)
        if s["pre"] is not None:
            dx = dx * _silu_slope(s["pre"].float())
        dw = torch.bmm(x.transpose(1, 2), g)
        return dx.to(torch.bfloat16), dw.to(torch.bfloat16)
    if c["mode"] == "e4m3":
        out = torch.bmm(x, s["w"].float().transpose(1, 2)) * s["ws"][:, None, :]
        out = _unpad(out, index) * s["xs"][:, None]
    else:
        out = _unpad(torch.bmm(x, s["w"].float()), index)
    return (_silu(out) if c["silu"] else out).to(torch.bfloat16)


_PLAIN = dict(norm=_plain_norm, route=_plain_route, combine=_plain_combine, proj=_plain_proj)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _sigmoid(x):
    return torch.sigmoid(x)


def _exact_norm(s, c):
    x = s["x"].double()
    h = x if s["res"] is None else x + s["res"].double()
    norm2 = torch.linalg.vector_norm(h, dim=1) ** 2
    rstd = (norm2 / h.shape[1] + _EPS).rsqrt()
    y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].double())
    total = h if c["residual"] else None
    if c["mode"] == "same":
        return dict(y=y, scales=None, sum=total)
    if c["mode"] == "e4m3":
        scales = torch.stack([p.abs().max(1).values for p in
                              torch.split(y, c["group"] or y.shape[1], dim=1)], 1) / 448
        of = torch.arange(y.shape[1], device=y.device) // (c["group"] or y.shape[1])
        return dict(y=_e4m3(y / scales[:, of]), scales=scales, sum=total)
    stored = h.to(s["x"].dtype).double()      # the gradients are those at the stored sum
    g = s["dy"].double() * s["weight"].double()
    dot = torch.einsum("rc,rc->r", g, stored)
    dx = g * rstd[:, None] - stored * (rstd ** 3 * dot / h.shape[1])[:, None]
    dw = torch.einsum("rc,rc,r->c", s["dy"].double(), stored, rstd)
    return dict(y=y, sum=total, rstd=rstd, dx=dx + s["dsum"].double(), dw=dw)


def _e4m3(v):
    """The e4m3 value nearest to each of v (ties to the even), as a double: 4 significant bits,
    steps of 2^-9 below 2^-6, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_route(s, c):
    k, e = c["choices"], c["experts"]
    ids = s["ids"].reshape(-1).cpu().numpy()
    lists = [[] for _ in range(e)]
    for p, i in enumerate(ids.tolist()):
        if i >= 0:
            lists[i].append(p)
    pairs = torch.tensor([p for one in lists for p in one], dtype=torch.int64)
    ends = torch.tensor([0] + [len(one) for one in lists], dtype=torch.int64).cumsum(0)
    slots = torch.full((ids.size,), -1, dtype=torch.int32)
    slots[pairs] = torch.arange(pairs.numel(), dtype=torch.int32)
    rows = torch.zeros(ids.size, dtype=torch.int64)
    rows[:pairs.numel()] = pairs // k
    xs = torch.zeros(ids.size, s["x"].shape[1], dtype=torch.float64)
    xs[:pairs.numel()] = s["x"].double().cpu()[pairs // k]
    scales = None
    if s["scales"] is not None:
        scales = torch.zeros(ids.size, 1, dtype=torch.float64)
        scales[:pairs.numel()] = s["scales"].double().cpu()[pairs // k]
    return dict(slots=slots.reshape(-1, k), offsets=ends, rows=rows, xs=xs, scales=scales)


def _exact_combine(s, c):
    y, res = s["y"].double(), s["res"].double()
    out = res.clone()
    train = c["mode"] == "train"
    dy = torch.zeros_like(y) if train else None
    dweights = torch.zeros_like(s["weights"], dtype=torch.float64) if train else None
    for j in range(c["choices"]):
        t = torch.nonzero(s["slots"][:, j] >= 0).squeeze(1)
        at, w = s["slots"][t, j].long(), s["weights"][t, j].double()
        out[t] += w[:, None] * y[at]
        if train:
            g = s["dout"][t].double()
            dy[at] = w[:, None] * g
            dweights[t, j] = torch.einsum("rc,rc->r", g, y[at])
    return dict(out=out, dy=dy, dweights=dweights) if train else dict(out=out)


def _exact_proj(s, c):
    ends = s["offsets"].tolist()
    x, dev = s["x"].double(), s["x"].device
    if c["mode"] == "bwd":
        g = s["dout"].double()
        dx = torch.zeros(c["rows"], c["k"], dtype=torch.float64, device=dev)
        dw = torch.zeros(c["experts"], c["k"], c["n"], dtype=torch.float64, device=dev)
        for i, (a, b) in enumerate(zip(ends, ends[1:])):
            dx[a:b] = g[a:b] @ s["w"][i].double().T
            dw[i] = x[a:b].T @ g[a:b]
        if s["pre"] is not None:
            p = s["pre"].double()
            dx *= _sigmoid(p) + p * _sigmoid(p) * _sigmoid(-p)
        return dx, dw
    out = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device=dev)
    for i, (a, b) in enumerate(zip(ends, ends[1:])):
        if c["mode"] == "e4m3":
            w = s["w"][i].double() * s["ws"][i].double()[:, None]
            out[a:b] = (x[a:b] * s["xs"][a:b].double()[:, None]) @ w.T
        else:
            out[a:b] = x[a:b] @ s["w"][i].double()
    return out * _sigmoid(out) if c["silu"] else out


_EXACT = dict(norm=_exact_norm, route=_exact_route, combine=_exact_combine, proj=_exact_proj)
