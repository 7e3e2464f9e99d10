"""The norm, the gated recurrence and the sorting of tokens by expert as measured cases.

What a sequence model has between its embedding and its logits beside the
convolution and the selective scan: the norm of its residual stream, a linear
recurrence with one gate per channel, and the way of tokens to their experts and
back.  `run` computes a case in plain torch operations, in 32 bits, or, where
`own` is true, through the library's public calls; `exact` gives the same
outputs from the definitions in 64 bits.

The definitions (t counts tokens, e channels, j choices of a token):

  norm      s[t] = x[t] + residual[t], rounded to the tensors' type, where there
            is a residual stream, else x[t];
            y[t,e] = (s[t,e] - m[t]) * r[t] * weight[e] + bias[e], m the mean of
            s[t] and r = 1 / sqrt(mean of (s[t] - m[t])^2 + eps); rms: m = 0
  gated     f[t,e] = sigmoid(gate[t,e]);  h[t,e] = f[t,e] * h[t-1,e] + (1 - f[t,e]) * x[t,e]
            activation "none": f = gate, and x enters as it is; the first term is
            dropped where a segment starts at t
  experts   the entries (t, j) in the order of their experts, entries of one
            expert in their own order, those of no expert (outside [0, experts))
            behind all others; a row of x for each of them, zeros for no expert;
            out[t] = sum over j of weights[t,j] * (the row of y that belongs to (t, j)),
            without the entries of no expert
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # the rows of one decoding step of 16 sequences, added to their stream: pure latency
        {"name": "norm_token", "op": "norm", "batch": 16, "length": 1, "channels": 4096, "dtype": "bf16", "rms": True,
         "bias": False, "residual": True, "grad": False},
        # one norm of a training step, forward and backward, within the residual stream
        {"name": "norm_train", "op": "norm", "batch": 4, "length": 4096, "channels": 4096, "dtype": "bf16",
         "rms": False, "bias": True, "residual": True, "grad": True},
        # odd sizes in 32 bits
        {"name": "norm_train_ragged", "op": "norm", "batch": 3, "length": 1001, "channels": 2047, "dtype": "f32",
         "rms": False, "bias": True, "residual": False, "grad": True},
        # a norm of each head of a layer: many short rows
        {"name": "norm_heads", "op": "norm", "batch": 64, "length": 4096, "channels": 128, "dtype": "f16", "rms": True,
         "bias": False, "residual": False, "grad": True},
        # one decoding step of one sequence, then that of a full serving batch
        {"name": "gated_token", "op": "gated_step", "batch": 1, "channels": 2048, "dtype": "bf16",
         "activation": "sigmoid", "idle": 0.0},
        {"name": "gated_token_batch", "op": "gated_step", "batch": 256, "channels": 4096, "dtype": "bf16",
         "activation": "sigmoid", "idle": 0.1},
        # one user's prompt: few channels for the machine, a long axis
        {"name": "gated_prompt", "op": "gated", "batch": 1, "length": 8192, "channels": 2048, "dtype": "bf16",
         "activation": "sigmoid", "grad": False, "packed": False},
        # a training step, forward and backward
        {"name": "gated_train", "op": "gated", "batch": 8, "length": 4096, "channels": 4096, "dtype": "bf16",
         "activation": "sigmoid", "grad": True, "packed": False},
        # packed documents that continue earlier context, odd sizes, decays given as they are, 32 bits
        {"name": "gated_train_packed", "op": "gated", "batch": 2, "length": 1000, "channels": 2047, "dtype": "f32",
         "activation": "none", "grad": True, "packed": True},
        # one decoding step of 64 sequences with 8 of 128 experts each
        {"name": "experts_token", "op": "experts", "tokens": 64, "choices": 8, "experts": 128, "dim": 2048,
         "dtype": "bf16", "ids": "int64", "dropped": 0.0, "grad": False},
        # a training step's tokens with 2 of 64 experts each, forward and backward
        {"name": "experts_train", "op": "experts", "tokens": 16384, "choices": 2, "experts": 64, "dim": 4096,
         "dtype": "bf16", "ids": "int64", "dropped": 0.0, "grad": True},
        # odd sizes in 32 bits, a tenth of the entries over their expert's capacity and so without one
        {"name": "experts_train_ragged", "op": "experts", "tokens": 5003, "choices": 3, "experts": 37, "dim": 1000,
         "dtype": "f32", "ids": "int32", "dropped": 0.1, "grad": True},
    ]


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 10


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A number of channels: more often than not a multiple of 64, else any."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.6 else n


def draw(rng):
    """A case of the ranges above: every operator, sizes log-uniform, odd ones among them."""
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "norm", "gated", "gated", "gated_step", "experts", "experts"])
        case = {"op": op}
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op == "norm":
            case |= {"batch": _log(rng, 1, 64), "length": _log(rng, 1, 8192), "channels": _width(rng, 32, 8192),
                     "dtype": dtype, "rms": rng.random() < 0.5, "bias": rng.random() < 0.5,
                     "residual": rng.random() < 0.5, "grad": rng.random() < 0.7}
        elif op == "gated_step":
            case |= {"batch": _log(rng, 1, 512), "channels": _width(rng, 64, 8192), "dtype": dtype,
                     "activation": rng.choice(["sigmoid", "sigmoid", "none"]), "idle": rng.choice([0.0, 0.1])}
        elif op == "gated":
            case |= {"batch": _log(rng, 1, 16), "length": _log(rng, 1, 16384), "channels": _width(rng, 64, 8192),
                     "dtype": dtype, "activation": rng.choice(["sigmoid", "sigmoid", "none"]),
                     "grad": rng.random() < 0.6, "packed": rng.random() < 0.3}
        else:
            experts = _log(rng, 2, 512)
            case |= {"tokens": _log(rng, 1, 32768), "choices": rng.randint(1, min(8, experts)), "experts": experts,
                     "dim": _width(rng, 64, 8192), "dtype": dtype, "ids": rng.choice(["int32", "int64"]),
                     "dropped": rng.choice([0.0, 0.0, 0.1]), "grad": rng.random() < 0.7}
        if _cost(case) <= most:
            return case


def work(case):
    """Each input read once, each output written once; products, sums and exponentials as one operation each."""
    b = BYTES[case["dtype"]]
    if case["op"] == "norm":
        rows, ch = case["batch"] * case["length"], case["channels"]
        parameters = ch * b * (2 if case["bias"] else 1)
        tensors = 4 if case["residual"] else 2  # x, (residual, sum), y
        flops = rows * ch * 8
        if case["grad"]:
            tensors += 4 if case["residual"] else 2  # dy, (dsum), dx, and s where it is the sum
            tensors += 0 if case["residual"] else 1
            parameters += ch * (b + (8 if case["bias"] else 4))
            flops += rows * ch * 14
        return {"bytes": tensors * rows * ch * b + parameters, "flops": flops}
    if case["op"] == "experts":
        rows = case["tokens"] * case["dim"] * b
        n = case["tokens"] * case["choices"]
        entries = n * case["dim"] * b
        small = n * ((4 if case["ids"] == "int32" else 8) + 4 + 4 + 4) + 8 * (case["experts"] + 1)
        if not case["grad"]:
            return {"bytes": 2 * rows + 2 * entries + small, "flops": 2 * n * case["dim"]}
        # backward: the gathered rows' gradient in, dx out; dout and y in, dy out; the weights' gradient out
        return {"bytes": 4 * rows + 5 * entries + small + 8 * n, "flops": 6 * n * case["dim"]}
    bt, ch = case["batch"], case["channels"]
    if case["op"] == "gated_step":
        return {"bytes": bt * ch * (3 * b + 8), "flops": bt * ch * 8}
    el, state = bt * case["length"] * ch, bt * ch * 4
    heads = bt * case["length"] if case["packed"] else 0
    if not case["grad"]:
        return {"bytes": 3 * el * b + 2 * state + heads, "flops": el * 8}
    # backward: x, gate and dy in, dx and dgate out
    return {"bytes": 8 * el * b + 2 * state + 2 * heads, "flops": el * 24}


# ------------------------------------------------------------------ inputs
def _heads(case, gen, batch, length):
    """Where documents start: about every 300 tokens, never at the first token (the rows continue a context)."""
    if not case["packed"]:
        return None
    heads = torch.rand(batch, length, generator=gen, device="cuda") < 1 / 300
    heads[:, 0] = False
    return heads


def _gate(case, normal, gen, tokens, ch):
    """Gates of channels that remember 2 to 1000 tokens; activation "none": the decays themselves."""
    span = 2 * torch.exp(torch.rand(ch, generator=gen, device="cuda") * math.log(500))
    v = torch.log(span - 1) + normal(*tokens, ch, dtype=torch.float32)
    return torch.sigmoid(v) if case["activation"] == "none" else v


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dtype, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        shape, ch = (case["batch"], case["length"], case["channels"]), case["channels"]
        s["x"] = normal(*shape) + normal(ch, scale=0.5)  # channels of a stream differ in their means
        s["residual"] = normal(*shape, scale=2.0) if case["residual"] else None
        s["weight"] = (1 + normal(ch, dtype=torch.float32, scale=0.1)).to(dtype)
        s["bias"] = normal(ch, scale=0.1) if case["bias"] else None
        if case["grad"]:
            s["dy"] = normal(*shape, scale=0.01)
            s["dsum"] = normal(*shape, scale=0.01) if case["residual"] else None
        return s
    if case["op"] == "experts":
        tokens, choices, experts, dim = case["tokens"], case["choices"], case["experts"], case["dim"]
        # experts differ in popularity, a token's choices are distinct
        score = torch.rand(tokens, experts, generator=gen, device="cuda").log_().neg_().log_().neg_()
        score += torch.randn(experts, generator=gen, device="cuda") * 0.7
        ids = score.topk(choices, dim=1).indices
        out = torch.rand(tokens, choices, generator=gen, device="cuda") < case["dropped"]
        s["ids"] = torch.where(out, -1, ids).to(torch.int32 if case["ids"] == "int32" else torch.int64)
        share = torch.rand(tokens, choices, generator=gen, device="cuda") + 0.1
        s["weights"] = share / share.sum(1, keepdim=True)
        s["x"] = normal(tokens, dim)
        s["y"] = normal(tokens * choices, dim)  # what the experts made of their rows
        if case["grad"]:
            s["dout"] = normal(tokens, dim, scale=0.01)
            s["drows"] = normal(tokens * choices, dim, scale=0.01)
        return s
    batch, ch = case["batch"], case["channels"]
    tokens = (batch,) if case["op"] == "gated_step" else (batch, case["length"])
    # x and the gate are the halves of one projection's output, as a model has them
    both = torch.cat([normal(*tokens, ch), _gate(case, normal, gen, tokens, ch).to(dtype)], -1)
    s["x"], s["gate"] = both[..., :ch], both[..., ch:]
    if case["op"] == "gated_step":
        pool = batch + max(4, batch // 8)
        slots = torch.randperm(pool, generator=gen, device="cuda")[:batch].to(torch.int32)
        idle = torch.rand(batch, generator=gen, device="cuda") < case["idle"]
        s["slots"] = torch.where(idle, torch.full_like(slots, -1), slots)
        s["pool"] = normal(pool + 1, ch, dtype=torch.float32)  # the last row takes the idle rows' writes of the plain form
        return s
    s["heads"] = _heads(case, gen, batch, case["length"])
    s["state"] = normal(batch, ch, dtype=torch.float32) if case["packed"] or not case["grad"] else None
    if case["grad"]:
        s["dy"] = normal(batch, case["length"], ch, scale=0.01)
    return s


# --------------------------------------------------------- the library's calls
def _run_own(s):
    import stream_compaction_gb300 as sc

    case = s["case"]
    if case["op"] == "norm":
        args = {"weight": s["weight"], "bias": s["bias"], "rms": case["rms"]}
        saved = sc.layer_norm_saved(s["x"]) if case["grad"] else None
        y = sc.layer_norm(s["x"], **args, eps=EPS, residual=s["residual"], saved=saved)
        out, stream = {}, s["x"]
        if case["residual"]:
            y, stream = y
            out["sum"] = stream
        out["y"] = y
        if case["grad"]:
            out["grads"] = sc.layer_norm_grad(s["dy"], stream, **args, saved=saved, dsum=s["dsum"])
        return out
    if case["op"] == "experts":
        order = sc.expert_sort(s["ids"], case["experts"])
        out = {"offsets": order.offsets, "order": order.order, "place": order.place,
               "rows": sc.expert_gather(s["x"], order), "out": sc.expert_combine(s["y"], order, s["weights"])}
        if case["grad"]:
            out["dx"] = sc.expert_gather_grad(s["drows"], order)
            out["grads"] = sc.expert_combine_grad(s["dout"], s["y"], order, s["weights"])
        return out
    activation = None if case["activation"] == "none" else case["activation"]
    if case["op"] == "gated_step":
        state = s["pool"][:-1]
        y = sc.gated_scan_step(s["x"], s["gate"], state, activation=activation, slots=s["slots"])
        return {"y": y, "state": state}
    more = {"activation": activation, "heads": s["heads"], "state": s["state"]}
    if not case["grad"]:
        final = torch.empty_like(s["state"])
        y = sc.gated_scan(s["x"], s["gate"], **more, final_state=final)
        return {"y": y, "state": final}
    saved = sc.gated_scan_saved(s["x"])
    y = sc.gated_scan(s["x"], s["gate"], **more, saved=saved)
    grads = sc.gated_scan_grad(s["dy"], s["x"], s["gate"], **more, saved=saved)
    return {"y": y, "grads": grads}


# ------------------------------------------------------------- the plain form
def _plain_norm(s):
    case, dtype = s["case"], s["x"].dtype
    out = {}
    v = s["x"].float()
    if case["residual"]:
        out["sum"] = (v + s["residual"].float()).to(dtype)
        v = out["sum"].float()
    w = s["weight"].float()
    c = v if case["rms"] else v - v.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)
    n = c * r
    y = n * w
    if case["bias"]:
        y = y + s["bias"].float()
    out["y"] = y.to(dtype)
    if not case["grad"]:
        return out
    dy = s["dy"].float()
    dn = dy * w
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if not case["rms"]:
        dx = dx - dn.mean(-1, keepdim=True)
    dx = dx * r
    if case["residual"]:
        dx = dx + s["dsum"].float()
    out["grads"] = {"x": dx.to(dtype), "weight": (dy * n).sum((0, 1))}
    if case["bias"]:
        out["grads"]["bias"] = dy.sum((0, 1))
    return out


def _plain_experts(s):
    case, dtype = s["case"], s["x"].dtype
    tokens, choices, experts = case["tokens"], case["choices"], case["experts"]
    ids = s["ids"].long().flatten()
    key = torch.where((ids >= 0) & (ids < experts), ids, experts)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device=order.device)
    before = key[None, :] < torch.arange(experts + 1, device=key.device)[:, None]
    offsets = before.sum(1)
    live = (key < experts).view(tokens, choices, 1)
    sorted_live = (key[order] < experts)[:, None]
    place2 = place.view(tokens, choices)
    weights = s["weights"].float()
    rows = torch.where(sorted_live, s["x"][order // choices], 0)
    mine = torch.where(live, s["y"][place2].float(), 0.0)
    out = {"offsets": offsets, "order": order.int(), "place": place2.int(), "rows": rows,
           "out": (mine * weights[..., None]).sum(1).to(dtype)}
    if case["grad"]:
        out["dx"] = torch.where(live, s["drows"][place2].float(), 0.0).sum(1).to(dtype)
        dout = s["dout"].float()
        dy = dout[order // choices] * weights.flatten()[order][:, None]
        out["grads"] = {"y": torch.where(sorted_live, dy, 0.0).to(dtype), "weights": (mine * dout[:, None]).sum(-1)}
    return out


def _plain_gates(s):
    """f, and what x is multiplied with."""
    g = s["gate"].float()
    if s["case"]["activation"] == "none":
        return g, torch.ones_like(g)
    return torch.sigmoid(g), torch.sigmoid(-g)


def _plain_gated_step(s):
    pool = s["pool"]
    ok = s["slots"] >= 0
    rows = torch.where(ok, s["slots"].long(), pool.shape[0] - 1)
    f, enters = _plain_gates(s)
    h = f * pool[rows] + enters * s["x"].float()
    pool.index_copy_(0, rows, h)
    return {"y": torch.where(ok[:, None], h, 0.0).to(s["x"].dtype), "state": pool[:-1]}


def _recurrence(a, b):
    """h[t] = a[t] * h[t-1] + b[t] along dimension 1, by doubling; overwrites both."""
    reach = 1
    while reach < b.shape[1]:
        b[:, reach:] = b[:, reach:] + a[:, reach:] * b[:, :-reach]
        a[:, reach:] = a[:, reach:] * a[:, :-reach]
        reach *= 2
    return b


def _plain_gated(s):
    case, dtype = s["case"], s["x"].dtype
    x = s["x"].float()
    f, enters = _plain_gates(s)
    kept = f if s["heads"] is None else torch.where(s["heads"][:, :, None], 0.0, f)
    h = enters * x
    if s["state"] is not None:
        h[:, 0] += kept[:, 0] * s["state"]
    h = _recurrence(kept.clone(), h)
    y = h.to(dtype)
    if not case["grad"]:
        return {"y": y, "state": h[:, -1].contiguous()}
    # the gradient of h runs back in time: dh[t] = kept[t+1] * dh[t+1] + dy[t]
    later = torch.cat([torch.zeros_like(f[:, :1]), kept[:, 1:].flip(1)], 1)
    dh = _recurrence(later, s["dy"].float().flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    if s["heads"] is not None:
        before = torch.where(s["heads"][:, :, None], 0.0, before)
    df = dh * before if case["activation"] == "none" else dh * (before - x) * f * enters
    grads = {"x": (dh * enters).to(dtype), "gate": df.to(dtype)}
    if s["state"] is not None:
        grads["state"] = dh[:, 0] * kept[:, 0]
    return {"y": y, "grads": grads}


def run(state):
    if own:
        return _run_own(state)
    plain = {"norm": _plain_norm, "gated": _plain_gated, "gated_step": _plain_gated_step, "experts": _plain_experts}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------- the definitions in 64 bits
def _exact_norm(s):
    case, ch = s["case"], s["case"]["channels"]
    flat = {k: v.reshape(-1, ch) for k, v in s.items() if k in ("x", "residual", "dy", "dsum") and v is not None}
    weight = s["weight"].double()
    bias = s["bias"].double() if case["bias"] else torch.zeros_like(weight)
    count = flat["x"].shape[0]
    dweight, dbias = torch.zeros_like(weight), torch.zeros_like(weight)
    parts = {"sum": [], "y": [], "x": []}
    for i in range(0, count, 4096):
        v = flat["x"][i:i + 4096].double()
        if case["residual"]:
            v = v + flat["residual"][i:i + 4096].double()
            parts["sum"].append(v)
            v = v.to(s["x"].dtype).double()  # the stream is what its type holds
        m = torch.zeros_like(v[:, :1]) if case["rms"] else v.sum(1, keepdim=True) / ch
        std = (((v - m) ** 2).sum(1, keepdim=True) / ch + EPS) ** 0.5
        z = (v - m) / std
        parts["y"].append(z * weight + bias)
        if case["grad"]:
            dy = flat["dy"][i:i + 4096].double()
            dweight += (dy * z).sum(0)
            dbias += dy.sum(0)
            dz = dy * weight
            back = dz - z * ((dz * z).sum(1, keepdim=True) / ch)
            if not case["rms"]:
                back = back - dz.sum(1, keepdim=True) / ch
            back = back / std
            parts["x"].append(back + flat["dsum"][i:i + 4096].double() if case["residual"] else back)
    shape = s["x"].shape
    out = {"sum": torch.cat(parts["sum"]).view(shape)} if case["residual"] else {}
    out["y"] = torch.cat(parts["y"]).view(shape)
    if case["grad"]:
        out["grads"] = {"x": torch.cat(parts["x"]).view(shape), "weight": dweight}
        if case["bias"]:
            out["grads"]["bias"] = dbias
    return out


def _exact_experts(s):
    case = s["case"]
    tokens, choices, experts, dim = case["tokens"], case["choices"], case["experts"], case["dim"]
    ids = s["ids"].flatten().tolist()
    bins = [[] for _ in range(experts + 1)]
    for entry, expert in enumerate(ids):
        bins[expert if 0 <= expert < experts else experts].append(entry)
    order = [entry for members in bins for entry in members]
    offsets = [0]
    for members in bins[:experts]:
        offsets.append(offsets[-1] + len(members))
    kept = offsets[-1]
    place = [0] * len(ids)
    for row, entry in enumerate(order):
        place[entry] = row
    as_int = {"dtype": torch.int64, "device": "cuda"}
    place = torch.tensor(place, **as_int)
    entries = torch.tensor(order, **as_int)[:kept]
    rows = torch.zeros(tokens * choices, dim, dtype=torch.float64, device="cuda")
    rows[:kept] = s["x"][entries // choices].double()
    total = torch.zeros(tokens, dim, dtype=torch.float64, device="cuda")
    out = {"offsets": torch.tensor(offsets, **as_int), "order": torch.tensor(order, **as_int).int(),
           "place": place.view(tokens, choices).int(), "rows": rows, "out": total}
    w = s["weights"].double().flatten()
    slots = [torch.arange(j, tokens * choices, choices, device="cuda") for j in range(choices)]
    if case["grad"]:
        dx = torch.zeros_like(total)
        dy = torch.zeros_like(rows)
        dw = torch.zeros(tokens, choices, dtype=torch.float64, device="cuda")
        out |= {"dx": dx, "grads": {"y": dy, "weights": dw}}
    for j, mine in enumerate(slots):  # the j-th choice of every token that has an expert
        at = place[mine]
        live = at < kept
        t, at = torch.nonzero(live).flatten(), at[live]
        y = s["y"][at].double()
        total[t] += w[mine[live], None] * y
        if case["grad"]:
            dx[t] += s["drows"][at].double()
            dout = s["dout"][t].double()
            dw[t, j] = (dout * y).sum(1)
            dy[at] = dout * w[mine[live], None]
    return out


def _exact_gated(s):
    case = s["case"]
    step = case["op"] == "gated_step"
    x, g = s["x"].double(), s["gate"].double()
    if step:
        x, g = x[:, None], g[:, None]
    if case["activation"] == "none":
        f, enters = g, torch.ones_like(g)
    else:
        f, enters = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    batch, length, ch = x.shape
    heads = None if step else s["heads"]
    h = torch.zeros(batch, ch, dtype=torch.float64, device="cuda")
    if step:
        pool, rows = s["pool"][:-1].double(), s["slots"].tolist()
        h = torch.stack([pool[max(r, 0)] for r in rows])
    elif s["state"] is not None:
        h = s["state"].double()
    y, before = torch.empty_like(x), torch.empty_like(x)
    for t in range(length):
        if heads is not None:
            h = h * (~heads[:, t]).double()[:, None]
        before[:, t] = h
        h = f[:, t] * h + enters[:, t] * x[:, t]
        y[:, t] = h
    if step:
        for row, r in enumerate(rows):
            if r >= 0:
                pool[r] = h[row]
            else:
                y[row] = 0
        return {"y": y[:, 0], "state": pool}
    if not case["grad"]:
        return {"y": y, "state": h}
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    carry = torch.zeros_like(h)
    for t in reversed(range(length)):
        dh = s["dy"][:, t].double() + carry
        dx[:, t] = dh * enters[:, t]
        if case["activation"] == "none":
            dg[:, t] = dh * before[:, t]
        else:
            dg[:, t] = dh * (before[:, t] - x[:, t]) * f[:, t] * enters[:, t]
        carry = dh * f[:, t]
        if heads is not None:
            carry = carry * (~heads[:, t]).double()[:, None]
    grads = {"x": dx, "gate": dg}
    if s["state"] is not None:
        grads["state"] = carry
    return {"y": y, "grads": grads}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_experts(s) if case["op"] == "experts" else _exact_gated(s)
