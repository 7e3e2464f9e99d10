"""The sequence-model operators of the library as measured cases.

Token embedding (lookup with scaling, and its gradient by sorted tokens), the
short causal convolution and the selective state space scan (prompts, training
steps, single tokens).  `run` computes a case in plain torch operations, in 32
bits, or, where `own` is true, through the library's public calls; `exact`
gives the same outputs from the definitions in 64 bits, token by token.

The definitions (t counts tokens, e channels, n states; g(e) the group of e):

  embedding    out[t] = scale * weight[ids[t]], a zero row for an id outside
               [0, vocab); dweight[v] = scale * sum of dout[t] over ids[t] = v
  convolution  pre[t,e] = bias[e] + sum_k w[e,k] * x[t-W+1+k, e], over the
               inputs of t's own segment; y = pre * sigmoid(pre)
  scan         d[t,e] = softplus(dt[t,e] + dt_bias[e])
               h[t,e,n] = exp(d[t,e] * A[e,n]) * h[t-1,e,n]
                          + d[t,e] * x[t,e] * B[t,g(e),n],
               the first term dropped where a segment starts at t
               y[t,e] = (sum_n C[t,g(e),n] * h[t,e,n] + D[e] * x[t,e])
                        * z[t,e] * sigmoid(z[t,e])
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # the rows of one decoding step of 16 sequences: pure latency
        {"name": "embed_token", "op": "embed", "tokens": 16, "vocab": 65536, "dim": 4096, "dtype": "bf16",
         "ids": "int64", "grad": False, "outside": 0.0},
        # a training step's tokens, Zipf-distributed, over a large vocabulary:
        # the gradient is a dense matrix of 1 GiB, mostly rows of absent tokens
        {"name": "embed_train", "op": "embed", "tokens": 16384, "vocab": 131072, "dim": 4096, "dtype": "bf16",
         "ids": "int64", "grad": True, "outside": 0.0},
        # odd sizes in 32 bits, a third of the positions padding (ids of -1)
        {"name": "embed_train_ragged", "op": "embed", "tokens": 5003, "vocab": 50021, "dim": 1000, "dtype": "f32",
         "ids": "int32", "grad": True, "outside": 0.33},
        # one decoding step's convolution for 64 sequences in a pool of states
        {"name": "conv_token", "op": "conv_step", "batch": 64, "channels": 4096, "width": 4, "dtype": "bf16",
         "idle": 0.1},
        # a prompt that continues earlier context, several documents packed in a row
        {"name": "conv_prompt_packed", "op": "conv", "batch": 3, "length": 1000, "channels": 2047, "width": 4,
         "dtype": "f32", "grad": False, "packed": True},
        # a training step's convolution, forward and backward
        {"name": "conv_train", "op": "conv", "batch": 8, "length": 4096, "channels": 4096, "width": 4,
         "dtype": "bf16", "grad": True, "packed": False},
        # one token of one sequence: the smallest call of a decoding loop
        {"name": "scan_token", "op": "scan_step", "batch": 1, "channels": 2048, "states": 16, "groups": 1,
         "dtype": "bf16", "idle": 0.0},
        # one decoding step of a full serving batch: bound by its states
        {"name": "scan_token_batch", "op": "scan_step", "batch": 256, "channels": 4096, "states": 16, "groups": 1,
         "dtype": "bf16", "idle": 0.1},
        # one user's prompt: few channels for the machine, a long axis
        {"name": "scan_prompt", "op": "scan", "batch": 1, "length": 4096, "channels": 4096, "states": 16,
         "groups": 1, "dtype": "bf16", "grad": False, "packed": False},
        # the prompts of a batch
        {"name": "scan_prompt_batch", "op": "scan", "batch": 8, "length": 4096, "channels": 4096, "states": 16,
         "groups": 1, "dtype": "f16", "grad": False, "packed": False},
        # a training step, forward and backward
        {"name": "scan_train", "op": "scan", "batch": 4, "length": 4096, "channels": 4096, "states": 16,
         "groups": 1, "dtype": "bf16", "grad": True, "packed": False},
        # packed documents, odd sizes, two groups of B and C, 32 bits
        {"name": "scan_train_packed", "op": "scan", "batch": 2, "length": 1000, "channels": 1002, "states": 24,
         "groups": 2, "dtype": "f32", "grad": True, "packed": True},
    ]


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 10


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the ranges above: every operator, sizes log-uniform, odd ones among them."""
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["embed", "conv", "conv_step", "scan", "scan", "scan_step"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op == "embed":
            case = {"op": op, "tokens": _log(rng, 1, 32768), "vocab": _log(rng, 1000, 131072),
                    "dim": _log(rng, 64, 4096), "dtype": dtype, "ids": rng.choice(["int32", "int64"]),
                    "grad": rng.random() < 0.7, "outside": rng.choice([0.0, 0.0, 0.2])}
        else:
            channels = _log(rng, 64, 4096)
            if rng.random() < 0.6:
                channels = max(64, channels // 64 * 64)
            case = {"op": op, "batch": _log(rng, 1, 256 if op.endswith("step") else 8), "channels": channels,
                    "dtype": dtype}
            if op.endswith("step"):
                case["idle"] = rng.choice([0.0, 0.1])
            else:
                case["length"] = _log(rng, 1, 8192)
                case["grad"] = rng.random() < 0.5
                case["packed"] = rng.random() < 0.3
            if op.startswith("conv"):
                case["width"] = rng.choice([2, 3, 4, 4])
            else:
                case["states"] = rng.choice([8, 16, 16, 16, 24, 32, 64])
                case["groups"] = rng.choice([1, 1, 2]) if channels % 2 == 0 else 1
        if _cost(case) <= most:
            return case


def work(case):
    """Each input read once, each output written once; products, sums and exponentials as one operation each."""
    b = BYTES[case["dtype"]]
    if case["op"] == "embed":
        rows = case["tokens"] * case["dim"] * b
        n = case["tokens"] * (4 if case["ids"] == "int32" else 8)
        if not case["grad"]:
            return {"bytes": n + 2 * rows, "flops": case["tokens"] * case["dim"]}
        return {"bytes": n + 3 * rows + case["vocab"] * case["dim"] * b, "flops": 3 * case["tokens"] * case["dim"]}
    bt, ch = case["batch"], case["channels"]
    if case["op"] == "conv_step":
        w = case["width"]
        return {"bytes": bt * ch * b * (2 + 2 * (w - 1)) + ch * (w + 1) * b, "flops": bt * ch * (2 * w + 4)}
    if case["op"] == "conv":
        w, el = case["width"], bt * case["length"] * ch
        if not case["grad"]:
            return {"bytes": 2 * el * b, "flops": el * (2 * w + 4)}
        return {"bytes": 5 * el * b, "flops": el * (8 * w + 16)}
    n, g = case["states"], case["groups"]
    if case["op"] == "scan_step":
        return {"bytes": bt * ch * (4 * b + 8 * n) + 2 * bt * g * n * b + ch * (4 * n + 8),
                "flops": bt * ch * (7 * n + 12)}
    el, bc = bt * case["length"] * ch, 2 * bt * case["length"] * g * n
    small, state = ch * (4 * n + 8), bt * ch * n * 4
    if not case["grad"]:
        return {"bytes": 4 * el * b + bc * b + small + 2 * state, "flops": el * (7 * n + 12)}
    # backward: x, dt, z, dy in, dx, ddt, dz out; B, C in and dB, dC out
    return {"bytes": (4 + 7) * el * b + 3 * bc * b + 3 * small + state, "flops": el * (24 * n + 40)}


# ------------------------------------------------------------------ inputs
def _heads(case, gen, batch, length):
    """Where documents start: about every 300 tokens, never at the first token (the rows continue a context)."""
    if not case["packed"]:
        return None
    heads = torch.rand(batch, length, generator=gen, device="cuda") < 1 / 300
    heads[:, 0] = False
    return heads


def _slots(case, gen, batch):
    """Rows of a pool of states in no order, -1 for the sequences that sit this step out."""
    pool = batch + max(4, batch // 8)
    slots = torch.randperm(pool, generator=gen, device="cuda")[:batch].to(torch.int32)
    idle = torch.rand(batch, generator=gen, device="cuda") < case["idle"]
    return pool, torch.where(idle, torch.full_like(slots, -1), slots)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dtype, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "embed":
        tokens, vocab, dim = case["tokens"], case["vocab"], case["dim"]
        ids_type = torch.int32 if case["ids"] == "int32" else torch.int64
        rank = torch.exp(torch.rand(tokens, generator=gen, device="cuda") * math.log(vocab + 1)).long() - 1
        ids = torch.randperm(vocab, generator=gen, device="cuda")[rank.clamp(0, vocab - 1)]
        out = torch.rand(tokens, generator=gen, device="cuda") < case["outside"]
        s["ids"] = torch.where(out, torch.full_like(ids, -1), ids).to(ids_type)
        s["weight"] = torch.randn(vocab, dim, generator=gen, device="cuda", dtype=dtype)
        s["scale"] = math.sqrt(dim)
        if case["grad"]:
            s["dout"] = normal(tokens, dim, scale=0.01)
        return s
    batch, ch = case["batch"], case["channels"]
    if case["op"].startswith("conv"):
        width = case["width"]
        s["weight"] = normal(ch, width, scale=0.5)
        s["bias"] = normal(ch, scale=0.1)
        if case["op"] == "conv_step":
            pool, s["slots"] = _slots(case, gen, batch)
            s["x"] = normal(batch, ch)
            s["pool"] = normal(pool + 1, width - 1, ch)  # the last row takes the idle rows' writes of the plain form
            return s
        # x is the first half of a projection's output, as the model has it
        s["x"] = normal(batch, case["length"], 2 * ch)[:, :, :ch]
        s["heads"] = _heads(case, gen, batch, case["length"])
        s["state"] = normal(batch, width - 1, ch) if case["packed"] else None
        if case["grad"]:
            s["dy"] = normal(batch, case["length"], ch, scale=0.01)
        return s
    n, g = case["states"], case["groups"]
    # steps between 0.001 and 0.1, decay rates 1 .. n, as such a model is set up
    step = torch.exp(torch.rand(ch, generator=gen, device="cuda") * math.log(100) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(torch.arange(1, n + 1, device="cuda").float() * (0.9 + 0.2 * torch.rand(ch, n, generator=gen, device="cuda")))
    s["D"] = 1 + normal(ch, dtype=torch.float32, scale=0.1)
    tokens = (batch,) if case["op"] == "scan_step" else (batch, case["length"])
    s["x"] = normal(*tokens, ch, scale=0.5)
    s["dt"] = normal(*tokens, ch, scale=0.3)
    s["z"] = normal(*tokens, 2 * ch)[..., ch:]
    bc = normal(*tokens, 64 + 2 * g * n)  # one projection's output, the low-rank part of dt in front
    s["B"] = bc[..., 64:64 + g * n].unflatten(-1, (g, n))
    s["C"] = bc[..., 64 + g * n:].unflatten(-1, (g, n))
    if case["op"] == "scan_step":
        pool, s["slots"] = _slots(case, gen, batch)
        s["pool"] = normal(pool + 1, ch, n, dtype=torch.float32, scale=0.1)
        return s
    s["heads"] = _heads(case, gen, batch, case["length"])
    s["state"] = normal(batch, ch, n, dtype=torch.float32, scale=0.1) if case["packed"] or not case["grad"] else None
    if case["grad"]:
        s["dy"] = normal(batch, case["length"], ch, scale=0.01)
    return s


# --------------------------------------------------------- the library's calls
def _run_own(s):
    import stream_compaction_gb300 as sc

    case = s["case"]
    if case["op"] == "embed":
        out = sc.embed(s["ids"], s["weight"], s["scale"])
        if not case["grad"]:
            return {"out": out}
        return {"out": out, "dweight": sc.embed_grad(s["ids"], s["dout"], case["vocab"], s["scale"])}
    if case["op"] == "conv_step":
        state = s["pool"][:-1]
        y = sc.causal_conv_step(s["x"], state, s["weight"], s["bias"], slots=s["slots"])
        return {"y": y, "state": state}
    if case["op"] == "conv":
        x, w, bias = s["x"], s["weight"], s["bias"]
        final = x.new_empty(case["batch"], case["width"] - 1, case["channels"])
        y = sc.causal_conv(x, w, bias, heads=s["heads"], state=s["state"], final_state=final)
        if not case["grad"]:
            return {"y": y, "state": final}
        grads = sc.causal_conv_grad(s["dy"], x, w, bias, heads=s["heads"], state=s["state"])
        return {"y": y, "state": final, "dx": grads["x"], "dweight": grads["weight"], "dbias": grads["bias"]}
    if case["op"] == "scan_step":
        state = s["pool"][:-1]
        y = sc.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], state, D=s["D"], z=s["z"],
                                   dt_bias=s["dt_bias"], slots=s["slots"])
        return {"y": y, "state": state}
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "heads": s["heads"], "state": s["state"]}
    if not case["grad"]:
        final = torch.empty_like(s["state"])
        y = sc.selective_scan(*args, **more, final_state=final)
        return {"y": y, "state": final}
    saved = sc.selective_scan_saved(s["x"], s["A"])
    y = sc.selective_scan(*args, **more, saved=saved)
    grads = sc.selective_scan_grad(s["dy"], *args, **more, saved=saved)
    return {"y": y, "grads": grads}


# ------------------------------------------------------------- the plain form
def _segments(heads, batch, length, device):
    """The number of the segment that each token belongs to; the inputs before the first token are of segment 0."""
    if heads is None:
        return torch.zeros(batch, length, dtype=torch.int64, device=device)
    return heads.long().cumsum(1)


def _plain_conv(s):
    case = s["case"]
    x, w = s["x"].float(), s["weight"].float()
    batch, length, ch = x.shape
    width = case["width"]
    before = torch.zeros(batch, width - 1, ch, device=x.device) if s["state"] is None else s["state"].float()
    padded = torch.cat([before, x], 1)
    seg = _segments(s["heads"], batch, length, x.device)
    seg_padded = torch.cat([seg.new_zeros(batch, width - 1), seg], 1)
    same = (seg_padded.unfold(1, width, 1) == seg[:, :, None]).float()[:, :, None, :]
    taps = padded.unfold(1, width, 1)
    pre = (taps * same * w).sum(-1) + s["bias"].float()
    gate = torch.sigmoid(pre)
    last = seg_padded[:, length:] == seg[:, -1:]
    state = torch.where(last[:, :, None], padded[:, length:], 0.0)
    dtype = s["x"].dtype
    out = {"y": (pre * gate).to(dtype), "state": state.to(dtype)}
    if not case["grad"]:
        return out
    dpre = s["dy"].float() * gate * (1 + pre * (1 - gate))
    out["dweight"] = (dpre[..., None] * taps * same).sum((0, 1))
    out["dbias"] = dpre.sum((0, 1))
    # dx[t] = sum_k w[k] * dpre[t + W-1-k]: the products, last tap first, read along a diagonal
    products = torch.nn.functional.pad((dpre[..., None] * w * same).flip(-1), (0, 0, 0, 0, 0, width - 1))
    out["dx"] = products.unfold(1, width, 1).diagonal(dim1=-2, dim2=-1).sum(-1).to(dtype)
    return out


def _plain_conv_step(s):
    pool = s["pool"]
    ok = s["slots"] >= 0
    rows = torch.where(ok, s["slots"].long(), pool.shape[0] - 1)
    window = torch.cat([pool[rows], s["x"][:, None]], 1)
    pre = (window.float() * s["weight"].float().T).sum(1) + s["bias"].float()
    pool.index_copy_(0, rows, window[:, 1:])
    y = torch.where(ok[:, None], pre * torch.sigmoid(pre), 0.0)
    return {"y": y.to(s["x"].dtype), "state": pool[:-1]}


def _recurrence(a, b):
    """h[t] = a[t] * h[t-1] + b[t] along dimension 1, by doubling; overwrites both."""
    reach = 1
    while reach < b.shape[1]:
        b[:, reach:] = b[:, reach:] + a[:, reach:] * b[:, :-reach]
        a[:, reach:] = a[:, reach:] * a[:, :-reach]
        reach *= 2
    return b


def _of_group(v, ch):
    """(..., groups, states) in 32 bits, each group's row for every channel of it."""
    g = v.shape[-2]
    return v.float().unsqueeze(-2).expand(*v.shape[:-1], ch // g, v.shape[-1]).reshape(*v.shape[:-2], ch, v.shape[-1])


def _plain_scan_step(s):
    pool, A = s["pool"], s["A"]
    ok = s["slots"] >= 0
    rows = torch.where(ok, s["slots"].long(), pool.shape[0] - 1)
    x, z = s["x"].float(), s["z"].float()
    d = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
    B, C = _of_group(s["B"], x.shape[-1]), _of_group(s["C"], x.shape[-1])
    h = torch.exp(d[..., None] * A) * pool[rows] + (d * x)[..., None] * B
    pool.index_copy_(0, rows, h)
    y = ((h * C).sum(-1) + s["D"] * x) * z * torch.sigmoid(z)
    return {"y": torch.where(ok[:, None], y, 0.0).to(s["x"].dtype), "state": pool[:-1]}


def _plain_scan(s):
    case = s["case"]
    x, z, A = s["x"].float(), s["z"].float(), s["A"]
    batch, length, ch = x.shape
    dtype, groups = s["x"].dtype, case["groups"]
    v = s["dt"].float() + s["dt_bias"]
    d = torch.nn.functional.softplus(v)
    a = torch.exp(d[..., None] * A)
    if s["heads"] is not None:
        a = torch.where(s["heads"][:, :, None, None], 0.0, a)
    h = (d * x)[..., None] * _of_group(s["B"], ch)
    if s["state"] is not None:
        h[:, 0] += a[:, 0] * s["state"]
    h = _recurrence(a.clone() if case["grad"] else a, h)
    C = _of_group(s["C"], ch)
    y0 = (h * C).sum(-1) + s["D"] * x
    gate = torch.sigmoid(z)
    y = (y0 * z * gate).to(dtype)
    if not case["grad"]:
        return {"y": y, "state": h[:, -1].contiguous()}
    dy = s["dy"].float()
    dz = dy * y0 * gate * (1 + z * (1 - gate))
    dy = dy * z * gate
    per_group = (batch, length, groups, ch // groups, case["states"])
    dC = (dy[..., None] * h).view(per_group).sum(3)
    # the gradient of h runs back in time: dh[t] = a[t+1] * dh[t+1] + C[t] * dy[t]
    later = torch.cat([torch.zeros_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    dh = _recurrence(later, (dy[..., None] * C).flip(1)).flip(1)
    del later, C
    first = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None]
    da = dh * torch.cat([first, h[:, :-1]], 1) * a  # the derivative by the exponent d * A
    dB = (dh * (d * x)[..., None]).view(per_group).sum(3)
    dinput = (dh * _of_group(s["B"], ch)).sum(-1)   # by d * x
    dA = (da * d[..., None]).sum((0, 1))
    dv = ((da * A).sum(-1) + dinput * x) * torch.sigmoid(v)
    grads = {"x": (dinput * d + dy * s["D"]).to(dtype), "dt": dv.to(dtype), "A": dA, "B": dB.to(dtype),
             "C": dC.to(dtype), "D": (dy * x).sum((0, 1)), "z": dz.to(dtype), "dt_bias": dv.sum((0, 1))}
    if s["state"] is not None:
        grads["state"] = dh[:, 0] * a[:, 0]
    return {"y": y, "grads": grads}


def _plain_embed(s):
    case = s["case"]
    ok = ((s["ids"] >= 0) & (s["ids"] < case["vocab"]))[:, None]
    rows = s["ids"].long().clamp(0, case["vocab"] - 1)
    dtype = s["weight"].dtype
    out = {"out": torch.where(ok, s["weight"][rows].float() * s["scale"], 0.0).to(dtype)}
    if case["grad"]:
        dweight = torch.zeros(case["vocab"], case["dim"], device=rows.device)
        dweight.index_add_(0, rows, torch.where(ok, s["dout"].float() * s["scale"], 0.0))
        out["dweight"] = dweight.to(dtype)
    return out


def run(state):
    if own:
        return _run_own(state)
    plain = {"embed": _plain_embed, "conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan,
             "scan_step": _plain_scan_step}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------- the definitions in 64 bits
def _exact_embed(s):
    ids, vocab, scale = s["ids"].long(), s["case"]["vocab"], float(s["scale"])
    kept = torch.nonzero((ids >= 0) & (ids < vocab)).flatten()
    out = torch.zeros(len(ids), s["case"]["dim"], dtype=torch.float64, device="cuda")
    out[kept] = s["weight"][ids[kept]].double().mul_(scale)
    if not s["case"]["grad"]:
        return {"out": out}
    order = kept[torch.argsort(ids[kept], stable=True)]
    tokens, counts = torch.unique_consecutive(ids[order], return_counts=True)
    dweight = torch.zeros(vocab, s["case"]["dim"], dtype=torch.float64, device="cuda")
    ends = counts.cumsum(0).tolist()
    sorted_rows = s["dout"][order].double()
    for token, begin, end in zip(tokens.tolist(), [0] + ends, ends):
        dweight[token] = sorted_rows[begin:end].sum(0) * scale
    return {"out": out, "dweight": dweight}


def _exact_conv(s):
    case = s["case"]
    x, w, width = s["x"].double(), s["weight"].double(), case["width"]
    batch, length, ch = x.shape
    pre = s["bias"].double().expand(batch, length, ch).clone()
    start = torch.zeros(batch, length, dtype=torch.int64, device="cuda")  # the first position that t may look at
    open_at = torch.full((batch,), -width, dtype=torch.int64, device="cuda")
    for t in range(length):
        if s["heads"] is not None:
            open_at = torch.where(s["heads"][:, t], torch.full_like(open_at, t), open_at)
        start[:, t] = open_at
    before = torch.zeros(batch, width - 1, ch, dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        before += s["state"].double()
    line = torch.cat([before, x], 1)
    at = torch.arange(length, device="cuda")
    sees = []
    for k in range(width):
        back = width - 1 - k
        sees.append(((at - back)[None] >= start).double()[..., None])
        pre += w[:, k] * line[:, k:k + length] * sees[k]
    pos = torch.arange(length - width + 1, length, device="cuda")
    state = line[:, length:] * (pos[None] >= start[:, -1:]).double()[..., None]
    gate = 1 / (1 + torch.exp(-pre))
    out = {"y": pre * gate, "state": state}
    if case["grad"]:
        dpre = s["dy"].double() * (gate + pre * gate * (1 - gate))
        dline = torch.zeros_like(line)
        dw = torch.zeros_like(w)
        for k in range(width):
            dline[:, k:k + length] += w[:, k] * dpre * sees[k]
            dw[:, k] = (dpre * line[:, k:k + length] * sees[k]).sum((0, 1))
        out |= {"dx": dline[:, width - 1:], "dweight": dw, "dbias": dpre.sum((0, 1))}
    return out


def _exact_conv_step(s):
    x, w, pool = s["x"].double(), s["weight"].double(), s["pool"][:-1].double()
    y = torch.zeros_like(x)
    for row, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        line = torch.cat([pool[slot], x[row][None]], 0)
        pre = s["bias"].double() + (line * w.T).sum(0)
        y[row] = pre / (1 + torch.exp(-pre))
        pool[slot] = line[1:]
    return {"y": y, "state": pool}


def _exact_scan(s):
    case = s["case"]
    n, ch = case["states"], case["channels"]
    x, z, A = s["x"].double(), s["z"].double(), s["A"].double()
    step = case["op"] == "scan_step"
    if step:
        x, z = x[:, None], z[:, None]
    dt = (s["dt"][:, None] if step else s["dt"]).double() + s["dt_bias"].double()
    d = torch.where(dt > 30, dt, torch.log1p(torch.exp(dt.clamp(max=30))))
    B, C = ((v[:, None] if step else v).double() for v in (s["B"], s["C"]))
    per = ch // case["groups"]
    B, C = (v.repeat_interleave(per, dim=2) for v in (B, C)) if case["groups"] > 1 else (B, C)
    batch, length = x.shape[:2]
    heads = None if step else s["heads"]
    if step:
        rows = s["slots"].tolist()
        pool = s["pool"][:-1].double()
        h0 = torch.stack([pool[max(r, 0)] for r in rows])
    else:
        h0 = torch.zeros(batch, ch, n, dtype=torch.float64, device="cuda")
        h0 = h0 if s["state"] is None else s["state"].double()
    h, y0, kept = h0, torch.empty_like(x), []
    for t in range(length):
        if heads is not None:
            h = h * (~heads[:, t]).double()[:, None, None]
        h = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * x[:, t])[..., None] * B[:, t]
        y0[:, t] = (h * C[:, t]).sum(-1) + s["D"].double() * x[:, t]
        if case.get("grad"):
            kept.append(h)
    gate = 1 / (1 + torch.exp(-z))
    y = y0 * z * gate
    if step:
        live = torch.tensor([r >= 0 for r in rows], device="cuda")
        for row, r in enumerate(rows):
            if r >= 0:
                pool[r] = h[row]
        return {"y": y[:, 0] * live[:, None], "state": pool}
    if not case["grad"]:
        return {"y": y, "state": h}
    dy, D = s["dy"].double(), s["D"].double()
    dz = dy * y0 * (gate + z * gate * (1 - gate))
    dy = dy * z * gate
    dd, dx, dA = torch.zeros_like(x), dy * D, torch.zeros_like(A)
    dB = torch.zeros(batch, length, case["groups"], n, dtype=torch.float64, device="cuda")
    dC = torch.zeros_like(dB)
    carry = torch.zeros_like(h0)
    for t in reversed(range(length)):
        dh = carry + dy[:, t, :, None] * C[:, t]
        dC[:, t] = (dy[:, t, :, None] * kept[t]).unflatten(1, (case["groups"], per)).sum(2)
        dB[:, t] = (dh * (d[:, t] * x[:, t])[..., None]).unflatten(1, (case["groups"], per)).sum(2)
        dbx = (dh * B[:, t]).sum(-1)
        dx[:, t] += dbx * d[:, t]
        decay = torch.exp(d[:, t, :, None] * A)
        if heads is not None:
            decay = decay * (~heads[:, t]).double()[:, None, None]
        carry = dh * decay
        by_exponent = carry * (kept[t - 1] if t else h0)
        dA += (by_exponent * d[:, t, :, None]).sum(0)
        dd[:, t] = (by_exponent * A).sum(-1) + dbx * x[:, t]
    dv = dd / (1 + torch.exp(-dt))
    grads = {"x": dx, "dt": dv, "A": dA, "B": dB, "C": dC, "D": (dy * x).sum((0, 1)), "z": dz,
             "dt_bias": dv.sum((0, 1))}
    if s["state"] is not None:
        grads["state"] = carry
    return {"y": y, "grads": grads}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        return _exact_embed(s)
    if case["op"] == "conv":
        return _exact_conv(s)
    return _exact_conv_step(s) if case["op"] == "conv_step" else _exact_scan(s)
