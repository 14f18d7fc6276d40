"""Timed cases of the dense operators that train and serve a model on looked-up
rows: layer norm, the gated feed-forward block and distillation from a
teacher's top logits.

run() computes them in their plain form (elementary torch operations in 32
bits, rounded once at the end) while `own` is false, and through the library's
public calls when it is true. Sizes are this repository's own (32,768 pooled
rows of the 11M-row table at dim 128; the 10^6-row and 1,000-row tables as
classes) or generic model widths.
"""
import math

import torch

own = False   # set from outside: false, the plain forms; true, the library's calls

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5

# --------------------------------------------------------------------------
# Cases. `mode`: "forward" is the serving form; "train" is the training step of
# the operator (forward and every gradient); "split" (distillation) is the
# forward and a later backward with the caller's own gradient of each loss.


def listed():
    return [
        # one looked-up row normalised before it is answered with: latency
        {"name": "norm-answer", "op": "norm", "mode": "forward", "dtype": "f32", "wdtype": "f32",
         "rows": 1, "dim": 128, "pad": 0, "bias": True},
        # the 11M-row table's pooled batch, normalised and trained through
        {"name": "norm-pooled-train", "op": "norm", "mode": "train", "dtype": "f32", "wdtype": "f32",
         "rows": 32768, "dim": 128, "pad": 0, "bias": True},
        # a training batch of a wide model, fp32 weights
        {"name": "norm-wide-train", "op": "norm", "mode": "train", "dtype": "bf16", "wdtype": "f32",
         "rows": 16384, "dim": 4096, "pad": 0, "bias": True},
        # ragged: odd width, rows cut out of a wider buffer, no bias
        {"name": "norm-odd", "op": "norm", "mode": "train", "dtype": "f16", "wdtype": "f16",
         "rows": 4099, "dim": 1021, "pad": 11, "bias": False},
        # one token through the block: the weights are read once
        {"name": "gate-token", "op": "gate", "mode": "forward", "dtype": "bf16", "act": "silu",
         "rows": 1, "dim": 4096, "hidden": 10240, "pad": 0},
        # the pooled batch at the table's dim, fp32, trained
        {"name": "gate-pooled-train", "op": "gate", "mode": "train", "dtype": "f32", "act": "gelu",
         "rows": 32768, "dim": 128, "hidden": 512, "pad": 0},
        # a training batch of a wide model: the largest
        {"name": "gate-wide-train", "op": "gate", "mode": "train", "dtype": "bf16", "act": "silu",
         "rows": 8192, "dim": 4096, "hidden": 10240, "pad": 0},
        # ragged prompt: no size a multiple of a tile, rows out of a wider buffer
        {"name": "gate-odd", "op": "gate", "mode": "forward", "dtype": "f16", "act": "silu",
         "rows": 1037, "dim": 1030, "hidden": 2731, "pad": 3},
        # seven answers over the 1,000-row table: latency
        {"name": "distill-small", "op": "distill", "mode": "forward", "dtype": "f32",
         "rows": 7, "classes": 1000, "top": 5, "pad": 0, "temperature": 1.0},
        # a training batch over a large vocabulary, loss and gradient together
        {"name": "distill-vocab-train", "op": "distill", "mode": "train", "dtype": "bf16",
         "rows": 4096, "classes": 131072, "top": 64, "pad": 0, "temperature": 2.0},
        # every row of the 10^6-row table as a class: few, very long rows
        {"name": "distill-items-train", "op": "distill", "mode": "train", "dtype": "f32",
         "rows": 96, "classes": 1000000, "top": 256, "pad": 0, "temperature": 1.0},
        # ragged: odd class count, the loss inside a larger objective
        {"name": "distill-odd-split", "op": "distill", "mode": "split", "dtype": "f16",
         "rows": 1021, "classes": 50021, "top": 20, "pad": 5, "temperature": 1.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size of [lo, hi]: half of them odd, the others 4 or 5 times a power of two."""
    n = _log_int(rng, lo, hi)
    if n < 64 or rng.random() < 0.5:
        return min(hi, n | 1)
    unit = 1 << (n.bit_length() - 3)
    return max(lo, (5 if n >= 5 * unit else 4) * unit)


def _limit(c):
    """The listed cases that bound a drawn one's work: the same operator's, and
    for products the same kind of type's."""
    return c["op"], c["op"] == "gate" and c["dtype"] == "f32"


def draw(rng):
    op = rng.choice(["norm", "gate", "distill"])
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(_limit(c), (0, 0))
        most[_limit(c)] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        dtype = rng.choice(["f32", "bf16", "f16"])
        pad = rng.choice([0, 0, 0, 1, 8, 24])
        if op == "norm":
            c = {"op": op, "mode": rng.choice(["forward", "train"]), "dtype": dtype,
                 "wdtype": rng.choice(["f32", dtype]), "rows": _size(rng, 1, 65536), "dim": _size(rng, 16, 16384),
                 "pad": pad, "bias": rng.random() < 0.7}
        elif op == "gate":
            c = {"op": op, "mode": rng.choice(["forward", "train"]), "dtype": dtype,
                 "act": rng.choice(["silu", "gelu", "relu"]), "rows": _size(rng, 1, 32768),
                 "dim": _size(rng, 64, 4096), "hidden": _size(rng, 64, 10240), "pad": pad}
        else:
            c = {"op": op, "mode": rng.choice(["forward", "train", "split"]), "dtype": dtype,
                 "rows": _size(rng, 1, 8192), "classes": _size(rng, 1000, 1000000), "top": _log_int(rng, 1, 256),
                 "pad": pad, "temperature": rng.choice([1.0, 1.5, 2.0, 4.0])}
        b, f = most[_limit(c)]
        w = work(c)
        if w["bytes"] <= b and w["flops"] <= f:
            return c


def work(case):
    c = case
    s = DTYPES[c["dtype"]].itemsize
    m = c["rows"]
    if c["op"] == "norm":
        n, ws = c["dim"], DTYPES[c["wdtype"]].itemsize
        k = 2 if c["bias"] else 1
        if c["mode"] == "forward":      # x in, y out; weights in
            return {"bytes": 2 * m * n * s + k * n * ws, "flops": 7 * m * n}
        # x and dy in, y and dx out; weights in, their gradients out
        return {"bytes": 4 * m * n * s + 2 * k * n * ws, "flops": 20 * m * n}
    if c["op"] == "gate":
        k, h = c["dim"], c["hidden"]
        if c["mode"] == "forward":      # x and both weights in, the product out; two products
            return {"bytes": (m * k + 2 * k * h + m * h) * s, "flops": 4 * m * k * h}
        # also the gradient in, dx and both weights' gradients out; four more products
        return {"bytes": (2 * m * k + 4 * k * h + 2 * m * h) * s, "flops": 12 * m * k * h}
    v, top = c["classes"], c["top"]
    lists = m * top * (8 + 4)
    if c["mode"] == "forward":          # logits in, a loss a row out
        return {"bytes": m * v * s + lists + 4 * m, "flops": 5 * m * v}
    # logits in and their gradient out, the row weights in, the losses out
    return {"bytes": 2 * m * v * s + lists + 8 * m, "flops": 8 * m * v}


# --------------------------------------------------------------------------
# Inputs.


def _rows(t, pad):
    """The same rows inside a buffer that is `pad` elements wider."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _inputs(case, seed):
    c = case
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device=DEV).manual_seed(seed * 2654435761 % (1 << 31) + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    m = c["rows"]
    if c["op"] == "norm":
        n, wdt = c["dim"], DTYPES[c["wdtype"]]
        x = normal(m, n)
        x *= torch.exp(0.5 * normal(m, 1))      # rows of unlike scale and offset
        x += normal(m, 1)
        s = {"x": _rows(x.to(dt), c["pad"]), "weight": (1 + 0.1 * normal(n)).to(wdt),
             "bias": (0.1 * normal(n)).to(wdt) if c["bias"] else None}
        if c["mode"] != "forward":
            s["dy"] = _rows(normal(m, n).to(dt), c["pad"])
        return s
    if c["op"] == "gate":
        k, h = c["dim"], c["hidden"]
        s = {"x": _rows(normal(m, k).to(dt), c["pad"]), "w_gate": (normal(h, k) / math.sqrt(k)).to(dt),
             "w_up": (normal(h, k) / math.sqrt(k)).to(dt)}
        if c["mode"] != "forward":
            s["dout"] = _rows(normal(m, h).to(dt), c["pad"])
        return s
    v, top = c["classes"], c["top"]
    # the teacher's list: distinct classes, falling logits; every tenth list is
    # cut short (-1 fills it up) and one of fifty is empty
    start = torch.randint(0, v, (m, 1), generator=g, device=DEV)
    step = torch.randint(1, max(2, v // max(top, 1)), (m, 1), generator=g, device=DEV)
    ids = (start + step * torch.arange(top, device=DEV)) % v
    drops = -torch.log(torch.rand(m, top, generator=g, device=DEV).clamp_min(1e-7))
    top_logits = 12.0 - 0.4 * torch.cumsum(drops, 1)
    kind = torch.rand(m, 1, generator=g, device=DEV)
    keep = torch.where(kind < 0.02, 0, torch.where(kind < 0.12, max(1, top // 2), top))
    ids = torch.where(torch.arange(top, device=DEV) < keep, ids, -1)
    z = torch.empty(m, v, dtype=dt, device=DEV)
    for a in range(0, m, 512):                  # student: noise, and a part of the teacher's shape
        b = min(m, a + 512)
        part = 1.5 * normal(b - a, v)
        part.scatter_add_(1, ids[a:b].clamp_min(0), torch.where(ids[a:b] >= 0, 0.6 * top_logits[a:b], 0.0))
        z[a:b] = part
    s = {"logits": _rows(z, c["pad"]), "ids": ids, "top_logits": top_logits}
    if c["mode"] != "forward":                  # each row's share of the loss (some rows padded out)
        w = torch.rand(m, generator=g, device=DEV) + 0.5
        s["row_weight"] = torch.where(torch.rand(m, generator=g, device=DEV) < 0.05, 0.0, w)
    return s


def prepare(case, seed):
    c = case
    s = _inputs(case, seed)
    s["case"] = c
    if not own:
        return s
    import tensor_train_compressed_amd as tte
    s["tte"] = tte
    m = c["rows"]
    f32 = dict(dtype=torch.float32, device=DEV)
    # the caller-owned outputs, kept statistics and workspaces of a program's loop
    if c["op"] == "norm":
        s["y"] = torch.empty_like(s["x"], memory_format=torch.contiguous_format)
        if c["mode"] != "forward":
            s["mean"], s["rstd"] = torch.empty(m, **f32), torch.empty(m, **f32)
            s["dx"] = torch.empty_like(s["y"])
            s["dweight"] = torch.empty_like(s["weight"])
            s["dbias"] = torch.empty_like(s["weight"]) if c["bias"] else None
            need = tte.tt_emb_norm_workspace_bytes(s["x"].dtype, m, c["dim"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    elif c["op"] == "gate":
        dt = s["x"].dtype
        s["out"] = torch.empty(m, c["hidden"], dtype=dt, device=DEV)
        if c["mode"] != "forward":
            s["gate"], s["up"] = torch.empty(m, c["hidden"], **f32), torch.empty(m, c["hidden"], **f32)
            s["dx"] = torch.empty(m, c["dim"], dtype=dt, device=DEV)
            s["dw_gate"], s["dw_up"] = torch.empty_like(s["w_gate"]), torch.empty_like(s["w_up"])
        need = tte.tt_emb_gate_workspace_bytes(dt, m, c["dim"], c["hidden"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    else:
        s["loss"] = torch.empty(m, **f32)
        need = tte.tt_emb_distill_workspace_bytes(s["logits"].dtype, m, c["classes"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        if c["mode"] != "forward":
            s["dlogits"] = torch.empty_like(s["logits"], memory_format=torch.contiguous_format)
        if c["mode"] == "split":
            s["stats"] = torch.empty(m, 2, **f32)
    return s


# --------------------------------------------------------------------------
# One pass.


def run(state):
    c = state["case"]
    return (_OWN if own else _PLAIN)[c["op"]](state, c)


def _own_norm(s, c):
    tte = s["tte"]
    if c["mode"] == "forward":
        tte.tt_emb_norm_forward(s["x"], s["weight"], s["bias"], s["y"], eps=EPS)
        return s["y"]
    tte.tt_emb_norm_forward(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=EPS)
    tte.tt_emb_norm_backward(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dweight"], s["dbias"],
                             workspace=s["workspace"])
    return [t for t in (s["y"], s["dx"], s["dweight"], s["dbias"]) if t is not None]


def _own_gate(s, c):
    tte = s["tte"]
    if c["mode"] == "forward":
        tte.tt_emb_gate_forward(s["x"], s["w_gate"], s["w_up"], s["out"], act=c["act"], workspace=s["workspace"])
        return s["out"]
    tte.tt_emb_gate_forward(s["x"], s["w_gate"], s["w_up"], s["out"], s["gate"], s["up"], act=c["act"],
                            workspace=s["workspace"])
    tte.tt_emb_gate_backward(s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["dout"], s["dx"], s["dw_gate"],
                             s["dw_up"], act=c["act"], workspace=s["workspace"])
    return [s["out"], s["dx"], s["dw_gate"], s["dw_up"]]


def _own_distill(s, c):
    tte, t = s["tte"], c["temperature"]
    if c["mode"] == "forward":
        tte.tt_emb_distill_forward(s["logits"], s["ids"], s["top_logits"], s["loss"], temperature=t,
                                   workspace=s["workspace"])
        return s["loss"]
    if c["mode"] == "train":
        tte.tt_emb_distill_train(s["logits"], s["ids"], s["top_logits"], s["row_weight"], s["loss"], s["dlogits"],
                                 temperature=t, workspace=s["workspace"])
    else:
        tte.tt_emb_distill_forward(s["logits"], s["ids"], s["top_logits"], s["loss"], s["stats"], temperature=t,
                                   workspace=s["workspace"])
        tte.tt_emb_distill_backward(s["logits"], s["ids"], s["top_logits"], s["stats"], s["row_weight"], s["dlogits"],
                                    temperature=t)
    return [s["loss"], s["dlogits"]]


def _plain_norm(s, c):
    x = s["x"].float()
    w = s["weight"].float()
    n = x.shape[1]
    d = x - x.sum(1, keepdim=True) / n
    rstd = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / n + EPS)
    xhat = d * rstd
    y = xhat * w
    if c["bias"]:
        y = y + s["bias"].float()
    y = y.to(s["x"].dtype)
    if c["mode"] == "forward":
        return y
    dy = s["dy"].float()
    a = dy * w
    dx = rstd * (a - a.sum(1, keepdim=True) / n - xhat * ((a * xhat).sum(1, keepdim=True) / n))
    out = [y, dx.to(s["x"].dtype), (dy * xhat).sum(0).to(s["weight"].dtype)]
    if c["bias"]:
        out.append(dy.sum(0).to(s["weight"].dtype))
    return out


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * (math.sqrt(0.5 / math.pi) * torch.exp(-0.5 * g * g))
    on = (g > 0).to(g.dtype)
    return g * on, on


def _plain_gate(s, c):
    dt = s["x"].dtype
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, c["act"])
    out = (a * u).to(dt)
    if c["mode"] == "forward":
        return out
    dout = s["dout"].float()
    dg, du = dout * u * da, dout * a
    return [out, (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)]


def _plain_distill(s, c):
    t = c["temperature"]
    z = s["logits"].float()
    v = z.shape[1]
    mx = z.max(1, keepdim=True).values
    e = torch.exp((z - mx) / t)
    total = e.sum(1, keepdim=True)
    present = (s["ids"] >= 0) & (s["ids"] < v)
    ids = torch.where(present, s["ids"], 0)
    tl = torch.where(present, s["top_logits"].float() / t, float("-inf"))
    some = present.any(1, keepdim=True)
    tl = tl - torch.where(some, tl.max(1, keepdim=True).values, 0.0)
    p = torch.exp(tl)
    norm = torch.where(some, p.sum(1, keepdim=True), 1.0)
    p = p / norm
    logq = (torch.gather(z, 1, ids) - mx) / t - torch.log(total)
    logp = tl - torch.log(norm)
    loss = t * t * torch.where(present, p * (logp - logq), 0.0).sum(1)
    if c["mode"] == "forward":
        return loss
    dz = e / total * some
    dz.scatter_add_(1, ids, torch.where(present, -p, 0.0))
    dz = dz * (t * s["row_weight"][:, None])
    return [loss, dz.to(s["logits"].dtype)]


_OWN = {"norm": _own_norm, "gate": _own_gate, "distill": _own_distill}
_PLAIN = {"norm": _plain_norm, "gate": _plain_gate, "distill": _plain_distill}


# --------------------------------------------------------------------------
# The same outputs in 64 bits, from the definitions and by differentiating
# them.


def exact(case, seed):
    c = case
    s = _inputs(case, seed)
    d = {k: v.double() for k, v in s.items() if v is not None and k not in ("logits", "ids")}
    if c["op"] == "norm":
        n = c["dim"]
        x = d["x"].requires_grad_()
        w = d["weight"].requires_grad_()
        b = d["bias"].requires_grad_() if c["bias"] else None
        y = torch.nn.functional.layer_norm(x, (n,), w, b, EPS)
        if c["mode"] == "forward":
            return y.detach()
        wrt = [x, w] + ([b] if c["bias"] else [])
        return [y.detach(), *torch.autograd.grad(y, wrt, d["dy"])]
    if c["op"] == "gate":
        x, wg, wu = (d[k].requires_grad_() for k in ("x", "w_gate", "w_up"))
        act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
               "relu": torch.nn.functional.relu}[c["act"]]
        out = act(torch.mm(x, wg.t())) * torch.mm(x, wu.t())
        if c["mode"] == "forward":
            return out.detach()
        return [out.detach(), *torch.autograd.grad(out, (x, wg, wu), d["dout"])]
    t = c["temperature"]
    m, v = s["logits"].shape
    losses, grads = [], []
    step = max(1, (1 << 26) // v)
    for a in range(0, m, step):
        z = s["logits"][a:a + step].double().requires_grad_()
        ids = s["ids"][a:a + step]
        present = (ids >= 0) & (ids < v)
        some = present.any(1, keepdim=True)
        tl = torch.where(present, d["top_logits"][a:a + step] / t, -torch.inf)
        p = torch.softmax(torch.where(some, tl, 0.0), 1) * present
        logq = torch.gather(torch.log_softmax(z / t, 1), 1, ids.clamp(0, v - 1))
        loss = t * t * (torch.special.xlogy(p, p) - p * logq).sum(1)
        losses.append(loss.detach())
        if c["mode"] != "forward":
            grads.append(torch.autograd.grad(loss, z, d["row_weight"][a:a + step])[0])
    if c["mode"] == "forward":
        return torch.cat(losses)
    return [torch.cat(losses), torch.cat(grads)]
