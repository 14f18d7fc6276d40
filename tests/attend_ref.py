"""64-bit definitions of the attention operators (norms of queries and keys with
the rotation by position, attention over packed prompts and over a paged cache)
with closed-form gradients, and the error bounds their tests allow.

Bounds count roundings, as those of tests/dense_ref.py do, of the steps the
kernels take: scores summed in fp32; weights e^(score - reference) in fp32, then
rounded to the operands' type for the product with the values; in the backward
the weights and weights x (dout . v - dout . out), rounded likewise."""
import math

import torch

from tests.dense_ref import BF16, F16, F32, LEVELS, TINY, U, U32, product_slack, rounded  # noqa: F401

# ------------------------------------------------------------------- rotation


def heads_of(x, dim):
    return x.double().reshape(x.shape[0], x.shape[1] // dim, dim)


def pair_index(rot, pairs):
    """Places of the pairs' first and second elements."""
    p = torch.arange(rot // 2)
    return (p, p + rot // 2) if pairs == "halves" else (2 * p, 2 * p + 1)


def turn(x, angle, pairs, sign=1.0):
    """x [rows, heads, dim], angle [rows, rot / 2]."""
    a, b = (i.to(x.device) for i in pair_index(2 * angle.shape[1], pairs))
    c, s = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def spread(x, rot, pairs):
    """|x| of an element and of its pair's other, summed: what bounds either after a rotation."""
    a, b = (i.to(x.device) for i in pair_index(rot, pairs))
    y = x.abs()
    z = y.clone()
    z[..., a] = z[..., b] = y[..., a] + y[..., b]
    return z


def rotate(x, w, positions, freq, dim, pairs, eps):
    """(y, n, r, angle) of one of q and k."""
    h = heads_of(x, dim)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    angle = positions.double()[:, None] * freq.double()
    return turn(h * r * w.double(), angle, pairs).flatten(1), h * r, r, angle


def rotate_grads(x, w, positions, freq, dim, pairs, eps, dy):
    _, n, r, angle = rotate(x, w, positions, freq, dim, pairs, eps)
    g = turn(heads_of(dy, dim), angle, pairs, -1.0)
    t = g * w.double()
    dx = r * (t - n * (t * n).mean(-1, keepdim=True))
    return dx.flatten(1), (g * n).sum((0, 1))


def rotate_bounds(x, w, positions, freq, dim, pairs, eps, dy, wt):
    """Bounds of y, and with dy of dx and dw. A head's sum of squares is a tree of some tens of roundings, its norm's
    error half of that; cosines and sines are good to 4 roundings and to what the angle's formation in fp64 leaves
    (three roundings of it, one of the definition's)."""
    t, rot = x.dtype, 2 * freq.numel()
    y, n, r, angle = rotate(x, w, positions, freq, dim, pairs, eps)
    far = (4 * 2.0 ** -52 * float(angle.abs().max())) if angle.numel() else 0.0
    u = spread(n * w.double(), rot, pairs).flatten(1)
    by = rounded(t, y) + (LEVELS / 2 * U32 + far) * u
    if dy is None:
        return by
    dx, dw = rotate_grads(x, w, positions, freq, dim, pairs, eps, dy)
    g = spread(heads_of(dy, dim), rot, pairs)
    tt, an = g * w.double().abs(), n.abs()
    bx = rounded(t, dx) + ((LEVELS * U32 + far) * r * (tt + an * (tt * an).mean(-1, keepdim=True))).flatten(1)
    bw = rounded(wt, dw) + ((2 * LEVELS * U32 + far) * g * an).sum((0, 1))
    return by, bx, bw


# ------------------------------------------------------------------ attention

def _one(q, k, v, dout, causal, scale, t):
    """One sequence and one key head: q, dout [group, n, D], k, v [m, D]; the last query sees the last key. Returns
    results and bounds."""
    n, m, d = q.shape[1], k.shape[0], k.shape[1]
    s = scale * q @ k.t()
    seen = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if causal:
        seen = seen.tril(m - n)
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - lse)
    out = p @ v
    w_round = U[t] if t != F32 else 0.0
    kd, kn = product_slack(d), product_slack(m)
    s0 = torch.where(seen, s, 0.0)
    # error of a score's exponent; of the weight, which f16 also rounds at 2^-33 of the largest (the bias is 2^8)
    e = kd * scale * (q.abs() @ k.abs().t()) + 4 * U32 * (1 + s0.abs())
    least = 2.0 ** -33 if t == F16 else 2.0 ** -126
    top = torch.exp(torch.where(seen, s, -math.inf).max(-1, keepdim=True).values - lse)   # the largest weight
    pe = p * (e + w_round) + least * top * seen
    el = (p * e).sum(-1, keepdim=True) + kn
    bo = rounded(t, out) + (pe + kn * p) @ v.abs() + out.abs() * el
    bl = el + 4 * U32 * (1 + lse.abs())
    if dout is None:
        return (out, lse), (bo, bl)
    dp = dout @ v.t()
    delta = (dout * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    e2 = e + bl + 4 * U32 * lse.abs()
    ddelta = (dout.abs() * bo).sum(-1, keepdim=True) + kd * (dout * out).abs().sum(-1, keepdim=True)
    tiny = TINY[t] * seen
    eds = p * (e2 * (dp - delta).abs() + kd * (dout.abs() @ v.abs().t()) + ddelta + 4 * U32 * (dp.abs() + delta.abs()))
    eds = eds + w_round * (ds.abs() + eds) + tiny
    ep = p * (e2 + w_round) + tiny
    kq = product_slack(q.shape[0] * n)
    dq, dk, dv = scale * ds @ k, scale * (ds.mT @ q).sum(0), (p.mT @ dout).sum(0)
    ads = ds.abs()
    bq = rounded(t, dq) + scale * (eds + kn * ads) @ k.abs()
    bk = rounded(t, dk) + scale * ((eds + kq * ads).mT @ q.abs()).sum(0)
    bv = rounded(t, dv) + ((ep + kq * p).mT @ dout.abs()).sum(0)
    return (out, lse, dq, dk, dv), (bo, bl, bq, bk, bv)


def attend(q, k, v, lengths, first, heads, kv, causal, scale, dout=None):
    """Results and bounds of every row, [rows, heads * dim] (lse: [heads, rows]); rows of no sequence hold NaN."""
    rows, dim, t = q.shape[0], q.shape[1] // heads, q.dtype
    g = heads // kv
    dev = q.device
    sizes = [(heads, dim), (heads, 1)] + ([(heads, dim), (kv, dim), (kv, dim)] if dout is not None else [])
    want, bound = ([torch.full((rows, *s), math.nan, dtype=torch.float64, device=dev) for s in sizes] for _ in range(2))
    q, k, v = (heads_of(x, dim) for x in (q, k, v))
    do = None if dout is None else dout.double().reshape(rows, heads, dim)
    at = first
    for n in lengths:
        r, at = slice(at, at + n), at + n
        for h in range(kv if n else 0):
            hs = slice(h * g, (h + 1) * g)
            a, b = _one(q[r, hs].transpose(0, 1), k[r, h], v[r, h], None if do is None else do[r, hs].transpose(0, 1),
                        causal, scale, t)
            for i in range(len(sizes)):
                for whole, part in ((want, a), (bound, b)):
                    if i < 3:
                        whole[i][r, hs] = part[i].transpose(0, 1)
                    else:
                        whole[i][r, h] = part[i]
    flat = lambda x: [x[0].flatten(1), x[1][:, :, 0].t().contiguous()] + [y.flatten(1) for y in x[2:]]   # noqa: E731
    return flat(want), flat(bound)


def paged(q, k_pages, v_pages, table, lengths, scale):
    """(out, bound) of one new token a sequence."""
    pages, size, kv, dim = k_pages.shape
    seqs, heads = q.shape[0], q.shape[1] // dim
    out, bound = (torch.zeros(seqs, heads, dim, dtype=torch.float64, device=q.device) for _ in range(2))
    for i, n in enumerate(lengths.tolist()):
        j = torch.arange(max(0, min(n, table.shape[1] * size)), device=q.device)
        page = table[i].long()[j // size]
        there = (page >= 0) & (page < pages)
        slot = (page * size + j % size)[there]
        if not slot.numel():
            continue
        k, v = (x.reshape(-1, kv, dim)[slot].double() for x in (k_pages, v_pages))
        g = heads // kv
        for h in range(kv):
            a, b = _one(q[i].double().reshape(kv, g, 1, dim)[h], k[:, h], v[:, h], None, False, scale, q.dtype)
            out[i, h * g:(h + 1) * g], bound[i, h * g:(h + 1) * g] = a[0][:, 0], b[0][:, 0]
    return out.flatten(1), bound.flatten(1)
