"""64-bit definitions of the dense operators (layer norm, gated feed-forward
block, distillation from a teacher's top logits) with closed-form gradients,
and the error bounds their tests allow.

Bounds count roundings. U[t] is half a step of type t relative to the value
(torch.finfo(t).eps / 2); TINY[t] half the smallest step of t, which is what a
rounding is off by near zero. Sums of fp32 terms formed as trees of some tens of
levels are off by at most LEVELS * U32 of the sum of magnitudes."""
import math

import torch

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
TINY = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -25}   # fp32: results below 2^-126 may be flushed
U32 = U[F32]
LEVELS = 64


def rounded(t, v):
    """Bound of one rounding of v to type t."""
    return U[t] * v.abs() + TINY[t]


def check(got, want, bound, what):
    got, want = got.double().cpu(), want.double().cpu()
    bound = bound.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert bool(torch.where(fine, True, same).all()), f"{what}: infinities or NaN differ"
    assert bool(torch.isfinite(got[fine]).all()), f"{what}: not finite"
    over = torch.where(fine, (got - want).abs() - bound, -1.0)
    if over.numel() and float(over.max()) > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} outside; worst at {i}: got "
                             f"{got.flatten()[i]!r} want {want.flatten()[i]!r} bound {bound.flatten()[i]!r}")


def rel(got, want):
    """2-norm of the error over the 2-norm of the result."""
    got, want = got.double().cpu(), want.double().cpu()
    n = float(want.norm())
    return float((got - want).norm()) / n if n else float(got.norm())


# ---------------------------------------------------------------- layer norm

def norm(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    xhat = (x - mean) * rstd
    y = xhat * w.double() + (0 if b is None else b.double())
    return y, mean, rstd, xhat


def norm_grads(x, w, dy, eps):
    _, mean, rstd, h = norm(x, w, None, eps)
    dy = dy.double()
    a = dy * w.double()
    dx = rstd * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def norm_bounds(x, w, b, dy, eps, wt):
    """Bounds of y, dx, dweight, dbias."""
    t = x.dtype
    y, mean, rstd, h = norm(x, w, b, eps)
    w = w.double()
    dh = LEVELS * U32 * (rstd * x.double().abs().mean(1, keepdim=True) + h.abs())    # error of xhat
    by = rounded(t, y) + w.abs() * dh + 4 * U32 * ((h * w).abs() + (0 if b is None else b.double().abs()))
    if dy is None:
        return by
    dx, dw, db = norm_grads(x, w, dy, eps)
    dy = dy.double()
    a = (dy * w).abs()
    q = (a * h.abs()).mean(1, keepdim=True)
    inner = a + a.mean(1, keepdim=True) + h.abs() * q
    bx = rounded(t, dx) + rstd * (LEVELS * U32 * inner + dh * q + h.abs() * (a * dh).mean(1, keepdim=True))
    bw = rounded(wt, dw) + 2 * LEVELS * U32 * (dy * h).abs().sum(0) + (dy.abs() * dh).sum(0)
    bb = rounded(wt, db) + 2 * LEVELS * U32 * dy.abs().sum(0)
    return by, bx, bw, bb


# ------------------------------------------------------- gated feed-forward

def act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        c = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    on = (g > 0).double()
    return torch.relu(g), on


def gate(x, wg, wu, kind):
    g, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    return act(g, kind)[0] * u, g, u


def gate_grads(x, wg, wu, dout, kind):
    _, g, u = gate(x, wg, wu, kind)
    a, da = act(g, kind)
    dout = dout.double()
    dg, du = dout * u * da, dout * a
    return dg @ wg.double() + du @ wu.double(), dg.t() @ x.double(), du.t() @ x.double()


def product_slack(n):
    """Of the sum of magnitudes: n products summed in fp32 by matrix cores,
    32 or fewer an instruction, at most six instructions a 32 (fp32's parts)."""
    return (n / 4 + LEVELS) * U32


def gate_bounds(x, wg, wu, dout, kind):
    """Bounds of out, g, u and (with dout) dx, dw_gate, dw_up."""
    t = x.dtype
    out, g, u = gate(x, wg, wu, kind)
    ax, ag, au = x.double().abs(), wg.double().abs(), wu.double().abs()
    k = product_slack(x.shape[1])
    eg, eu = k * (ax @ ag.t()), k * (ax @ au.t())
    a, da = act(g, kind)
    bo = rounded(t, out) + 1.2 * eg * (u.abs() + eu) + a.abs() * eu + LEVELS * U32 * (out.abs() + u.abs() * g.abs())
    if dout is None:
        return bo, eg, eu
    d = dout.double().abs()
    dg, du = (d * u.abs() * da.abs()), (d * a.abs())
    ft = U[t] if t != F32 else 2 * U32           # rounding of the factors dg and du
    # 0.8 bounds |act''|; relu's derivative jumps where g is within its error of 0
    jump = (g.abs() <= eg).double() * d * u.abs() if kind == "relu" else 0.0
    edg = ft * dg + d * (1.2 * eu + 0.8 * eg * u.abs() + LEVELS * U32 * u.abs()) + jump + TINY[t]
    edu = ft * du + d * (1.2 * eg + LEVELS * U32 * g.abs()) + TINY[t]
    dx, dwg, dwu = gate_grads(x, wg, wu, dout, kind)
    kh, km = product_slack(2 * wg.shape[0]), product_slack(x.shape[0])
    bx = rounded(t, dx) + edg @ ag + edu @ au + kh * (dg @ ag + du @ au)
    bg = rounded(t, dwg) + edg.t() @ ax + km * (dg.t() @ ax)
    bu = rounded(t, dwu) + edu.t() @ ax + km * (du.t() @ ax)
    return bo, eg, eu, bx, bg, bu


# ---------------------------------------------------------------- distillation

def distill(z, ids, tl, t):
    """(loss, gradient of each loss in its row's logits, bounds of both)."""
    z64, v = z.double(), z.shape[1]
    there = (ids >= 0) & (ids < v) & (tl != -math.inf)
    some = there.any(1, keepdim=True) if ids.shape[1] else torch.zeros(len(z), 1, dtype=torch.bool, device=z.device)
    x = torch.where(there, tl.double() / t, -math.inf)
    p = torch.where(there, torch.softmax(torch.where(some, x, 0.0), 1), 0.0) if ids.shape[1] else x
    lq = torch.log_softmax(z64 / t, 1)
    at = torch.gather(lq, 1, torch.where(there, ids, 0))
    lp = torch.log(torch.where(p > 0, p, 1.0))
    used = there & ~(p == 0)
    term = torch.where(used, p * (lp - at), 0.0)
    loss = t * t * term.sum(1)
    size = torch.where(used, p * (2 + lp.abs() + at.abs()), 0.0).sum(1)
    q = torch.exp(lq)
    taken = torch.zeros_like(q).scatter_add_(1, torch.where(there, ids, 0), p)
    grad = torch.where(some, t * (q - taken), 0.0)
    xs = torch.where(q > 0, lq.abs(), 0.0)
    bl = t * t * LEVELS * U32 * size + U32 * loss.abs() + TINY[F32]
    bg = t * U32 * ((LEVELS + 8 * xs) * q + LEVELS * taken)
    return loss, grad, bl, bg
