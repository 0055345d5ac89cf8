"""Plain 64-bit forms of the 8-bit operators and the block boundary, with bounds on what the
library's fp32 arithmetic may be off, each from its count of roundings."""
import torch

EPS32 = 2.0 ** -24        # half a step of fp32, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# smallest positive steps: a result that underflows is off by up to half of one
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
# A chain of fp32 additions in the row kernels: at most 64 entries of a thread (8 vectors of 8),
# 5 + 5 shuffle steps and a final scaling; positive terms, so the relative error of the sum is at
# most the number of roundings an entry passes through. 100 leaves room for the products.
CHAIN = 100 * EPS32


def hadamard(n, device):
    h = torch.ones(1, 1, dtype=torch.float64, device=device)
    while h.shape[0] < n:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h


def whiten(x, sign=None, chan_scale=None, block=0):
    """T(x) in fp64 and a bound on the error of its fp32 evaluation."""
    v = x.double()
    if not block:
        return v, torch.zeros_like(v)
    if chan_scale is not None:
        v = v * chan_scale.double()
    if sign is not None:
        v = torch.where(sign < 0, -v, v)
    b = v.reshape(-1, block)
    out = (b @ hadamard(block, x.device)) * block ** -0.5
    # log2(block) additions, the channel scale, 1/sqrt(block) and its own rounding
    steps = block.bit_length() - 1 + 3
    err = (steps * 2 * EPS32) * b.abs().sum(1, keepdim=True) * block ** -0.5 + TINY[torch.float32]
    return out.reshape(v.shape), err.expand_as(out).reshape(v.shape)


def codes(v):
    """int8 codes (fp64 values) and scales of fp64 rows: round half to even of 127 v / a."""
    a = v.abs().amax(1, keepdim=True)
    bad = ~torch.isfinite(v).all(1, keepdim=True)
    safe = torch.where((a > 0) & ~bad, a, torch.ones_like(a))
    q = torch.round(127 * torch.where(bad, torch.zeros_like(v), v) / safe)
    return q, torch.where(bad, torch.full_like(a, float("nan")), a / 127)[:, 0]


def norm(v, dv, kind, w, b, eps):
    """A norm in fp64 of rows known to within dv; returns (result, bound on the fp32 one)."""
    K = v.shape[1]
    d0 = dv
    if kind == "layer":
        mean_abs = v.abs().mean(1, keepdim=True)
        d0 = dv + dv.mean(1, keepdim=True) + CHAIN * (mean_abs + v.abs())
        v = v - v.mean(1, keepdim=True)
    ms = (v * v).sum(1, keepdim=True) / K + eps
    rs = ms.rsqrt()
    u = v * rs
    # error of the mean square from d0, relative to 2 * ms, and its own roundings
    dms = ((v.abs() * d0).mean(1, keepdim=True) + 0.5 * (d0 * d0).mean(1, keepdim=True)) / ms
    du = d0 * rs + u.abs() * (dms + CHAIN)
    if w is not None:
        u, du = u * w.double(), du * w.double().abs()
        du = du + 2 * EPS32 * u.abs()
    if b is not None:
        u = u + b.double()
        du = du + 2 * EPS32 * u.abs()
    return u, du


def boundary(h, r, post, pre, gate_rows, branch, resid):
    """(c, dc, n, dn): the boundary in fp64 with bounds. post, pre: (kind, w, b, eps) or None;
    gate_rows [rows][K or 1] or None."""
    u, du = h.double(), torch.zeros(h.shape, dtype=torch.float64, device=h.device)
    if post is not None:
        u, du = norm(u, du, *post)
    if gate_rows is not None:
        g = gate_rows.double()
        u, du = u * g, du * g.abs()
    b32 = torch.tensor(branch, dtype=torch.float32).item()     # the call takes them in fp32
    r32 = torch.tensor(resid, dtype=torch.float32).item()
    c, dc = u * b32, du * abs(b32)
    mag = c.abs()
    if r is not None:
        c = c + r32 * r.double()
        mag = mag + (r32 * r.double()).abs()
    dc = dc + 4 * EPS32 * mag
    if pre is None:
        return c, dc, c, dc
    n, dn = norm(c, dc, *pre)
    return c, dc, n, dn


def within(got, want, bound):
    """got (any type) against want (fp64) elementwise: the bound plus got's own rounding."""
    lim = bound * (1 + HALF_STEP[got.dtype]) + HALF_STEP[got.dtype] * want.abs() + TINY[got.dtype]
    bad = (got.double() - want).abs() > lim
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside the bound; worst "
                           f"{((got.double() - want).abs() / lim).max().item():.3g} x")


def product(xq, xs, wq, ws, K, bias):
    """The scaled product in fp64 and the bound: fl(acc), xs * ws, their product, the bias sum."""
    acc = xq[:, :K].double() @ wq[:, :K].double().t()
    y = acc * (xs.double()[:, None] * ws.double()[None, :])
    dy = 3.01 * EPS32 * y.abs()
    if bias is not None:
        y = y + bias.double()
        dy = dy + EPS32 * y.abs()
    return y, dy
