"""Plain float64 forms of the paged append and of latent attention, and the error bounds that the
kernels' roundings allow.  Used by the tests only; shares no code with the library.

Bounds.  u is half a step of the storage type relative to a value (bf16 2^-8, f16 2^-11), e = 2^-24
half a step of float32.
  logits   s = scale * sum of K products, accumulated in float32:
             |ds| <= (K + 4) e * scale * sum |q||k|   =: ds
           (each product of two 16-bit numbers is exact in float32; K sums, the scale, the
           conversion to powers of two and the subtraction of the maximum add one rounding each)
  weights  p = exp(s) / sum exp(s): each weight and the sum carry a relative error of ds plus a few
           roundings of float32 (exp2 1 step, n additions): dp = 2 ds + (n + 8) e; and each is
           rounded once to the storage type for the second product: u.  In f16 a weight below
           2^-14 has a step of 2^-24 instead, and the sum of weights is at least 1 there.
  output   sum p v, one rounding u of the result:
             |do| <= u |o| + (u + dp) sum p|v| (+ n 2^-24 max|v| in f16)
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
E32 = 2.0 ** -24
ROPE = 64


def rotate(x, start, row, neox):
    """float64: elements [start, start + rd) of x [N, D] rotated by the table row [rd]."""
    y = x.double().clone()
    half = row.shape[0] // 2
    c, s = row[:half].double(), row[half:].double()
    if neox:
        i, j = slice(start, start + half), slice(start + half, start + 2 * half)
    else:
        i, j = slice(start, start + 2 * half, 2), slice(start + 1, start + 2 * half, 2)
    a, b = y[:, i].clone(), y[:, j].clone()
    y[:, i], y[:, j] = a * c - b * s, b * c + a * s
    return y


def softmax_rows(s):
    """exp(s - lse), lse over the last axis; rows of -inf give zeros and -inf."""
    top = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full((*s.shape[:-1], 1), -math.inf,
                                                                   dtype=s.dtype, device=s.device)
    ref = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(s - ref)
    total = e.sum(-1, keepdim=True)
    lse = (ref + torch.log(total)).squeeze(-1)
    return torch.where(total > 0, e / total, torch.zeros_like(e)), lse


def output_bound(p, v, o, ds, u, n, f16):
    """Bound of the attention output's error, elementwise; p [.., n], v [n, d], o [.., d]."""
    dp = 2 * ds + (n + 8) * E32
    b = u * o.abs() + (u + dp)[..., None] * torch.matmul(p, v.abs()) + 2.0 ** -24  # subnormals
    if f16 and n:
        b = b + n * 2.0 ** -24 * v.abs().max()
    return b


def paged_reference(query, cache_rows, lens, counts, scale, latent, dtype):
    """cache_rows: list of [len, latent + 64] tensors; counts: query tokens of each sequence.
    Returns (out, lse, bound of out, bound of lse) in float64."""
    outs, lses, bounds, lbounds = [], [], [], []
    at = 0
    u, f16 = U[dtype], dtype == torch.float16
    for rows, n, c in zip(cache_rows, lens, counts):
        k = rows.double()
        q = query[at:at + c].double()
        at += c
        if c == 0:
            continue
        s = torch.matmul(q, k.t()) * scale  # [c, H, n]
        j = torch.arange(n, device=s.device)
        i = torch.arange(c, device=s.device)
        hidden = j[None, :] > i[:, None] + (n - c)
        s = s.masked_fill(hidden[:, None, :], -math.inf)
        p, lse = softmax_rows(s)
        v = k[:, :latent]
        o = torch.matmul(p, v)
        mag = torch.matmul(q.abs(), k.abs().t()) * abs(scale)
        ds = (k.shape[1] + 4) * E32 * (mag.amax(-1) if n else torch.zeros_like(lse))
        outs.append(o)
        lses.append(lse)
        bounds.append(output_bound(p, v, o, ds, u, n, f16))
        lbounds.append(ds + (n + 8) * E32 + 2 * E32 * torch.where(torch.isinf(lse), 0, lse).abs())
    cat = lambda x: torch.cat(x) if x else torch.empty(0)
    return cat(outs), cat(lses), cat(bounds), cat(lbounds)


def assert_within(got, want, bound, what):
    got = got.double()
    bad = ~((got - want).abs() <= bound) & ~((got == want) | (got.isnan() & want.isnan()))
    if bad.any():
        i = bad.nonzero()[0].tolist()
        err = ((got - want).abs() / bound)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at "
                             f"{i}: got {got[tuple(i)]:.9g}, want {want[tuple(i)]:.9g}, bound "
                             f"{bound[tuple(i)]:.3g}; worst {err[bad].max():.3g} x")


def expanded_reference(q, k, kr, v, scale, causal, dtype, grad=None):
    """One sequence in float64: q [n, H, dim + 64], k, v [m, H, dim], kr [m, 64], grad [n, H, dim].
    Returns a dict of (value, bound) pairs: out, lse and, with grad, dq, dk, dkr, dv.

    Backward bounds, beyond those of the module's head: dp_ij = <g, v_j> and D = <g, o> carry their
    float32 sums' errors and D the output's own error; ds = p (dp - D) is rounded once to the type;
    every gradient is a sum of products in float32, rounded once."""
    u, f16 = U[dtype], dtype == torch.float16
    n, m, h = q.shape[0], k.shape[0], q.shape[1]
    dim = k.shape[2]
    tiny = 2.0 ** -25 if f16 else 0.0
    q, v = q.double().transpose(0, 1), v.double().transpose(0, 1)
    k = torch.cat([k.double(), kr.double()[:, None, :].expand(m, h, ROPE)], dim=-1).transpose(0, 1)
    s = torch.matmul(q, k.transpose(1, 2)) * scale
    if causal:
        i, j = torch.arange(n, device=s.device), torch.arange(m, device=s.device)
        s = s.masked_fill(j[None, :] > i[:, None] + (m - n), -math.inf)
    p, lse = softmax_rows(s)
    o = torch.matmul(p, v)
    mag = torch.matmul(q.abs(), k.abs().transpose(1, 2)) * abs(scale)
    ds = (dim + ROPE + 4) * E32 * (mag.amax(-1) if m else torch.zeros_like(lse))
    ob = output_bound(p, v, o, ds, u, m, f16)
    flat_lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    lb = ds + (m + 8) * E32 + 2 * E32 * flat_lse.abs()
    back = lambda x: x.transpose(0, 1)
    r = {"out": (back(o), back(ob)), "lse": (back(lse), back(lb))}
    if grad is None:
        return r
    g = grad.double().transpose(0, 1)
    dP = torch.matmul(g, v.transpose(1, 2))
    D = (g * o).sum(-1, keepdim=True)
    dS = p * (dP - D)
    dp = (2 * ds + lb + 4 * E32 * flat_lse.abs() + 8 * E32)[..., None]  # weights from the saved lse
    eP = (dim + 4) * E32 * torch.matmul(g.abs(), v.abs().transpose(1, 2))
    eD = (g.abs() * (ob + (dim + 4) * E32 * o.abs())).sum(-1, keepdim=True)
    eS = p * (dp * (dP.abs() + D.abs()) + eP + eD + 4 * E32 * (dP.abs() + D.abs()))
    eS = eS + u * (dS.abs() + eS) + tiny
    sums = lambda a, b, eA, length: (torch.matmul(eA, b.abs()) +
                                     (length + 4) * E32 * torch.matmul(a.abs(), b.abs()))
    dq, eq = torch.matmul(dS, k) * scale, sums(dS, k, eS, m) * abs(scale)
    dSt, pt = dS.transpose(1, 2), p.transpose(1, 2)
    dk, ek = torch.matmul(dSt, q) * scale, sums(dSt, q, eS.transpose(1, 2), n) * abs(scale)
    dv = torch.matmul(pt, g)
    ev = sums(pt, g, ((u + dp) * p + tiny).transpose(1, 2), n)
    final = lambda x, e: (x, e + u * (x.abs() + e) + 2.0 ** -24)
    r["dq"] = final(back(dq), back(eq))
    r["dk"] = final(back(dk[..., :dim]), back(ek[..., :dim]))
    r["dv"] = final(back(dv), back(ev))
    r["dkr"] = final(dk[..., dim:].sum(0), ek[..., dim:].sum(0) + h * E32 * dk[..., dim:].abs().sum(0))
    return r
