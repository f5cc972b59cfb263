"""GPU: precision of latent attention where ordinary random data does not show it: keys and values
with a common offset, small and large gradients, weights far below the largest.

Bounds.  u is half a step of the storage type relative to a value (bf16 2^-8, f16 2^-11), e = 2^-24
half a step of float32.  A sum of n terms each of which was rounded on its own, by at most u
relative, is off by sum_j r_j x_j with |r_j| <= u.  Taken as independent with mean zero, Hoeffding's
inequality bounds that by T u sqrt(sum_j x_j^2) but for a probability of 2 exp(-T^2 / 2), 3e-8 with
T = 6 (elements: below 10^6 a call).  Errors of float32 are bounded at their worst:
  scores   (dim + 68) e scale sum |q||k|                                              =: a
  weights  p = exp(s - lse), relative: 2 a + (m + 16) e + 4 e |lse|                   =: r
  dP       (dim + 4) e sum |g||v|                                                     =: b
  D        sum_j p (r |dP| + b) + (m + 8) e sum_j p |dP|, D = sum_j p dP in float32   =: c
  ds       p (r (|dP| + |D|) + b + c + 4 e (|dP| + |D|)) before its rounding           =: f
A gradient then is off by
  T u sqrt(sum (ds k)^2) + sum f |k| + (n + 4) e sum |ds||k|, times scale, and its own rounding.
What is rounded to float16 is scaled by a power of two first, so that a value down to 2^-20 of the
largest of its sum keeps its bits; smaller ones are off by at most 2^-32 of that."""
import math

import pytest
import torch

import rope_partial_inplace_amd as ra
from attention_ref import ROPE, U, assert_within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16
E, T = 2.0 ** -24, 6.0
NAMES = ("dq", "dk", "dkr", "dv")


def randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def gradients_reference(q, k, kr, v, g, scale, causal, dtype):
    """(value, bound) of dq, dk, dkr and dv of one sequence, in float64."""
    u = U[dtype]
    step = 2.0 ** -25 if dtype == F16 else 0.0  # half a step of the smallest results
    n, m, h, dim = q.shape[0], k.shape[0], k.shape[1], k.shape[2]
    q, v, g = (x.double().transpose(0, 1) for x in (q, v, g))
    kr = kr.double()[:, None, :].expand(m, h, ROPE)
    k = torch.cat([k.double(), kr], dim=-1).transpose(0, 1).contiguous()
    s = torch.matmul(q, k.transpose(1, 2).contiguous()) * scale
    if causal:
        i, j = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
        s = s.masked_fill(j[None, :] > i[:, None] + (m - n), -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - lse)
    vt = v.transpose(1, 2).contiguous()
    dP = torch.matmul(g, vt)
    D = (p * dP).sum(-1, keepdim=True)
    dS = p * (dP - D)
    a = (dim + 68) * E * abs(scale) * torch.matmul(q.abs(), k.abs().transpose(1, 2).contiguous())
    r = 2 * a.amax(-1, keepdim=True) + (m + 16) * E + 4 * E * lse.abs()
    b = (dim + 4) * E * torch.matmul(g.abs(), vt.abs())
    c = (p * (r * dP.abs() + b)).sum(-1, keepdim=True) + (m + 8) * E * (p * dP.abs()).sum(-1, keepdim=True)
    f = p * (r * (dP.abs() + D.abs()) + b + c + 4 * E * (dP.abs() + D.abs()))
    low = 2.0 ** -32 if dtype == F16 else 0.0

    def product(x, err, y, length):
        """x y and its bound: x [h, a, length] rounded to the type, y [h, length, b]."""
        least = low * x.abs().amax(-1, keepdim=True) * y.abs().sum(-2, keepdim=True)
        bound = (T * u * torch.sqrt(torch.matmul(x * x, y * y)) + torch.matmul(err, y.abs()) +
                 (length + 4) * E * torch.matmul(x.abs(), y.abs()) + least)
        return torch.matmul(x, y), bound

    def final(x, e):
        return x, e + torch.clamp(u * (x.abs() + e), min=step) + 2.0 ** -130

    turned = lambda x: x.transpose(1, 2).contiguous()
    back = lambda x: x.transpose(0, 1)
    dq, eq = product(dS, f, k, m)
    dk, ek = product(turned(dS), turned(f), q, n)
    dv, ev = product(turned(p), turned(r * p), g, n)
    dq, eq, dk, ek = dq * scale, eq * abs(scale), dk * scale, ek * abs(scale)
    dkr, ekr = dk[..., dim:].sum(0), ek[..., dim:].sum(0) + h * E * dk[..., dim:].abs().sum(0)
    return {"dq": final(back(dq), back(eq)), "dk": final(back(dk[..., :dim]), back(ek[..., :dim])),
            "dkr": final(dkr, ekr), "dv": final(back(dv), back(ev))}


def check_gradients(q, k, kr, v, g, scale, causal, dtype):
    out, lse = ra.rope_latent_attention(q, k, kr, v, scale, causal)
    got = dict(zip(NAMES, ra.rope_latent_attention_backward(g, q, k, kr, v, out, lse, scale, causal)))
    torch.cuda.synchronize()
    for name, (want, bound) in gradients_reference(q, k, kr, v, g, scale, causal, dtype).items():
        assert_within(got[name], want, bound, name)


def data(gen, n, m, heads, dim, dtype, wide=1.0, small=1.0):
    """Inputs with keys `wide` times as large and queries that much smaller, gradients `small`
    times as large."""
    q, k, v = randn(gen, n, heads, dim + ROPE) / wide, randn(gen, m, heads, dim) * wide, randn(gen, m, heads, dim)
    kr, g = randn(gen, m, ROPE) * wide, randn(gen, n, heads, dim) * small
    return [x.to(dtype) for x in (q, k, kr, v, g)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,m,dim,causal", [(200, 2048, 128, False), (300, 1000, 64, True),
                                            (1100, 1100, 128, True), (70, 129, 64, False)])
@pytest.mark.parametrize("offset", [1.0, 3.0])
def test_gradients_of_keys_and_values_with_a_common_offset(offset, n, m, dim, causal, dtype):
    """Biased projections: every channel of keys, shared key parts and values has an offset of its
    own.  An error of D = sum_j p_j dP_j then reaches dq through sum_j p_j k_j, which no longer
    averages out (D from the rounded output: dq off by 5% of its norm at an offset of 1, by 45% at 3)."""
    g = gen_of(31)
    q, k, kr, v, grad = data(g, n, m, 2, dim, torch.float32)
    k, kr, v = k + offset * randn(g, 2, dim), kr + offset * randn(g, ROPE), v + offset * randn(g, 2, dim)
    check_gradients(*(x.to(dtype) for x in (q, k, kr, v, grad)), (dim + ROPE) ** -0.5, causal, dtype)


@pytest.mark.parametrize("small", [1e-1, 1e-3, 1e-4])
@pytest.mark.parametrize("wide", [8.0, 1 / 8])
@pytest.mark.parametrize("n,m,dim,causal", [(150, 2048, 128, False), (2048, 150, 64, False),
                                            (900, 900, 64, True)])
def test_float16_gradients_of_any_size(n, m, dim, causal, wide, small):
    """Small incoming gradients over long rows: p (dP - D) lies far below float16's normal range
    while the gradients do not."""
    check_gradients(*data(gen_of(32), n, m, 1, dim, F16, wide, small), (dim + ROPE) ** -0.5, causal, F16)


def test_float16_gradients_of_very_different_rows():
    """One row's gradient is 10^5 times the others'; keys that only the others see keep theirs."""
    q, k, kr, v, g = data(gen_of(33), 400, 400, 2, 128, torch.float32, 1.0, 1e-3)
    g[5] *= 1e5
    g[300:] *= 1e-1
    check_gradients(*(x.to(F16) for x in (q, k, kr, v, g)), 192 ** -0.5, True, F16)


def test_float16_gradients_whose_inner_values_pass_the_type():
    """|p (dP - D)| beyond 65504 with finite gradients."""
    gen = torch.Generator().manual_seed(LARGE_SEED)
    q, k, kr, v, g = large_data(gen)
    assert inner_and_results(q, k, kr, v, g)[0] > 66000
    check_gradients(*(x.to(DEV) for x in (q, k, kr, v, g)), 192 ** -0.5, True, F16)


LARGE_SEED = 45


def large_data(gen):
    r = lambda *shape: torch.randn(shape, generator=gen)
    return [x.to(F16) for x in (r(8, 1, 192), r(8, 1, 128), r(8, ROPE), r(8, 1, 128), r(8, 1, 128) * 8000)]


def inner_and_results(q, k, kr, v, g):
    """Largest |p (dP - D)|, and the largest gradient (float64, on the CPU)."""
    q, k, kr, v, g = (x.double() for x in (q[:, 0], k[:, 0], kr, v[:, 0], g[:, 0]))
    kk = torch.cat([k, kr], 1)
    s = (q @ kk.T * 192 ** -0.5).masked_fill(torch.ones(8, 8, dtype=torch.bool).triu(1), -math.inf)
    p = s.softmax(1)
    dP = g @ v.T
    dS = p * (dP - (p * dP).sum(1, keepdim=True))
    return (float(dS.abs().max()),
            max(float(x.abs().max()) for x in (dS @ kk * 192 ** -0.5, dS.T @ q * 192 ** -0.5, p.T @ g)))


@pytest.mark.parametrize("dim", [64, 128])
def test_float16_value_gradients_of_long_rows(dim):
    """Weights of 2^-19: dv is a sum of p g."""
    check_gradients(*data(gen_of(34), 8, 1 << 19, 1, dim, F16, 1.0, 100.0), (dim + ROPE) ** -0.5, False, F16)


def tail_scores(gen, m):
    """Scores (in powers of two) of one key at 0 and of the others near -23.5."""
    s = -23.5 + 0.4 * randn(gen, m)
    s[m // 3] = 0.0
    return s


def check_tail(out, lse, s, v):
    """One head: scores s [m] (natural), values v [m, d] of which the leading key's are zero.  Each
    weight keeps a relative error of half a step."""
    p = torch.exp(s - torch.logsumexp(s, 0))
    want = p @ v
    assert_within(lse.reshape(1), torch.logsumexp(s, 0).reshape(1), torch.full((1,), 2e-5, device=DEV, dtype=torch.float64), "lse")
    bound = (2 * U[F16] + 1e-3 * U[F16] + len(s) * E) * (p @ v.abs()) + 2.0 ** -25
    assert_within(out.reshape(-1), want, bound, "out")


def test_float16_weights_far_below_the_largest():
    """One key leads with weight near 1 and a value of zero; the result is the sum of many weights
    of 2^-23.5, which float16 holds with two bits at most."""
    g = gen_of(35)
    m, scale = 40000, 1.0
    goal = tail_scores(g, m) * math.log(2)
    v = (1 + 0.1 * randn(g, m, 128)) * 8
    v[m // 3] = 0
    # scores from two elements of the shared part, the second holding what the first rounds away
    kr = torch.zeros(m, ROPE, device=DEV)
    kr[:, 0] = goal.to(F16)
    kr[:, 1] = (goal - kr[:, 0]) * 1024
    q = torch.zeros(1, 1, 128 + ROPE, device=DEV)
    q[..., 128], q[..., 129] = 1, 1 / 1024
    q, kr, v = q.to(F16), kr.to(F16), v.to(F16)
    s = kr[:, 0].double() + kr[:, 1].double() / 1024
    out, lse = ra.rope_latent_attention(q, torch.zeros(m, 1, 128, dtype=F16, device=DEV), kr,
                                        v[:, None], scale)
    check_tail(out, lse, s, v.double())
    cache = torch.cat([v, kr], dim=1).reshape(-1, 64, 192)
    q[..., :128] = 0
    for heads in (1, 40):  # 32 and 64 rows a workgroup
        out, lse = ra.rope_latent_attention_paged(q.expand(1, heads, -1).contiguous(), cache,
                                                  torch.arange(m // 64, device=DEV)[None],
                                                  torch.tensor([m], device=DEV), 128, scale)
        for h in (0, heads - 1):
            check_tail(out[0, h], lse[0, h], s, v.double())


@pytest.mark.parametrize("causal", [True, False])
def test_scale_zero_with_large_scores(causal):
    """Scale 0: every visible key has the same weight, whatever the products."""
    g = gen_of(36)
    q, k, kr, v, grad = data(g, 40, 40, 1, 128, BF16)
    q, k, kr = ((x.float() * 1e17).to(BF16) for x in (q, k, kr))
    out, lse = ra.rope_latent_attention(q, k, kr, v, 0.0, causal)
    seen = torch.arange(1, 41, device=DEV) if causal else torch.full((40,), 40, device=DEV)
    mean = v[:, 0].double().cumsum(0) / seen[:, None] if causal else v[:, 0].double().mean(0).expand(40, -1)
    size = v[:, 0].double().abs().mean() * 8
    assert_within(lse[:, 0], seen.double().log(), torch.full((40,), 1e-5, device=DEV), "lse")
    assert ((out[:, 0].double() - mean).abs() <= 2.0 ** -7 * size).all()
    dq, dk, dkr, dv = ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, 0.0, causal)
    assert (dq == 0).all() and (dk == 0).all() and (dkr == 0).all()
    share = grad[:, 0].double() / seen[:, None]
    want = share.flip(0).cumsum(0).flip(0) if causal else share.sum(0).expand(40, -1)
    assert ((dv[:, 0].double() - want).abs() <= 2.0 ** -7 * share.abs().sum(0)).all()
    cache = torch.cat([(v[:, 0].float() * 1e17).to(BF16), kr], dim=1).reshape(1, 40, 192)
    out, lse = ra.rope_latent_attention_paged(q[-1:], cache, torch.zeros(1, 1, dtype=torch.int64, device=DEV),
                                              torch.tensor([40], device=DEV), 128, 0.0)
    assert abs(float(lse) - math.log(40)) < 1e-5
    assert ((out[0, 0].double() / 1e17 - cache[0, :, :128].double().mean(0) / 1e17).abs() <= 2.0 ** -7 * size).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_float16_non_finite_values_stay_in_their_sequence(value):
    """The factors that float16's p and ds are held with are a row's or a key's own.  A gradient that
    is not finite (a loss scaled too far) makes gradients of its sequence that are not."""
    from test_gpu_latent import inputs, offsets
    nq = nk = [70, 130, 65]
    q, k, kr, v, grad = inputs(nq, nk, 2, 64, F16, 9)
    where = dict(query_offsets=offsets(nq), key_offsets=offsets(nk))

    def both(q, k, kr, v, g):
        o, l = ra.rope_latent_attention(q, k, kr, v, 0.1, **where)
        return (o, l, *ra.rope_latent_attention_backward(g, q, k, kr, v, o, l, 0.1, **where))

    clean = both(q, k, kr, v, grad)
    for i in range(5):
        x = [t.clone() for t in (q, k, kr, v, grad)]
        x[i][70 + 129].view(-1)[0] = value  # the middle sequence's last token
        got = both(*x)
        for a, b in zip(got, clean):
            assert torch.equal(a[:70], b[:70]) and torch.equal(a[200:], b[200:])
        if i == 4:
            assert all(not torch.isfinite(t).all() for t in got[2:])
