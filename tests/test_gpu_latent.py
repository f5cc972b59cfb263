"""GPU: rope_latent_attention and its gradients against the formulas in float64
(tests/attention_ref.py, which derives the bounds) and against differences."""
import math

import pytest
import torch

import rope_partial_inplace_amd as ra
from attention_ref import ROPE, assert_within, expanded_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def randn(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def offsets(lengths, start=0):
    return torch.tensor([start] + (torch.tensor(lengths).cumsum(0) + start).tolist(), device=DEV)


def inputs(nq, nk, heads, dim, dtype, seed, spare=0, spread=1.0):
    """Packed inputs; `spare` rows before the first and behind the last sequence hold NaN."""
    g = gen_of(seed)
    tq, tk = sum(nq) + 2 * spare, sum(nk) + 2 * spare
    q = randn(g, dtype, tq, heads, dim + ROPE) * spread
    kv = randn(g, dtype, tk, heads, 2 * dim)
    kr = randn(g, dtype, tk, ROPE)
    grad = randn(g, dtype, tq, heads, dim)
    if spare:
        for x in (q, kv, kr, grad):
            x[:spare] = float("nan")
            x[-spare:] = float("nan")
    k, v = kv.split([dim, dim], dim=2)
    return q.to(dtype), k, kr, v, grad


NAMES = ("dq", "dk", "dkr", "dv")


def check(nq, nk, heads, dim, dtype, causal, seed=0, spare=2, scale=None, spread=1.0, use_offsets=True):
    q, k, kr, v, grad = inputs(nq, nk, heads, dim, dtype, seed, spare, spread)
    scale = scale if scale is not None else (dim + ROPE) ** -0.5
    where = dict(causal=causal)
    if use_offsets:
        where.update(query_offsets=offsets(nq, spare), key_offsets=offsets(nk, spare))
    else:
        where.update(num_sequences=len(nq))
    out = torch.full((q.shape[0], heads, dim), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((q.shape[0], heads), 7.0, device=DEV)
    ra.rope_latent_attention(q, k, kr, v, scale, out=out, lse=lse, **where)
    grads = ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, scale, **where)
    torch.cuda.synchronize()
    grads = dict(zip(NAMES, grads))
    qa = ka = spare
    for b, (n, m) in enumerate(zip(nq, nk)):
        qs, ks = slice(qa, qa + n), slice(ka, ka + m)
        ref = expanded_reference(q[qs], k[ks], kr[ks], v[ks], scale, causal, dtype, grad[qs])
        got = {"out": out[qs], "lse": lse[qs], "dq": grads["dq"][qs], "dk": grads["dk"][ks],
               "dkr": grads["dkr"][ks], "dv": grads["dv"][ks]}
        for name, (want, bound) in ref.items():
            assert_within(got[name], want, bound, f"sequence {b}: {name}")
        qa, ka = qa + n, ka + m
    if spare:  # rows outside all sequences
        for x in (out, lse):
            assert (x[:spare] == 7).all() and (x[-spare:] == 7).all()
        for name, x in grads.items():
            assert (x[:spare] == 0).all() and (x[-spare:] == 0).all(), name


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,heads", [
    ([1], [1], 1), ([63], [63], 3), ([64, 65], [64, 65], 2), ([127, 1, 130], [127, 1, 130], 2),
    ([1, 40, 200], [300, 41, 500], 3), ([129, 300], [129, 257], 9)])
def test_against_the_formulas(nq, nk, heads, causal, dim, dtype):
    if causal and any(n > m for n, m in zip(nq, nk)):
        nq = [min(n, m) for n, m in zip(nq, nk)]
    check(nq, nk, heads, dim, dtype, causal, seed=heads + dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_sequences_without_queries_or_keys(causal, dim):
    """Empty sequences among others, queries without any key, keys without any query, and causal
    rows before the first key (more queries than keys)."""
    check([0, 5, 0, 200, 70, 1], [0, 0, 130, 66, 70, 0], 3, dim, BF16, causal, seed=2)


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    nk = torch.randint(0, 40, (400,), generator=g).tolist()
    nq = [min(n, int(torch.randint(0, 40, (1,), generator=g))) for n in nk]
    q, k, kr, v, grad = inputs(nq, nk, 2, 64, F16, 3)
    where = dict(query_offsets=offsets(nq), key_offsets=offsets(nk))
    out, lse = ra.rope_latent_attention(q, k, kr, v, 0.1, **where)
    grads = ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, 0.1, **where)
    qa = ka = 0
    for n, m in zip(nq, nk):
        if n and m:
            one = [x.contiguous() for x in (q[qa:qa + n], k[ka:ka + m], kr[ka:ka + m], v[ka:ka + m])]
            o, l = ra.rope_latent_attention(*one, 0.1)
            gr = ra.rope_latent_attention_backward(grad[qa:qa + n], *one, o, l, 0.1)
            assert torch.equal(o, out[qa:qa + n]) and torch.equal(l, lse[qa:qa + n])
            assert torch.equal(gr[0], grads[0][qa:qa + n])
            for a, b in zip(gr[1:], grads[1:]):
                assert torch.equal(a, b[ka:ka + m])
        qa, ka = qa + n, ka + m


@pytest.mark.parametrize("count", [7, 64, 65])
def test_ragged_sequences_of_several_tiles(count):
    """The order in which workgroups take the sequences' tiles (longest first up to 64 sequences)
    reaches each of them once: packed, bit for bit what a call for each sequence gives."""
    g = torch.Generator().manual_seed(count)
    nk = torch.randint(0, 700, (count,), generator=g).tolist()
    nk[1], nk[-1] = 0, 1000
    nq = [n if i % 3 else n // 4 for i, n in enumerate(nk)]
    q, k, kr, v, grad = inputs(nq, nk, 3, 64, BF16, count)
    where = dict(query_offsets=offsets(nq), key_offsets=offsets(nk))
    out = torch.full((sum(nq), 3, 64), float("nan"), dtype=BF16, device=DEV)
    out, lse = ra.rope_latent_attention(q, k, kr, v, 0.1, out=out, **where)
    grads = ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, 0.1, **where)
    qa = ka = 0
    for n, m in zip(nq, nk):
        if n:
            one = [x.contiguous() for x in (q[qa:qa + n], k[ka:ka + m], kr[ka:ka + m], v[ka:ka + m])]
            o, l = ra.rope_latent_attention(*one, 0.1)
            gr = ra.rope_latent_attention_backward(grad[qa:qa + n], *one, o, l, 0.1)
            assert torch.equal(o, out[qa:qa + n]) and torch.equal(l, lse[qa:qa + n])
            for i, b in enumerate(grads):
                at = slice(qa, qa + n) if i == 0 else slice(ka, ka + m)
                assert torch.equal(gr[i], b[at]), (n, m, i)
        qa, ka = qa + n, ka + m


def test_equal_sequences_without_offsets():
    check([130] * 3, [200] * 3, 4, 128, BF16, True, seed=5, spare=0, use_offsets=False)
    check([1] * 5, [77] * 5, 4, 64, F16, False, seed=6, spare=0, use_offsets=False)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30])
def test_other_scales(scale):
    check([100, 7], [150, 7], 2, 64, BF16, True, seed=3, scale=scale)
    check([70], [200], 2, 128, F16, False, seed=4, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_large_scores_and_a_rising_maximum(dtype):
    """Scores of +-100 and more (weights down to zero), and keys ordered so that the running
    maximum rises from tile to tile."""
    check([300], [300], 2, 128, dtype, True, seed=7, spread=8.0)
    q, k, kr, v, grad = inputs([200], [700], 1, 64, dtype, 8)
    ramp = torch.linspace(-1, 1, 700, device=DEV)[:, None, None]
    k = (q[:1, :, :64].float() * ramp + k.float() * 0.1).to(dtype)
    q = (q[:1].float() + q.float() * 0.1).to(dtype)
    out, lse = ra.rope_latent_attention(q, k, kr, v, 0.5)
    grads = dict(zip(NAMES, ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, 0.5)))
    for name, (want, bound) in expanded_reference(q, k, kr, v, 0.5, True, dtype, grad).items():
        assert_within({"out": out, "lse": lse, **grads}[name], want, bound, name)


def test_non_finite_values_stay_in_their_sequence():
    nq = nk = [70, 130, 65]
    q, k, kr, v, grad = inputs(nq, nk, 2, 64, BF16, 9)
    where = dict(query_offsets=offsets(nq), key_offsets=offsets(nk))

    def both(*x):
        o, l = ra.rope_latent_attention(*x, 0.1, **where)
        return (o, l, *ra.rope_latent_attention_backward(grad, *x, o, l, 0.1, **where))

    clean = both(q, k, kr, v)
    for i, value in enumerate((float("nan"), float("inf"), -float("inf"))):
        x = [t.clone() for t in (q, k, kr, v)]
        x[i + 1][70 + 129].view(-1)[0] = value  # the middle sequence's last key
        got = both(*x)
        for a, b in zip(got, clean):
            assert torch.equal(a[:70], b[:70]) and torch.equal(a[200:], b[200:])
        assert not torch.isfinite(got[0][199]).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gradients_against_differences(dtype):
    """<gradient, d> against (L(x + e d) - L(x - e d)) / 2e of the loss L = <grad, out> computed
    in float64, for a direction d in each input."""
    n, m, heads, dim, scale = 37, 61, 3, 64, 0.1
    q, k, kr, v, grad = inputs([n], [m], heads, dim, dtype, 4)
    x = [t.clone().requires_grad_() for t in (q, k, kr, v)]
    out = ra.latent_attention(*x, scale)
    got = torch.autograd.grad(out, x, grad)
    bounds = expanded_reference(q, k, kr, v, scale, True, dtype, grad)

    def loss(*t):
        kk = torch.cat([t[1], t[2][:, None, :].expand(m, heads, ROPE)], dim=-1)
        s = torch.einsum("ihd,jhd->hij", t[0], kk) * scale
        hidden = torch.ones(n, m, dtype=torch.bool, device=DEV).triu(m - n + 1)
        p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
        return (torch.einsum("hij,jhd->ihd", p, t[3]) * grad.double()).sum()

    base = [t.double() for t in (q, k, kr, v)]
    g = gen_of(12)
    for i, name in enumerate(NAMES):
        d = torch.randn(base[i].shape, generator=g, device=DEV, dtype=torch.float64)
        up = [t + 1e-5 * d if j == i else t for j, t in enumerate(base)]
        down = [t - 1e-5 * d if j == i else t for j, t in enumerate(base)]
        slope = float(loss(*up) - loss(*down)) / 2e-5
        along = float((got[i].double() * d).sum())
        allowed = float((bounds[name][1] * d.abs()).sum()) + 1e-6 * abs(slope)
        assert abs(along - slope) <= allowed, (name, along, slope, allowed)


def test_autograd_layouts_and_unused_rows():
    """Gradients that arrive expanded or transposed, packed rows outside the sequences, inputs
    that are views of one projection, and a second backward pass."""
    nq = [50, 14]
    q, k, kr, v, _ = inputs(nq, nq, 2, 64, BF16, 10)
    kv = torch.cat([k, v], dim=2).requires_grad_()
    q, kr = q.clone().requires_grad_(), kr.clone().requires_grad_()
    off = offsets([40, 14])  # the last 10 rows belong to no sequence
    out = ra.latent_attention(q, kv[..., :64], kr, kv[..., 64:], 0.1, query_offsets=off,
                              key_offsets=off)
    assert (out[54:] == 0).all()
    one = torch.autograd.grad(out.sum(), (q, kv, kr), retain_graph=True)
    two = torch.autograd.grad(out, (q, kv, kr), torch.ones_like(out))
    for a, b in zip(one, two):
        assert torch.equal(a, b) and (a[54:] == 0).all()
    o2, l2 = ra.rope_latent_attention(q.detach(), kv.detach()[..., :64], kr.detach(),
                                      kv.detach()[..., 64:], 0.1, query_offsets=off, key_offsets=off)
    assert torch.equal(o2[:54], out[:54])


def test_gradients_without_heads_or_sequences_are_zero():
    q, k, kr, v, grad = inputs([40], [70], 2, 64, BF16, 11)
    none = torch.zeros(1, dtype=torch.int64, device=DEV)
    lse = torch.zeros(40, 2, device=DEV)
    torch.full((1 << 20,), float("nan"), device=DEV)  # freed again: new tensors find it
    grads = ra.rope_latent_attention_backward(grad, q, k, kr, v, grad, lse, 0.1,
                                              query_offsets=none, key_offsets=none)
    assert all((x == 0).all() for x in grads)
    torch.full((1 << 20,), float("nan"), device=DEV)
    grads = ra.rope_latent_attention_backward(*(x[:, :0] for x in (grad, q, k)), kr,
                                              *(x[:, :0] for x in (v, grad, lse)), 0.1)
    assert (grads[2] == 0).all() and all(grads[i].numel() == 0 for i in (0, 1, 3))


def test_autograd_takes_gradients_off_alignment_and_refuses_a_second_order():
    q, k, kr, v, grad = inputs([30], [30], 2, 64, BF16, 12)
    x = [t.clone().requires_grad_() for t in (q, k, kr, v)]
    odd = torch.zeros(3, dtype=BF16, device=DEV, requires_grad=True)
    out = ra.latent_attention(*x, 0.1)
    joined = torch.cat([odd, out.reshape(-1)])  # out's gradient begins 6 bytes into its memory
    one = torch.autograd.grad(joined, x, torch.cat([odd.detach(), grad.reshape(-1)]))
    two = torch.autograd.grad(ra.latent_attention(*x, 0.1), x, grad)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    first = torch.autograd.grad(ra.latent_attention(*x, 0.1).float().pow(2).sum(), x,
                                create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first[0].float().sum(), x)


def test_repeats_streams_and_graph_replays():
    """Bit-identical repeats, on another stream too; a captured forward and backward replayed with
    new inputs, eager work in between."""
    q, k, kr, v, grad = inputs([300, 77], [300, 99], 4, 128, BF16, 13)
    where = dict(query_offsets=offsets([300, 77]), key_offsets=offsets([300, 99]))

    def both(stream=None):
        o, l = ra.rope_latent_attention(q, k, kr, v, 0.08, stream=stream, **where)
        return (o, l, *ra.rope_latent_attention_backward(grad, q, k, kr, v, o, l, 0.08,
                                                         stream=stream, **where))

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (None, side, side.cuda_stream):
        again = both(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    g = gen_of(14)
    for i in range(4):
        q.copy_(randn(g, BF16, *q.shape))
        grad.copy_(randn(g, BF16, *grad.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in held]
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {i}"


def test_captured_autograd_step_replays():
    """Forward and backward through autograd inside one capture."""
    q, k, kr, v, grad = inputs([100], [100], 2, 64, F16, 15)
    x = [t.clone().requires_grad_() for t in (q, k, kr, v)]

    def step():
        return torch.autograd.grad(ra.latent_attention(*x, 0.1), x, grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        with torch.no_grad():
            x[0].copy_(randn(gen_of(20 + i), F16, *q.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), f"replay {i}"


def test_expanded_and_absorbed_forms_agree():
    """The same attention both ways: keys and values expanded from latent rows by W_k and W_v, and
    the absorbed query q W_k against the rows themselves, its output times W_v.  Compared in the
    expanded form's terms, with the extra rounding of the expanded keys, values and absorbed
    query."""
    g = gen_of(21)
    heads, dim, latent, n, m = 4, 64, 128, 5, 150
    c = randn(g, BF16, m, latent)
    kr = randn(g, BF16, m, ROPE)
    wk, wv = (randn(g, F16, heads, latent, dim).double() * latent ** -0.5 for _ in range(2))
    q = randn(g, BF16, n, heads, dim + ROPE)
    scale = (dim + ROPE) ** -0.5
    k = torch.einsum("jl,hld->jhd", c.double(), wk).to(BF16)
    v = torch.einsum("jl,hld->jhd", c.double(), wv).to(BF16)
    exp_out, exp_lse = ra.rope_latent_attention(q, k, kr, v, scale)
    qa = torch.cat([torch.einsum("ihd,hld->ihl", q[..., :dim].double(), wk).to(BF16),
                    q[..., dim:]], dim=-1)
    cache = torch.zeros(10, 16, latent + ROPE, dtype=BF16, device=DEV)
    cache.view(-1, latent + ROPE)[:m] = torch.cat([c, kr], dim=1)
    out, lse = ra.rope_latent_attention_paged(qa, cache, torch.arange(10, device=DEV)[None],
                                              torch.tensor([m], device=DEV), latent, scale)
    absorbed = torch.einsum("ihl,hld->ihd", out.double(), wv)
    # keys (or the absorbed query) off by half a step each: scores by at most u sum |q||k| on
    # either side; values by u |v|; the absorbed output by u |o| through W_v
    u = 2.0 ** -8
    ref = expanded_reference(q, k, kr, v, scale, True, BF16)
    dS = 2 * u * scale * (torch.einsum("ihd,jhd->hij", q[..., :dim].double().abs(),
                                       k.double().abs()).amax((0, 2))
                          + torch.einsum("ihl,jl->hij", qa[..., :latent].double().abs(),
                                         c.double().abs()).amax((0, 2)))[:, None, None]
    vmax = v.double().abs().amax()
    allowed = (2 * dS + 4 * u) * vmax + 2 * u * torch.einsum("ihl,hld->ihd", out.double().abs(), wv.abs())
    assert ((absorbed - exp_out.double()).abs() <= allowed + ref["out"][1]).all()
    assert ((lse - exp_lse).abs() <= dS[..., 0] + ref["lse"][1]).all()
