"""GPU: packed calls of latent attention over more sequences than a wavefront has lanes, bit for bit
what calls over 64 of the sequences at a time give (their tiles are found in another way)."""
import pytest
import torch

import rope_partial_inplace_amd as ra
from test_gpu_latent import BF16, DEV, inputs, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [65, 128, 4096, 4097, 9000])
@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences_as_in_calls_of_64(causal, count):
    g = torch.Generator().manual_seed(count)
    nk = torch.randint(0, 4, (count,), generator=g)
    nk[::97] = torch.randint(100, 300, (len(nk[::97]),), generator=g)  # several tiles
    nk[40:50] = 0
    nk[-3:] = torch.tensor([257, 0, 128])
    nq = torch.where(torch.arange(count) % 3 == 0, nk // 2, nk)
    nk, nq = nk.tolist(), nq.tolist()
    spare = 3  # rows of no sequence in front and behind
    q, k, kr, v, grad = inputs(nq, nk, 2, 64, BF16, count, spare)
    qo, ko = offsets(nq, spare), offsets(nk, spare)

    def both(qo, ko):
        out = torch.zeros(q.shape[0], 2, 64, dtype=BF16, device=DEV)
        lse = torch.zeros(q.shape[0], 2, device=DEV)
        where = dict(causal=causal, query_offsets=qo, key_offsets=ko)
        ra.rope_latent_attention(q, k, kr, v, 0.1, out=out, lse=lse, **where)
        return out, lse, *ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, 0.1, **where)

    got = both(qo, ko)
    for b in range(0, count, 64):
        e = min(count, b + 64)
        part = both(qo[b:e + 1], ko[b:e + 1])
        qs, ks = slice(int(qo[b]), int(qo[e])), slice(int(ko[b]), int(ko[e]))
        for i, (x, y) in enumerate(zip(got, part)):
            at = qs if i < 3 else ks
            assert torch.equal(x[at], y[at]), (b, i)
    for x in got:
        assert (x[:spare] == 0).all() and (x[-spare:] == 0).all()


@pytest.mark.parametrize("count", [3, 70])
def test_offsets_out_of_range_are_clamped(count):
    """As with the clamped values, bit for bit; gradients of every token come out."""
    n = [5] * count
    q, k, kr, v, grad = inputs(n, n, 2, 64, BF16, count)
    fixed = offsets(n)
    bad = fixed.clone()
    bad[0], bad[-1] = -(2 ** 62), 2 ** 62
    got = []
    for off in (fixed, bad):
        where = dict(query_offsets=off, key_offsets=off)
        out, lse = ra.rope_latent_attention(q, k, kr, v, 0.1, **where)
        got.append((out, lse, *ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, 0.1, **where)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("count", [6, 80])
def test_descending_offsets_write_no_rows_outside(count):
    """Results are not defined where offsets descend; rows of no sequence stay as they are."""
    n = [9] * count
    q, k, kr, v, grad = inputs(n, n, 2, 64, BF16, count, spare=4)
    for place, by in ((-2, 14), (2, 9), (count // 2, -200), (3, 1 << 40)):
        off = offsets(n, 4)
        off[place] -= by
        off.clamp_(4, 4 + 9 * count)
        out = torch.full((q.shape[0], 2, 64), 7.0, dtype=BF16, device=DEV)
        lse = torch.full((q.shape[0], 2), 7.0, device=DEV)
        ra.rope_latent_attention(q, k, kr, v, 0.1, out=out, lse=lse, query_offsets=off, key_offsets=off)
        for x in (out, lse):
            assert (x[:4] == 7).all() and (x[-4:] == 7).all()
        ra.rope_latent_attention_backward(grad, q, k, kr, v, out, lse, 0.1, query_offsets=off,
                                          key_offsets=off)
