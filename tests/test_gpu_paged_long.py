"""GPU: sharp checks of paged latent attention over long contexts.  Error bounds grow with the length
until they would let a lost row pass, so here the result depends on single rows: the same rows in
pages of different sizes give the same bits (the order of the sums is that of the lengths), and a key
that holds all the weight has to come out, wherever it lies."""
import pytest
import torch

import rope_partial_inplace_amd as ra
from attention_ref import ROPE

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def pages_of(rows, page, gen):
    """A cache that holds rows [n, width] in scattered pages of `page`, and its page table."""
    n, width = rows.shape
    count = -(-n // page)
    order = torch.randperm(count, generator=gen, device=DEV)
    cache = torch.full((count * page, width), float("nan"), dtype=rows.dtype, device=DEV)
    cache[:n] = rows
    placed = torch.empty(count, page, width, dtype=rows.dtype, device=DEV)
    placed[order] = cache.view(count, page, width)
    return placed, order


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("heads,latent", [(16, 512), (128, 512), (40, 128)])
@pytest.mark.parametrize("n", [20000, 40001])
def test_page_sizes_give_the_same_bits(n, heads, latent, dtype):
    """512 page places are held at a time: pages of 1 are refilled every 512 rows, of 5 every 2560,
    of 7 every 3584."""
    gen = torch.Generator(device=DEV).manual_seed(n + heads)
    lens = [n, 700, n // 3]
    rows = [torch.randn(m, latent + ROPE, generator=gen, device=DEV).to(dtype) for m in lens]
    q = torch.randn(3, heads, latent + ROPE, generator=gen, device=DEV).to(dtype)
    sl = torch.tensor(lens, device=DEV)
    first = None
    for page in (64, 1, 5, 7, 100, 4096):
        caches, tables, at = [], [], 0
        for r in rows:
            c, t = pages_of(r, page, gen)
            caches.append(c)
            tables.append(t + at)
            at += len(t)
        table = torch.zeros(3, max(map(len, tables)), dtype=torch.int64, device=DEV)
        for b, t in enumerate(tables):
            table[b, :len(t)] = t
        got = ra.rope_latent_attention_paged(q, torch.cat(caches), table, sl, latent, 0.05)
        if first is None:
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), page


@pytest.mark.parametrize("heads,latent", [(16, 512), (128, 512), (64, 256), (20, 128)])
@pytest.mark.parametrize("n,page", [(40001, 1), (40001, 64), (9999, 5), (2049, 16)])
def test_a_single_key_with_all_the_weight_comes_out(n, page, heads, latent):
    """Each query of a batch over the same context looks for one row: its score leads the others by
    more than 60 powers of two, so out is the row's latent part, exactly (its weight is 1 but for
    roundings of the score in float32, far below a step of the type).  Rows at the ends of tiles,
    of refills of the page places, and at and around every cut between the shares that clusters of
    workgroups take."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    rows = torch.randn(n, latent + ROPE, generator=gen, device=DEV).to(BF16)
    # a row's tail is a code of its number, +-1 for each of 32 bits (twice): another row's product
    # with it is smaller by 4 or more
    number = torch.arange(n, device=DEV) * 2654435761 % (1 << 32)
    bits = ((number[:, None] >> torch.arange(32, device=DEV)) & 1) * 2 - 1
    rows[:, latent:] = torch.cat([bits, bits], 1).to(BF16)
    cache, table = pages_of(rows, page, gen)
    tables = table[None]
    steps = -(-n // 64)
    at = {0, 1, 63, 64, 65, n // 2, n - 1, n - 2, n - 65, n // 64 * 64 - 1}
    for refill in range(0, n, 512 * page):
        at |= {refill - 1, refill, refill + 63, refill - 64}
    # cuts: the steps and the two that beginning an item costs, in even shares
    for groups in (256, 128):
        share = -(-(steps + 2) // groups)
        for g in range(1, groups):
            at |= {(g * share - 2) * 64 + d for d in (-1, 0, 63, 64)}
    at = torch.tensor(sorted(a for a in at if 0 <= a < n), device=DEV)
    sl = torch.tensor([n], device=DEV)
    for part in at.split(heads):
        q = torch.zeros(1, heads, latent + ROPE, dtype=BF16, device=DEV)
        q[0, :len(part), latent:] = rows[part, latent:]
        out, lse = ra.rope_latent_attention_paged(q, cache, tables, sl, latent, 12.0)
        assert torch.equal(out[0, :len(part)], rows[part, :latent]), part.tolist()
        # 64 * 12 in float32 powers of two: a few roundings of 1108, below 2^-13 each
        assert ((lse[0, :len(part)] - 64 * 12.0).abs() < 2.0 ** -10).all()
