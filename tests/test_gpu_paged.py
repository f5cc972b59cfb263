"""GPU: rope_append_paged_cache and rope_latent_attention_paged against plain float64 forms
(tests/attention_ref.py, which derives the bounds), and the two together."""
import math

import pytest
import torch

import rope_partial_inplace_amd as ra
import rope_workloads as W
from attention_ref import ROPE, U, assert_within, paged_reference, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def randn(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---- append -----------------------------------------------------------------------------------

def check_append(T, nq, nk, D, Dv, rd, dtype, neox, page, q_start=0, k_start=0, seed=0,
                 pages=None, layout="rows", in_place=False, skip=(), table_pad=0, view=False):
    g = gen_of(seed)
    pages = pages or -(-T // page) + 2
    pos = torch.randint(0, 300, (T,), generator=g, device=DEV)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].clone()
    for t, s in skip:
        slots[t] = s
    table = W.cos_sin_cache(300, rd, dtype).to(DEV)
    if table_pad:
        table = torch.cat([table, randn(g, dtype, 300, table_pad)], dim=1)[:, :rd]
    if view:  # columns of one projection
        full = randn(g, dtype, T, nq * D + nk * D + nk * Dv)
        q, k, v = full.split([nq * D, nk * D, nk * Dv], dim=1)
        q, k, v = q.unflatten(1, (nq, D)), k.unflatten(1, (nk, D)), v.unflatten(1, (nk, Dv))
    else:
        q, k, v = (randn(g, dtype, T, n, d) for n, d in ((nq, D), (nk, D), (nk, Dv)))
    if layout == "rows":
        kc, vc = randn(g, dtype, pages, page, nk, D), randn(g, dtype, pages, page, nk, Dv)
    elif layout == "heads":  # heads before rows
        kc = randn(g, dtype, pages, nk, page, D).transpose(1, 2)
        vc = randn(g, dtype, pages, nk, page, Dv).transpose(1, 2)
    else:  # one allocation, keys and values of a page side by side
        both = randn(g, dtype, pages, 2, page, nk, D)
        kc, vc = both[:, 0], both[:, 1]
    q0, k0, v0, kc0, vc0 = (x.clone() for x in (q, k, v, kc, vc))
    out = ra.rope_append_paged_cache(pos, slots, k, kc, table, value=v if Dv else None,
                                     value_cache=vc if Dv else None, query=q if nq else None,
                                     query_out=q if in_place else None, query_rot_start=q_start,
                                     key_rot_start=k_start, is_neox_style=neox)
    torch.cuda.synchronize()
    assert torch.equal(k, k0) and torch.equal(v, v0)
    want_k, want_v = kc0.clone(), vc0.clone()
    # two products and a sum, each rounded to float32, then one rounding to the type
    u = U[dtype] if dtype != F32 else 0.0
    for t in range(T):
        row = table[int(pos[t])]
        rows = [("key", k0[t], k_start)] + ([("query", q0[t], q_start)] if nq else [])
        for name, x, start in rows:
            want = rotate(x, start, row, neox)
            mag = x.double().abs().amax(1, keepdim=True) * 2
            if name == "query":
                got = out[t]
            else:
                s = int(slots[t])
                if not 0 <= s < pages * page:
                    continue
                got = kc[s // page, s % page]
                want_k[s // page, s % page] = got
            assert_within(got, want, u * want.abs() + 3 * 2.0 ** -24 * mag + 2.0 ** -25,
                          f"{name} of token {t}")
            keep = torch.ones(D, dtype=torch.bool, device=DEV)
            keep[start:start + rd] = False
            assert torch.equal(got[:, keep], x[:, keep]), f"{name} of token {t}: outside the slice"
        s = int(slots[t])
        if 0 <= s < pages * page:
            want_v[s // page, s % page] = v0[t]
    assert torch.equal(kc, want_k), "key cache: rows of other slots changed"
    if Dv:
        assert torch.equal(vc, want_v), "value cache"
    else:
        assert torch.equal(vc, vc0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("T,nq,nk,D,Dv,rd,page", [
    (1, 4, 1, 64, 64, 64, 16), (7, 32, 8, 128, 128, 128, 16), (33, 6, 2, 128, 64, 64, 1),
    (5, 3, 3, 96, 32, 32, 100)])
def test_append(T, nq, nk, D, Dv, rd, page, neox, dtype):
    check_append(T, nq, nk, D, Dv, rd, dtype, neox, page, seed=T)


@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("kw", [
    dict(D=576, Dv=0, rd=64, nk=1, q_start=512, k_start=512),    # a latent row with its tail
    dict(D=192, Dv=128, rd=64, nk=2, q_start=128, k_start=128),
    dict(D=50, Dv=7, rd=10, nk=2, q_start=3, k_start=5),         # nothing aligned: by elements
    dict(D=64, Dv=64, rd=64, nk=2, table_pad=3),                 # unaligned table rows
    dict(D=64, Dv=64, rd=32, nk=2, layout="heads"),
    dict(D=64, Dv=64, rd=64, nk=2, layout="pairs"),
    dict(D=64, Dv=64, rd=48, nk=2, q_start=16, in_place=True),
    dict(D=64, Dv=64, rd=64, nk=2, view=True, in_place=True),    # in place inside a projection
    dict(D=64, Dv=64, rd=64, nk=2, view=True, nq=0),
    dict(D=64, Dv=64, rd=64, nk=2, skip=((0, -1), (3, 10 ** 6), (4, -2 ** 62), (6, 2 ** 62)))],
    ids=lambda kw: "_".join(f"{a}{b}" for a, b in kw.items() if a not in ("skip",))[:60])
def test_append_layouts(kw, neox):
    check_append(**{**dict(T=9, nq=3, dtype=BF16, neox=neox, page=4, seed=5), **kw})


def test_append_out_of_range_positions_are_clamped():
    g = gen_of(3)
    table = W.cos_sin_cache(50, 64, BF16).to(DEV)
    k = randn(g, BF16, 3, 1, 64)
    pos = torch.tensor([-5, 10 ** 12, 7], device=DEV)
    slots = torch.arange(3, device=DEV)
    a, b = (torch.zeros(1, 4, 1, 64, dtype=BF16, device=DEV) for _ in range(2))
    ra.rope_append_paged_cache(pos, slots, k, a, table)
    ra.rope_append_paged_cache(pos.clamp(0, 49), slots, k, b, table)
    assert torch.equal(a, b)


def test_append_past_32_bit_offsets():
    """Rows of a cache of 5 GiB, addressed beyond 2^32 bytes and beyond 2^31 elements."""
    pages, page, D = 40000, 64, 1024
    kc = torch.zeros(pages, page, 1, D, dtype=BF16, device=DEV)
    g = gen_of(1)
    k = randn(g, BF16, 4, 1, D)
    slots = torch.tensor([pages * page - 1, 0, pages * page // 2 + 3, 33_554_432 // 16], device=DEV)
    pos = torch.zeros(4, dtype=torch.int64, device=DEV)
    table = W.cos_sin_cache(1, 64, BF16).to(DEV)  # position 0: no turn
    ra.rope_append_paged_cache(pos, slots, k, kc, table)
    flat = kc.view(-1, 1, D)
    assert torch.equal(flat[slots], k)
    assert int((flat != 0).any(-1).sum()) == 4


# ---- absorbed attention -----------------------------------------------------------------------

def paged_inputs(lens, counts, heads, latent, dtype, page, seed, extra_rows=0, spread=1.0):
    g = gen_of(seed)
    row = latent + ROPE
    need = [-(-n // page) for n in lens]
    cache = randn(g, dtype, max(1, sum(need)) + 2, page, row)
    order = torch.randperm(cache.shape[0], generator=g, device=DEV)
    table = torch.zeros(len(lens), max(1, max(need, default=1)), dtype=torch.int64, device=DEV)
    at, rows = 0, []
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        rows.append(cache[table[b, :c]].reshape(-1, row)[:lens[b]].clone())
        at += c
    # what lies past a sequence's end in its last page, and in pages of no one, is never used
    used = torch.zeros(cache.shape[:2], dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        for j in range(need[b]):
            used[table[b, j], :min(page, n - j * page)] = True
    cache[~used] = float("nan")
    query = randn(g, dtype, sum(counts) + extra_rows, heads, row) * spread
    return query.to(dtype), cache, table, torch.tensor(lens, device=DEV), rows


def check_paged(lens, counts, heads, latent, dtype, page, seed=0, scale=None, spread=1.0):
    extra = 3
    q, cache, table, sl, rows = paged_inputs(lens, counts, heads, latent, dtype, page, seed, extra,
                                             spread)
    scale = scale if scale is not None else 192 ** -0.5
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), device=DEV)
    T = sum(counts)
    out = torch.full((T + extra, heads, latent), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((T + extra, heads), 7.0, device=DEV)
    ra.rope_latent_attention_paged(q, cache, table, sl, latent, scale, query_offsets=off, out=out,
                                   lse=lse)
    torch.cuda.synchronize()
    want, wl, bound, lbound = paged_reference(q, rows, lens, counts, scale, latent, dtype)
    assert (out[T:] == 7).all() and (lse[T:] == 7).all(), "rows behind the last sequence"
    assert_within(lse[:T], wl, lbound, "lse")
    assert_within(out[:T], want, bound, "out")
    return out[:T]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("lens,counts,heads,page", [
    ([1], [1], 1, 16), ([63], [1], 16, 64), ([64], [1], 32, 64), ([65], [1], 33, 16),
    ([1000], [1], 16, 100), ([130, 1, 700, 64], [1, 1, 1, 1], 64, 16),
    ([129, 257], [1, 1], 128, 64), ([300, 5, 77], [4, 5, 2], 16, 1),
    ([200, 90], [40, 7], 20, 64)])
def test_paged_attention(lens, counts, heads, page, latent, dtype):
    check_paged(lens, counts, heads, latent, dtype, page, seed=len(lens) + heads)


@pytest.mark.parametrize("heads", [8, 48, 128])
def test_paged_sequences_without_rows_or_queries(heads):
    """No cached token, no query, more queries than cached tokens (the first ones see nothing)."""
    out = check_paged([0, 70, 3, 0, 129, 64], [2, 0, 5, 0, 1, 1], heads, 512, BF16, 16, seed=4)
    assert (out[:2] == 0).all() and (out[2:4] == 0).all()


def test_paged_many_ragged_sequences():
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 900, (300,), generator=g).tolist()
    counts = torch.randint(0, 3, (300,), generator=g).tolist()
    for heads, latent in ((16, 128), (40, 256), (128, 512)):
        first = check_paged(lens, counts, heads, latent, F16, 16, seed=9)
        for _ in range(5):
            assert torch.equal(first, check_paged(lens, counts, heads, latent, F16, 16, seed=9))


def test_paged_more_sequences_than_threads():
    """More sequences than a workgroup has threads, many of them without rows or queries, and
    offsets that descend behind the first 512."""
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 60, (1100,), generator=g).tolist()
    counts = torch.randint(0, 3, (1100,), generator=g).tolist()
    check_paged(lens, counts, 16, 128, F16, 16, seed=9)
    q, cache, table, sl, _ = paged_inputs(lens, counts, 16, 128, F16, 16, 9)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), device=DEV)
    off[900] += 5
    out = torch.full((q.shape[0], 16, 128), 3.0, dtype=F16, device=DEV)
    ra.rope_latent_attention_paged(q, cache, table, sl, 128, 0.1, query_offsets=off, out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("heads", [16, 128])
def test_paged_long_context(heads):
    """One sequence shared out over every compute unit, in pages of one token (whose numbers
    pass through LDS in several pieces) and of 64."""
    for page in (1, 64):
        check_paged([40001], [1], heads, 512, BF16, page, seed=2)


def test_paged_rising_and_falling_scores():
    """Scores whose maximum keeps rising along the sequence, and large ones: the running maximum
    is raised many times, and weights span the whole range of the type."""
    for dtype in (BF16, F16):
        lens, heads, latent = [2000], 16, 128
        q, cache, table, sl, rows = paged_inputs(lens, [1], heads, latent, dtype, 64, 3)
        ramp = torch.linspace(0, 3, 2048, device=DEV)
        for b in range(table.shape[1]):
            r = cache[table[0, b]]
            r[...] = torch.where(r.isnan(), r, (r.float() * 0.2 + q[0, 0].float()[None, :] *
                                                ramp[b * 64:(b + 1) * 64, None]).to(dtype))
        rows = [cache[table[0]].reshape(-1, latent + ROPE)[:2000].clone()]
        out, lse = ra.rope_latent_attention_paged(q, cache, table, sl, latent, 0.3)
        want, wl, bound, lb = paged_reference(q, rows, lens, [1], 0.3, latent, dtype)
        assert_within(lse, wl, lb, "lse")
        assert_within(out, want, bound, "out")


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30])
def test_paged_other_scales(scale):
    check_paged([300, 5, 77], [1, 2, 1], 16, 128, BF16, 16, seed=5, scale=scale)


def test_paged_without_offsets_and_strided_views():
    lens, heads, latent = [100, 260, 31], 12, 256
    q, cache, table, sl, rows = paged_inputs(lens, [2, 2, 2], heads, latent, BF16, 16, 8)
    wide = torch.zeros(6, heads, latent + ROPE + 16, dtype=BF16, device=DEV)
    wide[..., :latent + ROPE] = q
    spaced = torch.full((cache.shape[0], 16, 2, latent + ROPE), float("nan"), dtype=BF16, device=DEV)
    spaced[:, :, 0] = cache
    tt = torch.zeros(table.shape[1], 3, dtype=torch.int64, device=DEV).copy_(table.t()).t()
    assert not tt.is_contiguous()
    l2 = torch.zeros(3, 2, dtype=torch.int64, device=DEV)
    l2[:, 0] = sl
    a = ra.rope_latent_attention_paged(wide[..., :latent + ROPE], spaced[:, :, 0], tt, l2[:, 0],
                                       latent, 0.07)
    want, wl, bound, lb = paged_reference(q, rows, lens, [2, 2, 2], 0.07, latent, BF16)
    assert_within(a[0], want, bound, "out")
    assert_within(a[1], wl, lb, "lse")
    b = ra.rope_latent_attention_paged(q, cache[:, :, None], table, sl, latent, 0.07)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_paged_bad_pages_lengths_and_offsets_stay_inside():
    """Device data out of range is clamped: finite results of some rows, nothing faults."""
    lens, heads, latent = [100, 50], 16, 128
    q, cache, table, sl, _ = paged_inputs(lens, [1, 1], heads, latent, BF16, 16, 1)
    cache = torch.nan_to_num(cache)
    bad = table.clone()
    bad[0, 1], bad[0, 2], bad[1, 0] = -7, 10 ** 15, 2 ** 62
    fixed = bad.clamp(0, cache.shape[0] - 1)
    a = ra.rope_latent_attention_paged(q, cache, bad, sl, latent, 0.1)
    b = ra.rope_latent_attention_paged(q, cache, fixed, sl, latent, 0.1)
    assert torch.equal(a[0], b[0])
    cap = table.shape[1] * 16
    a = ra.rope_latent_attention_paged(q, cache, fixed, torch.tensor([10 ** 14, -3], device=DEV),
                                       latent, 0.1)
    b = ra.rope_latent_attention_paged(q, cache, fixed, torch.tensor([cap, 0], device=DEV), latent,
                                       0.1)
    assert torch.equal(a[0], b[0]) and (a[0][1] == 0).all()
    off = torch.tensor([-4, 1, 10 ** 10], device=DEV)
    a = ra.rope_latent_attention_paged(q, cache, fixed, sl, latent, 0.1, query_offsets=off)
    b = ra.rope_latent_attention_paged(q, cache, fixed, sl, latent, 0.1,
                                       query_offsets=torch.tensor([0, 1, 2], device=DEV))
    assert torch.equal(a[0], b[0])


def test_paged_descending_offsets_write_nothing():
    q, cache, table, sl, _ = paged_inputs([100, 50, 70], [2, 1, 1], 16, 128, BF16, 16, 1)
    for off in ([0, 4, 0, 4], [3, 2, 4, 4], [0, 1, 4, 3]):
        out = torch.full((4, 16, 128), 3.0, dtype=BF16, device=DEV)
        lse = torch.full((4, 16), 3.0, device=DEV)
        ra.rope_latent_attention_paged(q, cache, table, sl, 128, 0.1, out=out, lse=lse,
                                       query_offsets=torch.tensor(off, device=DEV))
        assert (out == 3).all() and (lse == 3).all()


def test_paged_repeats_are_identical():
    q, cache, table, sl, _ = paged_inputs([5000, 100, 3000], [1, 1, 1], 32, 512, BF16, 64, 6)
    first = ra.rope_latent_attention_paged(q, cache, table, sl, 512, 0.07)
    for _ in range(5):
        again = ra.rope_latent_attention_paged(q, cache, table, sl, 512, 0.07)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("page", [1, 5, 64])
def test_paged_past_32_bit_offsets(page):
    """A cache of 4.5 GiB whose used pages are scattered over all of it (neighbouring tokens of a
    sequence 2 GiB and more apart)."""
    latent, row_bytes, n = 512, 1152, 250
    pages = (9 << 29) // (row_bytes * page)
    cache = torch.zeros(pages, page, latent + ROPE, dtype=BF16, device=DEV)
    g = gen_of(2)
    need = -(-n // page)
    table = torch.randperm(pages, generator=g, device=DEV)[:need]
    table[0], table[-1] = pages - 1, 0
    cache[table] = randn(g, BF16, need, page, latent + ROPE)
    rows = [cache[table].reshape(-1, latent + ROPE)[:n]]
    q = randn(g, BF16, 1, 16, latent + ROPE)
    out, lse = ra.rope_latent_attention_paged(q, cache, table[None], torch.tensor([n], device=DEV),
                                              latent, 0.07)
    want, wl, bound, lb = paged_reference(q, rows, [n], [1], 0.07, latent, BF16)
    assert_within(out, want, bound, "out")
    assert_within(lse, wl, lb, "lse")


# ---- together ---------------------------------------------------------------------------------

def decode_step(q, k, pos, slots, table_cs, cache, q_full, page_table, lens):
    q_full[..., 512:] = 0
    ra.rope_append_paged_cache(pos, slots, k, cache, table_cs, query=q, query_out=q_full[..., 512:],
                               key_rot_start=512, is_neox_style=False)
    return ra.rope_latent_attention_paged(q_full, cache, page_table, lens, 512, 192 ** -0.5)


def decode_state(B=5, heads=16, page=16, seed=0):
    g = gen_of(seed)
    lens = torch.tensor([33, 1, 100, 64, 17][:B], device=DEV)  # the new token included
    need = [-(-int(n) // page) for n in lens]
    cache = torch.zeros(sum(need), page, 1, 576, dtype=BF16, device=DEV)
    table = torch.zeros(B, max(need), dtype=torch.int64, device=DEV)
    at = 0
    for b in range(B):
        table[b, :need[b]] = torch.arange(at, at + need[b], device=DEV)
        at += need[b]
    cs = W.cos_sin_cache(200, 64, BF16).to(DEV)
    return g, lens, cache, table, cs


def test_prompt_then_decoding_steps():
    """Prompts appended to the cache, then steps that append one token a sequence and attend,
    checked against rotating and attending in float64."""
    g, lens, cache, table, cs = decode_state()
    B, heads, page = 5, 16, 16
    rows = []
    for b in range(B):  # the prompt: everything but the last two tokens
        n = max(0, int(lens[b]) - 2)
        k = randn(g, BF16, n, 1, 576)
        pos = torch.arange(n, device=DEV)
        slots = table[b, pos // page] * page + pos % page
        ra.rope_append_paged_cache(pos, slots, k, cache, cs, key_rot_start=512, is_neox_style=False)
        rows.append([rotate(k[t], 512, cs[t], False)[0].to(BF16) for t in range(n)])
    for back in (1, 0):
        now = (lens - back).clamp(min=1)
        pos = now - 1
        slots = table[torch.arange(B, device=DEV), pos // page] * page + pos % page
        k, q = randn(g, BF16, B, 1, 576), randn(g, BF16, B, heads, 64)
        q_full = randn(g, BF16, B, heads, 576)
        out, lse = decode_step(q, k, pos, slots, cs, cache, q_full, table, now)
        for b in range(B):
            rows[b] = rows[b][:int(pos[b])] + [rotate(k[b], 512, cs[int(pos[b])], False)[0].to(BF16)]
            want_q = rotate(q[b], 0, cs[int(pos[b])], False)
            assert_within(q_full[b, :, 512:], want_q, 2.0 ** -8 * want_q.abs() + 1e-5, "query")
        ref = [torch.stack(r) for r in rows]
        want, wl, bound, lb = paged_reference(q_full, ref, now.tolist(), [1] * B, 192 ** -0.5, 512,
                                              BF16)
        # the cached rows may differ from the reference's by a rounding at ties
        assert_within(out, want, bound * 2, "out")
        assert_within(lse, wl, lb + 0.02, "lse")


def test_captured_decoding_step_replays():
    """A captured step (append and attention) replayed with new contents in its inputs, eager work
    in between, each replay against the eager result."""
    g, lens, cache, table, cs = decode_state(seed=3)
    B, heads, page = 5, 16, 16
    torch.nan_to_num_(cache)
    cache.copy_(randn(g, BF16, *cache.shape))
    pos = lens - 1
    slots = table[torch.arange(B, device=DEV), pos // page] * page + pos % page
    k, q = randn(g, BF16, B, 1, 576), randn(g, BF16, B, heads, 64)
    q_full = randn(g, BF16, B, heads, 576)
    now = lens.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        decode_step(q, k, pos, slots, cs, cache, q_full, table, now)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = decode_step(q, k, pos, slots, cs, cache, q_full, table, now)
    for i in range(4):
        k.copy_(randn(g, BF16, B, 1, 576))
        q.copy_(randn(g, BF16, B, heads, 64))
        if i == 2:
            now.copy_(torch.tensor([20, 1, 100, 5, 17], device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), cache.clone(), q_full.clone()
        eager = decode_step(q, k, pos, slots, cs, cache, q_full, table, now)
        torch.cuda.synchronize()
        for a, b in zip(got, (*eager, cache, q_full)):
            assert torch.equal(a, b), f"replay {i}"


def test_streams_given_and_current():
    """Calls on a stream that is not the current one, two at once, against the same calls alone."""
    q, cache, table, sl, _ = paged_inputs([3000, 700], [1, 1], 16, 512, BF16, 64, 11)
    q2 = randn(gen_of(5), BF16, *q.shape)
    want = [ra.rope_latent_attention_paged(x, cache, table, sl, 512, 0.07) for x in (q, q2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [ra.rope_latent_attention_paged(x, cache, table, sl, 512, 0.07, stream=s)
               for x, s in zip((q, q2), streams)]
        got3 = ra.rope_latent_attention_paged(q, cache, table, sl, 512, 0.07,
                                              stream=streams[0].cuda_stream)
        torch.cuda.synchronize()
        for a, b in zip(got + [got3], want + [want[0]]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
