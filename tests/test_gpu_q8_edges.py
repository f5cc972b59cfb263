"""GPU: single cases of the 8-bit cache's calls where they once went wrong."""
import math

import pytest
import torch

import rope_partial_inplace_amd as ra
from q8_ref import E4M3, I8, quantized_cache, rows_of
from test_gpu_q8_append import BF16, DEV, F16, F32, RAGGED, append, same, setup

pytestmark = pytest.mark.gpu


# ---- append: values of width 0 -----------------------------------------------------------------------

@pytest.mark.parametrize("codes", [I8, E4M3])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F16, 128), (F32, 30)])
@pytest.mark.parametrize("page,block", [(16, 16), (16, 4), (64, 64), (1, 1)])
def test_append_of_keys_alone(page, block, dtype, D, neox, codes):
    """As with values for keys and queries; the values' scales are those of top = 0."""
    size = dict(page=page, block=block, N=3, D=D, codes=codes, dtype=dtype)
    want, got = (setup(*RAGGED, Dv=Dv, **size) for Dv in (8, 0))
    for n in ("q", "k", "kc", "ks", "vs", "pos", "table"):
        got[n] = want[n].clone()
    vs = got["vs"].cpu().clone()
    q, w = append(got, neox=neox), append(want, neox=neox)
    torch.cuda.synchronize()
    same(q, w, "query")
    same(got["kc"], want["kc"], "kc")
    same(got["ks"], want["ks"], "ks")
    table = got["table"].tolist()
    for b, (n, m) in enumerate(zip(*RAGGED)):
        for t in range(max(n - m, 0), n):
            if t == max(n - m, 0) or t % block == 0:
                where = table[b][t // page], t % page // block
                old = vs[where] if t % block else torch.zeros(3)
                vs[where] = old.clamp_min(2.0 ** -120)
    same(got["vs"], vs, "vs")


# ---- fork: what dimension 1 of a cache means ---------------------------------------------------------

PAGE = 16
# what a cache is, its shape behind the pages, its type, and the part of a page x that n of its tokens are
LISTED = [("rows", (PAGE, 2, 24), BF16, lambda x, n: x[:n]),
          ("as many heads as rows", (PAGE, PAGE, 8), I8, lambda x, n: x[:n]),
          ("blocks of 4", (4, 3), F32, lambda x, n: x[:-(-n // 4)]),
          ("heads outermost", (8, PAGE, 64), BF16, lambda x, n: x[:, :n]),
          ("two heads outermost, codes", (2, PAGE, 128), E4M3, lambda x, n: x[:, :n]),
          ("more heads than rows", (32, PAGE, 16), I8, lambda x, n: x[:, :n]),
          ("keys and values", (2, PAGE * 40), F16, lambda x, n: x.view(2, PAGE, 40)[:, :n]),
          ("scales by head", (8,), F32, lambda x, n: x),
          ("scales of keys and values by head", (2, 1, 8), F32, lambda x, n: x)]
WHOLE = [("as many heads as rows, outermost", (PAGE, PAGE, 8), I8, lambda x, n: x[:, :n]),
         ("scales by head and token", (8, PAGE), F32, lambda x, n: x[:, :n]),
         ("scales of keys and values", (2, 8), F32, lambda x, n: x),
         ("rows", (PAGE, 40), F16, lambda x, n: x[:n])]


@pytest.mark.parametrize("listed", [True, False])
@pytest.mark.parametrize("tail", [1, 3, 8, 15])
def test_fork_copies_the_tokens_of_every_layout(tail, listed):
    """Each new row has its parent's tokens in all caches, by what the caches are."""
    g = torch.Generator(device=DEV).manual_seed(tail)
    ints = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)
    P, kinds = 24, LISTED if listed else WHOLE
    caches = [torch.randint(1, 100, (P, *shape), generator=g, device=DEV, dtype=torch.int8).to(dtype)
              for _, shape, dtype, _ in kinds]
    table, lens = [[5, 9, -1], [7, 2, 11], [3, -1, -1]], [PAGE + tail, 3 * PAGE, tail]
    refs = [0] * P
    for row in table:
        for q in row:
            if q >= 0:
                refs[q] += 1
    parents = [0, 0, 1, 2, 0, 2]
    handle = ra.PageCaches(caches) if listed else ra.PageCaches([], whole=caches)
    before = [x.clone() for x in caches]
    new, new_lens, _, short = ra.rope_fork_pages(ints(table), ints(lens), ints(parents), ints(refs), PAGE, handle)
    torch.cuda.synchronize()
    assert short.tolist() == [0] and new_lens.tolist() == [lens[p] for p in parents]
    new = new.tolist()
    assert len({r[-(-lens[p] // PAGE) - 1] for r, p in zip(new, parents) if lens[p] % PAGE}) == 5
    for (what, _, _, tokens), x, was in zip(kinds, caches, before):
        for row, p in zip(new, parents):
            for j in range(-(-lens[p] // PAGE)):
                n = min(PAGE, lens[p] - j * PAGE)
                a, b = (tokens(y, n).float() for y in (x[row[j]], was[table[p][j]]))
                assert torch.equal(a, b), (what, n)


# ---- attention: what a query does not see ------------------------------------------------------------

def packed(dtype, codes, D, heads, group, lens, counts, page, block, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n_pages = [-(-n // page) for n in lens]
    table = torch.zeros(len(lens), max(n_pages), dtype=torch.int64, device=DEV)
    order, at = torch.randperm(sum(n_pages), generator=g, device=DEV), 0
    for b, c in enumerate(n_pages):
        table[b, :c] = order[at:at + c]
        at += c
    kc, ks = quantized_cache(g, codes, sum(n_pages), page, block, heads, D)
    vc, vs = quantized_cache(g, codes, sum(n_pages), page, block, heads, D)
    q = torch.randn((sum(counts), heads * group, D), generator=g, device=DEV).to(dtype)
    ints = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)
    offsets = ints([0] + torch.tensor(counts).cumsum(0).tolist())
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=ints(lens), offsets=offsets)


def attend(s, **other):
    s = {**s, **other}
    out, lse = ra.rope_attention_paged_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"],
                                          s["q"].shape[2] ** -0.5, query_offsets=s["offsets"])
    torch.cuda.synchronize()
    return out, lse


# rows of a key head: 16, 32, and the kernel for more
ROWS = [(4, [4, 3, 4]), (8, [2, 1, 2]), (4, [8, 5, 8]), (16, [2, 2, 2]), (4, [40, 37, 70]), (1, [150, 200, 33])]
PLACES = [(16, 16), (16, 4), (16, 1), (64, 2), (5, 5), (5, 1)]  # page, block: scales of runs, of tokens; any page


@pytest.mark.parametrize("page,block", PLACES)
@pytest.mark.parametrize("group,counts", ROWS)
@pytest.mark.parametrize("dtype,codes,D", [(F16, I8, 128), (F16, E4M3, 64), (F16, E4M3, 256), (BF16, I8, 128)])
def test_scales_of_later_tokens_reach_no_query(dtype, codes, D, group, counts, page, block):
    """Values' scales of blocks that a query does not see, infinite or 2^40 times as large: not one bit of its
    output changes."""
    lens = [c + n for c, n in zip(counts, (203, 330, 64))]
    s = packed(dtype, codes, D, 2, group, lens, counts, page, block)
    want, want_lse = attend(s)
    touched = 0
    for factor in (math.inf, 2.0 ** 40):
        for back in (1, 2, 5):  # the poisoned block is that of the back-th token from the end
            vs = s["vs"].clone()
            same = torch.ones(sum(counts), dtype=torch.bool, device=DEV)
            at = 0
            for b, (n, c) in enumerate(zip(lens, counts)):
                begin = max(0, n - back) // block * block
                vs[s["table"][b, begin // page], begin % page // block] *= factor
                for i in range(c):
                    same[at + i] = n - c + 1 + i <= begin
                at += c
            out, lse = attend(s, vs=vs)
            assert torch.equal(lse, want_lse)
            assert torch.equal(out[same], want[same]), (factor, back)
            assert not torch.equal(out[~same], want[~same])
            touched += int(same.sum())
    assert touched > 0 or block == 16


@pytest.mark.parametrize("page,block", [(16, 4), (16, 1), (5, 1)])
@pytest.mark.parametrize("group,count", [(4, 4), (4, 8), (4, 60)])
@pytest.mark.parametrize("codes", [I8, E4M3])
def test_float16_beside_growing_scales(codes, group, count, page, block):
    """Values' scales that grow 2^30 fold over a sequence's last tokens: every query is within the bound (q8_ref.py)
    that the scales it sees give."""
    n, D, heads = 197 + count, 64, 2
    s = packed(F16, codes, D, heads, group, [n], [count], page, block, seed=3)
    t = torch.arange(n, device=DEV)
    where, row = s["table"][0][t // page], t % page // block
    grown = (t // block - (n - count) // block).clamp_min(0)
    grown = (grown * 30.0 / grown.max()).round()
    s["vs"].fill_(2.0 ** -24)
    s["vs"][where, row] = (2.0 ** (grown - 24))[:, None].expand(-1, heads)
    out, lse = attend(s)
    kc, kf = rows_of(s["kc"], s["ks"], s["table"][0], n)
    vc, vf = rows_of(s["vc"], s["vs"], s["table"][0], n)
    scale, u, e = D ** -0.5, 2.0 ** -11, 2.0 ** -24
    for i in range(count):
        m = n - count + 1 + i
        for h in range(heads * group):
            k = h // group
            q = s["q"][i, h].double()
            logits = (kc[:m, k] @ q) * kf[:m, k] * scale
            mag = ((kc[:m, k].abs() @ q.abs()) * kf[:m, k] * scale).max()
            v = vc[:m, k] * vf[:m, k, None]
            p = torch.softmax(logits, 0)
            ds = (D + 8) * e * mag
            dp = 2 * ds + (m + 10) * e
            want = p @ v
            bound = (u * want.abs() + (u + dp) * (p @ v.abs()) + 2.0 ** -25 +
                     m * 2.0 ** -35 * vf[:m, k].max() * vc[:m, k].abs().max())
            assert bool(((out[i, h].double() - want).abs() <= bound).all()), (i, h)
            assert abs(lse[i, h].double() - logits.logsumexp(0)) <= ds + (m + 10) * e + 4 * e * logits.abs().max()


def nan_where_seen(s, want, poisoned, lens, counts, block, D):
    """(mask of the output's elements that a NaN code of the values reaches) for poisoned (sequence, token, head,
    element) quadruples."""
    heads = s["kc"].shape[2]
    group = s["q"].shape[1] // heads
    reach = torch.zeros_like(want, dtype=torch.bool)
    for b, token, h, d in poisoned:
        at = sum(counts[:b])
        for i in range(counts[b]):
            if token < lens[b] - counts[b] + 1 + i:
                reach[at + i, h * group:(h + 1) * group, d] = True
    return reach


@pytest.mark.parametrize("page,block", PLACES)
@pytest.mark.parametrize("group,counts", ROWS)
@pytest.mark.parametrize("dtype,D", [(F16, 128), (BF16, 64), (BF16, 128), (BF16, 256), (F16, 256)])
def test_nan_codes_of_later_tokens_reach_no_query(dtype, D, group, counts, page, block):
    """Values' codes that are NaN: those elements of the queries that see the token are NaN, and not one bit of
    anything else changes."""
    lens = [c + n for c, n in zip(counts, (203, 330, 64))]
    s = packed(dtype, E4M3, D, 2, group, lens, counts, page, block, seed=5)
    want, want_lse = attend(s)
    for backs in ([1], [2], [5, 1], list(range(1, 9)), [70]):
        poisoned = [(b, n - back, (b + back) % 2, d) for b, n in enumerate(lens) for back in backs
                    if back <= n for d in ((7 * back) % D, D - 1 - back % D, (13 * back + b) % D)]
        vc = s["vc"].clone()
        raw = vc.view(torch.uint8)
        for k, (b, t, h, d) in enumerate(poisoned):
            raw[s["table"][b, t // page], t % page, h, d] = 0x7f | (k & 1) << 7
        out, lse = attend(s, vc=vc)
        reach = nan_where_seen(s, want, poisoned, lens, counts, block, D)
        assert torch.equal(lse, want_lse)
        assert bool(torch.isnan(out[reach]).all()) and bool(reach.any()), backs
        assert torch.equal(out[~reach], want[~reach]), backs


@pytest.mark.parametrize("group,count", [(4, 4), (4, 8), (4, 50)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_one_bad_value_of_a_piece(bad, dtype, group, count):
    """A non-finite value element, appended and attended to with the queries before and behind it."""
    n, D, at = 150 + count, 128, count // 2
    s = packed(dtype, E4M3, D, 2, group, [n], [count], 16, 16, seed=7)
    g = torch.Generator(device=DEV).manual_seed(8)
    k, v = (torch.randn((count, 2, D), generator=g, device=DEV).to(dtype) for _ in range(2))
    cs = torch.cat([torch.ones(300, 32, device=DEV), torch.zeros(300, 32, device=DEV)], 1).to(dtype)
    results = []
    for x in (0.0, bad):
        v[at, 1, 77] = x
        c = {m: s[m].clone() for m in ("kc", "vc", "ks", "vs")}
        ra.rope_append_paged_cache_q8(torch.arange(n - count, n, device=DEV), k, v, c["kc"], c["vc"], c["ks"], c["vs"],
                                      s["table"], s["lens"], cs)
        results.append(attend(s, **c)[0])
    clean, out = results
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[at:, group:, 77] = True
    assert bool(torch.isnan(out[hit]).all()) and torch.equal(out[~hit], clean[~hit])


def test_whole_pages_of_other_orders():
    """Copies, forks and compactions of caches given as `whole`, whose pages are dense in another order."""
    g = torch.Generator(device=DEV).manual_seed(2)
    ints = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)
    base = [torch.randint(0, 100, (12, PAGE, 3, 8), generator=g, device=DEV, dtype=torch.int8),
            torch.rand((12, 2, PAGE, 4), generator=g, device=DEV)]
    views = [base[0].permute(0, 3, 1, 2), base[1][:, 1], base[1][:, 0].transpose(1, 2)]
    handle = ra.PageCaches([], whole=views)
    want = [x.clone() for x in base]

    def move(pairs):
        was = [w.clone() for w in want]
        for w, x in zip(want, was):
            for a, b in pairs:
                w[b] = x[a]

    ra.rope_copy_pages(ints([3, 5]), ints([4, 9]), handle)
    move([(3, 4), (5, 9)])
    # pages 6 and 2 of one sequence, whose tail is copied to page 0
    refs = [0, 1, 1, 1, 1, 1, 1, 0, 0, 0, 1, 0]
    rows, lens, counts, _ = ra.rope_fork_pages(ints([[6, 2]]), ints([PAGE + 3]), ints([0, 0]), ints(refs), PAGE, handle)
    move([(2, 0)])
    assert rows.tolist() == [[6, 2], [6, 0]]
    rows, counts, _, live = ra.rope_compact_pages(rows, counts, handle)
    move([(10, 7)])
    assert live.tolist() == [8] and rows.tolist() == [[6, 2], [6, 0]]
    torch.cuda.synchronize()
    for x, w in zip(base, want):
        assert torch.equal(x, w)
