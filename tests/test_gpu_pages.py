"""GPU: rope_copy_pages, rope_fork_pages and rope_compact_pages against lists on the host."""
import random

import pytest
import torch

import rope_partial_inplace_amd as ra
from q8_ref import compact_reference, fork_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def pool(gen, pages, dtype, *shape):
    x = torch.randint(0, 256, (pages, *shape, torch.empty(0, dtype=dtype).element_size()),
                      generator=gen, device=DEV, dtype=torch.uint8)
    return x.flatten(-2).view(dtype).view(pages, *shape)


def raw(x):
    return x.contiguous().view(torch.uint8)


def layers(gen, pages, page, kinds):
    """Caches of several kinds: rows first, heads first, scales, odd sizes, keys beside values."""
    out = []
    for k in kinds:
        if k == "kv":
            both = pool(gen, pages, torch.bfloat16, 2, page, 2, 24)
            out += [both[:, 0], both[:, 1]]
        elif k == "heads":
            out.append(pool(gen, pages, torch.int8, 3, page, 16).transpose(1, 2))
        elif k == "scales":
            out.append(pool(gen, pages, torch.float32, max(1, page // 4), 3))
        elif k == "odd":
            out.append(pool(gen, pages, torch.int8, page, 7, 3))
        elif k == "wide":
            out.append(pool(gen, pages, torch.float8_e4m3fn, page, 8, 128))
        elif k == "vector":
            out.append(pool(gen, pages, torch.int64))
        elif k == "off":  # two bytes off every larger boundary
            out.append(pool(gen, pages, torch.float16, page * 6 + 1)[:, 1:].view(pages, page, 6))
    return out


KINDS = ["kv", "heads", "scales", "odd", "wide", "vector", "off"]


@pytest.mark.parametrize("page", [1, 4, 16, 33])
@pytest.mark.parametrize("kinds", [["wide"], KINDS, ["wide"] * 100 + ["scales"] * 100, ["odd"], []])
@pytest.mark.parametrize("n", [0, 1, 37])
def test_copy(n, kinds, page):
    g = torch.Generator(device=DEV).manual_seed(n + page)
    pages = 90
    caches = layers(g, pages, page, kinds)
    want = [x.clone() for x in caches]
    order = torch.randperm(pages, generator=g, device=DEV)
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    if n > 4:  # padding
        src[1], dst[2], src[3], dst[4] = -1, pages, 1 << 60, -(1 << 40)
    for x, w in zip(caches, want):
        for a, b in zip(src.tolist(), dst.tolist()):
            if 0 <= a < pages and 0 <= b < pages:
                w[b] = x[a]
    ra.rope_copy_pages(src, dst, caches if n % 2 else ra.PageCaches(caches))
    torch.cuda.synchronize()
    for x, w in zip(caches, want):
        assert torch.equal(raw(x), raw(w))


def test_copy_strided_lists_and_onto_itself():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = pool(g, 20, torch.bfloat16, 16, 2, 64)
    w = x.clone()
    both = ints([[3, 4], [5, 6], [7, 7]])
    w[4], w[6] = x[3], x[5]
    ra.rope_copy_pages(both[:, 0], both[:, 1], [x])
    torch.cuda.synchronize()
    assert torch.equal(raw(x), raw(w))


def random_batch(r, B, R, page, width, pages, external=False, holes=True):
    """A table whose pages are held by one row each, or (forked before) by several."""
    free = list(range(pages))
    r.shuffle(free)
    refs, table, lens = [0] * pages, [], []
    for b in range(B):
        n = r.choice([0, r.randint(0, width * page), r.randint(0, width) * page])
        used = -(-n // page)
        share = r.randint(0, min(used, -(-lens[-1] // page))) if table and r.random() < 0.3 else 0
        if share and lens[-1] % page and share == -(-lens[-1] // page) and r.random() < 0.5:
            share -= 1
        if len(free) < used - share + (pages // 4 if holes else 0):
            n, used, share = 0, 0, 0
        row = (table[-1][:share] if share else []) + [free.pop() for _ in range(used - share)]
        for q in row:
            refs[q] += 1
        lens.append(n)
        table.append(row + [r.choice([-1, 0, pages + 7]) for _ in range(width - used)])
    if external:
        for q in r.sample(range(pages), min(pages, 5)):
            refs[q] += 1
    parents = [r.choice([-1, B, r.randrange(max(B, 1))]) if r.random() < 0.2 else r.randrange(max(B, 1))
               for _ in range(R)]
    grow = [r.choice([0, 1, 1, 5, page, -3]) for _ in range(R)]
    return table, lens, parents, grow, refs


def run_fork(r, B, R, page, width, pages, kinds, wider=0, grow_given=True, in_place=False, **more):
    g = torch.Generator(device=DEV).manual_seed(r.randrange(1 << 30))
    table, lens, parents, grow, refs = random_batch(r, B, R, page, width, pages, **more)
    if not grow_given:
        grow = [0] * R
    caches = layers(g, pages, page, kinds)
    before = [x.clone() for x in caches]
    rows, new_lens, counts, short, copies = fork_reference(table, lens, parents, grow, refs, page,
                                                           width + wider)
    t = ints(table).view(B, width)
    rc = ints(refs)
    out = torch.full((R, width + wider), -77, dtype=torch.int64, device=DEV)
    got = ra.rope_fork_pages(t, ints(lens).view(B), ints(parents).view(R), rc, page,
                             ra.PageCaches(caches), grow=ints(grow).view(R) if grow_given else None,
                             page_table_out=out if wider else None,
                             ref_counts_out=rc if in_place else None)
    torch.cuda.synchronize()
    assert got[0].tolist() == rows
    assert got[1].tolist() == new_lens
    assert got[2].tolist() == counts
    assert got[3].tolist() == [short]
    assert t.tolist() == table and (in_place or rc.tolist() == refs)
    for x, w, k in zip(caches, before, range(len(caches))):
        first = w.clone()
        rows_first = w.dim() > 1 and (w.shape[1] == 1 or w.stride(1) >= max(w.stride()[2:], default=1))
        splits = w.dim() > 1 and (page % w.shape[1] == 0 or w.shape[1] % page == 0)
        for a, b, tokens in copies:
            if b >= 0:
                n = -(-tokens * w.shape[1] // page) if rows_first and splits else None
                if n is None:
                    w[b] = first[a]
                else:
                    w[b, :n] = first[a, :n]
        assert torch.equal(raw(x), raw(w)), k


@pytest.mark.parametrize("seed", range(30))
def test_fork(seed):
    r = random.Random(seed)
    page = r.choice([1, 3, 4, 16, 64])
    width = r.randint(1, 9)
    B, R = r.randint(1, 20), r.randint(1, 40)
    run_fork(r, B, R, page, width, B * width + r.choice([0, 10, 300]),
             r.sample(KINDS, r.randint(0, 4)), wider=r.choice([0, 0, 3]),
             grow_given=r.random() < 0.8, in_place=r.random() < 0.5, external=r.random() < 0.5,
             holes=r.random() < 0.7)


@pytest.mark.parametrize("B,R,pages", [(1, 1, 1), (4, 0, 9), (0, 3, 9), (1030, 2500, 9000), (5000, 3000, 40000),
                                       (2, 1025, 4096), (3, 5, 4097)])
def test_fork_sizes(B, R, pages):
    """Rows past a workgroup's threads, sequences past what LDS holds, pages past a chunk."""
    run_fork(random.Random(B + R), B, R, 4, 6, pages, ["scales"])


def test_fork_without_pages_or_places():
    t = ra.rope_fork_pages(torch.empty(3, 0, dtype=torch.int64, device=DEV), ints([5, 0, 1]),
                           ints([2, 0]), ints([0, 1]), 16)
    assert t[0].shape == (2, 0) and t[1].tolist() == [0, 0] and t[2].tolist() == [0, 1]
    t = ra.rope_fork_pages(ints([[0], [0]]), ints([0, 0]), ints([0, 1, 1]),
                           torch.empty(0, dtype=torch.int64, device=DEV), 16, grow=ints([1, 1, 0]))
    assert t[0].tolist() == [[-1], [-1], [-1]] and t[3].tolist() == [2] and t[1].tolist() == [1, 1, 0]


def test_fork_refuses_narrower_tables_and_overlaps():
    t, n, c = ints([[0, 1]]), ints([20]), ints([1, 1, 0])
    with pytest.raises(ra.RopeError):
        ra.rope_fork_pages(t, n, ints([0]), c, 16, page_table_out=ints([[0]]))
    with pytest.raises(ra.RopeError):
        ra.rope_fork_pages(t, n, ints([0]), c, 16, page_table_out=t)
    with pytest.raises(ra.RopeError):
        ra.rope_fork_pages(t, n, ints([0]), c, 16, [torch.zeros(4, 16, device=DEV)])


def run_compact(r, B, width, pages, kinds, share, in_place=False):
    g = torch.Generator(device=DEV).manual_seed(r.randrange(1 << 30))
    used = r.sample(range(pages), min(pages, int(pages * share)))
    refs = [0] * pages
    for q in used:
        refs[q] = r.randint(1, 3)
    pick = lambda: r.choice(used) if used and r.random() < 0.9 else r.choice([-1, pages, 1 << 50, -9])
    table = [[pick() for _ in range(width)] for _ in range(B)]
    caches = layers(g, pages, 8, kinds)
    before = [x.clone() for x in caches]
    rows, counts, page_map, live, moves = compact_reference(table, refs)
    t, c = ints(table).view(B, width), ints(refs).view(pages)
    got = ra.rope_compact_pages(t, c, caches, page_table_out=t if in_place else None,
                                ref_counts_out=c if in_place else None)
    torch.cuda.synchronize()
    assert got[0].tolist() == rows
    assert got[1].tolist() == counts
    assert got[2].tolist() == page_map
    assert got[3].tolist() == [live]
    for x, w in zip(caches, before):
        first = w.clone()
        for a, b in moves:
            w[b] = first[a]
        assert torch.equal(raw(x), raw(w))


@pytest.mark.parametrize("seed", range(20))
def test_compact(seed):
    r = random.Random(seed)
    run_compact(r, r.randint(0, 20), r.randint(0, 12), r.randint(1, 500),
                r.sample(KINDS, r.randint(0, 4)), r.choice([0.0, 0.1, 0.5, 0.9, 1.0]), r.random() < 0.5)


@pytest.mark.parametrize("pages,share", [(4095, 0.5), (4096, 0.5), (4097, 0.99), (8192, 0.5), (20000, 0.3),
                                         (12288, 1 / 3), (1, 1.0), (0, 0.0)])
def test_compact_sizes(pages, share):
    """Borders of the chunks that pages are counted in."""
    run_compact(random.Random(pages), 7, 5, pages, ["scales", "odd"] if pages < 9000 else ["scales"],
                share)


@pytest.mark.parametrize("pages", [8 * 4096, 8 * 4096 + 1, 70000, 300001])
def test_large_pools(pages):
    """Pools whose free pages are counted chunk by chunk first."""
    run_compact(random.Random(pages), 7, 5, pages, ["vector"], 0.4, in_place=pages % 2 == 1)
    run_fork(random.Random(pages), 40, 70, 4, 6, pages, ["vector"], in_place=pages % 2 == 0)


def test_pages_beyond_4_gib():
    pages, words = 70, 1 << 26  # 64 MiB each
    x = torch.zeros(pages, words, dtype=torch.int8, device=DEV)
    for p in (0, 31, 32, 33, 63, 64, 65, 69):
        x[p] = p
    ra.rope_copy_pages(ints([0, 31, 69, 64]), ints([68, 34, 1, 66]), [x])
    torch.cuda.synchronize()
    for p, v in ((68, 0), (34, 31), (1, 69), (66, 64), (65, 65), (67, 0), (35, 0)):
        assert bool((x[p] == v).all()), p


def spread(x, columns=False):
    """The same numbers, other strides: every second element of a larger tensor, or column by column."""
    if columns:
        return x.t().contiguous().t()
    wide = torch.full((*x.shape, 2), -55, dtype=x.dtype, device=DEV)
    wide[..., 1] = x
    return wide[..., 1]


@pytest.mark.parametrize("columns", [False, True])
def test_strided_tables_and_vectors(columns):
    r = random.Random(11)
    B, R, page, width, pages = 7, 12, 4, 6, 90
    table, lens, parents, grow, refs = random_batch(r, B, R, page, width, pages)
    want = fork_reference(table, lens, parents, grow, refs, page, width + 1)
    out = spread(torch.zeros(R, width + 1, dtype=torch.int64, device=DEV), not columns)
    vectors = [spread(ints(x)) for x in (lens, parents, grow, refs, [0] * R, [0] * pages, [0])]
    got = ra.rope_fork_pages(spread(ints(table), columns), vectors[0], vectors[1], vectors[3], page,
                             grow=vectors[2], page_table_out=out, seq_lens_out=vectors[4],
                             ref_counts_out=vectors[5], shortage=vectors[6])
    torch.cuda.synchronize()
    assert [x.tolist() for x in got] == [want[0], want[1], want[2], [want[3]]]
    want = compact_reference(got[0].tolist(), got[2].tolist())
    moved = ra.rope_compact_pages(got[0], got[2], page_table_out=got[0], ref_counts_out=got[2],
                                  page_map=spread(ints([0] * pages)), live=spread(ints([0])))
    torch.cuda.synchronize()
    assert [x.tolist() for x in moved] == [want[0], want[1], want[2], [want[3]]]
    assert moved[0].data_ptr() == out.data_ptr()


def test_graphs_replay():
    """A step's fork and compaction captured together; every replay on other lengths."""
    r = random.Random(5)
    B, R, page, width, pages = 6, 9, 4, 7, 120
    g = torch.Generator(device=DEV).manual_seed(3)
    caches = layers(g, pages, page, ["wide", "scales"])
    start = [x.clone() for x in caches]
    table, lens, parents, grow, refs = (torch.zeros(B, width, dtype=torch.int64, device=DEV),
                                        ints([0] * B), ints([0] * R), ints([0] * R), ints([0] * pages))
    handle = ra.PageCaches(caches)

    def step():
        new = ra.rope_fork_pages(table, lens, parents, refs, page, handle, grow=grow)
        return new, ra.rope_compact_pages(new[0], new[2], handle)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for n in range(4):
        inputs = random_batch(r, B, R, page, width, pages)
        for t, v in zip((table, lens, parents, grow, refs), inputs):
            t.copy_(ints(v).view_as(t))
        for x, w in zip(caches, start):
            x.view(torch.uint8).copy_(w.view(torch.uint8))
        want = step()
        torch.cuda.synchronize()
        kept = [x.clone() for x in caches]
        for x, w in zip(caches, start):
            x.view(torch.uint8).copy_(w.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
        for x, y in zip(caches, kept):
            assert torch.equal(raw(x), raw(y))


def test_other_streams():
    """Outputs and workspaces belong to the stream that the call is given."""
    r = random.Random(8)
    table, lens, parents, grow, refs = random_batch(r, 5, 7, 4, 6, 60)
    want = fork_reference(table, lens, parents, grow, refs, 4, 6)
    t, n, p, gr, c = ints(table), ints(lens), ints(parents), ints(grow), ints(refs)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = [ra.rope_fork_pages(t, n, p, c, 4, grow=gr, stream=stream) for _ in range(20)]
    stream.synchronize()
    for g in got:
        assert g[0].tolist() == want[0] and g[2].tolist() == want[2]
