"""GPU: rope_attention_paged_q8 against float64 within derived bounds, and the cache's calls together as
a serving loop makes them."""
import math
import random

import pytest
import torch

import rope_partial_inplace_amd as ra
import rope_workloads as W
from q8_ref import E4M3, I8, attention_reference, quantized_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def offsets_of(counts, first=0):
    return torch.tensor([first] + (torch.tensor(counts).cumsum(0) + first).tolist(), device=DEV)


def setup(lens, counts, page, block, heads, N, D, codes, dtype, seed=0, spread=1.0, spare=2):
    g = gen_of(seed)
    T = sum(counts)
    n_pages = [max(1, -(-max(n, 0) // page)) for n in lens]
    pages = sum(n_pages) + spare
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.randint(-3, pages + 3, (len(lens), max(n_pages)), generator=g, device=DEV)
    at = 0
    for b, c in enumerate(n_pages):
        table[b, :c] = order[at:at + c]
        at += c
    kc, ks = quantized_cache(g, codes, pages, page, block, N, D, spread=spread)
    vc, vs = quantized_cache(g, codes, pages, page, block, N, D, spread=spread)
    # whatever lies behind the last tokens reaches no result
    for b, n in enumerate(lens):
        last = int(table[b, n_pages[b] - 1])
        rest = n - (n_pages[b] - 1) * page
        for c, s in ((kc, ks), (vc, vs)):
            c.view(I8)[last, rest:] = 127  # a NaN, or the largest code
            s[last, -(-rest // block):] = math.nan
    for x in order[at:].tolist():
        kc.view(I8)[x], vc.view(I8)[x], ks[x], vs[x] = 127, 127, math.nan, math.inf
    q = torch.randn((T, heads, D), generator=g, device=DEV).to(dtype)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=torch.tensor(lens, device=DEV),
                offsets=offsets_of(counts), counts=list(counts), scale=D ** -0.5)


def attend(s, offsets=True, **more):
    return ra.rope_attention_paged_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"],
                                      s["scale"], query_offsets=s["offsets"] if offsets else None, **more)


def close(got, want, bound, what):
    top, eps = torch.finfo(got.dtype).max, torch.finfo(got.dtype).eps
    limit = top / (1 - eps / 2) * (1 - eps / 4)
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), what + ": NaN"
    same = (got == want) | want.isnan()
    # from half a step above the largest number (2 - eps) 2^k on, at (2 - eps / 2) 2^k, the nearest is an
    # infinity: 65520 in float16
    same |= got.isinf() & (got.sign() == want.sign()) & (want.abs() + bound >= limit)
    err = torch.where(same, 0.0, (got - want).abs() - bound)
    assert float(err.max() if err.numel() else 0.0) <= 0.0, \
        f"{what}: {float(err.max())} past the bound at {(err == err.max()).nonzero()[0].tolist()}"


def check(s, offsets=True, firsts=None):
    held = {n: x.clone() for n, x in s.items() if isinstance(x, torch.Tensor)}
    T, H, D = s["q"].shape
    out = torch.full((T, H, D), 7.0, dtype=s["q"].dtype, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    attend(s, offsets, out=out, lse=lse)
    width = s["table"].shape[1] * s["kc"].shape[1]
    lens = [min(max(n, 0), width) for n in s["lens"].tolist()]
    table = s["table"].clamp(0, s["kc"].shape[0] - 1)
    o, l, bo, bl = attention_reference(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], table, lens,
                                       s["counts"], s["scale"], firsts)
    inside = torch.zeros(T, dtype=torch.bool, device=DEV)
    at = 0
    for b, c in enumerate(s["counts"]):
        f = at if firsts is None else firsts[b]
        inside[f:f + c] = True
        at += c
    assert bool((out[~inside] == 7.0).all()) and bool((lse[~inside] == 7.0).all())
    close(out[inside], o[inside], bo[inside], "out")
    close(lse[inside], l[inside], bl[inside], "lse")
    again = attend(s, offsets)
    assert torch.equal(again[0][inside].view(torch.int16), out[inside].view(torch.int16))
    assert torch.equal(again[1][inside].view(torch.int32), lse[inside].view(torch.int32))
    for n, x in held.items():
        a, b = (y.contiguous().view(torch.uint8) for y in (s[n], x))
        assert torch.equal(a, b), n


LENS = [35, 1, 16, 0, 130, 65, 257, 2]
SINGLE = [1, 1, 1, 1, 1, 1, 1, 1]
FEW = [3, 1, 4, 2, 3, 0, 4, 4]          # two of them longer than their sequences
MANY = [35, 1, 16, 9, 60, 65, 100, 0]


@pytest.mark.parametrize("codes", [I8, E4M3])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("counts,heads,N", [(SINGLE, 8, 2), (SINGLE, 6, 6), (SINGLE, 32, 1), (FEW, 10, 2),
                                            (MANY, 4, 2), (MANY, 7, 1)])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 4), (5, 5), (32, 2), (1, 1), (12, 4)])
def test_attention(page, block, counts, heads, N, D, dtype, codes):
    check(setup(LENS, counts, page, block, heads, N, D, codes, dtype, seed=page + heads))


@pytest.mark.parametrize("page,block", [(15, 3), (100, 100), (100, 1), (128, 128), (48, 6), (256, 64)])
@pytest.mark.parametrize("counts", [SINGLE, FEW, MANY])
def test_pages_and_blocks(page, block, counts):
    check(setup(LENS, counts, page, block, 12, 3, 128, E4M3, BF16, seed=page))
    check(setup(LENS, counts, page, block, 12, 3, 64, I8, F16, seed=page))


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    r = random.Random(seed)
    page = r.choice([1, 3, 16, 32, 64, 80])
    block = r.choice([d for d in range(1, page + 1) if page % d == 0])
    N, group = r.randint(1, 4), r.choice([1, 2, 3, 4, 7, 8, 16, 40])
    lens, counts = [], []
    for _ in range(r.randint(1, 20)):
        lens.append(r.choice([0, 1, r.randint(1, 64), r.randint(1, 900)]))
        counts.append(r.choice([0, 1, 1, 1, r.randint(0, 12), min(lens[-1], r.randint(0, 300))]))
    check(setup(lens, counts, page, block, N * group, N, r.choice([64, 128, 256]), r.choice([I8, E4M3]),
                r.choice([BF16, F16]), seed=seed))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("heads,N,count", [(8, 1, 1), (32, 8, 1), (8, 8, 3), (64, 2, 2)])
def test_long_sequences_are_split(heads, N, count, dtype):
    check(setup([70001, 5, 30000], [count] * 3, 64, 64, heads, N, 128, E4M3, dtype))
    check(setup([40000], [count], 16, 1, heads, N, 64, I8, dtype))


def test_long_prompts():
    check(setup([1500, 2100], [1500, 700], 64, 64, 8, 2, 128, E4M3, BF16))
    check(setup([1300], [1300], 16, 4, 4, 1, 256, I8, F16))
    check(setup([6000], [257], 16, 16, 6, 2, 64, I8, BF16))


@pytest.mark.parametrize("B", [255, 256, 257, 700, 3000])
def test_many_sequences(B):
    r = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 70, (B,), generator=r).tolist()
    counts = torch.randint(0, 3, (B,), generator=r).tolist()
    check(setup(lens, counts, 16, 16, 2, 1, 64, I8, BF16))
    counts = [c * 20 for c in counts]
    check(setup(lens, counts, 16, 16, 2, 1, 64, E4M3, F16))


def test_no_sequence_has_rows_or_tokens():
    check(setup([0, 0, 0], [1, 2, 1], 16, 16, 4, 2, 64, I8, BF16))
    s = setup([40, 3], [0, 0], 16, 16, 4, 2, 64, I8, BF16)
    assert attend(s)[0].shape == (0, 4, 64)
    s = setup([40, 3], [2, 1], 16, 16, 4, 2, 64, I8, BF16)
    s["offsets"] = torch.zeros_like(s["offsets"])
    s["counts"] = [0, 0]
    check(s)
    s = setup([40, 3], [2, 1], 16, 16, 4, 2, 64, E4M3, BF16)
    s["kc"], s["vc"], s["ks"], s["vs"] = (s[n][:0] for n in ("kc", "vc", "ks", "vs"))
    out, lse = attend(s)  # a cache without pages
    assert not out.any() and bool((lse == -math.inf).all())
    s["table"] = s["table"][:, :0]
    out, lse = attend(s)
    assert not out.any() and bool((lse == -math.inf).all())


def test_without_offsets():
    check(setup([35, 1, 200], [1, 1, 1], 16, 16, 8, 2, 128, I8, BF16), offsets=False)
    check(setup([35, 20, 200], [20, 20, 20], 16, 16, 8, 2, 128, E4M3, F16), offsets=False)


@pytest.mark.parametrize("counts", [SINGLE, MANY])
def test_rows_outside_all_sequences_stay(counts):
    s = setup(LENS, counts, 16, 16, 4, 2, 64, I8, BF16)
    s["q"] = torch.cat([s["q"], s["q"][:5]])
    s["offsets"] = offsets_of(counts, first=3)
    firsts = s["offsets"][:-1].tolist()
    check(s, firsts=firsts)


@pytest.mark.parametrize("counts", [SINGLE, MANY])
def test_descending_offsets_write_nothing(counts):
    s = setup(LENS, counts, 16, 16, 4, 2, 64, I8, BF16)
    s["offsets"] = s["offsets"].flip(0)
    out, lse = torch.full_like(s["q"], 7.0), torch.full(s["q"].shape[:2], 7.0, device=DEV)
    attend(s, out=out, lse=lse)
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


def test_values_out_of_range_are_clamped():
    s = setup([35, 200, 16], [1, 3, 1], 16, 16, 4, 2, 64, E4M3, BF16, spare=0)
    # pages whose rows are all live, in the places of entries out of range
    s["kc"], s["vc"] = (torch.ones(x.shape, device=DEV).to(E4M3) for x in (s["kc"], s["vc"]))
    s["ks"], s["vs"] = torch.rand_like(s["ks"]), torch.rand_like(s["vs"])
    s["table"][1, 3], s["table"][1, 5] = -1, 1 << 50
    s["lens"][1], s["lens"][2] = 1 << 40, -3
    check(s)


@pytest.mark.parametrize("counts", [SINGLE, MANY])
def test_layouts(counts):
    """Heads before rows, keys and values in one allocation, scales, tables and queries in any order."""
    s = setup(LENS, counts, 16, 4, 6, 3, 64, E4M3, BF16)
    pages = s["kc"].shape[0]
    both = torch.zeros(pages, 2, 3, 16, 80, dtype=I8, device=DEV)
    for n, k in (("kc", 0), ("vc", 1)):
        view = both[:, k].transpose(1, 2)[..., 16:]
        view.copy_(s[n].view(I8))
        s[n] = view.view(E4M3)
    s["ks"] = s["ks"].permute(2, 0, 1).contiguous().permute(1, 2, 0)
    wide = torch.empty(*s["vs"].shape, 2, device=DEV)
    wide[..., 1] = s["vs"]
    s["vs"] = wide[..., 1]
    s["table"] = s["table"].t().contiguous().t()
    s["lens"] = torch.stack([s["lens"], s["lens"]], 1)[:, 0]
    s["q"] = torch.cat([s["q"].flatten(1), s["q"].flatten(1)], 1)[:, :6 * 64].unflatten(1, (6, 64))
    check(s)


@pytest.mark.parametrize("counts", [SINGLE, MANY])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("factor", [1e-30, 1e-6, 300.0])
def test_scales_of_any_size(factor, dtype, counts):
    """Value scales far from 1 and from each other, logits that vanish or pick one token."""
    s = setup(LENS, counts, 16, 4, 4, 2, 64, E4M3, dtype, spread=8.0)
    s["vs"] *= min(factor, 1.0)
    s["scale"] *= factor
    s["ks"] /= s["ks"].nan_to_num(0.0, 0.0).mean()  # of size 1
    check(s)


@pytest.mark.parametrize("counts", [SINGLE, MANY])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_negative_and_zero_scales(dtype, counts):
    for c in (0.0, -0.3):
        s = setup(LENS, counts, 16, 4, 4, 2, 128, I8, dtype)
        s["scale"] = c
        s["ks"] *= torch.randint(-1, 2, s["ks"].shape, generator=gen_of(3), device=DEV)
        s["vs"] *= torch.randint(-1, 2, s["vs"].shape, generator=gen_of(4), device=DEV)
        check(s)


@pytest.mark.parametrize("counts", [[1, 1, 1], [4, 2, 9], [30, 20, 64]])
@pytest.mark.parametrize("dtype,codes", [(BF16, E4M3), (F16, I8)])
def test_nan_where_it_belongs(dtype, codes, counts):
    """A poisoned scale in tokens that a row sees makes it NaN, in later ones it does not; other
    sequences stay."""
    s = setup([70, 20, 64], counts, 16, 4, 4, 2, 64, codes, dtype)
    clean = attend(s)
    page, block = int(s["table"][0, 4]), 1  # tokens 68 and 69
    s["vs"][page, block, 1] = math.nan
    out, _ = attend(s)
    first = 70 - counts[0]
    for i in range(counts[0]):
        sees = first + i >= 68
        assert bool(out[i, 2:].isnan().all()) == sees
        assert torch.equal(out[i, :2], clean[0][i, :2])
        assert sees or torch.equal(out[i, 2:], clean[0][i, 2:])
    assert torch.equal(out[counts[0]:], clean[0][counts[0]:])
    s["q"][counts[0], 1, 5] = math.nan
    out2, lse2 = attend(s)
    assert bool(out2[counts[0], 1].isnan().all()) and bool(lse2[counts[0], 1].isnan())
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device=DEV)
    keep[counts[0], 1] = False
    assert torch.equal(out2[keep].view(torch.int16), out[keep].view(torch.int16))


def test_scores_that_grow_along_the_sequence():
    """Every tile raises the maximum, by less and by more than what is carried."""
    for step in (0.5, 3.0, 30.0):
        for counts in ([1], [40]):
            s = setup([300], counts, 16, 1, 2, 1, 64, I8, F16)
            s["kc"][:] = 1
            s["q"][:] = 1.0
            t = torch.arange(304, device=DEV).view(19, 16)
            s["ks"][s["table"][0, :19], :, 0] = t.float() * step / 64
            s["scale"] = 1.0
            check(s)


def test_beyond_4_gib():
    page, N, D = 64, 8, 128
    pages = (1 << 32) // (page * N * D) + 40
    s = setup([150, 300, 64], [1, 1, 1], page, 16, 16, N, D, E4M3, BF16)
    small = s["kc"].shape[0]
    where = torch.tensor([pages // 2 - 1, pages // 2, pages - 1, 0, pages - 2, 7, pages - 41, pages - 39,
                          pages // 2 + 1, 5, 9, 11, pages - 20], device=DEV)[:small]
    assert len(where) == small
    big = dict(s)
    for n in ("kc", "vc"):
        big[n] = torch.empty(pages, page, N, D, dtype=I8, device=DEV).view(E4M3)
        big[n].view(I8)[where] = s[n].view(I8)
    for n in ("ks", "vs"):
        big[n] = torch.zeros(pages, 4, N, device=DEV)
        big[n][where] = s[n]
    table = s["table"].clamp(0, small - 1)
    big["table"] = where[table]
    s["table"] = table
    for counts in ([1, 1, 1], [50, 64, 64]):
        for x in (s, big):
            x["q"] = torch.randn((sum(counts), 16, D), generator=gen_of(1), device=DEV).to(BF16)
            x["offsets"] = offsets_of(counts)
        a, b = attend(s), attend(big)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))
        assert torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


def test_streams_and_graphs():
    """Calls on two streams at once, and replays of a captured one between eager calls."""
    a = setup(LENS, SINGLE, 16, 16, 8, 2, 128, I8, BF16)
    b = setup([20000, 3], [1, 1], 16, 16, 8, 2, 128, E4M3, BF16)
    want = attend(a), attend(b)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((attend(a, stream=one), attend(b, stream=two)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], want[0][0]) and torch.equal(y[0], want[1][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend(a), attend(b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attend(a), attend(b)
    for n in range(4):
        a["lens"].add_(n)  # lengths are read by the replay
        a["lens"].clamp_(max=256)
        a["ks"].nan_to_num_(0.01), a["vs"].nan_to_num_(0.01, 0.01, 0.01)
        eager = attend(a), attend(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, eager):
            assert torch.equal(x[0].view(torch.int16), y[0].view(torch.int16))
            assert torch.equal(x[1].view(torch.int32), y[1].view(torch.int32))


@pytest.mark.parametrize("codes,block", [(E4M3, 16), (I8, 1), (I8, 16)])
@pytest.mark.parametrize("page", [16, 20])
def test_serving_loop(page, codes, block):
    """A prompt, samples of it, single tokens with forks of beams, a compaction: every layer's
    attention is that of unquantised copies within the codes' steps, and the same after the pages
    have moved."""
    block = math.gcd(block, page)
    layers, heads, N, D, pages, width = 2, 8, 2, 64, 120, 8
    g = gen_of(7)
    caches = []
    for _ in range(layers):
        for _ in range(2):
            caches.append(torch.zeros(pages, page, N, D, device=DEV).to(codes))
            caches.append(torch.zeros(pages, page // block, N, device=DEV))
    handle = ra.PageCaches(caches)
    cs = W.cos_sin_cache(512, D, BF16).to(DEV)
    refs = torch.zeros(pages, dtype=torch.int64, device=DEV)
    table = torch.full((1, width), -1, dtype=torch.int64, device=DEV)
    lens = torch.zeros(1, dtype=torch.int64, device=DEV)
    history = [[(torch.zeros(0, N, D, dtype=torch.float64, device=DEV),) * 2 for _ in range(layers)]]
    steps = [([0], [45]), ([0, 0, 0], [1, 1, 1]), ([0, 1, 2], [1, 1, 1]), ([1, 1, 0, 2], [1, 1, 1, 1]),
             ([3, 0, 0], [17, 1, 1]), ([2, 0], [1, 1]), ([1], [5])]
    for parents, grow in steps:
        p, n = torch.tensor(parents, device=DEV), torch.tensor(grow, device=DEV)
        table, lens, refs, short = ra.rope_fork_pages(table, lens, p, refs, page, handle, grow=n,
                                                      ref_counts_out=refs)
        assert short.item() == 0
        used = table[table >= 0]
        assert int(refs.sum()) == used.numel()
        T = sum(grow)
        offsets = offsets_of(grow)
        pos = torch.cat([torch.arange(int(l) - c, int(l)) for l, c in zip(lens.tolist(), grow)]).to(DEV)
        history = [list(history[x]) for x in parents]
        outs = []
        for i in range(layers):
            kc, ks, vc, vs = caches[4 * i:4 * i + 4]
            q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(BF16) for h in (heads, N, N))
            rotated = ra.rope_append_paged_cache_q8(pos, k, v, kc, vc, ks, vs, table, lens, cs,
                                                    query_offsets=offsets, query=q)
            out, lse = ra.rope_attention_paged_q8(rotated, kc, vc, ks, vs, table, lens, D ** -0.5,
                                                  query_offsets=offsets)
            o, l, bo, bl = attention_reference(rotated, kc, vc, ks, vs, table.clamp(min=0),
                                               lens.tolist(), grow, D ** -0.5)
            close(out, o, bo, "out"), close(lse, l, bl, "lse")
            # what the cache holds is what was given, within its steps
            half = D // 2
            row = cs[pos].double()[:, None]
            kd = k.double()
            turned = torch.cat([kd[..., :half] * row[..., :half] - kd[..., half:] * row[..., half:],
                                kd[..., half:] * row[..., :half] + kd[..., :half] * row[..., half:]], -1)
            at = 0
            for b, c in enumerate(grow):
                hk, hv = history[b][i]
                history[b][i] = (torch.cat([hk, turned[at:at + c]]), torch.cat([hv, v[at:at + c].double()]))
                at += c
                for cache, scales, want in ((kc, ks, history[b][i][0]), (vc, vs, history[b][i][1])):
                    t = torch.arange(int(lens[b]), device=DEV)
                    where, off = table[b][t // page], t % page
                    held = cache.view(I8)[where, off].view(codes).double()
                    s = scales[where, off // block].double()[..., None]
                    # int8: half a step when coded, and half a (smaller) step each time a scale
                    # grew, at most once a token of the block; e4m3: half a step of the number, or of the
                    # smallest normal one; 2^-20: the float32 operations
                    step = (s * 0.5 * (1 + block) if codes == I8 else
                            torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10))
                    assert bool(((held * s - want).abs() <= step + want.abs() * 2.0 ** -20 + s * 2.0 ** -16).all())
            outs.append((rotated, out))
        moved = ra.rope_compact_pages(table, refs, handle)
        table, refs = moved[0], moved[1]
        live = moved[3].item()
        assert bool((refs[:live] > 0).all()) and not refs[live:].any()
        for i, (rotated, out) in enumerate(outs):
            kc, ks, vc, vs = caches[4 * i:4 * i + 4]
            again, _ = ra.rope_attention_paged_q8(rotated, kc, vc, ks, vs, table, lens, D ** -0.5,
                                                  query_offsets=offsets)
            assert torch.equal(again, out)
