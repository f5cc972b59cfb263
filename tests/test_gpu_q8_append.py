"""GPU: rope_append_paged_cache_q8 against the definition in float32, bit for bit, everything outside the
appended tokens unchanged."""
import math

import pytest
import torch

import rope_partial_inplace_amd as ra
import rope_workloads as W
from q8_ref import E4M3, I8, append_reference, quantized_cache, rotate32

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def same(a, b, what):
    a, b = (x.cpu().contiguous() for x in (a, b))
    if a.dtype == E4M3:  # a NaN is a NaN
        x, y = a.view(torch.int8), b.view(torch.int8)
        ok = (x == y) | (((x & 127) == 127) & ((y & 127) == 127))
    else:
        ok = (a == b) | ((a != a) & (b != b))
    assert a.dtype == b.dtype and bool(ok.all()), \
        f"{what}: {int((~ok).sum())} of {ok.numel()} differ, first at {(~ok).nonzero()[0].tolist()}"


def setup(lens, counts, page, block, N, D, Dv, codes, dtype, seed=0, nq=4, rd=None, layout="rows",
          spare=2, magnitude=1.0, view=False):
    g = gen_of(seed)
    T = sum(counts)
    rd = rd or D
    n_pages = [max(1, -(-max(n, 0) // page)) for n in lens]
    pages = sum(n_pages) + spare
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.zeros(len(lens), max(n_pages), dtype=torch.int64, device=DEV)
    at = 0
    for b, c in enumerate(n_pages):
        table[b, :c] = order[at:at + c]
        at += c
    kc, ks = quantized_cache(g, codes, pages, page, block, N, D)
    vc, vs = quantized_cache(g, codes, pages, page, block, N, Dv)
    if codes == E4M3:  # scales as the append leaves them
        ks, vs = (torch.exp2(torch.round(torch.log2(x))) for x in (ks, vs))
    if layout == "heads":
        kc, vc = (x.view(torch.int8).transpose(1, 2).contiguous().transpose(1, 2).view(codes)
                  for x in (kc, vc))
        ks, vs = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (ks, vs))
    randn = lambda *s: (torch.randn(s, generator=g, device=DEV) * magnitude).to(dtype)
    if view:  # columns of one projection
        q, k, v = randn(T, nq * D + N * D + N * Dv).split([nq * D, N * D, N * Dv], dim=1)
        q, k, v = q.unflatten(1, (nq, D)), k.unflatten(1, (N, D)), v.unflatten(1, (N, Dv))
    else:
        q, k, v = randn(T, nq, D), randn(T, N, D), randn(T, N, Dv)
    pos = torch.randint(0, 300, (T,), generator=g, device=DEV)
    cs = W.cos_sin_cache(300, rd, dtype).to(DEV)
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), device=DEV)
    return dict(pos=pos, q=q, k=k, v=v, kc=kc, vc=vc, ks=ks, vs=vs, table=table, cs=cs,
                lens=torch.tensor(lens, device=DEV), offsets=offsets)


def append(s, start=0, neox=True, offsets=True, query=True, in_place=False, **more):
    return ra.rope_append_paged_cache_q8(
        s["pos"], s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["cs"],
        query_offsets=s["offsets"] if offsets else None, query=s["q"] if query else None,
        query_out=s["q"] if in_place else None, query_rot_start=start, key_rot_start=start,
        is_neox_style=neox, **more)


def check(s, start=0, neox=True, **more):
    h = {n: x.cpu().clone() for n, x in s.items()}
    out = append(s, start, neox, **more)
    torch.cuda.synchronize()
    rows = h["cs"][h["pos"].clamp(0, h["cs"].shape[0] - 1)]
    lens, offsets = h["lens"].tolist(), h["offsets"].tolist()
    append_reference(rotate32(h["k"], start, rows, neox), h["kc"], h["ks"], h["table"], lens, offsets)
    append_reference(h["v"].float(), h["vc"], h["vs"], h["table"], lens, offsets)
    for n in ("ks", "vs", "kc", "vc"):
        same(s[n], h[n], n)
    if out is not None:
        want = rotate32(h["q"], start, rows, neox).to(h["q"].dtype)
        rd = rows.shape[1]
        want[..., :start], want[..., start + rd:] = h["q"][..., :start], h["q"][..., start + rd:]
        same(out, want, "query")
    for n in ("k", "v", "table", "lens", "pos", "offsets"):
        same(s[n], h[n], n)


RAGGED = [35, 1, 16, 0, 70, 5, 64], [3, 1, 16, 0, 41, 7, 0]  # lengths, new tokens (7 of 5: two are cut)


@pytest.mark.parametrize("codes", [I8, E4M3])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("page,block", [(16, 16), (16, 4), (64, 64), (5, 5), (12, 3), (1, 1), (32, 1)])
def test_append(page, block, dtype, neox, codes):
    check(setup(*RAGGED, page, block, 3, 64, 64, codes, dtype, seed=page + block), neox=neox)


@pytest.mark.parametrize("codes", [I8, E4M3])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("D,Dv,rd,start", [(128, 64, 128, 0), (128, 128, 64, 64), (96, 96, 96, 0),
                                           (80, 48, 32, 16), (256, 256, 64, 0), (72, 40, 24, 7),
                                           (130, 66, 66, 2), (576, 16, 64, 512), (88, 64, 64, 8),
                                           (136, 40, 32, 24), (160, 128, 64, 32)])
def test_widths_and_slices(D, Dv, rd, start, neox, codes):
    s = setup(*RAGGED, 16, 8, 2, D, Dv, codes, BF16, seed=D, rd=rd)
    check(s, start, neox)


@pytest.mark.parametrize("block", [4, 16, 32, 64, 128])
@pytest.mark.parametrize("dtype,codes", [(BF16, E4M3), (F16, I8), (F32, I8)])
def test_prompts(block, dtype, codes):
    """Long runs of tokens: places numbered by block, blocks of several wavefronts."""
    check(setup([300, 777, 64, 129], [300, 500, 64, 1], 128, block, 2, 128, 128, codes, dtype, seed=block))


@pytest.mark.parametrize("layout", ["rows", "heads"])
@pytest.mark.parametrize("view", [False, True])
def test_layouts(layout, view):
    check(setup(*RAGGED, 16, 4, 3, 64, 64, I8, BF16, layout=layout, view=view))
    s = setup(*RAGGED, 16, 4, 3, 64, 64, E4M3, BF16, layout=layout, view=view)
    both = torch.zeros(s["kc"].shape[0], 2, 16, 3, 64, dtype=torch.int8, device=DEV)
    both[:, 0], both[:, 1] = s["kc"].view(I8), s["vc"].view(I8)
    s["kc"], s["vc"] = both[:, 0].view(E4M3), both[:, 1].view(E4M3)
    s["table"] = s["table"].t().contiguous().t()
    s["lens"] = torch.stack([s["lens"], s["lens"]], 1)[:, 0]
    s["pos"] = torch.stack([s["pos"], s["pos"]], 1)[:, 1]
    check(s, in_place=True)


def test_codes_off_alignment():
    """Rows and codes that are not on vector boundaries go element by element."""
    s = setup(*RAGGED, 16, 4, 3, 64, 64, I8, BF16)
    wide = torch.zeros(*s["kc"].shape[:3], 67, dtype=torch.int8, device=DEV)
    wide[..., 3:] = s["kc"]
    s["kc"] = wide[..., 3:]
    check(s)
    assert not wide[..., :3].any()
    s = setup(*RAGGED, 16, 4, 3, 64, 64, I8, F16)
    k = torch.zeros(s["k"].numel() + 1, dtype=F16, device=DEV)
    k[1:] = s["k"].flatten()
    s["k"] = k[1:].view_as(s["k"])
    check(s)


def test_even_batches_without_offsets():
    check(setup([20, 33, 4], [4, 4, 4], 16, 4, 2, 64, 64, I8, BF16), offsets=False)
    check(setup([1] * 70, [1] * 70, 16, 16, 2, 64, 64, E4M3, BF16), offsets=False, query=False)
    check(setup([200, 333], [100, 100], 16, 16, 2, 64, 64, E4M3, BF16), offsets=False)


@pytest.mark.parametrize("B", [63, 64, 65, 300, 5000])
def test_many_sequences(B):
    """The place's sequence is found 64 offsets at a time."""
    r = torch.Generator().manual_seed(B)
    counts = torch.randint(0, 4, (B,), generator=r).tolist()
    lens = [c + int(x) for c, x in zip(counts, torch.randint(0, 9, (B,), generator=r))]
    check(setup(lens, counts, 4, 2, 1, 16, 16, I8, F32, nq=1))
    check(setup(lens, [7 * c for c in counts], 64, 64, 1, 16, 16, E4M3, F32, nq=1))


def test_tokens_outside_the_cache_are_skipped():
    s = setup(*RAGGED, 16, 4, 3, 64, 64, I8, BF16)
    s["table"][0, 0], s["table"][4, 2], s["table"][2, 0] = -1, s["kc"].shape[0], 1 << 40
    s["lens"][1], s["lens"][5] = -5, 1 << 50
    s["pos"][3], s["pos"][4] = -7, 1 << 40
    check(s)


def test_rows_outside_all_sequences():
    s = setup(*RAGGED, 16, 4, 3, 64, 64, E4M3, BF16)
    s["offsets"][0] += 2
    check(s)
    s = setup(*RAGGED, 16, 4, 3, 64, 64, E4M3, BF16)
    s["offsets"][-1] += 100  # past the batch: cut there
    h = s["offsets"].clone()
    h[-1] -= 100
    t = {n: x.clone() for n, x in s.items()} | {"offsets": h}
    append(s), append(t)
    for n in ("kc", "vc", "ks", "vs"):
        same(s[n], t[n], n)


def test_descending_offsets_stay_inside():
    s = setup(*RAGGED, 16, 4, 3, 64, 64, I8, BF16)
    s["offsets"] = s["offsets"].flip(0)
    append(s)
    torch.cuda.synchronize()


@pytest.mark.parametrize("codes", [I8, E4M3])
def test_scale_grows_token_by_token(codes):
    """A block filled by single tokens of growing and falling size; the codes of earlier ones follow."""
    for n, size in enumerate([1e-3, 1.0, 0.5, 30.0, 0.0, 1e4, 1.0, 3e4, 5.0]):
        s2 = setup([n + 1, n + 1], [1, 1], 8, 8, 2, 64, 64, codes, F32, seed=n, nq=1, magnitude=size)
        if n:
            for x in ("kc", "vc", "ks", "vs", "table"):
                s2[x] = s[x]
        else:
            s2["table"] = torch.tensor([[2, 4], [3, 1]], device=DEV)
            for x, w in (("kc", 64), ("vc", 64)):
                s2[x] = quantized_cache(gen_of(1), codes, 5, 8, 8, 2, w)[0]
            for x in ("ks", "vs"):
                s2[x] = quantized_cache(gen_of(1), codes, 5, 8, 8, 2, 8)[1]
        s = s2
        check(s)


def test_e4m3_scales_are_powers_of_two_and_codes_stay_exact():
    """Growth from 2^-4 to 2^10 leaves the codes' values as they were."""
    s = setup([1], [1], 16, 16, 1, 64, 64, E4M3, F32, nq=1, magnitude=2.0 ** -4)
    append(s)
    values = lambda: (s["vc"][s["table"][0, 0], 0].float() *
                      s["vs"][s["table"][0, 0], 0][:, None])
    first = values().clone()
    for n in range(1, 8):
        t = setup([n + 1], [1], 16, 16, 1, 64, 64, E4M3, F32, nq=1, magnitude=2.0 ** (2 * n - 4), seed=n)
        for x in ("kc", "vc", "ks", "vs", "table"):
            t[x] = s[x]
        s = t
        append(s)
        scale = s["vs"][s["table"][0, 0], 0]
        assert torch.equal(torch.exp2(torch.round(torch.log2(scale))), scale)
        # codes fall into the subnormal numbers below 2^-6 / 2^10
        still = first.abs() >= 2.0 ** -6 * scale[:, None]
        assert torch.equal(values()[still], first[still])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("codes", [I8, E4M3])
def test_non_finite_and_extreme_values(codes, dtype):
    for bad in (math.nan, math.inf, -math.inf):
        s = setup(*RAGGED, 16, 4, 3, 64, 64, codes, dtype, rd=32)
        s["k"][5, 1, 40] = bad   # outside the slice, inside it, and a value
        s["k"][20, 0, 3] = bad
        s["v"][30, 2, 17] = bad
        check(s)
    for size in (0.0, 1e-38, 1e30):
        s = setup(*RAGGED, 16, 4, 3, 64, 64, codes, dtype, magnitude=size)
        check(s)
    s = setup(*RAGGED, 16, 4, 3, 64, 64, codes, dtype)
    s["ks"][s["table"][0, 2], 0] = math.nan  # an earlier NaN stays while its tokens do
    check(s)


@pytest.mark.parametrize("dtype,block,width", [(BF16, 32, 128), (F16, 128, 64), (F32, 64, 128), (BF16, 128, 128)])
@pytest.mark.parametrize("codes", [I8, E4M3])
def test_non_finite_values_in_long_blocks(codes, dtype, block, width):
    """Blocks of two and four wavefronts, which meet twice where one of them has such a value; places that
    fill a workgroup partly."""
    for heads in (1, 3):
        s = setup([300, 777, 64, 129], [299, 500, 64, 1], 128, block, heads, width, width, codes, dtype, seed=block)
        s["k"][5, 0, 40], s["k"][400, heads - 1, 3], s["v"][798, 0, 17] = math.nan, math.inf, -math.inf
        check(s, neox=heads == 1)


def test_negative_zero_and_ties():
    s = setup([4], [4], 4, 4, 1, 16, 16, I8, F32, nq=1, rd=2)
    v = torch.arange(64, device=DEV, dtype=F32).view(4, 1, 16) - 31.5
    v[0, 0, 0], v[1, 0, 1] = 127.0, -0.0
    s["v"] = v  # a scale of 1 (127 / 127 rounds to it): halves go to even
    check(s)


def test_graph_replays_and_repeats():
    s = setup(*RAGGED, 16, 4, 3, 64, 64, I8, BF16)
    fresh = {n: x.clone() for n, x in s.items()}
    append(s)
    want = {n: s[n].clone() for n in ("kc", "vc", "ks", "vs")}
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        append(s)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = append(s)
    for n in range(3):
        for x in want:
            s[x].copy_(fresh[x])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x in want:
            same(s[x], want[x], x)
        assert out.abs().sum() > 0


def test_beyond_4_gib():
    """Pages on both sides of 2^31 and 2^32 bytes, and of 2^32 elements of the scales' extent."""
    page, N, D = 64, 8, 128
    pages = (1 << 32) // (page * N * D) + 40
    kc = torch.empty(pages, page, N, D, dtype=torch.int8, device=DEV)
    vc = torch.empty_like(kc)
    s = setup([50, 65, 130, 7], [3, 1, 66, 7], page, 16, N, D, D, I8, BF16)
    small = [s["kc"], s["vc"], s["ks"], s["vs"]]
    half = pages // 2
    where = torch.tensor([half - 1, half, pages - 1, pages - 2, half + 1, 3, pages - 30, pages - 40, 17, 1],
                         device=DEV)[:s["kc"].shape[0]]
    ks = torch.zeros(pages, 4, N, device=DEV)
    vs = torch.zeros_like(ks)
    for big, x in zip((kc, vc, ks, vs), small):
        big[where] = x
    t = dict(s, kc=kc, vc=vc, ks=ks, vs=vs, table=where[s["table"]])
    append(t)
    append(s)
    torch.cuda.synchronize()
    for big, x, n in zip((kc, vc, ks, vs), small, ("kc", "vc", "ks", "vs")):
        same(big[where], x, n)
