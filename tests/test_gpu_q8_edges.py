"""GPU: single cases of the 8-bit cache's calls where they once went wrong."""
import math

import pytest
import torch

import rope_partial_inplace_amd as ra
from q8_ref import E4M3, I8
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
