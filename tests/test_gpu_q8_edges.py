"""GPU: single cases of the 8-bit cache's calls where they once went wrong."""
import math

import pytest
import torch

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
