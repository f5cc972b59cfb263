"""Plain forms of the 8-bit paged cache's operators and of the operators on pages.  Used by the tests
only; shares no code with the library.

Append: every step of the definition is one float32 operation, so codes and scales are compared bit
for bit.  Attention: float64 from the codes and scales, with the bounds that the kernel's roundings
allow.  u is half a step of the query's type relative to a value (bf16 2^-8, f16 2^-11), e = 2^-24.
  logits   s_j = scale ks_j <q, kc_j>: products of a 16-bit number and a code are exact in float32;
           D sums, the scale to powers of two, its product with ks, that with the sum, and the
           subtraction of the maximum add a rounding each: |ds| <= (D + 8) e max_j |scale ks_j| <|q|, |kc_j|>
  weights  exp2 (1 step), n additions, the product with vs: dp = 2 ds + (n + 10) e, and one rounding u
           for the second product.  float16 takes weights times 2^11 or more beside a sum of at least
           2^11, and vs over a power of two at most twice the largest: where a weight is subnormal its
           error is half of 2^-24 of that: n 2^-25 2^-11 2 max vs max|vc|
  output   |do| <= u |o| + (u + dp) sum p |v|
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E32 = 2.0 ** -24
E4M3, I8 = torch.float8_e4m3fn, torch.int8


def quantized_cache(gen, dtype, pages, page, block, heads, width, device="cuda", spread=1.0):
    """Random codes with scales that differ from block to block."""
    if dtype == I8:
        c = torch.randint(-127, 128, (pages, page, heads, width), generator=gen, device=device,
                          dtype=torch.int8)
    else:
        c = (torch.randn((pages, page, heads, width), generator=gen, device=device) * 60).to(E4M3)
    s = torch.rand((pages, page // block, heads), generator=gen, device=device) * 0.02 + 0.002
    s = s * torch.exp(spread * torch.randn(s.shape, generator=gen, device=device) * 0.5)
    return c, s.float()


def rows_of(cache, scales, pages, n):
    """float64 [n, heads, width]: a sequence's first n tokens, codes times scales."""
    page = cache.shape[1]
    block = page // scales.shape[1]
    t = torch.arange(n, device=cache.device)
    where, off = pages[t // page], t % page
    x = cache.view(torch.int8)[where, off].view(cache.dtype).to(torch.float64)
    return x, scales[where, off // block].double()


def attention_reference(query, key, value, ks, vs, table, lens, counts, scale, firsts=None):
    """(out, lse, bound of out, bound of lse) in float64 for the packed batch; rows outside all
    sequences are zero."""
    T, H, D = query.shape
    N = key.shape[2]
    G = H // N
    u, f16 = U[query.dtype], query.dtype == torch.float16
    out = torch.zeros(T, H, D, dtype=torch.float64, device=query.device)
    lse = torch.zeros(T, H, dtype=torch.float64, device=query.device)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    at = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        first = at if firsts is None else firsts[b]
        at += c
        if c == 0:
            continue
        kc, kf = rows_of(key, ks, table[b], n)
        vc, vf = rows_of(value, vs, table[b], n)
        i, j = torch.arange(c, device=query.device), torch.arange(n, device=query.device)
        hidden = (j[None, :] > i[:, None] + (n - c))[:, None, :]
        for h in range(N):
            q = query[first:first + c, h * G:(h + 1) * G].double()
            k, v = kc[:, h], vc[:, h] * vf[:, h, None]
            s = torch.matmul(q, k.t()) * kf[:, h] * scale
            mag = torch.matmul(q.abs(), k.abs().t()) * (kf[:, h].abs() * abs(scale))
            s = s.masked_fill(hidden, -math.inf)
            mag = mag.masked_fill(hidden, 0.0)
            top = s.amax(-1, keepdim=True) if n else torch.full((c, G, 1), -math.inf,
                                                                dtype=torch.float64, device=s.device)
            ref = torch.where(torch.isinf(top), torch.zeros_like(top), top)
            e = torch.exp(s - ref)
            total = e.sum(-1, keepdim=True)
            p = torch.where(total > 0, e / total, torch.zeros_like(e))
            l = (ref + torch.log(total)).squeeze(-1)
            ds = (D + 8) * E32 * (mag.amax(-1) if n else torch.zeros_like(l))
            o = torch.matmul(p, v)
            dp = 2 * ds + (n + 10) * E32
            b_out = u * o.abs() + (u + dp)[..., None] * torch.matmul(p, v.abs()) + 2.0 ** -126
            if f16 and n:  # and the output's own subnormal step
                b_out = b_out + 2.0 ** -25 + n * 2.0 ** -35 * vf[:, h].abs().max() * vc[:, h].abs().max()
            rows = slice(first, first + c), slice(h * G, (h + 1) * G)
            out[rows], lse[rows], bo[rows] = o, l, b_out
            finite = torch.where(torch.isinf(l), torch.zeros_like(l), l)
            bl[rows] = ds + (n + 10) * E32 + 4 * E32 * finite.abs()
    return out, lse, bo, bl


# ---- append, in float32 on the host ----------------------------------------------------------------

def rotate32(x, start, rows, neox):
    """x [T, N, D], rows [T, rd]: float32, every product and sum rounded by itself."""
    y = x.float().clone()
    half = rows.shape[1] // 2
    c, s = rows[:, None, :half].float(), rows[:, None, half:].float()
    i, j = ((slice(start, start + half), slice(start + half, start + 2 * half)) if neox else
            (slice(start, start + 2 * half, 2), slice(start + 1, start + 2 * half, 2)))
    a, b = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def needed_scale(top, codes):
    """top: float32 scalars."""
    if codes == I8:
        return torch.maximum(top * torch.tensor(1.0 / 127, dtype=torch.float32),
                             torch.tensor(2.0 ** -120))
    out = torch.empty_like(top)
    for i, t in enumerate(top.flatten().tolist()):
        k = -120
        while t > 448 * 2.0 ** k:
            k += 1
        out.view(-1)[i] = 2.0 ** k
    return out


def encode(x, codes):
    if codes == I8:
        return torch.round(x).clamp(-127, 127).to(torch.int8)
    return torch.where(torch.isfinite(x), x, math.nan).to(E4M3)


def append_reference(x, cache, scales, table, lens, offsets):
    """One of keys and values: x [T, N, D] float32 (host), cache and scales changed in place."""
    codes = cache.dtype
    pages, page = cache.shape[:2]
    blocks = scales.shape[1]
    block = page // blocks
    raw = cache.view(torch.int8)
    for b, n in enumerate(lens):
        n = min(max(n, 0), table.shape[1] * page)
        o0, o1 = offsets[b], offsets[b + 1]
        start = n - (o1 - o0)
        place = max(start, 0)
        while place < n:
            begin = place // block * block
            end = min(n, begin + block)
            where, row0 = int(table[b, begin // page]), begin % page
            if 0 <= where < pages:
                new = x[o0 + place - start:o0 + end - start]  # [m, N, D]
                finite = torch.isfinite(new)
                top = torch.where(finite, new.abs(), 0.0).amax(dim=(0, 2))
                now = needed_scale(top, codes)
                if codes == I8:
                    now = torch.where(finite.all(0).all(-1), now, math.nan)
                before = place - begin
                old = scales[where, row0 // block].clone()
                if before:
                    now = torch.where(torch.isnan(now) | torch.isnan(old), math.nan,
                                      torch.maximum(now, old))
                    earlier = cache[where, row0:row0 + before].float()
                    anew = encode(earlier * (old / now)[None, :, None], codes).view(torch.int8)
                    grown = (now != old)[None, :, None]
                    raw[where, row0:row0 + before] = torch.where(
                        grown, anew, raw[where, row0:row0 + before])
                coded = encode(new * (1.0 / now)[None, :, None], codes)
                raw[where, row0 + before:row0 + end - begin] = coded.view(torch.int8)
                scales[where, row0 // block] = now
            place = end


# ---- pages ---------------------------------------------------------------------------------------------

def fork_reference(table, lens, parents, grow, refs, page, width):
    """Lists in, lists out: (table, lens, refs, shortage, [(source, target, tokens)])."""
    pages = len(refs)
    ok = lambda q: 0 <= q < pages
    lens = [min(max(n, 0), len(table[0]) * page if table else 0) for n in lens]
    counts, free = list(refs), [p for p, n in enumerate(refs) if n == 0]
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            if ok(table[b][j]):
                counts[table[b][j]] -= 1
    begun, rows, new_lens, copies, short = set(), [], [], [], 0
    for p, g in zip(parents, grow):
        if not 0 <= p < len(lens):
            rows.append([-1] * width)
            new_lens.append(0)
            continue
        n = lens[p]
        total = n + min(max(g, 0), width * page - n)
        row = list(table[p][:-(-n // page)])

        def take():
            nonlocal short
            short += not free
            return free.pop(0) if free else -1

        if n % page and ok(row[-1]) and (p in begun or refs[row[-1]] > 1):
            got = take()
            copies.append((row[-1], got, n % page))
            row[-1] = got
        begun.add(p)
        while len(row) < -(-total // page):
            row.append(take())
        for q in row:
            if ok(q):
                counts[q] += 1
        rows.append(row + [-1] * (width - len(row)))
        new_lens.append(total)
    return rows, new_lens, counts, short, copies


def compact_reference(table, refs):
    live = sum(n > 0 for n in refs)
    holes = [p for p in range(live) if refs[p] <= 0]
    moves = list(zip([p for p in range(live, len(refs)) if refs[p] > 0], holes))
    page_map = [p if n > 0 else -1 for p, n in enumerate(refs)]
    refs = list(refs)
    for a, b in moves:
        page_map[a] = b
        refs[a], refs[b] = 0, refs[a]
    return [[page_map[p] if 0 <= p < len(refs) else p for p in r] for r in table], refs, page_map, live, moves
