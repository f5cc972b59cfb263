"""Measured calls of the 8-bit paged cache and of the operators on a cache's pages.

Five operators, as a decoder with grouped-query heads uses them around the rotary position
embedding:

  append8    rope_append_paged_cache_q8: a batch of new tokens' keys is rotated by position, and keys
             and values are written to a paged cache of 8-bit codes with a float32 scale for each
             block of tokens and head; the queries are rotated by the same launch
  attend8    rope_attention_paged_q8: grouped-query attention over that cache
  copy       rope_copy_pages: listed pages of every layer's caches are copied to other pages
  fork       rope_fork_pages: the sequences of the next step continue sequences of this one; full
             pages are shared, a last page that is not full is copied, new pages are taken for the
             tokens to come, and holds that end are given back
  compact    rope_compact_pages: the pages in use move to the lowest numbers

Cases are plain dicts.  `prepare` draws the inputs of a case from a seed, `run` makes one call
(the plain form in elementary torch operations, or the library's entry points where `own` is
set), `exact` gives the same outputs from the definitions in float64, `work` the bytes and
operations a call cannot do without.  A cache in 8 bits is returned as its codes (a tensor of
float8_e4m3fn or int8 values) and its scales.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "int8": 1}
SMALLEST = 2.0 ** -120  # of a scale


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # -- append8
        # one decoding step of 64 conversations, grouped-query heads (32 query, 8 key) of 128
        dict(name="append8_decode", op="append8", dtype="bf16", codes="e4m3", batch=64, min_new=1,
             max_new=1, min_old=100, max_old=2000, nq=32, nk=8, head=128, rd=128, neox=True,
             page=16, block=16, max_seq=32768, lens_seed=1),
        # prompts, half of each head rotated in pairs; some go on behind a cached beginning
        dict(name="append8_prompt", op="append8", dtype="f16", codes="int8", batch=7, min_new=300,
             max_new=3000, min_old=0, max_old=500, nq=32, nk=8, head=128, rd=64, neox=False,
             page=64, block=32, max_seq=32768, lens_seed=2),
        # -- attend8
        # one token of one conversation: latency
        dict(name="attend8_single", op="attend8", dtype="bf16", codes="e4m3", batch=1, nq=16, nk=4,
             head=128, min_len=1001, max_len=1001, min_q=1, max_q=1, page=16, block=16,
             lens_seed=3),
        # a decoding step of 64 conversations of very different lengths, 32 query and 8 key heads
        dict(name="attend8_batch", op="attend8", dtype="bf16", codes="e4m3", batch=64, nq=32, nk=8,
             head=128, min_len=200, max_len=9000, min_q=1, max_q=1, page=16, block=16,
             lens_seed=4),
        # few long contexts, a scale for every token
        dict(name="attend8_long", op="attend8", dtype="f16", codes="int8", batch=6, nq=40, nk=8,
             head=128, min_len=60000, max_len=131072, min_q=1, max_q=1, page=64, block=1,
             lens_seed=5),
        # the next piece of two prompts against a cached beginning
        dict(name="attend8_piece", op="attend8", dtype="bf16", codes="int8", batch=2, nq=16, nk=4,
             head=128, min_len=5500, max_len=5777, min_q=500, max_q=777, page=64, block=64,
             lens_seed=6),
        # -- copy
        # a shared beginning of some pages gets a second copy, 4 layers in 16 bits
        dict(name="copy_few", op="copy", dtype="bf16", layers=4, pages=100, page=64, nk=8, head=128,
             block=64, moved=8),
        # a sequence of 8000 tokens goes to pages set apart, 32 layers in 8 bits
        dict(name="copy_many", op="copy", dtype="e4m3", layers=32, pages=1200, page=16, nk=8,
             head=128, block=16, moved=500),
        # -- fork
        # four beams each of 4 sequences after a step: some beams end, others go on twice
        dict(name="fork_beams", op="fork", dtype="bf16", layers=2, pages=800, page=16, nk=8,
             head=128, block=16, batch=16, rows=16, min_len=40, max_len=500, lens_seed=7),
        # 128 prompts sampled twice each, 32 layers in 8 bits
        dict(name="fork_samples", op="fork", dtype="e4m3", layers=32, pages=6000, page=16, nk=4,
             head=128, block=16, batch=128, rows=256, min_len=100, max_len=2000, lens_seed=8),
        # -- compact
        # a small pool in 16 bits
        dict(name="compact_small", op="compact", dtype="f16", layers=2, pages=333, page=16, nk=2,
             head=64, block=16, batch=8, min_len=10, max_len=700, spread=0.6, lens_seed=9),
        # a large pool of which a good half is in use
        dict(name="compact_large", op="compact", dtype="int8", layers=16, pages=6000, page=16, nk=8,
             head=128, block=16, batch=100, min_len=100, max_len=2000, spread=0.6, lens_seed=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _page_and_block(rng):
    page = rng.choice([1, 8, 16, 16, 32, 64, 64, 100, 128])
    return page, rng.choice([b for b in (1, 4, 5, 16, 32, 64, page) if page % b == 0])


def _draw_append8(rng):
    page, block = _page_and_block(rng)
    head = rng.choice([64, 96, 128, 256])
    nk = rng.choice([1, 2, 5, 8])
    decode = rng.random() < 0.5
    most = 1 if decode else _log_int(rng, 2, 3000)
    return dict(op="append8", dtype=rng.choice(["bf16", "f16", "f32"]),
                codes=rng.choice(["e4m3", "int8"]),
                batch=_log_int(rng, 1, 256 if decode else 16), min_new=max(1, most // 10),
                max_new=most, min_old=rng.choice([0, 1, 100]), max_old=_log_int(rng, 100, 2000),
                nq=nk * rng.choice([1, 3, 4]), nk=nk, head=head,
                rd=rng.choice([r for r in (32, 64, 96, 128, 256) if r <= head]),
                neox=rng.random() < 0.5, page=page, block=block, max_seq=8192,
                lens_seed=rng.randrange(1 << 20))


def _draw_attend8(rng):
    page, block = _page_and_block(rng)
    longest = _log_int(rng, 1, 131072)
    nk = rng.choice([1, 2, 4, 8])
    most = rng.choice([1, 1, 1, 2, 6, _log_int(rng, 2, 777)])
    return dict(op="attend8", dtype=rng.choice(["bf16", "f16"]),
                codes=rng.choice(["e4m3", "int8"]), batch=_log_int(rng, 1, 64),
                nq=nk * rng.choice([1, 4, 5, 8, 16]), nk=nk, head=rng.choice([64, 128, 128, 256]),
                min_len=max(most, longest // 10), max_len=max(most, longest), min_q=1, max_q=most,
                page=page, block=block, lens_seed=rng.randrange(1 << 20))


def _draw_pool(rng):
    page, block = _page_and_block(rng)
    return dict(dtype=rng.choice(["e4m3", "int8", "bf16", "f16", "f32"]),
                layers=_log_int(rng, 1, 32), page=page, nk=rng.choice([1, 2, 4, 8]),
                head=rng.choice([64, 96, 128]), block=block)


def _draw_copy(rng):
    moved = _log_int(rng, 1, 500)
    return dict(op="copy", **_draw_pool(rng), pages=2 * moved + _log_int(rng, 1, 200), moved=moved)


def _draw_fork(rng):
    pool = _draw_pool(rng)
    batch, rows, longest = _log_int(rng, 1, 128), _log_int(rng, 1, 256), _log_int(rng, 10, 2000)
    used = batch * (-(-longest // pool["page"]))
    return dict(op="fork", **pool, pages=used + 7 * rows + rng.randrange(100), batch=batch,
                rows=rows, min_len=max(1, longest // 20), max_len=longest,
                lens_seed=rng.randrange(1 << 20))


def _draw_compact(rng):
    pool = _draw_pool(rng)
    batch, longest = _log_int(rng, 1, 100), _log_int(rng, 10, 2000)
    spread = rng.uniform(0.3, 1.0)
    used = batch * (-(-longest // pool["page"]))
    return dict(op="compact", **pool, pages=int(used / spread) + 1, batch=batch,
                min_len=max(1, longest // 20), max_len=longest, spread=spread,
                lens_seed=rng.randrange(1 << 20))


def _padded(case):
    """Elements that the plain form of a case's attention lays out (sequences are padded to the longest)."""
    if case["op"] != "attend8":
        return 0
    nk, nq = _lengths(case)
    wide = -(-max(nk) // case["page"]) * case["page"]
    return len(nk) * wide * (case["nk"] * case["head"] + case["nq"] * max(nq))


def _pool_bytes(case):
    if "pages" not in case:
        return 0
    return 2 * case["layers"] * case["pages"] * case["page"] * case["nk"] * case["head"] * BYTES[case["dtype"]]


def _cost(case):
    """Memory traffic and products of a case on one scale (bytes)."""
    w = work(case)
    return w["bytes"] + w["flops"] / 100


def draw(rng):
    """A case of the listed ranges that costs no more than the largest listed one of its kind."""
    make = {"append8": _draw_append8, "attend8": _draw_attend8, "copy": _draw_copy,
            "fork": _draw_fork, "compact": _draw_compact}
    op = rng.choice(list(make))
    alike = [c for c in listed() if c["op"] == op]
    while True:
        case = make[op](rng)
        if (_cost(case) <= max(map(_cost, alike)) and _padded(case) <= max(map(_padded, alike)) and
                _pool_bytes(case) <= max(map(_pool_bytes, alike))):
            return case


# ---- sizes ----------------------------------------------------------------------------------

def _lengths(case):
    """(cached tokens, query tokens) of the case's sequences; append8: (all tokens, new tokens)."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "append8":
        new = [_log_int(rng, case["min_new"], case["max_new"]) for _ in range(case["batch"])]
        return [n + rng.randint(case["min_old"], max(case["min_old"], case["max_old"]))
                for n in new], new
    full = [_log_int(rng, case["min_len"], case["max_len"]) for _ in range(case["batch"])]
    if case["op"] != "attend8":
        return full, None
    return full, [min(n, rng.randint(case["min_q"], case["max_q"])) for n in full]


def _counts(case, lengths):
    return [-(-n // case["page"]) for n in lengths]


def _parents(case):
    """fork: (the sequence that each new row continues, -1 for an empty row; tokens to come)."""
    rng = random.Random(case["lens_seed"] + 1)
    batch, rows = case["batch"], case["rows"]
    if rows >= 2 * batch:  # every sequence goes on rows // batch times
        parents = [i * batch // rows for i in range(rows)]
    else:  # beams: some end, some go on more than once, a few rows stay empty
        parents = [-1 if rng.random() < 0.05 else rng.randrange(batch) for _ in range(rows)]
    return parents, [rng.choice([1, 1, 1, 2, 5]) for _ in range(rows)]


def _tail_rows(case):
    """fork: cached tokens of the pages that have to be copied."""
    lens, _ = _lengths(case)
    seen, total = set(), 0
    for p in _parents(case)[0]:
        if p in seen:
            total += lens[p] % case["page"]
        elif p >= 0:
            seen.add(p)
    return total


def _moves(case):
    """compact: pages in use behind the place where all of them would end."""
    used = _used_pages(case)
    return int((used >= len(used)).sum())


def _used_pages(case):
    """compact: the pages in use, spread over the pool."""
    n = sum(_counts(case, _lengths(case)[0]))
    pool = min(case["pages"], max(n, int(n / case["spread"])))
    return np.random.RandomState(case["lens_seed"]).permutation(pool)[:n]


def _token_bytes(case):
    """Bytes of a token in all caches of a case on pages, the scales with their share."""
    row = case["nk"] * case["head"] * BYTES[case["dtype"]]
    if case["dtype"] in CODES:
        row += case["nk"] * 4 / case["block"]
    return 2 * case["layers"] * row


def work(case):
    if case["op"] == "append8":
        es = BYTES[case["dtype"]]
        total, new = _lengths(case)
        t, head, nk = sum(new), case["head"], case["nk"]
        q = 2 * t * case["nq"] * head * es
        kv = 2 * t * nk * head * (es + 1)
        blocks = sum((n - 1) // case["block"] - (n - m) // case["block"] + 1
                     for n, m in zip(total, new))
        rows = min(t, case["max_seq"]) * case["rd"] * es
        return {"bytes": q + kv + 2 * blocks * nk * 8 + rows + 8 * t + 16 * case["batch"],
                "flops": 3 * t * case["rd"] * (case["nq"] + nk) + 4 * t * nk * head}
    if case["op"] == "attend8":
        es = BYTES[case["dtype"]]
        nk, nq = _lengths(case)
        heads, head = case["nk"], case["head"]
        kv = 2 * sum(nk) * heads * head
        scales = 2 * sum(-(-n // case["block"]) for n in nk) * heads * 4
        qo = sum(nq) * case["nq"] * (2 * head * es + 4)
        pairs = sum(q * k - q * (q - 1) // 2 for k, q in zip(nk, nq))
        return {"bytes": kv + scales + qo + 8 * sum(_counts(case, nk)) + 16 * case["batch"],
                "flops": 4 * pairs * case["nq"] * head}
    if case["op"] == "copy":
        return {"bytes": 2 * case["moved"] * (case["page"] * _token_bytes(case) + 8), "flops": 0}
    lens, _ = _lengths(case)
    if case["op"] == "fork":
        wide = max(_counts(case, lens)) + -(-5 // case["page"])
        tables = 8 * (sum(_counts(case, lens)) + case["rows"] * wide)
        return {"bytes": 2 * _tail_rows(case) * _token_bytes(case) + tables + 16 * case["pages"] +
                16 * case["batch"] + 24 * case["rows"], "flops": 0}
    tables = 16 * case["batch"] * max(_counts(case, lens))
    return {"bytes": 2 * _moves(case) * case["page"] * _token_bytes(case) + tables +
            24 * case["pages"], "flops": 0}


# ---- inputs ---------------------------------------------------------------------------------

def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int64, device=DEVICE)


def _offsets(lengths):
    return _ints(np.concatenate([[0], np.cumsum(lengths)]).tolist())


def _table(max_seq, rd, dtype):
    inv = 10000.0 ** (-2.0 * np.arange(rd // 2, dtype=np.float64) / rd)
    a = np.arange(max_seq, dtype=np.float64)[:, None] * inv[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1)).to(DEVICE).to(dtype)


def _filled(gen, codes, pages, page, block, heads, head):
    """A cache of normal values, some channels larger, as codes and scales."""
    x = torch.randn((pages, page // block, block, heads, head), generator=gen, device=DEVICE)
    x *= torch.rand((heads, head), generator=gen, device=DEVICE).pow(4) * 6 + 0.5
    top = x.abs().amax(dim=(2, 4))
    scales = torch.exp2(torch.ceil(torch.log2(top / 448))) if codes == "e4m3" else top / 127
    x /= scales[:, :, None, :, None]
    x = (x if codes == "e4m3" else x.round_()).to(CODES[codes])
    return x.view(pages, page, heads, head), scales


def _page_table(gen, case, lens, spare=0, within=None):
    """Pages of the sequences in no order, and the table's unused places 0."""
    counts = _counts(case, lens)
    table = torch.zeros(len(lens), max(counts) + spare, dtype=torch.int64, device=DEVICE)
    order = torch.randperm(within or sum(counts), generator=gen, device=DEVICE)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table


def _pool(gen, case):
    """The key and value caches of all layers in one allocation, with a list of them as layers
    hold them (and of their scales)."""
    shape = (2 * case["layers"], case["pages"], case["page"], case["nk"], case["head"])
    if case["dtype"] in CODES:
        # bytes as an e4m3 cache may hold them: up to 240 in size, no NaN among them
        x = torch.randint(0, 240, shape, generator=gen, device=DEVICE, dtype=torch.uint8)
        x += (x >= 120) * torch.tensor(8, dtype=torch.uint8, device=DEVICE)
        scales = torch.rand((*shape[:2], case["page"] // case["block"], case["nk"]), generator=gen,
                            device=DEVICE) + 0.5
        x = x.view(CODES[case["dtype"]])
        return {"caches": x, "scales": scales, "list": [*x.unbind(0), *scales.unbind(0)]}
    x = torch.randn(shape, generator=gen, device=DEVICE, dtype=DTYPES[case["dtype"]])
    return {"caches": x, "list": list(x.unbind(0))}


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "append8":
        total, new = _lengths(case)
        dt, t, nq, nk, d = DTYPES[case["dtype"]], sum(new), case["nq"], case["nk"], case["head"]
        s["lens"], s["new"] = total, new
        s["seq_lens"], s["query_offsets"] = _ints(total), _offsets(new)
        s["page_table"] = _page_table(gen, case, total)
        s["positions"] = _ints([p for n, m in zip(total, new) for p in range(n - m, n)])
        s["table"] = _table(case["max_seq"], case["rd"], dt)
        pages = sum(_counts(case, total)) + 3
        for name in ("key", "value"):
            s[name + "_cache"], s[name + "_scales"] = _filled(gen, case["codes"], pages, case["page"],
                                                              case["block"], nk, d)
        qkv = _normal(gen, dt, t, nq + 2 * nk, d)  # one projection's output
        s["query"], s["key"], s["value"] = qkv.split([nq, nk, nk], dim=1)
        s["query_out"] = torch.empty(t, nq, d, dtype=dt, device=DEVICE)
        return s
    if case["op"] == "attend8":
        nk, nq = _lengths(case)
        s["lens"], s["new"] = nk, nq
        s["seq_lens"], s["query_offsets"] = _ints(nk), _offsets(nq)
        s["page_table"] = _page_table(gen, case, nk)
        for name in ("key", "value"):
            s[name + "_cache"], s[name + "_scales"] = _filled(
                gen, case["codes"], sum(_counts(case, nk)), case["page"], case["block"], case["nk"],
                case["head"])
        s["query"] = _normal(gen, DTYPES[case["dtype"]], sum(nq), case["nq"], case["head"])
        s["scale"] = case["head"] ** -0.5
        return s
    s.update(_pool(gen, case))
    if own:  # the description of its caches that a program makes once
        import rope_partial_inplace_amd as ra
        s["list"] = ra.PageCaches(s["list"])
    if case["op"] == "copy":
        order = torch.randperm(case["pages"], generator=gen, device=DEVICE)
        s["sources"] = order[:case["moved"]].contiguous()
        s["targets"] = order[case["moved"]:2 * case["moved"]].contiguous()
        return s
    lens, _ = _lengths(case)
    s["seq_lens"] = _ints(lens)
    if case["op"] == "fork":
        s["page_table"] = _page_table(gen, case, lens, spare=-(-5 // case["page"]),
                                      within=case["pages"])
        parents, grow = _parents(case)
        s["parents"], s["grow"] = _ints(parents), _ints(grow)
    else:
        used = torch.from_numpy(_used_pages(case)).to(DEVICE)
        used = used[torch.randperm(len(used), generator=gen, device=DEVICE)]
        s["page_table"] = _page_table(gen, case, lens)
        s["page_table"] = used[s["page_table"]]
    s["ref_counts"] = torch.zeros(case["pages"], dtype=torch.int64, device=DEVICE)
    held = (torch.arange(s["page_table"].shape[1], device=DEVICE)[None, :] <
            _ints(_counts(case, lens))[:, None])
    s["ref_counts"].index_add_(0, s["page_table"][held], torch.ones_like(s["page_table"][held]))
    return s


# ---- one pass -------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append8": _own_append8, "attend8": _own_attend8, "copy": _own_copy,
                "fork": _own_fork, "compact": _own_compact}[op](state)
    return {"append8": _plain_append8, "attend8": _plain_attend8, "copy": _plain_copy,
            "fork": _plain_fork, "compact": _plain_compact}[op](state)


def _append8_outputs(s):
    return {n: s[n] for n in ("query_out", "key_cache", "key_scales", "value_cache",
                              "value_scales")}


def _pool_outputs(s):
    return {n: s[n] for n in ("caches", "scales") if n in s}


def _own_append8(s):
    import rope_partial_inplace_amd as ra
    ra.rope_append_paged_cache_q8(s["positions"], s["key"], s["value"], s["key_cache"],
                                  s["value_cache"], s["key_scales"], s["value_scales"],
                                  s["page_table"], s["seq_lens"], s["table"],
                                  query_offsets=s["query_offsets"], query=s["query"],
                                  query_out=s["query_out"], is_neox_style=s["case"]["neox"])
    return _append8_outputs(s)


def _own_attend8(s):
    import rope_partial_inplace_amd as ra
    out, lse = ra.rope_attention_paged_q8(s["query"], s["key_cache"], s["value_cache"],
                                          s["key_scales"], s["value_scales"], s["page_table"],
                                          s["seq_lens"], s["scale"],
                                          query_offsets=s["query_offsets"])
    return {"out": out, "lse": lse}


def _own_copy(s):
    import rope_partial_inplace_amd as ra
    ra.rope_copy_pages(s["sources"], s["targets"], s["list"])
    return _pool_outputs(s)


def _own_fork(s):
    import rope_partial_inplace_amd as ra
    table, lens, counts, shortage = ra.rope_fork_pages(s["page_table"], s["seq_lens"], s["parents"],
                                                       s["ref_counts"], s["case"]["page"],
                                                       s["list"], grow=s["grow"])
    return {"page_table": table, "seq_lens": lens, "ref_counts": counts, "shortage": shortage,
            **_pool_outputs(s)}


def _own_compact(s):
    import rope_partial_inplace_amd as ra
    table, counts, page_map, live = ra.rope_compact_pages(s["page_table"], s["ref_counts"],
                                                          s["list"])
    return {"page_table": table, "ref_counts": counts, "page_map": page_map, "live": live,
            **_pool_outputs(s)}


# A scale is the smallest power of two that brings a block's largest value into e4m3's range (so
# that a larger one later costs the block's codes no second rounding), or for int8 a 127th of that
# value; codes are the values times 1 / scale, all in float32, so that both sides round alike.

def _needed_scale(top, codes):
    if codes == "int8":
        return (top * (1.0 / 127)).clamp_min(SMALLEST)
    fraction, exponent = torch.frexp(top)  # top = fraction 2^exponent, 0.5 <= fraction < 1
    exponent = torch.where(top > 0, exponent - 9 + (fraction > 0.875), -120).clamp_min(-120)
    return ((exponent.int() + 127) << 23).view(torch.float32)  # 2^exponent


def _encode(x, codes):
    if codes == "int8":
        return torch.round(x).clamp(-127, 127).to(torch.int8)
    return x.to(torch.float8_e4m3fn)


def _plain_rotate(x, cos, sin, neox):
    """x [T, N, D] in float32, its first 2 cos.shape[1] elements rotated."""
    rd = 2 * cos.shape[-1]
    r, c, s = x[..., :rd], cos[:, None, :], sin[:, None, :]
    if neox:
        a, b = r[..., :rd // 2], r[..., rd // 2:]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rd:]], dim=-1)


def _sequence_of(s):
    """Of every query (or new) token: its sequence, and its place there."""
    t = torch.arange(sum(s["new"]), device=DEVICE)
    b = torch.searchsorted(s["query_offsets"][1:], t, right=True)
    i = t - s["query_offsets"][b]
    return b, i, s["seq_lens"][b] - (s["query_offsets"][b + 1] - s["query_offsets"][b]) + i


def _plain_quantized(s, x, name, b, at):
    """The tokens x [T, heads, D] (float32) into their blocks, whose earlier tokens are coded anew
    where the scale grows."""
    c = s["case"]
    page, block = c["page"], c["block"]
    cache, scales = s[name + "_cache"], s[name + "_scales"]
    codes = cache.view(torch.int8).view(-1, block, *cache.shape[2:])  # [blocks, block, heads, D]
    flat = scales.view(-1, scales.shape[-1])
    unit = s["page_table"][b, at // page] * (page // block) + at % page // block
    top = torch.zeros_like(flat)
    top.scatter_reduce_(0, unit[:, None].expand(-1, top.shape[1]), x.abs().amax(-1), "amax")
    # a sequence's first new token is the only one that may have earlier tokens in its block
    start = s["seq_lens"] - (s["query_offsets"][1:] - s["query_offsets"][:-1])
    unit0 = s["page_table"][torch.arange(len(start), device=DEVICE), start // page]
    unit0 = unit0 * (page // block) + start % page // block
    old = torch.where((start % block != 0)[:, None], flat[unit0], 0.0)
    floor = torch.zeros_like(flat).index_copy_(0, unit0, old)
    now = torch.maximum(_needed_scale(top, c["codes"]), floor)
    earlier = codes[unit0]
    anew = earlier.view(cache.dtype).float() * (old / now[unit0])[:, None, :, None]
    anew = _encode(anew, c["codes"]).view(torch.int8)
    live = torch.arange(block, device=DEVICE)[None, :] < (start % block)[:, None]
    codes[unit0] = torch.where(live[:, :, None, None], anew, earlier)
    flat[unit] = now[unit]
    codes[unit, at % block] = _encode(x * (1.0 / now[unit])[..., None], c["codes"]).view(torch.int8)


def _plain_append8(s):
    c = s["case"]
    rows = s["table"][s["positions"]].float()
    cos, sin = rows[:, :c["rd"] // 2], rows[:, c["rd"] // 2:]
    s["query_out"].copy_(_plain_rotate(s["query"].float(), cos, sin, c["neox"]))
    b, _, at = _sequence_of(s)
    _plain_quantized(s, _plain_rotate(s["key"].float(), cos, sin, c["neox"]), "key", b, at)
    _plain_quantized(s, s["value"].float(), "value", b, at)
    return _append8_outputs(s)


def _plain_rows(s, name):
    """The sequences' keys or values [B, heads, tokens, D] in float32, padded to the longest."""
    c, table = s["case"], s["page_table"]
    cache, scales = s[name + "_cache"], s[name + "_scales"]
    x = cache.view(torch.int8)[table].view(cache.dtype).float()  # [B, pages, page, heads, D]
    x = x.unflatten(2, (-1, c["block"])) * scales[table][:, :, :, None, :, None]
    return x.flatten(1, 3).transpose(1, 2).contiguous()


def _plain_attend8(s):
    c = s["case"]
    batch, most, group, dt = len(s["new"]), max(s["new"]), c["nq"] // c["nk"], s["query"].dtype
    b, i, _ = _sequence_of(s)
    q = torch.zeros(batch, most, c["nq"], c["head"], device=DEVICE)
    q[b, i] = s["query"].float()
    q = q.unflatten(2, (c["nk"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3).contiguous()
    scores = torch.matmul(q, _plain_rows(s, "key").transpose(2, 3).contiguous()) * s["scale"]
    # query i of n sees the first len - n + 1 + i tokens
    seen = (s["seq_lens"] - (s["query_offsets"][1:] - s["query_offsets"][:-1]) + 1)[:, None]
    seen = (seen + torch.arange(most, device=DEVICE)).clamp_min(1)
    hidden = torch.arange(scores.shape[-1], device=DEVICE) >= seen.repeat_interleave(group, 1)[..., None]
    scores.masked_fill_(hidden[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - top)
    del scores
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, _plain_rows(s, "value")) / total
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.unflatten(2, (most, group))[b, :, i].flatten(1, 2).to(dt)
    return {"out": out, "lse": lse.unflatten(2, (most, group))[b, :, i].flatten(1, 2)}


def _as_bytes(x):
    return x.view(torch.int8) if x.element_size() == 1 else x


def _plain_copy(s):
    for x in _pool_outputs(s).values():
        x = _as_bytes(x)
        x[:, s["targets"]] = x[:, s["sources"]]
    return _pool_outputs(s)


def _plain_fork(s):
    page, table, counts = s["case"]["page"], s["page_table"], s["ref_counts"]
    batch, rows, pages = table.shape[0], len(s["parents"]), len(counts)
    row, place = torch.arange(rows, device=DEVICE), torch.arange(table.shape[1], device=DEVICE)
    some = (s["parents"] >= 0) & (s["parents"] < batch)
    parent = torch.where(some, s["parents"], 0)
    length = torch.where(some, s["seq_lens"][parent], 0)
    grown = length + torch.where(some, s["grow"], 0)
    used, wanted, tail = -(-length // page), -(-grown // page), length % page
    last = table[parent, (used - 1).clamp_min(0)]
    # the first row that continues a sequence keeps its last page, unless something else holds it too
    first = torch.full((batch + 1,), rows, device=DEVICE)
    first.scatter_reduce_(0, torch.where(some, parent, batch), row, "amin")
    keep = some & (first[parent] == row) & (counts[last] <= 1)
    copied = some & (tail > 0) & ~keep
    need = copied + wanted - used
    base = need.cumsum(0) - need
    free = counts == 0
    order = torch.full((pages + rows * table.shape[1] + 1,), -1, device=DEVICE)
    order.scatter_(0, torch.where(free, free.cumsum(0) - 1, pages + rows * table.shape[1]),
                   torch.arange(pages, device=DEVICE))
    order[-1] = -1
    # the new table
    fresh = (place >= (used - copied.long())[:, None]) & (place < wanted[:, None])
    rank = base[:, None] + place - (used - copied.long())[:, None]
    taken = torch.where(fresh, order[torch.where(fresh, rank, 0)], -1)
    new_table = torch.where(fresh, taken, torch.where(place < used[:, None], table[parent], -1))
    # holds: a sequence's full pages go on once for every row, its last page if it is kept
    children = torch.zeros(batch + 1, dtype=torch.int64, device=DEVICE)
    children.index_add_(0, torch.where(some, parent, batch), torch.ones_like(parent))
    kept = torch.zeros(batch, dtype=torch.int64, device=DEVICE)
    kept.scatter_reduce_(0, parent, (keep & some).long(), "amax")
    held = -(-s["seq_lens"] // page)
    partial = (place == held[:, None] - 1) & (s["seq_lens"] % page != 0)[:, None]
    delta = torch.where(partial, kept[:, None], children[:batch, None]) - 1
    delta = torch.where(place < held[:, None], delta, 0)
    new_counts = counts.clone()
    new_counts.index_add_(0, table.flatten(), delta.flatten())
    got = taken.flatten()
    new_counts.index_add_(0, got.clamp_min(0), (got >= 0).long())
    # the copies: a row without one writes its own page (page 0 where it has none) onto itself
    target = torch.where(copied, order[base], last)
    for name, x in _pool_outputs(s).items():
        x = _as_bytes(x)
        live = -(-tail * x.shape[2] // page)
        mask = torch.arange(x.shape[2], device=DEVICE) < live[:, None]
        mask = mask.view(rows, x.shape[2], *[1] * (x.dim() - 3))
        x[:, target] = torch.where(mask, x[:, last], x[:, target])
    short = (need.sum() - free.sum()).clamp_min(0)
    return {"page_table": new_table, "seq_lens": grown, "ref_counts": new_counts,
            "shortage": short.view(1), **_pool_outputs(s)}


def _plain_compact(s):
    counts = s["ref_counts"]
    page = torch.arange(len(counts), device=DEVICE)
    used = counts > 0
    live = used.sum()
    sources = torch.nonzero(used & (page >= live)).squeeze(1)
    targets = torch.nonzero(~used & (page < live)).squeeze(1)
    page_map = torch.where(used, page, -1)
    page_map[sources] = targets
    new_counts = counts.clone()
    new_counts[targets] = counts[sources]
    new_counts[sources] = 0
    for x in _pool_outputs(s).values():
        x = _as_bytes(x)
        x[:, targets] = x[:, sources]
    return {"page_table": page_map[s["page_table"]], "ref_counts": new_counts,
            "page_map": page_map, "live": live.view(1), **_pool_outputs(s)}


# ---- from the definitions, in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append8":
        return _exact_append8(case, s)
    if case["op"] == "attend8":
        return _exact_attend8(case, s)
    return {"copy": _exact_copy, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](case, s)


_E4M3 = np.array([(-1.0 if b & 128 else 1.0) * (
    math.nan if b & 127 == 127 else
    (b & 7) * 2.0 ** -9 if b & 120 == 0 else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10))
    for b in range(256)])


def _nearest(x, codes):
    """x (float64) rounded to the nearest value of the codes' type, ties to even."""
    if codes == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append8(c, s):
    half, page, block = c["rd"] // 2, c["page"], c["block"]
    turn = s["table"].double()[s["positions"]]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None, :]

    def rotated(x):
        y = x.double().clone()
        a, b = ((slice(0, half), slice(half, 2 * half)) if c["neox"] else
                (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
        z = torch.complex(y[..., a], y[..., b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
        return y

    out = {"query_out": rotated(s["query"])}
    levels = torch.from_numpy(_E4M3).to(DEVICE)
    limit = 127.0 if c["codes"] == "int8" else 448.0
    for name, x in (("key", rotated(s["key"])), ("value", s["value"].double())):
        cache, scales = s[name + "_cache"], s[name + "_scales"].double()
        if c["codes"] == "int8":
            codes = cache.double()
        else:
            codes = levels[cache.view(torch.uint8).long()]
        at = 0
        for b, (n, m) in enumerate(zip(s["lens"], s["new"])):
            pages = s["page_table"][b, :-(-n // page)]
            # the blocks from the one of the first new token on, as rows of this sequence
            first = (n - m) // block * block
            many = -(-(n - first) // block)
            where = first + torch.arange(many * block, device=DEVICE)
            where, off = pages[where // page], where % page
            rows = codes[where, off].view(many, block, *x.shape[1:])
            place = where.view(many, block)[:, 0], off.view(many, block)[:, 0] // block
            new = torch.zeros(many * block, *x.shape[1:], dtype=torch.float64, device=DEVICE)
            new[n - m - first:n - first] = x[at:at + m]
            new = new.view_as(rows)
            need = new.abs().amax(dim=(1, 3)) / limit
            if c["codes"] == "e4m3":
                need = torch.exp2(torch.ceil(torch.log2(need.clamp_min(SMALLEST))))
            need = need.clamp_min(SMALLEST)
            before = n - m - first  # earlier tokens of the first block
            now = need.clone()
            if before:
                old = scales[place][0]
                now[0] = torch.maximum(need[0], old)
                rows[0, :before] = _nearest(rows[0, :before] * (old / now[0])[:, None], c["codes"])
            coded = _nearest(new / now[:, None, :, None], c["codes"])
            flat, coded = rows.view(-1, *x.shape[1:]), coded.view(-1, *x.shape[1:])
            flat[before:before + m] = coded[before:before + m]
            codes[where, off] = flat
            scales[place] = now
            at += m
        out[name + "_cache"], out[name + "_scales"] = codes, scales
    return out


def _exact_attend8(c, s):
    page, block, group = c["page"], c["block"], c["nq"] // c["nk"]
    f64 = dict(dtype=torch.float64, device=DEVICE)
    levels = torch.from_numpy(_E4M3).to(DEVICE)
    out = torch.empty(sum(s["new"]), c["nq"], c["head"], **f64)
    lse = torch.empty(sum(s["new"]), c["nq"], **f64)
    at = 0
    for b, (nk, nq) in enumerate(zip(s["lens"], s["new"])):
        token = torch.arange(nk, device=DEVICE)
        where, off = s["page_table"][b, token // page], token % page
        hidden = torch.ones(nq, nk, dtype=torch.bool, device=DEVICE).triu(nk - nq + 1)
        hidden = hidden.repeat_interleave(group, 0)
        for h in range(c["nk"]):
            k, v = (x[where, off, h] for x in (s["key_cache"].view(torch.uint8),
                                               s["value_cache"].view(torch.uint8)))
            if c["codes"] == "int8":
                k, v = k.view(torch.int8).double(), v.view(torch.int8).double()
            else:
                k, v = levels[k.long()], levels[v.long()]
            k = k * s["key_scales"][where, off // block, h].double()[:, None]
            v = v * s["value_scales"][where, off // block, h].double()[:, None]
            heads = slice(h * group, (h + 1) * group)
            logits = s["query"][at:at + nq, heads].double().flatten(0, 1) @ k.t() * s["scale"]
            logits[hidden] = -math.inf
            total = torch.logsumexp(logits, dim=1)
            lse[at:at + nq, heads] = total.view(nq, group)
            out[at:at + nq, heads] = (torch.exp(logits - total[:, None]) @ v).view(nq, group, -1)
        at += nq
    return {"out": out, "lse": lse}


# The operators on pages move data and count: their outputs are whole numbers, or copies, whose
# definition is written with lists of pages here.

def _exact_pool(s, pairs, rows=None):
    """The caches after the copies (source, target), of `rows` tokens each where given."""
    out = {}
    for name, x in _pool_outputs(s).items():
        x = x.clone()
        raw = _as_bytes(x)
        before = raw.clone()
        for k, (a, b) in enumerate(pairs):
            n = raw.shape[2] if rows is None else -(-rows[k] * raw.shape[2] // s["case"]["page"])
            raw[:, b, :n] = before[:, a, :n]
        out[name] = x.double() if x.dtype != torch.int8 else x
    return out


def _exact_copy(c, s):
    return _exact_pool(s, list(zip(s["sources"].tolist(), s["targets"].tolist())))


def _exact_fork(c, s):
    page, counts, table = c["page"], s["ref_counts"].tolist(), s["page_table"].tolist()
    lens, wide = s["seq_lens"].tolist(), s["page_table"].shape[1]
    held_before = list(counts)
    free = [p for p, n in enumerate(counts) if n == 0]
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            counts[table[b][j]] -= 1
    begun, rows, new_lens, pairs, tails, short = set(), [], [], [], [], 0
    for p, g in zip(s["parents"].tolist(), s["grow"].tolist()):
        if not 0 <= p < len(lens):
            rows.append([])
            new_lens.append(0)
            continue
        n = lens[p]
        row = table[p][:-(-n // page)]
        if n % page and (p in begun or held_before[row[-1]] > 1):
            short += not free
            got = free.pop(0) if free else -1
            pairs.append((row[-1], got))
            tails.append(n % page)
            row[-1] = got
        begun.add(p)
        while len(row) < -(-(n + g) // page):
            short += not free
            row.append(free.pop(0) if free else -1)
        for q in row:
            if q >= 0:
                counts[q] += 1
        rows.append(row)
        new_lens.append(n + g)
    rows = [r + [-1] * (wide - len(r)) for r in rows]
    return {"page_table": _ints(rows), "seq_lens": _ints(new_lens), "ref_counts": _ints(counts),
            "shortage": _ints([short]), **_exact_pool(s, pairs, tails)}


def _exact_compact(c, s):
    counts = s["ref_counts"].tolist()
    live = sum(n > 0 for n in counts)
    holes = [p for p in range(live) if counts[p] == 0]
    pairs = list(zip((p for p in range(live, len(counts)) if counts[p] > 0), holes))
    moved = [p if n > 0 else -1 for p, n in enumerate(counts)]
    for a, b in pairs:
        moved[a], counts[b], counts[a] = b, counts[a], 0
    table = [[moved[p] for p in row] for row in s["page_table"].tolist()]
    return {"page_table": _ints(table), "ref_counts": _ints(counts), "page_map": _ints(moved),
            "live": _ints([live]), **_exact_pool(s, pairs)}
