"""Measured calls of the paged-cache append and the latent attention operators.

Three families, as a latent-attention or grouped-query decoder uses them around the rotary
position embedding:

  append    rope_append_paged_cache: a batch of new tokens' keys (and values) is rotated by
            position and written to its slots of a paged cache; the queries are rotated by the
            same launch
  absorbed  rope_latent_attention_paged: every head of a query attends to one shared latent row
            per cached token (key = the whole row, value = its first latent_dim elements)
  expanded  rope_latent_attention and its backward: keys and values of every head expanded from
            the latent, with one rotated key part shared by the heads

Cases are plain dicts.  `prepare` draws the inputs of a case from a seed, `run` makes one call
(the plain form in elementary torch operations, or the library's entry points where `own` is
set), `exact` gives the same outputs from the definitions in float64, `work` the bytes and
operations a call cannot do without.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
ROPE = 64  # rotated elements of a latent row, and of an expanded query head


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # -- append
        # one decoding step of 64 sequences, grouped-query heads (32 query, 8 key) of 128
        dict(name="append_decode", op="append", dtype="bf16", tokens=64, nq=32, nk=8, head=128,
             value=True, rd=128, q_start=0, k_start=0, neox=True, page=16, max_seq=32768),
        # a prompt of 8192 tokens, half of each head rotated in pairs
        dict(name="append_prompt", op="append", dtype="f16", tokens=8192, nq=32, nk=8, head=128,
             value=True, rd=64, q_start=0, k_start=0, neox=False, page=64, max_seq=32768),
        # latent rows of 8 x 4096 tokens: 512 latent elements and a rotated tail of 64; the
        # queries' rotated parts go to the tail of the absorbed query
        dict(name="append_latent", op="append", dtype="bf16", tokens=32768, nq=16, nk=1, head=576,
             value=False, rd=64, q_start=128, k_start=512, neox=False, page=64, max_seq=8192),
        # -- absorbed
        # one token of one conversation, 16 heads: latency
        dict(name="absorbed_single", op="absorbed", dtype="bf16", batch=1, heads=16, latent=512,
             min_len=1001, max_len=1001, min_q=1, max_q=1, page=64, lens_seed=1),
        # a decoding step of 64 conversations of very different lengths, 32 heads
        dict(name="absorbed_batch", op="absorbed", dtype="bf16", batch=64, heads=32, latent=512,
             min_len=200, max_len=9000, min_q=1, max_q=1, page=64, lens_seed=2),
        # drafted tokens being verified: up to 5 queries a sequence, 16 heads, small pages
        dict(name="absorbed_draft", op="absorbed", dtype="f16", batch=24, heads=16, latent=512,
             min_len=100, max_len=5000, min_q=1, max_q=5, page=16, lens_seed=3),
        # few long contexts with all 128 heads
        dict(name="absorbed_long", op="absorbed", dtype="bf16", batch=6, heads=128, latent=512,
             min_len=60000, max_len=131072, min_q=1, max_q=1, page=64, lens_seed=4),
        # -- expanded
        # a batch of prompts, packed one behind the other
        dict(name="expanded_prompts", op="expanded", dtype="bf16", batch=7, heads=32, dim=128,
             min_len=300, max_len=6000, prefix=0, causal=True, train=False, lens_seed=5),
        # the next piece of a prompt against a cached beginning
        dict(name="expanded_piece", op="expanded", dtype="f16", batch=2, heads=16, dim=128,
             min_len=500, max_len=777, prefix=5000, causal=True, train=False, lens_seed=6),
        # one training step's attention, 4 x 2048 tokens of 32 heads, forward and gradients
        dict(name="expanded_train", op="expanded", dtype="bf16", batch=4, heads=32, dim=128,
             min_len=2048, max_len=2048, prefix=0, causal=True, train=True, lens_seed=7),
        # a small unmasked one (an encoder over short ragged texts), narrow heads
        dict(name="expanded_train_small", op="expanded", dtype="f16", batch=5, heads=8, dim=64,
             min_len=17, max_len=333, prefix=0, causal=False, train=True, lens_seed=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_append(rng):
    tokens = _log_int(rng, 1, 32768)
    dtype = rng.choice(["bf16", "f16", "f32"])
    if rng.random() < 0.4:
        return dict(op="append", dtype=dtype, tokens=tokens, nq=rng.choice([4, 8, 16]), nk=1,
                    head=rng.choice([576, 320]), value=False, rd=64, q_start=128,
                    k_start=rng.choice([0, 256]), neox=rng.random() < 0.5,
                    page=rng.choice([1, 16, 64, 100]), max_seq=8192)
    head = rng.choice([64, 96, 128])
    rd = rng.choice([r for r in (32, 64, 96, 128) if r <= head])
    nk = rng.choice([1, 2, 5, 8])
    return dict(op="append", dtype=dtype, tokens=tokens, nq=nk * rng.choice([1, 3, 4]), nk=nk,
                head=head, value=True, rd=rd, q_start=0, k_start=0, neox=rng.random() < 0.5,
                page=rng.choice([1, 16, 64, 100]), max_seq=32768)


def _draw_absorbed(rng):
    max_len = _log_int(rng, 1, 131072)
    max_q = rng.choice([1, 1, 1, 2, 6])
    return dict(op="absorbed", dtype=rng.choice(["bf16", "f16"]), batch=_log_int(rng, 1, 64),
                heads=rng.choice([4, 8, 16, 24, 32, 64, 128]),
                latent=rng.choice([512, 512, 256, 128]), min_len=max(max_q, max_len // 10),
                max_len=max(max_q, max_len), min_q=1, max_q=max_q,
                page=rng.choice([1, 16, 64, 100]), lens_seed=rng.randrange(1 << 20))


def _draw_expanded(rng):
    max_len = _log_int(rng, 1, 6000)
    train = rng.random() < 0.5
    return dict(op="expanded", dtype=rng.choice(["bf16", "f16"]), batch=rng.randint(1, 7),
                heads=rng.choice([1, 4, 8, 16, 31]), dim=rng.choice([128, 128, 64]),
                min_len=max(1, max_len // 8), max_len=max_len,
                prefix=rng.choice([0, 0, _log_int(rng, 1, 5000)]), causal=rng.random() < 0.7,
                train=train, lens_seed=rng.randrange(1 << 20))


def _cost(case):
    """Memory traffic and products of a case on one scale (bytes)."""
    w = work(case)
    return w["bytes"] + w["flops"] / 100


def draw(rng):
    """A case of the listed ranges that costs no more than the largest listed one of its kind."""
    op = rng.choice(["append", "absorbed", "expanded"])
    make = {"append": _draw_append, "absorbed": _draw_absorbed, "expanded": _draw_expanded}[op]
    while True:
        case = make(rng)
        alike = [c for c in listed() if c["op"] == op and c.get("train") == case.get("train")]
        if _cost(case) <= max(_cost(c) for c in alike):
            return case


# ---- sizes ----------------------------------------------------------------------------------

def _lengths(case):
    """(key lengths, query lengths) of the case's sequences."""
    rng = random.Random(case["lens_seed"])
    full = [_log_int(rng, case["min_len"], case["max_len"]) for _ in range(case["batch"])]
    if case["op"] == "absorbed":
        return full, [min(n, rng.randint(case["min_q"], case["max_q"])) for n in full]
    return [n + case["prefix"] for n in full], full


def _pairs(case):
    """Visible (query, key) pairs of all sequences."""
    total = 0
    for nk, nq in zip(*_lengths(case)):
        causal = case["op"] == "absorbed" or case["causal"]
        total += nq * nk - (nq * (nq - 1) // 2 if causal else 0)
    return total


def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "append":
        t, rd = case["tokens"], case["rd"]
        latent = not case["value"]
        q = t * case["nq"] * (rd if latent else case["head"])
        k = t * case["nk"] * case["head"] * (2 if case["value"] else 1)
        rows = min(t, case["max_seq"])  # each table row is needed once
        rotated = t * rd * (case["nq"] + case["nk"])
        return {"bytes": 2 * (q + k) * es + rows * rd * es + 16 * t, "flops": 3 * rotated}
    if case["op"] == "absorbed":
        nk, nq = _lengths(case)
        row, h = case["latent"] + ROPE, case["heads"]
        kv = sum(nk) * row * es
        qo = sum(nq) * h * ((row + case["latent"]) * es + 4)
        table = 8 * sum(-(-n // case["page"]) for n in nk) + 16 * case["batch"]
        return {"bytes": kv + qo + table, "flops": 2 * _pairs(case) * h * (row + case["latent"])}
    nk, nq = _lengths(case)
    h, d = case["heads"], case["dim"]
    q = sum(nq) * h * (d + ROPE) * es
    k = sum(nk) * (h * 2 * d + ROPE) * es
    o = sum(nq) * h * d * es
    lse = sum(nq) * h * 4
    n_bytes, flops = q + k + o + lse, 2 * _pairs(case) * h * (2 * d + ROPE)
    if case["train"]:  # backward: all of it again, the incoming gradient, three gradients out;
        n_bytes += q + k + o + lse + o + q + k  # five products
        flops += 2 * _pairs(case) * h * (3 * (d + ROPE) + 2 * d)
    return {"bytes": n_bytes, "flops": flops}


# ---- inputs ---------------------------------------------------------------------------------

def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)


def _offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int64,
                        device=DEVICE)


def _table(max_seq, rd, dtype):
    inv = 10000.0 ** (-2.0 * np.arange(rd // 2, dtype=np.float64) / rd)
    a = np.arange(max_seq, dtype=np.float64)[:, None] * inv[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1)).to(DEVICE).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "append":
        t, nq, nk, d = case["tokens"], case["nq"], case["nk"], case["head"]
        pages = -(-t // case["page"]) + 3
        s["positions"] = torch.randint(0, case["max_seq"], (t,), generator=gen, device=DEVICE)
        s["slots"] = torch.randperm(pages * case["page"], generator=gen, device=DEVICE)[:t]
        # sequences own whole pages, so neighbouring tokens mostly share one
        s["slots"] = s["slots"].sort().values.contiguous()
        s["table"] = _table(case["max_seq"], case["rd"], dt)
        s["key_cache"] = _normal(gen, dt, pages, case["page"], nk, d)
        if case["value"]:
            qkv = _normal(gen, dt, t, nq + 2 * nk, d)  # one projection's output
            s["query"], s["key"], s["value"] = qkv.split([nq, nk, nk], dim=1)
            s["value_cache"] = _normal(gen, dt, pages, case["page"], nk, d)
            s["query_out"] = torch.empty(t, nq, d, dtype=dt, device=DEVICE)
        else:
            s["key"] = _normal(gen, dt, t, 1, d)
            s["query"] = _normal(gen, dt, t, nq, case["q_start"] + case["rd"])[..., case["q_start"]:]
            # the tail of the absorbed query, whose first d - rd elements a product fills
            s["query_full"] = torch.zeros(t, nq, d, dtype=dt, device=DEVICE)
            s["query_out"] = s["query_full"][..., d - case["rd"]:]
        return s
    nk, nq = _lengths(case)
    s["nk"], s["nq"] = nk, nq
    s["query_offsets"] = _offsets(nq)
    if case["op"] == "absorbed":
        row, page = case["latent"] + ROPE, case["page"]
        counts = [-(-n // page) for n in nk]
        s["cache"] = _normal(gen, dt, sum(counts), page, row)
        order = torch.randperm(sum(counts), generator=gen, device=DEVICE)
        table = torch.zeros(len(nk), max(counts), dtype=torch.int64, device=DEVICE)
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = order[at:at + c]
            at += c
        s["page_table"] = table
        s["seq_lens"] = torch.tensor(nk, dtype=torch.int64, device=DEVICE)
        s["query"] = _normal(gen, dt, sum(nq), case["heads"], row)
        s["scale"] = (128 + ROPE) ** -0.5
        return s
    h, d = case["heads"], case["dim"]
    s["key_offsets"] = _offsets(nk)
    s["query"] = _normal(gen, dt, sum(nq), h, d + ROPE)
    # one up-projection's output holds a head's key and value side by side
    s["key"], s["value"] = _normal(gen, dt, sum(nk), h, 2 * d).split([d, d], dim=2)
    s["key_rope"] = _normal(gen, dt, sum(nk), ROPE)
    if case["train"]:
        s["grad"] = _normal(gen, dt, sum(nq), h, d)
    s["scale"] = (d + ROPE) ** -0.5
    return s


# ---- one pass -------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "absorbed": _own_absorbed, "expanded": _own_expanded}[op](state)
    return {"append": _plain_append, "absorbed": _plain_absorbed,
            "expanded": _plain_expanded}[op](state)


def _own_append(s):
    import rope_partial_inplace_amd as ra
    c = s["case"]
    ra.rope_append_paged_cache(s["positions"], s["slots"], s["key"], s["key_cache"], s["table"],
                               value=s.get("value"), value_cache=s.get("value_cache"),
                               query=s["query"], query_out=s["query_out"],
                               key_rot_start=c["k_start"], is_neox_style=c["neox"])
    return _append_outputs(s)


def _append_outputs(s):
    out = {"query": s["query_out"], "key_cache": s["key_cache"]}
    if "value" in s:
        out["value_cache"] = s["value_cache"]
    return out


def _own_absorbed(s):
    import rope_partial_inplace_amd as ra
    out, lse = ra.rope_latent_attention_paged(s["query"], s["cache"], s["page_table"],
                                              s["seq_lens"], s["case"]["latent"], s["scale"],
                                              query_offsets=s["query_offsets"])
    return {"out": out, "lse": lse}


def _own_expanded(s):
    import rope_partial_inplace_amd as ra
    c = s["case"]
    where = dict(causal=c["causal"], query_offsets=s["query_offsets"],
                 key_offsets=s["key_offsets"])
    args = (s["query"], s["key"], s["key_rope"], s["value"])
    out, lse = ra.rope_latent_attention(*args, s["scale"], **where)
    res = {"out": out, "lse": lse}
    if c["train"]:
        dq, dk, dkr, dv = ra.rope_latent_attention_backward(s["grad"], *args, out, lse,
                                                            s["scale"], **where)
        res.update(dquery=dq, dkey=dk, dkey_rope=dkr, dvalue=dv)
    return res


def _plain_rotate(x, start, cos, sin, neox):
    """x [T, N, D] in float32, its elements [start, start + rd) rotated."""
    rd = 2 * cos.shape[-1]
    r = x[..., start:start + rd]
    c, s = cos[:, None, :], sin[:, None, :]
    if neox:
        a, b = r[..., :rd // 2], r[..., rd // 2:]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    return torch.cat([x[..., :start], turned, x[..., start + rd:]], dim=-1)


def _plain_append(s):
    c = s["case"]
    rows = s["table"][s["positions"]].float()
    cos, sin = rows[:, :c["rd"] // 2], rows[:, c["rd"] // 2:]
    dt = s["key"].dtype
    s["query_out"].copy_(_plain_rotate(s["query"].float(), 0, cos, sin, c["neox"]).to(dt))
    k = _plain_rotate(s["key"].float(), c["k_start"], cos, sin, c["neox"]).to(dt)
    s["key_cache"].view(-1, *k.shape[1:])[s["slots"]] = k
    if "value" in s:
        s["value_cache"].view(-1, *k.shape[1:])[s["slots"]] = s["value"]
    return _append_outputs(s)


def _plain_softmax(scores):
    """Probabilities and log-sum-exp over the last axis (every row sees something)."""
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    return e / total, (top + torch.log(total)).squeeze(-1)


def _plain_mask(nq, nk):
    """True where query i of nq may not see key j of nk: the last query sees all keys."""
    i = torch.arange(nq, device=DEVICE)[:, None]
    return torch.arange(nk, device=DEVICE)[None, :] > i + (nk - nq)


def _plain_absorbed(s):
    c, dt = s["case"], s["query"].dtype
    outs, lses, at = [], [], 0
    for b, (nk, nq) in enumerate(zip(s["nk"], s["nq"])):
        pages = s["page_table"][b, :-(-nk // c["page"])]
        rows = s["cache"][pages].reshape(-1, s["cache"].shape[-1])[:nk].float()
        q = s["query"][at:at + nq].float()
        scores = (q @ rows.t()) * s["scale"]  # [nq, heads, nk]
        if nq > 1:
            scores.masked_fill_(_plain_mask(nq, nk)[:, None, :], -math.inf)
        p, lse = _plain_softmax(scores)
        outs.append(p @ rows[:, :c["latent"]])
        lses.append(lse)
        at += nq
    return {"out": torch.cat(outs).to(dt), "lse": torch.cat(lses)}


def _plain_expanded(s):
    c, dt, scale = s["case"], s["query"].dtype, s["scale"]
    d, h = c["dim"], c["heads"]
    parts = {"out": [], "lse": [], "dquery": [], "dkey": [], "dkey_rope": [], "dvalue": []}
    qa = ka = 0
    for nk, nq in zip(s["nk"], s["nq"]):
        q = s["query"][qa:qa + nq].float().transpose(0, 1)
        kr = s["key_rope"][ka:ka + nk].float()
        k = torch.cat([s["key"][ka:ka + nk].float(), kr[:, None, :].expand(nk, h, ROPE)], dim=-1)
        k = k.transpose(0, 1).contiguous()
        v = s["value"][ka:ka + nk].float().transpose(0, 1).contiguous()
        scores = torch.matmul(q, k.transpose(1, 2)) * scale
        if c["causal"]:
            scores.masked_fill_(_plain_mask(nq, nk), -math.inf)
        p, lse = _plain_softmax(scores)
        del scores
        o = torch.matmul(p, v)
        parts["out"].append(o.transpose(0, 1))
        parts["lse"].append(lse.transpose(0, 1))
        if c["train"]:
            g = s["grad"][qa:qa + nq].float().transpose(0, 1)
            dp = torch.matmul(g, v.transpose(1, 2))
            ds = p * (dp - (g * o).sum(-1, keepdim=True)) * scale
            del dp
            dk = torch.matmul(ds.transpose(1, 2), q).transpose(0, 1)
            parts["dquery"].append(torch.matmul(ds, k).transpose(0, 1))
            parts["dkey"].append(dk[..., :d])
            parts["dkey_rope"].append(dk[..., d:].sum(1))
            parts["dvalue"].append(torch.matmul(p.transpose(1, 2), g).transpose(0, 1))
        qa += nq
        ka += nk
    return {name: torch.cat(p).to(torch.float32 if name == "lse" else dt)
            for name, p in parts.items() if p}


# ---- from the definitions, in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_absorbed(case, s) if case["op"] == "absorbed" else _exact_expanded(case, s)


def _exact_append(c, s):
    """The rotation as a product of complex numbers, one for each pair of elements."""
    half = c["rd"] // 2
    turn = s["table"].double()[s["positions"]]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None, :]

    def rotated(x, start):
        y = x.double().clone()
        if c["neox"]:
            first, second = slice(start, start + half), slice(start + half, start + 2 * half)
        else:
            first = slice(start, start + 2 * half, 2)
            second = slice(start + 1, start + 2 * half, 2)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"query": rotated(s["query"], 0)}
    new = {"key_cache": rotated(s["key"], c["k_start"])}
    if c["value"]:
        new["value_cache"] = s["value"].double()
    page, offset = s["slots"] // c["page"], s["slots"] % c["page"]
    for name, rows in new.items():
        cache = s[name].double()
        cache[page, offset] = rows
        out[name] = cache
    return out


def _exact_absorbed(c, s):
    page = c["page"]
    out = torch.empty(sum(s["nq"]), c["heads"], c["latent"], dtype=torch.float64, device=DEVICE)
    lse = torch.empty(sum(s["nq"]), c["heads"], dtype=torch.float64, device=DEVICE)
    at = 0
    for b, (nk, nq) in enumerate(zip(s["nk"], s["nq"])):
        where = torch.arange(nk, device=DEVICE)
        keys = s["cache"][s["page_table"][b, where // page], where % page].double()
        for i in range(nq):
            seen = keys[:nk - nq + 1 + i]
            logits = s["query"][at].double() @ seen.t() * s["scale"]
            lse[at] = torch.logsumexp(logits, dim=1)
            out[at] = torch.exp(logits - lse[at][:, None]) @ seen[:, :c["latent"]]
            at += 1
    return {"out": out, "lse": lse}


def _exact_expanded(c, s):
    d, h = c["dim"], c["heads"]
    f64 = dict(dtype=torch.float64, device=DEVICE)
    tq, tk = sum(s["nq"]), sum(s["nk"])
    r = {"out": torch.empty(tq, h, d, **f64), "lse": torch.empty(tq, h, **f64)}
    if c["train"]:
        r.update(dquery=torch.empty(tq, h, d + ROPE, **f64), dkey=torch.empty(tk, h, d, **f64),
                 dkey_rope=torch.zeros(tk, ROPE, **f64), dvalue=torch.empty(tk, h, d, **f64))
    qa = ka = 0
    for nk, nq in zip(s["nk"], s["nq"]):
        qs, ks = slice(qa, qa + nq), slice(ka, ka + nk)
        rope = s["key_rope"][ks].double()
        hidden = None
        if c["causal"]:
            hidden = torch.ones(nq, nk, dtype=torch.bool, device=DEVICE).triu(nk - nq + 1)
        for head in range(h):
            q, k = s["query"][qs, head].double(), s["key"][ks, head].double()
            v = s["value"][ks, head].double()
            logits = (q[:, :d] @ k.t() + q[:, d:] @ rope.t()) * s["scale"]
            if hidden is not None:
                logits[hidden] = -math.inf
            lse = torch.logsumexp(logits, dim=1, keepdim=True)
            p = torch.exp(logits - lse)
            r["lse"][qs, head] = lse[:, 0]
            r["out"][qs, head] = p @ v
            if c["train"]:
                g = s["grad"][qs, head].double()
                dp = g @ v.t()
                dl = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
                r["dquery"][qs, head, :d] = dl @ k
                r["dquery"][qs, head, d:] = dl @ rope
                r["dkey"][ks, head] = dl.t() @ q[:, :d]
                r["dkey_rope"][ks] += dl.t() @ q[:, d:]
                r["dvalue"][ks, head] = p.t() @ g
        qa += nq
        ka += nk
    return r
