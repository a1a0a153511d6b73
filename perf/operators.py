"""Cases of the attention operators: normed and rotated heads appended to a paged cache, attention over packed
prompts, and attention of a batch whose sequences share a prefix of that cache.

``own`` false computes each operator in elementary torch operations in 32 bits (64 for angles), rounded once at the
end; ``own`` true calls the library's entry points.  Sizes: 8 query heads on one key/value head of 256 with 10 and 50
action rows and 768 encoder tokens are this library's decoder and encoder row counts; the other head layouts are
generic grouped-head ones.
"""
import itertools
import math
import random

import torch

own = False

PAGE = 16                       # cache rows per page unless a case says otherwise
# (query heads, key/value heads, head size)
HEADS = ((8, 1, 256), (32, 8, 128), (16, 2, 64), (28, 4, 128), (16, 16, 72), (12, 12, 80), (40, 8, 128), (8, 8, 64))


# ---------------------------------------------------------------- cases

def _append(name, tokens, heads, rot, interleaved, norm, base, factor, first, padding, keep_k):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads[0], "kv_heads": heads[1], "dim": heads[2],
            "rot": rot, "interleaved": interleaved, "norm": norm, "base": base, "factor": factor, "first": first,
            "padding": padding, "keep_k": keep_k}


def _prompt(name, sequences, rows, context, padding, heads, causal):
    return {"name": name, "op": "prompt", "sequences": sequences, "rows": rows, "context": context,
            "padding": padding, "heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "causal": causal}


def _shared(name, sequences, rows, prefix, suffix, page, heads, causal):
    return {"name": name, "op": "shared", "sequences": sequences, "rows": rows, "prefix": prefix, "suffix": suffix,
            "page": page, "heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "causal": causal}


def listed():
    return [
        # one generated token of one sequence: pure latency
        _append("append one token", 1, HEADS[0], 256, False, False, 10000.0, 1.0, 801, 0, False),
        # the action decoder's rows, positions behind the encoder's tokens
        _append("append 50 action rows", 50, HEADS[0], 256, False, False, 10000.0, 1.0, 768, 0, False),
        # a packed prompt with normed heads, part of each head rotated in pairs, a padded tail
        _append("append 2049 tokens", 2049, HEADS[3], 64, True, True, 500000.0, 1.0, 0, 3, True),
        # a long document's chunk far from the start, frequencies stretched for the long context
        _append("append 16387 far tokens", 16387, HEADS[1], 128, False, True, 1000000.0, 32.0, 1000003, 0, True),
        # the action rows among themselves, no cache
        _prompt("prompt 50 rows", 1, 50, 0, 0, HEADS[0], False),
        # the encoder's tokens, every token sees every other
        _prompt("prompt 768 tokens", 1, 768, 0, 0, HEADS[0], False),
        # a serving batch: 16 ragged causal prompts, some with keys of an earlier chunk before them, a padded tail
        _prompt("prompt 16 ragged", 16, 9001, 700, 5, HEADS[3], True),
        # one long causal prompt
        _prompt("prompt 8191 tokens", 1, 8191, 0, 0, HEADS[1], True),
        # one denoising step: 10 action rows over the encoder's cached keys and their own
        _shared("shared 10 rows", 1, 10, 768, 10, PAGE, HEADS[0], False),
        # one token of one sequence with a very long cache and no shared prefix
        _shared("shared one token long", 1, 1, 0, 131071, 64, HEADS[1], True),
        # 64 sequences decode one token each behind one long shared prompt
        _shared("shared 64 sequences", 64, 1, 8195, 300, PAGE, HEADS[1], True),
        # 32 sampled action chunks of 50 rows over one encoder prefix
        _shared("shared 32 chunks", 32, 50, 800, 50, PAGE, HEADS[0], False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    heads = rng.choice(HEADS)
    op = rng.choice(("append", "prompt", "shared"))
    if op == "append":
        tokens = _spread(rng, 1, 16384 * 48 // (heads[0] + 2 * heads[1]) * 128 // max(heads[2], 128))
        tokens = min(tokens, 16384)
        rots = [r for r in (heads[2], 64, 32, 16) if r <= heads[2]]
        case = _append("", tokens, heads, rng.choice(rots), rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice((10000.0, 500000.0)), rng.choice((1.0, 8.0)), rng.randrange(0, 1 << 20),
                       rng.randrange(0, 1 + min(4, tokens - 1)), rng.random() < 0.5)
    elif op == "prompt":
        causal = rng.random() < 0.7
        sequences = _spread(rng, 1, 24)
        rows = _spread(rng, max(16, sequences), 6000 if causal else 4000)
        context = rng.choice((0, 0, _spread(rng, 1, 600)))
        case = _prompt("", sequences, rows, context, rng.randrange(0, 4), heads, causal)
    else:
        rows = rng.choice((1, 1, 1, 2, 5, 10, 50))
        sequences = _spread(rng, 1, 64 if rows < 50 else 32)
        prefix = rng.choice((0, _spread(rng, 17, 8000)))
        most = max(64, min(60000, 120000 * 8 // (sequences * heads[1]))) if rows == 1 else 400
        suffix = max(rows, _spread(rng, 1, most))
        case = _shared("", sequences, rows, prefix, suffix, rng.choice((8, 16, 64)), heads, rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(total, parts, empty):
    """`total` split into `parts` ragged lengths, always the same ones for the same numbers; with `empty`, one part
    of three or more is 0 and one is 1."""
    if parts == 1:
        return [total]
    rng = random.Random("%d in %d" % (total, parts))
    weights = [math.exp(rng.gauss(0.0, 0.8)) for _ in range(parts)]
    if empty and parts >= 3:
        weights[0] = weights[1] = 0.0
    whole = sum(weights)
    lengths = [int(total * w / whole) for w in weights]
    if empty and parts >= 3:
        lengths[1] = min(1, total)
    lengths[-1] += total - sum(lengths)
    if lengths[-1] < 0:
        lengths[lengths.index(max(lengths))] += lengths[-1]
        lengths[-1] = 0
    rng.shuffle(lengths)
    return lengths


def _prompt_lengths(case):
    """(rows, keys) of each sequence: the rows of a chunk and, in some sequences, keys of earlier chunks before it."""
    rows = _lengths(case["rows"], case["sequences"], True)
    rng = random.Random("context %d %d" % (case["rows"], case["sequences"]))
    extra = [rng.randint(0, case["context"]) if rng.random() < 0.6 else 0 for _ in rows]
    return rows, [r + x for r, x in zip(rows, extra)]


def _suffix_lengths(case):
    """Cached rows of each sequence behind the prefix, the call's own rows among them."""
    if case["sequences"] == 1:
        return [case["suffix"]]
    rng = random.Random("suffix %d %d" % (case["suffix"], case["sequences"]))
    return [rng.randint(case["rows"], case["suffix"]) for _ in range(case["sequences"])]


def _pairs(rows, keys, causal):
    """Visible (row, key) pairs of one sequence whose ends are aligned."""
    if not causal:
        return rows * keys
    return sum(max(0, min(keys, i + 1 + keys - rows)) for i in range(rows))


def work(case):
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        kept = case["tokens"] - case["padding"]
        read = case["tokens"] * (hq + 2 * hk) * d * 2 + case["tokens"] * 12 + case["rot"] * 2
        written = case["tokens"] * (hq + (hk if case["keep_k"] else 0)) * d * 2 + kept * 2 * hk * d * 2
        return {"bytes": read + written, "flops": case["tokens"] * (hq + hk) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "prompt":
        rows, keys = _prompt_lengths(case)
        pairs = sum(_pairs(r, k, case["causal"]) for r, k in zip(rows, keys))
        return {"bytes": 2 * d * (2 * sum(rows) * hq + 2 * sum(keys) * hk), "flops": 4 * d * hq * pairs}
    lengths = _suffix_lengths(case)
    rows = case["rows"]
    pairs = sum(rows * case["prefix"] + _pairs(rows, n, case["causal"]) for n in lengths)
    cached = case["prefix"] + sum(lengths)
    return {"bytes": 2 * d * (2 * len(lengths) * rows * hq + 2 * cached * hk), "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------- inputs

def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(torch.bfloat16)


def _offsets(lengths):
    return torch.tensor([0] + list(itertools.accumulate(lengths)), dtype=torch.int32, device="cuda")


def _prepare_append(case, gen):
    t, hq, hk, d, rot = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["rot"]
    pages = -(-t // PAGE) + 5
    table = torch.randperm(pages, device="cuda", generator=gen)
    at = torch.arange(t, device="cuda")
    slots = table[at // PAGE] * PAGE + at % PAGE
    slots[t - case["padding"]:] = -1
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    qkv = _normal(gen, t, (hq + 2 * hk) * d)
    s = {"qkv": qkv, "q": qkv[:, :hq * d], "k": qkv[:, hq * d:(hq + hk) * d], "v": qkv[:, (hq + hk) * d:],
         "inv_freq": (case["base"] ** (-2.0 * j / rot) / case["factor"]).float(),
         "rot_scale": 0.1 * math.log(case["factor"]) + 1.0, "eps": 1e-6,
         "positions": (at + case["first"]).to(torch.int32), "slots": slots,
         "q_weight": None, "k_weight": None,
         "q_out": torch.zeros(t, hq, d, dtype=torch.bfloat16, device="cuda"),
         "k_out": torch.zeros(t, hk, d, dtype=torch.bfloat16, device="cuda") if case["keep_k"] else None,
         "k_cache": _normal(gen, pages * PAGE, hk, d), "v_cache": _normal(gen, pages * PAGE, hk, d)}
    if case["norm"]:
        s["q_weight"], s["k_weight"] = (1 + _normal(gen, d, scale=0.2) for _ in range(2))
    return s


def _prepare_prompt(case, gen):
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    rows, keys = _prompt_lengths(case)
    total_q, total_k = sum(rows) + case["padding"], sum(keys) + case["padding"]
    # logits of a few units: rows attend to a minority of their keys
    return {"q": _normal(gen, total_q, hq, d, scale=2.0), "k": _normal(gen, total_k, hk, d),
            "v": _normal(gen, total_k, hk, d), "cu_q": _offsets(rows), "cu_k": _offsets(keys),
            "longest": (max(rows), max(keys)), "scale": 1.0 / math.sqrt(d),
            "out": torch.zeros(total_q, hq, d, dtype=torch.bfloat16, device="cuda")}


def _prepare_shared(case, gen):
    hq, hk, d, page, b = case["heads"], case["kv_heads"], case["dim"], case["page"], case["sequences"]
    lengths = _suffix_lengths(case)
    shared, each = -(-case["prefix"] // page), -(-case["suffix"] // page)
    pages = shared + each * b + 3
    table = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    s = {"q": _normal(gen, b * case["rows"], hq, d, scale=2.0),
         "k_cache": _normal(gen, pages * page, hk, d), "v_cache": _normal(gen, pages * page, hk, d),
         "prefix_pages": table[:shared].clone() if shared else None,
         "prefix_len": torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda") if shared else None,
         "block_table": table[shared:shared + each * b].reshape(b, each).clone(),
         "seq_lens": torch.tensor(lengths, dtype=torch.int32, device="cuda"),
         "pages": (pages, shared, each), "scale": 1.0 / math.sqrt(d),
         "out": torch.zeros(b * case["rows"], hq, d, dtype=torch.bfloat16, device="cuda")}
    if own:
        import bf16_gemm_vla_amd as vla

        n = vla.vla_attn_shared_prefix_workspace_bytes(b, case["rows"], hq, hk, d, shared * page, each * page)
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")      # kept by the program, zero-filled once
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"append": _prepare_append, "prompt": _prepare_prompt, "shared": _prepare_shared}[case["op"]]
    return dict(make(case, gen), case=case)


# ---------------------------------------------------------- plain forms

def _plain_heads(x, weight, cos, sin, rot, interleaved, eps):
    """Normed and rotated heads of x (tokens x heads x size), in fp32, rounded once."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    return torch.cat((turned, x[..., rot:]), -1).to(torch.bfloat16)


def _plain_append(s):
    case = s["case"]
    t, hq, hk, d, rot = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["rot"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = (torch.cos(angle) * s["rot_scale"]).float(), (torch.sin(angle) * s["rot_scale"]).float()
    s["q_out"].copy_(_plain_heads(s["q"].reshape(t, hq, d), s["q_weight"], cos, sin, rot, case["interleaved"], s["eps"]))
    k = _plain_heads(s["k"].reshape(t, hk, d), s["k_weight"], cos, sin, rot, case["interleaved"], s["eps"])
    if s["k_out"] is not None:
        s["k_out"].copy_(k)
    kept = s["slots"] >= 0
    s["k_cache"][s["slots"][kept]] = k[kept]
    s["v_cache"][s["slots"][kept]] = s["v"].reshape(t, hk, d)[kept]


def _plain_attend(q, k, v, seen, scale):
    """Attention of q (batch x rows x heads x size) over k and v (batch x keys x kv heads x size); seen: batch x rows
    x keys.  fp32 throughout; a row that sees nothing gives 0."""
    b, n, hq, d = q.shape
    hk = k.shape[2]
    q = q.float().reshape(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    k, v = (x.float().permute(0, 2, 1, 3).contiguous() for x in (k, v))
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale).reshape(b, hk, hq // hk, n, -1)
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True).clamp_(min=1e-38)
    out = torch.matmul(scores.reshape(b, hk, -1, scores.shape[-1]), v).reshape(b, hk, hq // hk, n, d) / total
    return out.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)


def _plain_prompt(s):
    most_q, most_k = s["longest"]
    nq, nk = (s[c][1:] - s[c][:-1] for c in ("cu_q", "cu_k"))
    i, j = torch.arange(most_q, device="cuda"), torch.arange(most_k, device="cuda")
    row = (s["cu_q"][:-1, None] + i).clamp_(max=s["q"].shape[0] - 1)
    key = (s["cu_k"][:-1, None] + j).clamp_(max=s["k"].shape[0] - 1)
    seen = (j < nk[:, None])[:, None, :] & (i < nq[:, None])[:, :, None]
    if s["case"]["causal"]:
        seen = seen & (j <= i[:, None] + (nk - nq)[:, None, None])
    out = _plain_attend(s["q"][row], s["k"][key], s["v"][key], seen, s["scale"])
    real = i < nq[:, None]
    s["out"][row[real]] = out[real].to(torch.bfloat16)


def _plain_shared(s):
    case = s["case"]
    b, rows, page = case["sequences"], case["rows"], case["page"]
    inside = torch.arange(page, device="cuda")
    slot = (s["block_table"].long()[:, :, None] * page + inside).reshape(b, -1)
    j, i = torch.arange(slot.shape[1], device="cuda"), torch.arange(rows, device="cuda")
    length = s["seq_lens"][:, None, None]
    seen = (j < length).expand(b, rows, -1)
    if case["causal"]:
        seen = seen & (j <= i[:, None] + length - rows)
    if s["prefix_pages"] is not None:
        shared = (s["prefix_pages"].long()[:, None] * page + inside).reshape(1, -1).expand(b, -1)
        there = torch.arange(shared.shape[1], device="cuda") < s["prefix_len"]
        slot, seen = torch.cat((shared, slot), 1), torch.cat((there.expand(b, rows, -1), seen), 2)
    q = s["q"].reshape(b, rows, case["heads"], case["dim"])
    out = _plain_attend(q, s["k_cache"][slot], s["v_cache"][slot], seen, s["scale"])
    s["out"].copy_(out.reshape(s["out"].shape).to(torch.bfloat16))


def run(state):
    s, case = state, state["case"]
    if own:
        import bf16_gemm_vla_amd as vla

        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        if case["op"] == "append":
            stride = s["qkv"].shape[1]
            vla.vla_qk_norm_rope_append(
                s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["inv_freq"], s["positions"], s["slots"],
                s["q_out"], s["k_out"], s["k_cache"], s["v_cache"], case["tokens"], hq, hk, d, case["rot"],
                stride, stride, stride, hq * d, hk * d, s["k_cache"].shape[0],
                vla.VLA_ROPE_INTERLEAVED if case["interleaved"] else vla.VLA_ROPE_HALF, s["rot_scale"], s["eps"])
        elif case["op"] == "prompt":
            vla.vla_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], case["sequences"],
                                s["q"].shape[0], s["k"].shape[0], hq, hk, d, hq * d, hk * d, hk * d, hq * d,
                                case["causal"], s["scale"])
        else:
            pages, shared, each = s["pages"]
            vla.vla_attn_shared_prefix(
                s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"], s["prefix_len"], s["block_table"],
                s["seq_lens"], s["out"], s["ws"], s["ws"].numel(), case["sequences"], case["rows"], hq, hk, d,
                pages, case["page"], shared, each, hq * d, hq * d, case["causal"], s["scale"])
    elif case["op"] == "append":
        _plain_append(s)
    elif case["op"] == "prompt":
        _plain_prompt(s)
    else:
        _plain_shared(s)
    if case["op"] == "append":
        out = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if s["k_out"] is not None:
            out["k"] = s["k_out"]
        return out
    return {"out": s["out"]}


# ------------------------------------------------------- 64-bit results

def _exact_append(s):
    case = s["case"]
    t, rot = case["tokens"], case["rot"]
    turn = torch.polar(torch.full((t, 1, rot // 2), s["rot_scale"], dtype=torch.float64, device="cuda"),
                       (s["positions"].double()[:, None] * s["inv_freq"].double())[:, None, :])

    def head(x, weight):
        x = x.double().reshape(t, -1, case["dim"])
        if weight is not None:
            x = weight.double() * x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt()
        y = x.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k, v = head(s["k"], s["k_weight"]), s["v"].double().reshape(t, -1, case["dim"])
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    kept = torch.nonzero(s["slots"] >= 0)[:, 0]
    k_cache.index_copy_(0, s["slots"][kept], k[kept])
    v_cache.index_copy_(0, s["slots"][kept], v[kept])
    out = {"q": head(s["q"], s["q_weight"]), "k_cache": k_cache, "v_cache": v_cache}
    if case["keep_k"]:
        out["k"] = k
    return out


def _exact_rows(q, k, v, limits, scale):
    """Rows q (n x heads x size) in 64 bits, row i seeing the first limits[i] keys, one key/value head at a time."""
    n, hq, d = q.shape
    hk = k.shape[1]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    if k.shape[0] == 0 or n == 0:
        return out
    hidden = torch.arange(k.shape[0], device="cuda")[None, :] >= limits[:, None]
    some = (limits > 0).double()[:, None]
    for h in range(hq):
        kh, vh = k[:, h * hk // hq].double(), v[:, h * hk // hq].double()
        weight = torch.softmax((q[:, h].double() @ kh.t() * scale).masked_fill_(hidden, -1e300), -1)
        out[:, h] = weight @ vh * some
    return out


def _exact_prompt(s):
    out = s["out"].double()
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cq) - 1):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        limits = torch.full((nq,), nk, device="cuda")
        if s["case"]["causal"]:
            limits = (torch.arange(nq, device="cuda") + 1 + nk - nq).clamp(0, nk)
        keys = slice(ck[b], ck[b + 1])
        out[cq[b]:cq[b + 1]] = _exact_rows(s["q"][cq[b]:cq[b + 1]], s["k"][keys], s["v"][keys], limits, s["scale"])
    return {"out": out}


def _exact_shared(s):
    case = s["case"]
    rows, page, prefix = case["rows"], case["page"], case["prefix"]
    out = s["out"].double()

    def cached(cache, pages, n):
        return cache.reshape(-1, page, *cache.shape[1:])[pages.long()].flatten(0, 1)[:n]

    for b, n in enumerate(s["seq_lens"].tolist()):
        k, v = (cached(s[c], s["block_table"][b], n) for c in ("k_cache", "v_cache"))
        if prefix:
            k, v = (torch.cat((cached(s[c], s["prefix_pages"], prefix), x)) for c, x in (("k_cache", k), ("v_cache", v)))
        limits = torch.full((rows,), prefix + n, device="cuda")
        if case["causal"]:
            limits = prefix + (torch.arange(rows, device="cuda") + 1 + n - rows).clamp(0, n)
        out[b * rows:(b + 1) * rows] = _exact_rows(s["q"][b * rows:(b + 1) * rows], k, v, limits, s["scale"])
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "prompt": _exact_prompt, "shared": _exact_shared}[case["op"]](s)
